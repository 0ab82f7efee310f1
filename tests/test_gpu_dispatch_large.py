"""Dispatch of more choices than 256 runs of 2048: a workgroup of the sort takes several runs in turn.  All outputs are
equal bit for bit to the definition, the rows to fp8_quant_act_1x128."""
import numpy as np
import pytest

from decoder_util import dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


@pytest.mark.parametrize("tokens,k,experts", [(65536, 8, 256), (65537, 8, 256), (70001, 8, 384), (131099, 9, 64), (40001, 32, 1024), (600_011, 1, 1), (530_000, 1, 7)])
def test_many_runs(tokens, k, experts):
    banner(f"dispatch {tokens} tokens x {k} of {experts} experts")
    rng = np.random.default_rng(120)
    ids = rng.integers(0, experts, (tokens, k)).astype(np.int32)
    ids[rng.random((tokens, k)) < 0.4] = experts // 2      # one expert is asked for by many
    ids[rng.random(tokens) < 0.05] = -1
    ids[rng.random((tokens, k)) < 0.02] = experts
    g = torch.Generator(device="cuda").manual_seed(121)
    x = torch.randn(tokens, 128, device="cuda", generator=g).bfloat16()
    q, scale, offsets, order, position = fb.fp8_moe_dispatch(x, dev(ids), experts)
    flat = ids.reshape(-1).astype(np.int64)
    flat = np.where((flat >= 0) & (flat < experts), flat, experts)
    want = np.argsort(flat, kind="stable")
    assert np.array_equal(order.cpu().numpy(), want)
    back = np.empty(tokens * k, np.int32)
    back[want] = np.arange(tokens * k)
    assert np.array_equal(position.cpu().numpy().reshape(-1), back)
    assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(flat[want], np.arange(experts + 1)))
    codes, s = fb.fp8_quant_act_1x128(x)
    token, dead = dev(want // k), dev(flat[want] == experts)
    assert torch.equal(q, codes[token].masked_fill_(dead[:, None], 0))
    assert torch.equal(scale, s[token].masked_fill_(dead[:, None], 1.0))
