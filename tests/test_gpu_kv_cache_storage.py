"""A cache whose tensors got another storage: calls use the new one, and the old one keeps its bytes."""
import copy

import numpy as np
import pytest

import oracle.kv_cache as kv
from decoder_util import Batch, bf16, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def test_calls_follow_a_new_storage():
    banner("append and attention after set_")
    b = Batch(90, [3, 1], [20, 33], 2, 64, 16)
    cache, cu, lens, table = b.on_gpu()
    held = [t.detach() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]      # the old storages
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        t.set_(t.clone())
    rng = np.random.default_rng(91)
    q, k, v = (bf16(rng.standard_normal((b.tokens, h, 64))) for h in (4, 2, 2))
    got = fb.fp8_kv_append(*[dev(x, torch.bfloat16) for x in (q, k, v)], cache, cu, lens, table, b.max_new)
    out = fb.fp8_kv_attention(got, cache, cu, lens, table, b.max_new, b.max_len)
    for i, y in enumerate((k, v)):
        wc, ws = kv.append(b.codes[i], b.scales[i], y.astype(np.float64), b.cu, b.lens, b.table, 16)
        assert np.array_equal((cache.k, cache.v)[i].cpu().numpy(), wc) and np.array_equal((cache.k_scale, cache.v_scale)[i].cpu().numpy(), ws)
        assert np.array_equal(held[i].cpu().numpy(), b.codes[i]) and np.array_equal(held[2 + i].cpu().numpy(), b.scales[i])
    other = copy.deepcopy(cache)
    assert other.k.data_ptr() != cache.k.data_ptr() and copy.copy(cache).k is cache.k
    cache.k.zero_()
    cache.k.copy_(other.k)
    assert torch.equal(out, fb.fp8_kv_attention(got, other, cu, lens, table, b.max_new, b.max_len))
