"""Appends to a cache of more than 2^32 bytes whose used pages lie at its end: codes and scales of all positions are those
of the definition, and every page before them keeps its zeros (an address cut to 32 bits would fall among them)."""
import numpy as np
import pytest

import oracle.kv_cache as kv
from decoder_util import Batch, bf16, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


@pytest.mark.parametrize("new,total", [([1, 40], [300, 40]), ([300, 7], [300, 135])])
def test_offsets_beyond_32_bits(new, total):
    banner(f"append to a cache of 4.4 GB, new {new}")
    pages, size, dim = 270_000, 128, 128
    assert (pages - 10) * size * dim > 1 << 32
    cache = fb.KVCache.empty(pages, 1, size, dim)
    b = Batch(130, new, total, 1, dim, size)
    first = pages - b.pages
    for far, near in zip(cache.args, (*b.codes, *b.scales)):
        far[first:] = dev(near)
    k, v = (bf16(np.random.default_rng(131 + i).standard_normal((b.tokens, 1, dim)) * 3) for i in range(2))
    table = np.where(b.table >= 0, b.table + first, -1).astype(np.int32)
    assert fb.fp8_kv_append(None, dev(k, torch.bfloat16), dev(v, torch.bfloat16), cache, dev(b.cu), dev(b.lens), dev(table), b.max_new) is None
    for i, (y, c, s) in enumerate(((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale))):
        wc, ws = kv.append(b.codes[i], b.scales[i], y.astype(np.float64), b.cu, b.lens, b.table, size)
        assert not np.array_equal(wc, b.codes[i])
        assert np.array_equal(c[first:].cpu().numpy(), wc) and np.array_equal(s[first:].cpu().numpy(), ws)
        assert not bool(c[:first].any()) and bool((s[:first] == 1).all())
