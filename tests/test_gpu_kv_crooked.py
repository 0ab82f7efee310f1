"""Attention over tables that hold anything: nothing outside out, lse and the workspace is written, rows of sequences
whose entries are sound are what they are alone, and a row before position 0 sees nothing."""
import numpy as np
import pytest

from decoder_util import Batch, bf16, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

GUARD = 4096


class Guarded:
    """Device bytes between two guards."""

    def __init__(self, size):
        self.size = size
        self.all = torch.full((2 * GUARD + size,), 0xa5, dtype=torch.uint8, device="cuda")
        self.ptr = self.all.data_ptr() + GUARD

    def view(self, dtype, *shape):
        return self.all[GUARD:GUARD + self.size].view(dtype).view(shape)

    def check(self):
        assert bool((self.all[:GUARD] == 0xa5).all()) and bool((self.all[GUARD + self.size:] == 0xa5).all())


def attend(cache, q, cu, lens, table, max_new, max_len, window=0):
    """The library's call with guarded outputs and workspace: (out, lse)."""
    from fp8_block_scaled_05_amd import decoder
    t, hq, d = q.shape
    pages, heads, size, _ = cache.k.shape
    c = decoder._CACHE.pack(*(x.data_ptr() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)), pages, heads, size, d)
    b = decoder._BATCH.pack(cu.data_ptr(), lens.data_ptr(), table.data_ptr(), table.stride(0), table.shape[1], lens.numel(), t, max_new, max_len)
    args = lambda o, l, w, n: decoder._ATTEND.pack(q.data_ptr(), o, l, w, n, hq * d, d, hq, window, d ** -0.5)   # noqa: E731
    need = fb.lib().fp8_kv_attention_workspace(c, b, args(0, 0, 0, 0))
    assert need >= 0
    out, lse, room = Guarded(2 * t * hq * d), Guarded(4 * t * hq), Guarded(need)
    fb._check(fb.lib().fp8_kv_attention(c, b, args(out.ptr, lse.ptr, room.ptr if need else 0, need), fb._stream()))
    torch.cuda.synchronize()
    for g in (out, lse, room):
        g.check()
    return out.view(torch.bfloat16, t, hq, d), lse.view(torch.float32, t, hq)


# 16-row tiles, unsplit and split, and 128-row tiles: new tokens a sequence, cached tokens
SIZES = [(1, 90), (1, 5000), (3, 700), (300, 1200), (700, 3000)]


@pytest.mark.parametrize("new,total", SIZES)
@pytest.mark.parametrize("window", [0, 50])
def test_crooked_lengths(new, total, window):
    banner(f"attend crooked lengths {new} {total} window {window}")
    b = Batch(95, [new] * 6, [total] * 6, 2, 64, 16)
    cache, cu, _, table = b.on_gpu()
    q = dev(bf16(np.random.default_rng(96).standard_normal((b.tokens, 8, 64))), torch.bfloat16)
    want, wlse = attend(cache, q, cu, dev(b.lens), table, new, total, window)
    lens = b.lens.copy()
    lens[1], lens[2], lens[3], lens[4] = -5, np.iinfo(np.int32).min, np.iinfo(np.int32).max, new // 2
    out, lse = attend(cache, q, cu, dev(lens), table, new, total, window)
    for s in (0, 5):
        rows = slice(s * new, (s + 1) * new)
        assert torch.equal(out[rows], want[rows]) and torch.equal(lse[rows], wlse[rows])
    for s, n in ((1, new), (2, new), (4, new - new // 2)):     # rows before position 0
        rows = slice(s * new, s * new + n)
        assert bool((out[rows] == 0).all()) and bool(torch.isneginf(lse[rows]).all())
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("new,total", SIZES)
def test_crooked_offsets(new, total):
    """Offsets that fall, that are negative and that lie beyond the tokens, and a bound of new tokens that is too small."""
    banner(f"attend crooked offsets {new} {total}")
    b = Batch(97, [new] * 6, [total] * 6, 2, 64, 16)
    cache, cu, lens, table = b.on_gpu()
    q = dev(bf16(np.random.default_rng(98).standard_normal((b.tokens, 8, 64))), torch.bfloat16)
    want, wlse = attend(cache, q, cu, lens, table, new, total)
    t = b.tokens
    for crooked in ([0, t, 0, t, 0, t, 0], [t, 0, t, 0, t, 0, t], [-5, t // 2, -(1 << 31), (1 << 31) - 1, 7, t + 9, 3], [0] * 7,
                    [(1 << 31) - 1] * 7, [-(1 << 31)] * 7):
        attend(cache, q, dev(np.array(crooked, np.int64).astype(np.int32)), lens, table, new, total)
    straight = b.cu.copy()
    straight[0], straight[6] = -9, t + 1000            # clamped: the same rows
    out, lse = attend(cache, q, dev(straight), lens, table, new, total)
    assert torch.equal(out, want) and torch.equal(lse, wlse)
    attend(cache, q, cu, lens, table, max(1, new // 2), total // 2)


def test_many_sequences_claim_all_rows():
    """Each second of 4000 sequences claims every row: tiles number far more than the launch has."""
    banner("attend 4000 sequences, falling offsets")
    new, n = 600, 4000
    b = Batch(99, [new], [900], 1, 64, 16)
    cache, _, _, table = b.on_gpu()
    q = dev(bf16(np.random.default_rng(100).standard_normal((new, 4, 64))), torch.bfloat16)
    cu = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = new
    lens = torch.full((n,), 900, dtype=torch.int32, device="cuda")
    tables = table.expand(n, -1).contiguous()
    # the same sizes, so the same tiles: the first sequence owns all rows
    want, _ = attend(cache, q, torch.full_like(cu, new).index_fill_(0, torch.zeros(1, dtype=torch.int64, device="cuda"), 0), lens, tables, new, 900)
    out, _ = attend(cache, q, cu, lens, tables, new, 900)
    # whatever was written is the rows' own result
    same = (out == want).all(-1) | (out.view(torch.uint8).view(new, 4, 128) == 0xa5).all(-1)
    assert bool(same.all())
