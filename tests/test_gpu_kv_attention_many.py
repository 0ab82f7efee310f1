"""Attention over many sequences and long caches, against float64 on the GPU: row tiles of more than 64 sequences are
found among all of them, a split spans more tiles than one look at the block table serves, and few or many splits are
joined.  Tolerances as in test_gpu_kv_attention.py."""
import numpy as np
import pytest

from decoder_util import Batch, bf16, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _check(b, hq, window=0, seed=70):
    q = dev(bf16(np.random.default_rng(seed).standard_normal((b.tokens, hq, b.dim))), torch.bfloat16)
    cache, cu, lens, table = b.on_gpu()
    out, lse = fb.fp8_kv_attention(q, cache, cu, lens, table, b.max_new, b.max_len, window=window, return_lse=True)
    scale = b.dim ** -0.5
    at = 0
    for s, (n, total) in enumerate(zip(b.new, b.lens.tolist())):
        if not n:
            continue
        pages = table[s, :-(-total // b.page)].long()
        k, v = ((c[pages].view(torch.float8_e4m3fn).double() * x[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :total]
                for c, x in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        seen, mine = torch.arange(total, device="cuda")[None], torch.arange(total - n, total, device="cuda")[:, None]
        ok = seen <= mine
        if window:
            ok &= mine - seen < window
        for h in range(hq):
            g = h // (hq // b.heads)
            x = q[at:at + n, h].double()
            z = torch.where(ok, x @ k[g].t().contiguous() * scale, -float("inf"))
            absz = torch.where(ok, x.abs() @ k[g].abs().t().contiguous() * scale, 0.0).amax(1)
            want = torch.logsumexp(z, 1)
            w = torch.exp(z - want[:, None])
            dz = 2.0 ** -18 * absz + 2.0 ** -16
            ref = w @ v[g]
            tol = (2.0 ** -8 + 2 * dz[:, None]) * (w @ v[g].abs()) + 2.0 ** -8 * ref.abs() + 1e-30
            assert bool(((out[at:at + n, h].double() - ref).abs() <= tol).all()), (s, h)
            assert bool(((lse[at:at + n, h].double() - want).abs() <= dz + 2.0 ** -22 * want.abs()).all()), (s, h)
        at += n


def test_more_sequences_than_lanes():
    banner("attend 150 sequences of 0 to 90 new tokens")
    rng = np.random.default_rng(71)
    new = [int(n) for n in rng.integers(0, 91, 150)]
    new[3] = new[77] = 0
    total = [n + int(t) for n, t in zip(new, rng.integers(0, 400, 150))]
    _check(Batch(72, new, total, 2, 64, 16), 4)


@pytest.mark.parametrize("dim,page,window", [(128, 64, 0), (64, 16, 0), (128, 32, 5000)])
def test_more_tiles_than_one_look(dim, page, window):
    """100 and more 64-key tiles of one workgroup: 512 tiles of rows leave the keys unsplit."""
    banner(f"attend 8 x 2048 new rows over 7000 tokens, dim {dim} window {window}")
    new = [512, 500, 511, 300, 512, 40, 1, 512]
    total = [7000, 6500, 600, 4100, 4500, 6999, 6000, 5001]
    _check(Batch(73, new, total, 8, dim, page), 32, window)


@pytest.mark.parametrize("new,total,hq,hk,dim", [([70, 9], [3000, 2500], 8, 2, 64), ([33], [9000], 4, 1, 128), ([300, 0, 200], [2000, 5, 1300], 16, 4, 128),
                                                ([1], [40000], 16, 1, 64), ([2, 1, 1], [1500, 1, 2048], 8, 1, 128), ([1], [2100], 8, 8, 128), ([1, 1], [130, 6000], 16, 2, 128)])
def test_splits_of_the_keys(new, total, hq, hk, dim):
    banner(f"attend splits new {new} total {total}")
    _check(Batch(74, new, total, hk, dim, 64), hq)


def test_missing_pages_in_a_long_cache():
    """Page numbers that are no pages hide their tokens, in every kernel, wherever they lie in a tile."""
    for new, total in ((1, 9000), (64, 9000), (1200, 9000)):
        b = Batch(75, [new], [total], 2, 64, 16)
        gone = [0, 5, 63, 64, 250, 251, 252, 253, 300]
        holed = b.table.copy()
        b.table[0, gone] = b.table[0, 10]              # so that the reference may read them; masked below
        q = dev(bf16(np.random.default_rng(76).standard_normal((new, 4, 64))), torch.bfloat16)
        holed[0, gone[::2]] = -1
        holed[0, gone[1::2]] = b.pages + 7
        cache, cu, lens, _ = b.on_gpu()
        out = fb.fp8_kv_attention(q, cache, cu, lens, dev(holed), new, total)
        pages = dev(b.table)[0].long()
        k, v = ((c[pages].view(torch.float8_e4m3fn).double() * x[pages].double()[..., None, None]).transpose(0, 1).flatten(1, 2)[:, :total]
                for c, x in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
        there = torch.ones(-(-total // 16), dtype=torch.bool, device="cuda")
        there[gone] = False
        ok = there.repeat_interleave(16)[:total][None] & (torch.arange(total, device="cuda")[None] <= torch.arange(total - new, total, device="cuda")[:, None])
        for h in range(4):
            z = torch.where(ok, q[:, h].double() @ k[h // 2].t().contiguous() / 8, -float("inf"))
            w = torch.softmax(z, 1)
            tol = (2.0 ** -8 + 2.0 ** -10) * (w @ v[h // 2].abs()) + 2.0 ** -8 * (w @ v[h // 2]).abs() + 1e-30
            assert bool(((out[:, h].double() - w @ v[h // 2]).abs() <= tol).all()), (new, h)


@pytest.mark.parametrize("new,total", [(1, 5000), (1, 1000), (90, 5000), (1500, 5000)])
def test_a_nan_value_is_its_rows(new, total):
    """A NaN among the values makes whole rows NaN where they see it, far from any edge, with the keys split or not."""
    b = Batch(77, [new], [total], 2, 128, 64)
    b.codes[1][b.table[0][333 // 64], 1, 333 % 64, 17] = 0x7f
    q = dev(bf16(np.random.default_rng(78).standard_normal((new, 4, 128))), torch.bfloat16)
    cache, cu, lens, table = b.on_gpu()
    out, lse = fb.fp8_kv_attention(q, cache, cu, lens, table, new, total, return_lse=True)
    assert torch.isnan(out[:, 2:]).all() and torch.isnan(lse[:, 2:]).all()
    assert not torch.isnan(out[:, :2]).any() and not torch.isnan(lse[:, :2]).any()


@pytest.mark.parametrize("which", [0, 1])
def test_a_nan_in_a_late_token_of_a_prompt(which):
    """The 1700th of 3000 new tokens has a NaN in its key (or value) for kv head 0: rows before it, in its own tile too, and
    the other kv head do not notice."""
    b = Batch(79, [3000], [3210], 2, 64, 16)
    place = 210 + 1700
    b.codes[which][b.table[0][place // 16], 0, place % 16, 5] = 0xff
    q = dev(bf16(np.random.default_rng(80).standard_normal((3000, 4, 64))), torch.bfloat16)
    cache, cu, lens, table = b.on_gpu()
    out, _ = fb.fp8_kv_attention(q, cache, cu, lens, table, 3000, 3210, return_lse=True)
    assert torch.isnan(out[1700:, :2]).all()
    assert not torch.isnan(out[:1700]).any() and not torch.isnan(out[:, 2:]).any()


def test_a_small_window_over_a_long_prompt():
    banner("attend 6000 new tokens, window 100")
    _check(Batch(81, [6000], [6100], 8, 64, 32), 32, 100)


@pytest.mark.parametrize("new,hq,hk,dim", [([2], 64, 4, 128), ([3, 7], 16, 1, 64), ([17], 3, 1, 128), ([40, 0, 33], 10, 2, 64), ([500], 4, 2, 128)])
def test_several_tiles_of_16_rows(new, hq, hk, dim):
    banner(f"attend 16-row tiles new {new} heads {hq}/{hk}")
    _check(Batch(82, new, [n + 1111 * (i % 2) for i, n in enumerate(new)], hk, dim, 16), hq)
