"""The cache append against its float64 definition.

Tolerances.  Without norm and rotation the stored values are the bf16 inputs: codes and scales are equal bit for
bit.  Otherwise y is computed in float32: a rotation adds two products (error at most 2^-22 (|x1| + |x2|)), a norm
has a sum of up to 128 squares and a few more roundings (relative 2^-19 in all); its bf16 or E4M3 rounding adds
half a step (2^-8 or 2^-4 of the value, or half the smallest E4M3 step, 2^-10, times the scale)."""
import numpy as np
import pytest

import oracle.kv_cache as kv
from decoder_util import Batch, angles, bf16, dev
from gpu_util import banner
from oracle import e4m3_decode

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

BATCHES = {
    "one token": ([1], [1]),
    "decode": ([1, 1, 0, 1], [17, 64, 9, 33]),
    "mid page": ([5, 3], [9, 130]),
    "many pages": ([200, 1, 33], [200, 77, 128]),
    "page boundary": ([16, 17, 1], [32, 33, 129]),
}


def _inputs(b, q_heads, seed, spread=1.0):
    rng = np.random.default_rng(seed)
    width = (q_heads + 2 * b.heads) * b.dim
    qkv = bf16(rng.standard_normal((b.tokens, width)) * spread)
    qkv[rng.random(qkv.shape) < 1e-3] *= 16
    return bf16(qkv)


def _split(b, qkv, q_heads):
    a, c = q_heads * b.dim, (q_heads + b.heads) * b.dim
    return (qkv[:, :a].reshape(b.tokens, q_heads, b.dim), qkv[:, a:c].reshape(b.tokens, b.heads, b.dim),
            qkv[:, c:].reshape(b.tokens, b.heads, b.dim))


def _run(b, qkv, q_heads, **kw):
    cache, cu, lens, table = b.on_gpu()
    g = dev(qkv, torch.bfloat16)                      # q, k, v are slices of one buffer
    a, c = q_heads * b.dim, (q_heads + b.heads) * b.dim
    q = fb.fp8_kv_append(g[:, :a].unflatten(1, (q_heads, b.dim)), g[:, a:c].unflatten(1, (b.heads, b.dim)),
                         g[:, c:].unflatten(1, (b.heads, b.dim)), cache, cu, lens, table, b.max_new, **kw)
    torch.cuda.synchronize()
    return q.float().cpu().numpy(), cache


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", BATCHES)
def test_plain_store_is_bit_exact(name, dim, page):
    new, total = BATCHES[name]
    b = Batch(1, new, total, 2, dim, page)
    banner(f"append {name} dim {dim} page {page}")
    qkv = _inputs(b, 4, 2, spread=8.0)
    q, k, v = _split(b, qkv, 4)
    got_q, cache = _run(b, qkv, 4)
    assert np.array_equal(got_q, q)
    for y, codes, scale, gc, gs in ((k, b.codes[0], b.scales[0], cache.k, cache.k_scale), (v, b.codes[1], b.scales[1], cache.v, cache.v_scale)):
        wc, ws = kv.append(codes, scale, y.astype(np.float64), b.cu, b.lens, b.table, page)
        assert np.array_equal(gs.cpu().numpy(), ws)
        assert np.array_equal(gc.cpu().numpy(), wc)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dim,rot,q_heads,with_norm", [(128, 128, 8, True), (128, 64, 10, False), (64, 64, 2, True), (64, 32, 3 * 2, True),
                                                       (128, 16, 2, False), (64, 48, 4, True), (128, 0, 4, True)])
def test_norm_and_rotation(layout, dim, rot, q_heads, with_norm):
    b = Batch(3, [40, 1, 0, 70], [100, 33, 5, 70], 2, dim, 32)
    banner(f"append {layout} dim {dim} rot {rot} norm {with_norm}")
    qkv = _inputs(b, q_heads, 4)
    q, k, v = _split(b, qkv, q_heads)
    rng = np.random.default_rng(5)
    qw, kw = (bf16(1 + 0.2 * rng.standard_normal(dim)) for _ in range(2)) if with_norm else (None, None)
    rope = angles(128, rot) if rot else None
    got_q, cache = _run(b, qkv, q_heads, rope=dev(rope) if rot else None, rope_layout=layout,
                        q_weight=dev(qw, torch.bfloat16) if with_norm else None, k_weight=dev(kw, torch.bfloat16) if with_norm else None, eps=1e-5)
    want = kv.treat(q, qw, 1e-5, rope, layout, b.cu, b.lens)
    size = np.abs(kv.norm(q, qw, 1e-5))
    other = size.max(-1, keepdims=True)               # a pair's other member is at most this
    assert (np.abs(got_q - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * (size + other)).all()
    yk = kv.treat(k, kw, 1e-5, rope, layout, b.cu, b.lens)
    wc, ws = kv.append(b.codes[0], b.scales[0], yk, b.cu, b.lens, b.table, 32)
    assert np.array_equal(cache.k_scale.cpu().numpy(), ws)
    got, was = cache.k.cpu().numpy(), b.codes[0]
    wv, ws_v = kv.append(b.codes[1], b.scales[1], v.astype(np.float64), b.cu, b.lens, b.table, 32)
    assert np.array_equal(cache.v.cpu().numpy(), wv) and np.array_equal(cache.v_scale.cpu().numpy(), ws_v)
    fresh = np.zeros(got.shape[:1] + got.shape[2:3], bool)
    for r, s, p in kv.rows_of(b.cu, b.lens):
        page, off = b.table[s][p // 32], p % 32
        fresh[page, off] = True
        value = e4m3_decode(got[page, :, off]).astype(np.float64) * ws[page][:, None]
        y = yk[r]
        tol = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * ws[page][:, None] + 2.0 ** -18 * np.abs(y).max(-1, keepdims=True)
        assert (np.abs(value - y) <= tol).all()
    old = ~np.broadcast_to(fresh[:, None, :, None], got.shape)
    assert np.array_equal(got[old], wc[old])          # older tokens and untouched bytes


def test_scales_follow_the_data():
    """Exponents at both ends: a page of zeros gets the smallest scale, large values a large one, and an older
    small scale grows without losing what it held (values that the new scale can hold exactly)."""
    b = Batch(6, [2, 2, 2], [34, 2, 2], 1, 64, 32)
    b.scales[0][:] = 2.0 ** -9
    k = np.zeros((6, 1, 64), np.float32)
    k[0:2] = bf16(3e4)
    k[4:6] = bf16(1e-30)
    qkv = np.concatenate([np.zeros((6, 64), np.float32), k[:, 0], k[:, 0]], 1)
    _, cache = _run(b, qkv, 1)
    wc, ws = kv.append(b.codes[0], b.scales[0], k.astype(np.float64), b.cu, b.lens, b.table, 32)
    assert np.array_equal(cache.k_scale.cpu().numpy(), ws) and np.array_equal(cache.k.cpu().numpy(), wc)
    assert ws[b.table[1, 0], 0] == 2.0 ** -32 and ws[b.table[2, 0], 0] == 2.0 ** -32


def test_growing_scale_token_by_token():
    """Forty appends of one token each: the pages end as the definition says after each of them."""
    b = Batch(7, [1], [40], 2, 128, 16)
    rng = np.random.default_rng(8)
    cache, cu, _, table = b.on_gpu()
    codes, scales = [c.copy() for c in b.codes], [s.copy() for s in b.scales]
    for n in range(1, 41):
        lens = np.array([n], np.int32)
        k, v = (bf16(rng.standard_normal((1, 2, 128)) * 2.0 ** rng.integers(-3, 5)) for _ in range(2))
        assert fb.fp8_kv_append(None, dev(k, torch.bfloat16), dev(v, torch.bfloat16), cache, cu, dev(lens), table, 1) is None
        for i, y in ((0, k), (1, v)):
            codes[i], scales[i] = kv.append(codes[i], scales[i], y.astype(np.float64), b.cu, lens, b.table, 16)
    for i, (c, s) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert np.array_equal(s.cpu().numpy(), scales[i]) and np.array_equal(c.cpu().numpy(), codes[i])


def test_pitched_heads_and_head_major_rows():
    """[H, T, D] inputs seen as [T, H, D]: the head pitch is the larger one."""
    b = Batch(9, [7, 20], [7, 33], 2, 64, 16)
    rng = np.random.default_rng(10)
    q, k, v = (bf16(rng.standard_normal((h, b.tokens, 64))) for h in (4, 2, 2))
    cache, cu, lens, table = b.on_gpu()
    got = fb.fp8_kv_append(*[dev(x, torch.bfloat16).transpose(0, 1) for x in (q, k, v)], cache, cu, lens, table, b.max_new)
    assert np.array_equal(got.float().cpu().numpy(), q.transpose(1, 0, 2))
    for y, i, c in ((k, 0, cache.k), (v, 1, cache.v)):
        wc, _ = kv.append(b.codes[i], b.scales[i], y.transpose(1, 0, 2).astype(np.float64), b.cu, b.lens, b.table, 16)
        assert np.array_equal(c.cpu().numpy(), wc)


def test_bad_tables_leave_other_pages_alone():
    """Page numbers that are not pages, lengths beyond the table and below the new tokens, positions outside the
    angles: those tokens are not stored, everything else is as it would be."""
    b = Batch(11, [3, 3, 3, 3], [20, 20, 20, 20], 1, 64, 16)
    rng = np.random.default_rng(12)
    q, k, v = (bf16(rng.standard_normal((12, 1, 64))) for _ in range(3))
    table, lens = b.table.copy(), b.lens.copy()
    table[1, 1] = b.pages                     # one past the last page
    lens[2] = 10_000                          # beyond its row of the table
    lens[3] = 1                               # two of its three tokens would lie before position 0
    cache, cu, _, _ = b.on_gpu()
    rope = angles(32, 64)
    got = fb.fp8_kv_append(dev(q, torch.bfloat16), dev(k, torch.bfloat16), dev(v, torch.bfloat16), cache, cu, dev(lens), dev(table), 3,
                           rope=dev(rope))
    torch.cuda.synchronize()
    got = got.float().cpu().numpy()
    assert np.all(got[6:11] == 0) and np.all(np.any(got[[0, 1, 2, 3, 4, 5, 11]] != 0, axis=-1))
    page0, page3 = b.table[0, 1], b.table[3, 0]
    wc, ws = kv.append(b.codes[1], b.scales[1], v[:3].astype(np.float64), b.cu[:2], b.lens[:1], b.table[:1], 16)
    wc, ws = kv.append(wc, ws, v[11:].astype(np.float64), np.array([0, 1]), np.array([1]), b.table[3:], 16)
    assert np.array_equal(cache.v.cpu().numpy(), wc) and np.array_equal(cache.v_scale.cpu().numpy(), ws)
    changed = np.argwhere((wc != b.codes[1]).any((1, 2, 3)))[:, 0]
    assert set(changed) <= {page0, page3}
