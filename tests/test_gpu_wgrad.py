"""The experts' weight gradients against float64.

Tolerance: every product of two widened codes is exact in float32's 24 bits, and each of an expert's `depth` products joins
a sum by at most one rounding: depth * 2^-24 of the products' magnitudes; a result in bf16 adds half a step, 2^-8, an
accumulated one a rounding of the sum.  Small integers with scales of one size are exact."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import e4m3_encode, train
from train_util import BF16, F32, HALF, dev, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _operand(rng, rows, columns, spread=8):
    codes = rng.integers(0, 256, (rows, columns)).astype(np.uint8)
    codes = np.where(codes & 0x7f == 0x7f, 0x30, codes).astype(np.uint8)      # no NaN
    return codes, (2.0 ** rng.integers(-spread, spread + 1, (rows, columns // 128))).astype(np.float32)


def _wide(t, pad):
    """The same matrix with a larger pitch, NaN codes between its rows."""
    w = torch.full((t.shape[0], t.shape[1] + pad), 0x7f, dtype=torch.uint8, device="cuda")
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def _check(n, k, padded, columns, dtype=F32, was=None, pad=0, seed=0):
    rng = np.random.default_rng(seed + n + k)
    a, sa = _operand(rng, n, columns)
    b, sb = _operand(rng, k, columns)
    da, db = dev(a), dev(b)
    if pad:
        da, db = _wide(da, pad), _wide(db, 2 * pad)
    y = None if was is None else dev(was).to(dtype)
    got = fb.fp8_blockscaled_grouped_wgrad(dev(np.asarray(padded, np.int32)), da, dev(sa), db, dev(sb), out_dtype=dtype, y=y,
                                           accumulate=was is not None)
    want, size, depth = train.wgrad(padded, train.values(a, sa), train.values(b, sb))
    slack = np.array(depth)[:, None, None] * 2.0 ** -24 * size
    if was is not None:
        assert got is y
        want = want + was
        slack = slack + 2.0 ** -24 * (np.abs(want) + slack)
    off = np.abs(f64(got) - want)
    most = slack * (1 + 2 * HALF[dtype]) + HALF[dtype] * np.abs(want)
    assert (off <= most).all(), (np.argwhere(off > most)[:3].tolist(), off.max())


SIZES = [(16, 16), (48, 80), (128, 128), (144, 112), (256, 400), (512, 272), (400, 656)]
TABLES = [([0, 128], 128), ([0, 384], 384), ([0, 256, 256, 640, 768], 896), ([0, 0, 0], 128), ([0, 128, 256, 384, 512, 640], 640),
          ([128, 640, 1152], 1280), ([0, 1664], 1664)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,k", SIZES)
def test_weight_gradient(n, k, dtype):
    for i, (padded, columns) in enumerate(TABLES):
        banner(f"weight gradient {n}x{k} {dtype} experts {padded}")
        _check(n, k, padded, columns, dtype, pad=16 * (i % 3))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_accumulates(dtype):
    rng = np.random.default_rng(1)
    for n, k, padded in ((48, 80, [0, 256, 256, 384]), (272, 144, [0, 128, 512, 512])):
        banner(f"accumulated weight gradient {n}x{k} {dtype}")
        was = (1000 * rng.standard_normal((3, n, k))).astype(np.float32)
        was = dev(was).to(dtype).float().cpu().numpy()
        _check(n, k, padded, padded[-1], dtype, was=was)


def test_large_tiles():
    """Enough tiles for the larger kernel: ragged edges, an expert without rows, one of a single block."""
    for dtype in (F32, BF16):
        banner(f"weight gradient in large tiles {dtype}")
        padded = [0, 384, 384, 512, 1152, 1280, 1280, 2048, 2176]
        _check(1808, 2064, padded, 2304, dtype, seed=3)
    was = np.random.default_rng(4).standard_normal((8, 1808, 2064)).astype(np.float32) * 1000
    _check(1808, 2064, padded, 2304, F32, was=was, seed=5)


@pytest.mark.parametrize("n,k,experts", [(1808, 2032, 8), (1808, 2048, 8), (784, 1040, 60)])
def test_largest_tiles(n, k, experts):
    """512 tiles of 256, with rows of y that are whole lines or not, and 1200: both ways to the largest kernel."""
    rng = np.random.default_rng(9)
    for dtype in (F32, BF16):
        banner(f"weight gradient {n}x{k} of {experts} experts {dtype}")
        padded = np.concatenate([[0], np.cumsum(128 * rng.integers(0, 5, experts))])
        columns = max(int(padded[-1]), 128 * experts) + 128
        _check(n, k, padded, columns, dtype, seed=7)
    _check(n, k, padded, columns, F32, was=np.random.default_rng(8).standard_normal((experts, n, k)).astype(np.float32) * 100, seed=8)


def test_shallow_experts():
    """About a block an expert and 1890 tiles of 128: their kernel for experts like these."""
    rng = np.random.default_rng(10)
    padded = np.concatenate([[0], np.cumsum(128 * rng.integers(0, 3, 30))])
    for dtype in (F32, BF16):
        banner(f"weight gradient of 30 shallow experts {dtype}")
        _check(784, 1040, padded, int(padded[-1]) + 128, dtype, seed=11)
    banner("the same, in whole lines")
    _check(784, 1024, padded, int(padded[-1]) + 128, F32, seed=12)


def test_middle_tiles():
    """504 tiles of 128 over deep experts, in whole lines or not."""
    for k in (1040, 1152):
        for dtype in (F32, BF16):
            banner(f"weight gradient 784x{k} of 8 experts {dtype}")
            _check(784, k, [0, 384, 384, 512, 1152, 1280, 1280, 2048, 2432], 2560, dtype, seed=13)
    banner("added to")
    _check(784, 1040, [0, 384, 384, 512, 1152, 1280, 1280, 2048, 2432], 2560, F32,
           was=np.random.default_rng(14).standard_normal((8, 784, 1040)).astype(np.float32) * 100, seed=15)


def test_many_experts():
    rng = np.random.default_rng(2)
    padded = np.concatenate([[0], np.cumsum(128 * rng.integers(0, 3, 300))])
    banner("weight gradient of 300 experts")
    _check(32, 48, padded, int(padded[-1]) + 128)
    banner("weight gradient of 1024 experts")
    _check(16, 16, np.arange(1025) // 2 * 128, 128 * 512)


def test_integers_are_exact():
    rng = np.random.default_rng(3)
    a, b = rng.integers(-8, 9, (96, 1280)), rng.integers(-8, 9, (160, 1280))
    ones = [np.ones((len(m), 10), np.float32) for m in (a, b)]
    y = fb.fp8_blockscaled_grouped_wgrad(dev(np.array([0, 512, 1280], np.int32)), dev(e4m3_encode(a.astype(np.float32))), dev(ones[0]),
                                         dev(e4m3_encode(b.astype(np.float32))), dev(ones[1] * 2))
    assert np.array_equal(y.cpu().numpy(), np.stack([2 * a[:, :512] @ b[:, :512].T, 2 * a[:, 512:] @ b[:, 512:].T]))


def test_crooked_tables_stay_inside():
    """Falling, negative and far offsets, and ones that are no multiples of 128."""
    for padded in ([0, 200, 300], [-500, 130, 2 ** 31 - 1], [2 ** 31 - 1, -2 ** 31, 0], [384, 128, 512, 0, 640], [0, 127, 128]):
        banner(f"weight gradient, crooked table {padded}")
        _check(48, 32, padded, 640)


def test_scales_at_their_limits():
    a, b = np.full((32, 256), 0x38, np.uint8), np.full((16, 256), 0x40, np.uint8)       # 1 and 2
    for x, z in ((2.0 ** -100, 2.0 ** 100), (2.0 ** 100, 1.0), (2.0 ** -60, 2.0 ** -60), (2.0 ** 120, 2.0 ** -50), (1.0, 2.0 ** 115)):
        y = fb.fp8_blockscaled_grouped_wgrad(dev(np.array([0, 256], np.int32)), dev(a), dev(np.full((32, 2), x, np.float32)), dev(b),
                                             dev(np.full((16, 2), z, np.float32)))
        assert (y.cpu().numpy() == np.float32(512 * x * z)).all()


@pytest.mark.parametrize("bad", [3.0, 0.1, 0.0, -1.0, float("nan"), float("inf"), 2.0 ** -101, 2.0 ** 121])
def test_a_scale_that_is_no_power_of_two_gives_nan(bad):
    """At its own row or column, for either operand; experts whose blocks it is not in are untouched."""
    rng = np.random.default_rng(6)
    padded = dev(np.array([0, 256, 640], np.int32))
    a, sa = _operand(rng, 144, 640)
    b, sb = _operand(rng, 160, 640)
    fine = fb.fp8_blockscaled_grouped_wgrad(padded, dev(a), dev(sa), dev(b), dev(sb))
    for which, row, block in (("a", 140, 3), ("b", 7, 4), ("a", 0, 2)):
        s = [sa.copy(), sb.copy()]
        s["ab".index(which)][row, block] = bad
        y = fb.fp8_blockscaled_grouped_wgrad(padded, dev(a), dev(s[0]), dev(b), dev(s[1]))
        assert torch.equal(y[0], fine[0])
        line = y[1, row] if which == "a" else y[1, :, row]
        assert line.isnan().all()
        assert (y[1].isnan() | (y[1] == fine[1])).all()


def test_nan_codes_stay_in_their_row():
    rng = np.random.default_rng(7)
    a, sa = _operand(rng, 64, 256)
    b, sb = _operand(rng, 48, 256)
    args = [dev(np.array([0, 256], np.int32)), dev(a), dev(sa), dev(b), dev(sb)]
    fine = fb.fp8_blockscaled_grouped_wgrad(*args)
    args[1][5, 200] = 0x7f
    y = fb.fp8_blockscaled_grouped_wgrad(*args)
    assert y[0, 5].isnan().all()
    rest = torch.arange(64, device="cuda") != 5
    assert torch.equal(y[0, rest], fine[0, rest])


def test_nothing_to_do():
    z = dev(np.array([0, 0, 0], np.int32))
    u8, f32 = dict(dtype=torch.uint8, device="cuda"), dict(device="cuda")
    y = fb.fp8_blockscaled_grouped_wgrad(z, torch.zeros(32, 0, **u8), torch.zeros(32, 0, **f32), torch.zeros(16, 0, **u8), torch.zeros(16, 0, **f32),
                                         y=torch.full((2, 32, 16), 5.0, **f32))
    assert (y == 0).all()
    y = fb.fp8_blockscaled_grouped_wgrad(z, torch.zeros(32, 0, **u8), torch.zeros(32, 0, **f32), torch.zeros(16, 0, **u8), torch.zeros(16, 0, **f32),
                                         y=torch.full((2, 32, 16), 5.0, **f32), accumulate=True)
    assert (y == 5).all()
    assert fb.fp8_blockscaled_grouped_wgrad(z, torch.zeros(0, 128, **u8), torch.zeros(0, 1, **f32), torch.zeros(16, 128, **u8),
                                            torch.zeros(16, 1, **f32)).shape == (2, 0, 16)


def test_from_rows_to_gradients():
    """Quantizer and GEMM together against the float64 product of the rows: each operand is off by at most 2^-4 of its value
    and 2^-10 of its tile's scale."""
    banner("weight gradients from rows")
    rng = np.random.default_rng(8)
    counts = [130, 0, 7, 260]
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    x, dy = rng.standard_normal((397, 160)).astype(np.float32), (1e-3 * rng.standard_normal((397, 96))).astype(np.float32)
    a, sa, padded = fb.fp8_quant_grouped_t(dev(dy), dev(off))
    b, sb, again = fb.fp8_quant_grouped_t(dev(x), dev(off))
    assert torch.equal(padded, again)
    y = f64(fb.fp8_blockscaled_grouped_wgrad(padded, a, sa, b, sb))
    for e in range(4):
        rows = slice(off[e], off[e + 1])
        want = dy[rows].astype(np.float64).T @ x[rows]
        noise = (np.abs(dy[rows]).T + 2.0 ** -6 * 1e-3) @ (np.abs(x[rows]) + 2.0 ** -6)
        assert (np.abs(y[e] - want) <= (2.0 ** -3 + 2.0 ** -8) * noise).all()
        if counts[e]:
            assert np.linalg.norm(y[e] - want) <= 0.06 * np.linalg.norm(want)


def test_the_same_bits_every_time():
    rng = np.random.default_rng(9)
    a, sa = _operand(rng, 512, 1024)
    b, sb = _operand(rng, 512, 1024)
    args = dev(np.array([0, 384, 1024], np.int32)), dev(a), dev(sa), dev(b), dev(sb)
    first = fb.fp8_blockscaled_grouped_wgrad(*args)
    assert all(torch.equal(first, fb.fp8_blockscaled_grouped_wgrad(*args)) for _ in range(5))
