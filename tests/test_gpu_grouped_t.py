"""Transposed tiles of experts' rows: codes, scales and padded offsets are bit-exact, and nothing else is written."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import train
from train_util import BF16, F32, dev, on_gpu, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

I32 = torch.int32
COUNTS = [[1], [128], [129, 0, 1], [0, 0, 5], [127, 128, 1, 0, 300], [0], [0, 0], [3] * 70, [0] * 64 + [1, 0, 129], [40, 0] * 130]


def _values(rng, rows, cols, dtype):
    """Rows whose columns have sizes of their own, with zeros, and maxima on either side of 448 times a power of two."""
    x = rng.standard_normal((rows, cols)) * 2.0 ** rng.integers(-110, 60, cols)
    x[:, ::7] = 0
    if cols > 20 and rows:
        x[0, 1], x[0, 2], x[0, 3], x[0, 4] = 448 * 2.0 ** -3, 450 * 2.0 ** -3, 447 * 2.0 ** -3, 2.0 ** -100
        x[1:, 1:5] = 0
        x[-1, 5] = -0.0
    return rounded(x, dtype)


def _buffers(cols, columns):
    return torch.full((cols, columns), 0x55, dtype=torch.uint8, device="cuda"), torch.full((cols, columns // 128), 7.0, device="cuda")


def _check(x, off, order, top_k, dtype, extra=0, pad=0):
    places = len(x) if order is None else len(order)
    columns = fb.lib().fp8_quant_grouped_t_columns(places, len(off) - 1) + extra
    q, scale = _buffers(x.shape[1], columns)
    want = train.tiles(x, off, order, top_k, q.cpu().numpy(), scale.cpu().numpy())
    got = fb.fp8_quant_grouped_t(on_gpu(x, dtype, pad), dev(np.asarray(off, np.int32)), order=None if order is None else dev(order), top_k=top_k,
                                 q=q, scale=scale)
    for a, b, name in zip(got, want, ("codes", "scales", "padded")):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), np.ascontiguousarray(b).view(np.uint8)), name
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{sum(c)}")
def test_tiles(counts, dtype):
    rng = np.random.default_rng(len(counts))
    for cols in (16, 144) if sum(counts) > 400 else (16, 144, 400):
        banner(f"tiles {sum(counts)} rows of {len(counts)} experts, {cols} columns, {dtype}")
        x = _values(rng, sum(counts), cols, dtype)
        _check(x, np.concatenate([[0], np.cumsum(counts)]), None, 1, dtype, extra=128 * (cols == 144), pad=16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("top_k", [1, 2, 3, 8])
def test_gathered(top_k, dtype):
    rng = np.random.default_rng(top_k)
    banner(f"gathered tiles, top_k {top_k}, {dtype}")
    x = _values(rng, 60, 80, dtype)
    order = rng.permutation(60 * top_k).astype(np.int32)
    off = [0, 20, 20, 45, 50]
    _check(x, off, order, top_k, dtype)
    order[3:40:5] = [-1, 60 * top_k, 2 ** 31 - 1, -2 ** 31, 60 * top_k + 1, 0, 0, 59 * top_k]      # rows of zeros, and rows twice
    _check(x, off, order, top_k, dtype)
    _check(x, off, order[:48].copy(), top_k, dtype)


def test_places_behind_the_last_expert_and_crooked_offsets():
    rng = np.random.default_rng(5)
    x = _values(rng, 300, 48, F32)
    for off in ([0, 100], [7, 150, 299], [-5, 20, 4000], [10, 5, 200, 100, 300], [300, 0], [2 ** 31 - 1, -2 ** 31, 5], [0, 300, 0, 300]):
        banner(f"crooked offsets {off}")
        _check(x, off, None, 1, F32)


def test_no_places_and_no_columns():
    off = dev(np.array([0, 0, 0], np.int32))
    q, scale, padded = fb.fp8_quant_grouped_t(torch.zeros(0, 64, device="cuda"), off)
    assert q.shape == (64, 0) and scale.shape == (64, 0) and padded.tolist() == [0, 0, 0]
    q, scale, padded = fb.fp8_quant_grouped_t(torch.zeros(5, 0, device="cuda"), dev(np.array([0, 2, 5], np.int32)))
    assert q.shape == (0, 256) and padded.tolist() == [0, 128, 256]
    # places that all stand for zeros
    q, scale, padded = fb.fp8_quant_grouped_t(torch.zeros(0, 64, device="cuda"), dev(np.array([0, 3], np.int32)),
                                              order=dev(np.array([0, 1, -1], np.int32)), top_k=2)
    assert (q == 0).all() and (scale == 1).all() and padded.tolist() == [0, 128]


def test_wide_strips():
    """Many column blocks a workgroup, and one expert of many blocks; the GEMM's dequantizer reads the result."""
    banner("tiles in wide strips")
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(5000, 7168, device="cuda", generator=g).to(BF16)
    off = torch.tensor([0, 4200, 4200, 5000], dtype=I32, device="cuda")
    q, scale, padded = fb.fp8_quant_grouped_t(x, off)
    assert padded.tolist() == [0, 4224, 4224, 4224 + 896]
    back = fb.fp8_dequant(q, scale)
    for lo, hi, at in ((0, 4200, 0), (4200, 5000, 4224)):
        v = x[lo:hi].float().t()
        step = scale[:, at // 128:at // 128 + -(-(hi - lo) // 128)].repeat_interleave(128, 1)[:, :hi - lo]
        assert (back[:, at:at + hi - lo] - v).abs().le(2.0 ** -4 * v.abs() + 2.0 ** -10 * step).all()
        assert (back[:, at + hi - lo:at + -(-(hi - lo) // 128) * 128] == 0).all()
    s, m = scale[:, :padded[-1] // 128], torch.frexp(scale[:, :padded[-1] // 128])[0]
    assert (m == 0.5).all() and (s > 0).all()


def test_a_broken_value_stays_in_its_tile():
    x = np.random.default_rng(7).standard_normal((256, 32)).astype(np.float32)
    off = dev(np.array([0, 256], np.int32))
    a = fb.fp8_quant_grouped_t(dev(x), off)
    x[5, 3], x[200, 9] = np.nan, np.inf
    b = fb.fp8_quant_grouped_t(dev(x), off)
    keep = torch.ones(32, 2, dtype=torch.bool, device="cuda")
    keep[3, 0] = keep[9, 1] = False
    assert torch.equal(a[1][keep], b[1][keep])
    codes = keep.repeat_interleave(128, 1)
    assert torch.equal(a[0][codes], b[0][codes])
