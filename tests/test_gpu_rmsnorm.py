"""The norm and its gradient against float64.

Tolerances, counted in roundings of float32 (2^-24 each).  A row's sum of squares: at most 32 additions in a thread, 6 of
the wave, 16 of the waves, one multiplication each before; its relative error enters 1/root by half: 28.  The mean, the
root and the two products: 8 with the root's own two steps.  Together under 64 = 2^-18.  dx: the same for both of its
terms and the mean of g h, measured against their magnitudes: 2^-17.  dweight: a sum over the rows, one rounding a row and
one a worker, its terms as above."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import quant_1x128, train
from train_util import BF16, F32, check_near, check_quantized, dev, f64, on_gpu, rounded, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

Y, DX = 2.0 ** -18, 2.0 ** -17
COLS = [128, 384, 512, 640, 1024, 1152, 2048, 2176, 4096, 7168, 8192, 8320, 16384, 16512, 32768]


def _rows(rng, rows, cols, dtype):
    x = rng.standard_normal((rows, cols)) * np.where(rng.random((rows, cols)) < 0.01, 20.0, 1.0)
    return rounded(x, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_norm(cols, dtype):
    rows = 5 if cols < 8192 else 3
    rng = np.random.default_rng(cols)
    x, res = _rows(rng, rows, cols, dtype), _rows(rng, rows, cols, dtype)
    for wtype, with_res in ((None, True), (BF16, False), (F32, True)):
        banner(f"norm {rows}x{cols} {dtype} weight {wtype} residual {with_res}")
        w = rounded(1 + 0.3 * rng.standard_normal(cols), wtype) if wtype else None
        q, scale, y, out = fb.fp8_rmsnorm_quant(on_gpu(x, dtype, 8), dev(w).to(wtype) if wtype else None,
                                                residual=on_gpu(res, dtype, 16) if with_res else None, eps=1e-5, with_y=True)
        h = rounded(x + res, dtype) if with_res else x
        assert (out is None) == (not with_res)
        if with_res:
            assert np.array_equal(f64(out), h)
        want = train.rmsnorm(h, w, np.float32(1e-5))
        check_near(y, want, Y * np.abs(want), dtype, "y")
        check_quantized(q, scale, want, Y * np.abs(want), "q")
        if dtype is F32:                       # the codes are exactly those of the float32 y
            for a, b in zip(quant_1x128(y.cpu().numpy()), (q, scale)):
                assert np.array_equal(a.view(np.uint8), b.cpu().numpy().view(np.uint8))


@pytest.mark.parametrize("cols", [128, 2048, 7168])
def test_norm_of_bf16_is_that_of_the_same_float32(cols):
    """Codes come from the float32 y, whatever the rows' type."""
    rng = np.random.default_rng(1)
    x = _rows(rng, 40, cols, BF16)
    w = dev(rounded(1 + 0.3 * rng.standard_normal(cols), BF16)).to(BF16)
    a = fb.fp8_rmsnorm_quant(on_gpu(x, BF16), w)
    b = fb.fp8_rmsnorm_quant(on_gpu(x, F32), w, with_y=True)
    assert same_bits(a[0], b[0]) and same_bits(a[1], b[1]) and a[2] is None and a[3] is None
    c = fb.fp8_quant_act_1x128(b[2])
    assert same_bits(c[0], b[0]) and same_bits(c[1], b[1])


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 63, 1000, 5001, 12289])
def test_norm_many_rows(rows):
    """Workers with several rows: every row as if it stood alone."""
    banner(f"norm of {rows} rows")
    for cols, dtype in ((256, F32), (2560, BF16)):
        g = torch.Generator(device="cuda").manual_seed(rows)
        x = torch.randn(rows, cols, device="cuda", generator=g).to(dtype)
        w = torch.randn(cols, device="cuda", generator=g)
        q, scale, y, _ = fb.fp8_rmsnorm_quant(x, w, with_y=True)
        z = x.double() * torch.rsqrt(x.double().square().mean(1, keepdim=True) + 1e-6) * w.double()
        assert (y.double() - z).abs().le(Y * 1.01 * z.abs() + (2.0 ** -8 if dtype is BF16 else 2.0 ** -23) * z.abs()).all()
        for r in {0, rows // 2, rows - 1}:
            one = fb.fp8_rmsnorm_quant(x[r:r + 1], w, with_y=True)
            assert same_bits(one[0], q[r:r + 1]) and same_bits(one[1], scale[r:r + 1]) and same_bits(one[2], y[r:r + 1])


def test_norm_outputs_asked_for_one_by_one():
    rng = np.random.default_rng(2)
    x, res = on_gpu(_rows(rng, 7, 384, BF16), BF16), on_gpu(_rows(rng, 7, 384, BF16), BF16)
    full = fb.fp8_rmsnorm_quant(x, residual=res, with_y=True)
    only_y = fb.fp8_rmsnorm_quant(x, residual=res, with_y=True, quantize=False)
    only_q = fb.fp8_rmsnorm_quant(x, residual=res)
    assert only_y[0] is None and only_y[1] is None and only_q[2] is None
    assert same_bits(only_y[2], full[2]) and same_bits(only_q[0], full[0]) and same_bits(only_q[1], full[1])
    # in place of the residual, and of x
    for target in ("residual", "x"):
        a, b = x.clone(), res.clone()
        out = fb.fp8_rmsnorm_quant(a, residual=b, residual_out=b if target == "residual" else a)
        assert out[3] is (b if target == "residual" else a) and same_bits(out[3], full[3]) and same_bits(out[0], full[0])
    # into slices of wider buffers, whose other columns stay
    wide_q, wide_y = torch.full((7, 512), 9, dtype=torch.uint8, device="cuda"), torch.full((7, 512), 3.0, dtype=BF16, device="cuda")
    scale = torch.empty(7, 3, device="cuda")
    out = fb.fp8_rmsnorm_quant(x, residual=res, q=wide_q[:, 64:448], y=wide_y[:, 64:448], scale=scale)
    assert same_bits(out[0].contiguous(), full[0]) and same_bits(out[2].contiguous(), full[2]) and same_bits(scale, full[1])
    assert (wide_q[:, :64] == 9).all() and (wide_q[:, 448:] == 9).all() and (wide_y[:, :64] == 3).all() and (wide_y[:, 448:] == 3).all()


def test_norm_values_at_the_edges():
    """Rows of zeros, tiles of zeros, tiny and huge values, a single large value; non-finite values stay in their row."""
    x = np.zeros((8, 512), np.float32)
    x[1, :128] = 1e-30
    x[2] = 2.0 ** 59
    x[3, 300] = 1.0
    x[4] = np.linspace(-1e-6, 1e-6, 512)
    x[5, 7], x[5, 9] = np.nan, 1.0
    x[6, 200] = np.inf
    x[7] = np.tile([1.0, -0.0], 256)
    q, scale, y, _ = fb.fp8_rmsnorm_quant(on_gpu(x, F32), eps=1e-12, with_y=True)
    fine = [0, 1, 2, 3, 4, 7]
    want = train.rmsnorm(x[fine], None, float(np.float32(1e-12)))
    check_near(y[fine], want, Y * np.abs(want), F32)
    codes, scales = quant_1x128(y[fine].cpu().numpy())
    assert np.array_equal(q[fine].cpu().numpy(), codes) and np.array_equal(scale[fine].cpu().numpy(), scales)
    assert (q[7].cpu().numpy()[1::2] == 0x80).all()


def test_norm_no_rows():
    q, scale, y, out = fb.fp8_rmsnorm_quant(torch.zeros(0, 256, device="cuda"), residual=torch.zeros(0, 256, device="cuda"), with_y=True)
    assert q.shape == (0, 256) and scale.shape == (0, 2) and y.shape == (0, 256) and out.shape == (0, 256)
    dx, dw = fb.fp8_rmsnorm_backward(torch.zeros(0, 256, device="cuda"), torch.zeros(0, 256, device="cuda"), torch.ones(256, device="cuda"),
                                     dweight=torch.full((256,), 5.0, device="cuda"))
    assert dx.shape == (0, 256) and (dw == 0).all()


def _check_backward(rows, cols, dtype, wtype, with_res, pad=0):
    banner(f"norm gradient {rows}x{cols} {dtype} weight {wtype} residual {with_res}")
    rng = np.random.default_rng(rows * 131 + cols)
    h, dy = _rows(rng, rows, cols, dtype), rounded(1e-3 * rng.standard_normal((rows, cols)), dtype)
    res = rounded(1e-3 * rng.standard_normal((rows, cols)), dtype) if with_res else None
    w = rounded(1 + 0.3 * rng.standard_normal(cols), wtype) if wtype else None
    dx, dw = fb.fp8_rmsnorm_backward(on_gpu(dy, dtype, pad), on_gpu(h, dtype, pad), dev(w).to(wtype) if wtype else None,
                                     dresidual=on_gpu(res, dtype, pad) if with_res else None, eps=1e-5)
    want, want_w, size, size_w = train.rmsnorm_grad(dy, h, w, np.float32(1e-5), res)
    check_near(dx, want, DX * size, dtype, "dx")
    assert (dw is None) == (w is None)
    if w is not None:
        assert (np.abs(f64(dw) - want_w) <= (Y + (rows + 64) * 2.0 ** -24) * size_w).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_norm_gradient(cols, dtype):
    for wtype, with_res in ((None, True), (BF16, False), (F32, True)):
        _check_backward(5 if cols < 8192 else 3, cols, dtype, wtype, with_res, pad=8)


@pytest.mark.parametrize("rows", [1, 2, 64, 769, 1537, 4099])
def test_norm_gradient_many_rows(rows):
    _check_backward(rows, 256, BF16, F32, True)
    if rows <= 1537:
        _check_backward(rows, 2304, F32, BF16, True)


def test_norm_gradient_in_place_and_again():
    """dx over each of its inputs, and the same bits at every call."""
    g = torch.Generator(device="cuda").manual_seed(0)
    dy, h, res = (torch.randn(1500, 1024, device="cuda", generator=g).to(BF16) for _ in range(3))
    w = torch.randn(1024, device="cuda", generator=g)
    dx, dw = fb.fp8_rmsnorm_backward(dy, h, w, dresidual=res)
    for i in range(3):
        args = [dy.clone(), h.clone(), res.clone()]
        a, b = fb.fp8_rmsnorm_backward(args[0], args[1], w, dresidual=args[2], dx=args[i])
        assert a is args[i] and same_bits(a, dx) and same_bits(b, dw)


def test_norm_gradient_against_differences():
    """The calls themselves: a step of h and of the weight along their gradients changes <y, dy> as they say.  Differences
    of float32 outputs of size 1: 2^-18 each over a step of 2^-6 of 512 terms."""
    g = torch.Generator(device="cuda").manual_seed(3)
    h, dy, way = (torch.randn(4, 128, device="cuda", generator=g) for _ in range(3))
    w, wway = (torch.randn(128, device="cuda", generator=g) for _ in range(2))
    dx, dw = fb.fp8_rmsnorm_backward(dy, h, w)

    def value(step):
        y = fb.fp8_rmsnorm_quant(h + step * way, w + step * wway, quantize=False, with_y=True)[2]
        return float((y.double() * dy.double()).sum())

    step = 2.0 ** -6
    got, want = float((dx.double() * way.double()).sum() + (dw.double() * wway.double()).sum()), (value(step) - value(-step)) / (2 * step)
    size = float((dx * way).abs().sum() + (dw * wway).abs().sum())
    # the differences' third order: below 64 step^2 of the terms' size
    assert abs(got - want) <= size * (64 * step ** 2 + 2.0 ** -18 / step)
