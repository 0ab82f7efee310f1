"""The gated activation and its gradient against float64.

Tolerances in float32 roundings (2^-24): exp2 of the hardware 2, its corrected argument 2, 1 + e one, the reciprocal 2, the
products 4: under 16 = 2^-20, relative to y and, for the gradient, to the magnitudes of its terms (one addition more:
2^-19).  An exponential that leaves float32's normal range (|gate| above 87) may be 0: 2^-125 |up| (1 + |gate|)."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import quant_1x128, train
from train_util import BF16, F32, check_near, check_quantized, f64, on_gpu, rounded, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

Y, D = 2.0 ** -20, 2.0 ** -19
SIZES = [(1, 128), (1, 2048), (3, 384), (7, 640), (33, 1408), (130, 2048), (1, 18432)]


def _halves(rng, rows, cols, dtype):
    g, u = rng.standard_normal((2, rows, cols)) * 3
    g.flat[:12] = [0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 88.0, -88.0, 105.0, -105.0, 1e4, -1e4]
    return rounded(g, dtype), rounded(u, dtype)


def _tiny(g, *others):
    return 2.0 ** -125 * (1 + np.abs(g.astype(np.float64))) * np.prod([1 + np.abs(o.astype(np.float64)) for o in others], axis=0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_activation(rows, cols, dtype):
    banner(f"activation {rows}x{cols} {dtype}")
    g, u = _halves(np.random.default_rng(rows + cols), rows, cols, dtype)
    both = on_gpu(np.concatenate([g, u], 1), dtype)
    q, scale, y = fb.fp8_swiglu_quant(both[:, :cols], both[:, cols:], with_y=True)
    want = train.swiglu(g, u)
    slack = Y * np.abs(want) + _tiny(g, u)
    check_near(y, want, slack, dtype)
    check_quantized(q, scale, want, slack)
    if dtype is F32:
        for a, b in zip(quant_1x128(y.cpu().numpy()), (q, scale)):
            assert np.array_equal(a.view(np.uint8), b.cpu().numpy().view(np.uint8))
    else:
        wide = both.float()
        other = fb.fp8_swiglu_quant(wide[:, :cols], wide[:, cols:])
        assert same_bits(other[0], q) and same_bits(other[1], scale) and other[2] is None


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_activation_gradient(rows, cols, dtype):
    banner(f"activation gradient {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    g, u = _halves(rng, rows, cols, dtype)
    dy = rounded(rng.standard_normal((rows, cols)), dtype)
    both = on_gpu(np.concatenate([g, u], 1), dtype)
    q, scale, d = fb.fp8_swiglu_backward(on_gpu(dy, dtype, 8), both[:, :cols], both[:, cols:], with_d=True)
    want, size = train.swiglu_grad(dy, g, u)
    slack = D * size + np.tile(_tiny(g, u, dy), (1, 2))
    check_near(d, want, slack, dtype)
    check_quantized(q, scale, want, slack)
    if dtype is F32:
        for a, b in zip(quant_1x128(d.cpu().numpy()), (q, scale)):
            assert np.array_equal(a.view(np.uint8), b.cpu().numpy().view(np.uint8))
    # over the matrix that holds gate and up
    again = fb.fp8_swiglu_backward(on_gpu(dy, dtype), both[:, :cols], both[:, cols:], d=both)
    assert again[2] is both and same_bits(both, d) and same_bits(again[0], q) and same_bits(again[1], scale)


@pytest.mark.parametrize("rows", [1023, 16385, 40001])
def test_many_tiles(rows):
    """Waves of one and of two steps, tiles that do not fill the last workgroup: every row as if it stood alone."""
    banner(f"activation of {rows} rows")
    g = torch.Generator(device="cuda").manual_seed(rows)
    gate, up, dy = (torch.randn(rows, 384, device="cuda", generator=g).to(BF16) for _ in range(3))
    got = fb.fp8_swiglu_quant(gate, up, with_y=True) + fb.fp8_swiglu_backward(dy, gate, up, with_d=True)
    x, u, d = gate.double(), up.double(), dy.double()
    s = torch.sigmoid(x)
    for y, want, size in ((got[2], x * s * u, (x * s * u).abs()),
                          (got[5], torch.cat([d * u * s * (1 + x * (1 - s)), d * x * s], 1),
                           torch.cat([(d * u).abs() * s * (1 + x.abs() * (1 - s)), (d * x).abs() * s], 1))):
        assert (y.double() - want).abs().le((2.0 ** -8 + 2.0 ** -15) * want.abs() + 2.0 ** -18 * size).all()
    for r in (0, 517, rows - 1):
        one = slice(r, r + 1)
        alone = fb.fp8_swiglu_quant(gate[one], up[one], with_y=True) + fb.fp8_swiglu_backward(dy[one], gate[one], up[one], with_d=True)
        assert all(same_bits(a, b[one].contiguous()) for a, b in zip(alone, got))


def test_outputs_asked_for_one_by_one():
    g = torch.Generator(device="cuda").manual_seed(0)
    gate, up, dy = (torch.randn(9, 256, device="cuda", generator=g) for _ in range(3))
    full, back = fb.fp8_swiglu_quant(gate, up, with_y=True), fb.fp8_swiglu_backward(dy, gate, up, with_d=True)
    y = fb.fp8_swiglu_quant(gate, up, with_y=True, quantize=False)
    d = fb.fp8_swiglu_backward(dy, gate, up, with_d=True, quantize=False)
    assert y[:2] == (None, None) and d[:2] == (None, None) and same_bits(y[2], full[2]) and same_bits(d[2], back[2])
    q = torch.full((9, 640), 9, dtype=torch.uint8, device="cuda")
    out = fb.fp8_swiglu_backward(dy, gate, up, q=q[:, 64:576])
    assert out[2] is None and same_bits(out[0].contiguous(), back[0]) and (q[:, :64] == 9).all() and (q[:, 576:] == 9).all()


def test_no_rows_and_bad_tiles():
    z = torch.zeros(0, 256, device="cuda")
    assert fb.fp8_swiglu_quant(z, z)[0].shape == (0, 256) and fb.fp8_swiglu_backward(z, z, z, with_d=True)[2].shape == (0, 512)
    g = torch.Generator(device="cuda").manual_seed(1)
    gate, up = (torch.randn(4, 384, device="cuda", generator=g) for _ in range(2))
    want = fb.fp8_swiglu_quant(gate, up)
    gate[1, 130], gate[2, 5], up[3, 383] = float("nan"), float("-inf"), float("inf")
    got = fb.fp8_swiglu_quant(gate, up)
    keep = np.ones((4, 3), bool)
    keep[1, 1] = keep[2, 0] = keep[3, 2] = False
    for r, t in np.argwhere(keep):
        assert same_bits(got[0][r, 128 * t:128 * t + 128].contiguous(), want[0][r, 128 * t:128 * t + 128].contiguous())
        assert float(got[1][r, t]) == float(want[1][r, t])


def test_gradient_against_differences():
    """Central differences of the call's own float32 outputs, whose rounding is 2^-20 of them over the step."""
    g = torch.Generator(device="cuda").manual_seed(2)
    gate, up, dy, wg, wu = (torch.randn(4, 128, device="cuda", generator=g) for _ in range(5))
    d = fb.fp8_swiglu_backward(dy, gate, up, quantize=False, with_d=True)[2].double()

    def value(step):
        return float((fb.fp8_swiglu_quant(gate + step * wg, up + step * wu, quantize=False, with_y=True)[2].double() * dy.double()).sum())

    step = 2.0 ** -6
    way = torch.cat([wg, wu], 1).double()
    size = float((d * way).abs().sum())
    assert abs(float((d * way).sum()) - (value(step) - value(-step)) / (2 * step)) <= size * (16 * step ** 2 + 2.0 ** -18 / step)


def test_extreme_gates_match_float64():
    x = np.concatenate([np.linspace(-120, 120, 4000), np.linspace(-2, 2, 96)]).astype(np.float32).reshape(32, 128)
    ones = np.ones_like(x)
    y = fb.fp8_swiglu_quant(on_gpu(x, F32), on_gpu(ones, F32), quantize=False, with_y=True)[2]
    want = train.swiglu(x, ones)
    assert (np.abs(f64(y) - want) <= Y * np.abs(want) + _tiny(x)).all()
