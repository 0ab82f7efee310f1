"""The activation and its gradient for finite inputs of every size, against float64: what float64 says is within the type's
range is finite, and what is beyond it is infinite.

Tolerances: 2^-19 of a result's terms (the float32 roundings, under 32 of them).  Below gates of -87 an exponential may count
as 0: 88 * 2^-126 < 2^-119 of the other factors.  A product on the way that falls below float32's normal range is off by at
most 2^-149, times the factors that follow: |up| (|gate|'s own part is within 2^-149 |dy|)."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import train
from train_util import BF16, F32, HALF, f64, on_gpu, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

MOST = {F32: float(np.finfo(np.float32).max), BF16: float(torch.finfo(BF16).max)}
GATES = [1e30, 1e20, 1e10, 105.0, 100.0, 88.5, 87.5, 87.0, 86.5, 80.0, 30.0, 2.4, 1.278, 1e-20, 1e-38, 0.0]
UPS = [1e38, 1e30, 1e20, 1e10, 1.0, 1e-10, 1e-30, 1e-38]


def _grid(dtype):
    gates = np.array([s * v for v in [MOST[dtype], *GATES] for s in (1, -1)])
    ups = np.array([s * v for v in [MOST[dtype], *UPS] for s in (1, -1)])
    g, u = (x.ravel() for x in np.meshgrid(gates, ups))
    n = -(-g.size // 128) * 128
    return [rounded(np.resize(x, n).reshape(-1, 128), dtype) for x in (g, u)]


def _check(got, want, slack, dtype):
    got, most = f64(got), MOST[dtype]
    near = HALF[dtype] * np.abs(want) + slack
    inside, outside = np.abs(want) + near <= most, np.abs(want) - near >= most * (1 + 2 * HALF[dtype])
    bad = np.argwhere(inside & ~(np.abs(got - want) <= near * (1 + 2.0 ** -7)))
    assert bad.size == 0, [(tuple(i), got[tuple(i)], want[tuple(i)]) for i in bad[:4]]
    assert (got[outside] == np.sign(want[outside]) * np.inf).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_activation(dtype):
    banner(f"activation of values of all sizes, {dtype}")
    g, u = _grid(dtype)
    y = fb.fp8_swiglu_quant(on_gpu(g, dtype), on_gpu(u, dtype), quantize=False, with_y=True)[2]
    want = train.swiglu(g, u)
    _check(y, want, 2.0 ** -19 * np.abs(want) + 2.0 ** -119 * np.abs(u.astype(np.float64)) + 2.0 ** -133, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1.0, 2.0 ** 127, 1e30, 1e10, 0.01, 1e-10, 1e-30])
def test_gradient(size, dtype):
    banner(f"activation gradient of values of all sizes, dy of {size}, {dtype}")
    g, u = _grid(dtype)
    dy = rounded(np.where(np.arange(g.size).reshape(g.shape) % 2, size, -size), dtype)
    d = fb.fp8_swiglu_backward(on_gpu(dy, dtype), on_gpu(g, dtype), on_gpu(u, dtype), quantize=False, with_d=True)[2]
    want, terms = train.swiglu_grad(dy, g, u)
    a, b = np.abs(dy.astype(np.float64)), np.abs(u.astype(np.float64))
    slack = 2.0 ** -19 * terms + 2.0 ** -133 + np.concatenate([2.0 ** -119 * a * b + 2.0 ** -148 * b, 2.0 ** -119 * a], 1)
    _check(d, want, slack, dtype)


def test_a_masked_gate_leaves_its_tile():
    """Gates of the type's lowest value next to ordinary ones: zeros, and the tile's codes and scale as with gates of -200."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    for dtype in (F32, BF16):
        g, u, dy = (torch.randn(6, 256, device="cuda", generator=gen).to(dtype) for _ in range(3))
        u *= 100
        masked = torch.rand(6, 256, device="cuda", generator=gen) < 0.3
        low, plain = g.masked_fill(masked, torch.finfo(dtype).min), g.masked_fill(masked, -200.0)
        for call in (lambda x: fb.fp8_swiglu_quant(x, u, with_y=True), lambda x: fb.fp8_swiglu_backward(dy, x, u, with_d=True)):
            for a, b in zip(call(low), call(plain)):
                assert torch.equal(a, b)
        assert (fb.fp8_swiglu_quant(low, u, with_y=True)[2][masked] == 0).all()
