"""The norm and its gradient up to the sizes that the header states, at every way to share a row out, and beyond them.
Tolerances as in test_gpu_rmsnorm.py: nothing on the way leaves float32's normal range."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import train
from train_util import BF16, F32, check_near, check_quantized, dev, f64, on_gpu, rounded, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

Y, DX = 2.0 ** -18, 2.0 ** -17
COLS = [128, 512, 640, 1408, 2048, 2176, 7168, 8192, 16384, 32768]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", COLS)
def test_largest_values(cols, dtype):
    """All values of a row at 2^60, some smaller, one alone; the weight's gradient of the same."""
    banner(f"norm of values of 2^60, {cols} columns, {dtype}")
    rng = np.random.default_rng(cols)
    h = 2.0 ** 60 * rng.choice([-1.0, 1.0], (4, cols))
    h[1] *= rng.random(cols)
    h[2] = 0
    h[2, cols // 2] = 2.0 ** 60
    h[3] = rng.standard_normal(cols)
    h, dy = rounded(h, dtype), rounded(2.0 ** 60 * rng.uniform(-1, 1, (4, cols)), dtype)
    w = rng.uniform(0.1, 1.0, cols).astype(np.float32)
    q, scale, y, _ = fb.fp8_rmsnorm_quant(on_gpu(h, dtype), dev(w), with_y=True)
    want = train.rmsnorm(h, w, float(np.float32(1e-6)))
    check_near(y, want, Y * np.abs(want), dtype)
    check_quantized(q, scale, want, Y * np.abs(want))
    dx, dw = fb.fp8_rmsnorm_backward(on_gpu(dy, dtype), on_gpu(h, dtype), dev(w))
    want, want_w, size, size_w = train.rmsnorm_grad(dy, h, w, float(np.float32(1e-6)))
    check_near(dx, want, DX * size, dtype)
    assert (np.abs(f64(dw) - want_w) <= (Y + 68 * 2.0 ** -24) * size_w).all()


@pytest.mark.parametrize("cols", COLS)
def test_beyond_them(cols):
    """A row of 2^64 is not passed off as zeros, and its neighbours do not see it."""
    banner(f"norm of values of 2^64, {cols} columns")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x, dy, w = (torch.randn(n, cols, device="cuda", generator=g) for n in (6, 6, 1))
    fine = fb.fp8_rmsnorm_quant(x, w[0], with_y=True) + fb.fp8_rmsnorm_backward(dy, x, w[0])
    x[2] = 2.0 ** 64
    got = fb.fp8_rmsnorm_quant(x, w[0], with_y=True) + fb.fp8_rmsnorm_backward(dy, x, w[0])
    rest = [0, 1, 3, 4, 5]
    for i in (0, 1, 2, 4):
        assert same_bits(got[i][rest], fine[i][rest])
    assert got[2][2].isnan().all() and got[4][2].isnan().all() and got[5].isnan().all()
    assert (got[0][2] & 0x7f == 0x7f).all()
