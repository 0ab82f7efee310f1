"""How far a NaN or an infinity reaches in the norm's gradient: in h, its row of dx and the weight's gradient as a whole (the
row's root is a factor of each of its parts); in dy, its row of dx and its column of the weight's gradient."""
import pytest

from gpu_util import banner
from train_util import BF16, F32, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [256, 2048, 7168, 16384, 32768])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_norm_gradient(bad, cols, dtype):
    banner(f"norm gradient with {bad}, {cols} columns, {dtype}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    h, dy, res = (torch.randn(37, cols, device="cuda", generator=g).to(dtype) for _ in range(3))
    w = torch.randn(cols, device="cuda", generator=g)
    dx, dw = fb.fp8_rmsnorm_backward(dy, h, w, dresidual=res)
    rows = torch.arange(37, device="cuda") != 20
    for at in (0, cols // 2 + 3, cols - 1):
        other = h.clone()
        other[20, at] = bad
        got = fb.fp8_rmsnorm_backward(dy, other, w, dresidual=res)
        assert same_bits(got[0][rows], dx[rows]) and not got[1].isfinite().all()
        other = dy.clone()
        other[20, at] = bad
        got = fb.fp8_rmsnorm_backward(other, h, w, dresidual=res)
        columns = torch.arange(cols, device="cuda") != at
        assert same_bits(got[0][rows], dx[rows]) and same_bits(got[1][columns], dw[columns]) and not got[1][at].isfinite()
        other = res.clone()
        other[20, at] = bad
        got = fb.fp8_rmsnorm_backward(dy, h, w, dresidual=other)
        columns[at] = False
        assert same_bits(got[0][rows], dx[rows]) and same_bits(got[0][20][columns], dx[20][columns]) and same_bits(got[1], dw)
