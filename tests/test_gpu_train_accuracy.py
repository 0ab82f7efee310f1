"""The float32 results of the norm and the activation are no further from float64 (root mean square of the relative errors)
than those of elementary float32 operations, each rounded by itself: the same number of roundings of a value or fewer, and
of a row's mean and root fewer."""
import pytest

from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _rms(got, want):
    real = want != 0
    return float(((got.double() - want)[real] / want[real]).square().mean().sqrt()) * 2 ** 24


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("rows,cols", [(2048, 7168), (2048, 2048), (512, 16384), (8192, 128), (4096, 1408)])
def test_norm(rows, cols, weighted):
    banner(f"accuracy of the norm, {rows}x{cols}")
    g = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, device="cuda", generator=g) * torch.exp2(4 * torch.rand(rows, 1, device="cuda", generator=g))
    w = torch.randn(cols, device="cuda", generator=g) if weighted else None
    want = x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    plain = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    if weighted:
        want, plain = want * w.double(), plain * w
    got = fb.fp8_rmsnorm_quant(x, w, quantize=False, with_y=True)[2]
    assert _rms(got, want) <= _rms(plain, want)
