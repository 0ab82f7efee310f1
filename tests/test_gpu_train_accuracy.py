"""The float32 results of the norm and the activation are no further from float64 (root mean square of the relative errors)
than those of elementary float32 operations, each rounded by itself: the same number of roundings of a value or fewer, and
of a row's mean and root fewer.  The activation's gradient in up has one rounding fewer on float32 rows; on bf16 rows the
elementary dy * gate is exact, so that it has one more, and that of gate has as many as elementary operations at its size."""
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


def _act(dtype, spread):
    g = torch.Generator(device="cuda").manual_seed(5)
    return [(spread * torch.randn(4096, 2048, device="cuda", generator=g)).to(dtype).float() for _ in range(3)]


@pytest.mark.parametrize("spread", [1.0, 4.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_activation(dtype, spread):
    banner(f"accuracy of the activation, {dtype} values of {spread}")
    gate, up, _ = _act(dtype, spread)
    want = gate.double() * torch.sigmoid(gate.double()) * up.double()
    plain = gate / (1 + torch.exp(-gate)) * up
    assert _rms(fb.fp8_swiglu_quant(gate, up, quantize=False, with_y=True)[2], want) <= _rms(plain, want)


@pytest.mark.parametrize("spread", [1.0, 4.0])
def test_activation_gradient(spread):
    """Of gate against the size of its terms: near the slope's zero they cancel."""
    banner(f"accuracy of the activation's gradient, values of {spread}")
    gate, up, dy = _act(torch.float32, spread)
    d = fb.fp8_swiglu_backward(dy, gate, up, quantize=False, with_d=True)[2]
    g, u, e = gate.double(), up.double(), dy.double()
    s, plain = torch.sigmoid(g), 1 / (1 + torch.exp(-gate))
    assert _rms(d[:, 2048:], e * g * s) <= _rms(dy * gate * plain, e * g * s)
    size, want = e * u * s * (1 + g.abs() * (1 - s)), e * u * s * (1 + g * (1 - s))
    assert _rms(size + (d[:, :2048].double() - want), size) <= _rms(size + ((dy * up * plain * (1 + gate * (1 - plain))).double() - want), size)
