"""The example layer's gradients against float64 autograd of the same layer with its dequantized weights, the choice of
experts held.

Each gradient passes at most four E4M3 roundings on its way (the activations in front of the first product, the output's
gradient, the activation's, and the operands of its own product), each by at most 2^-4 of a value: 0.25 of the norm.  A wrong
row, expert, factor or transpose is off by the norm itself."""
import os
import sys

import pytest

from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def _plain(layer, x, router, up, down, norm, ids):
    """float64, on the CPU: the layer's output for a given choice of experts."""
    a = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6) * norm
    s = torch.sigmoid(a @ router.t()).gather(1, ids)
    w = s / (s.sum(1, keepdim=True) + 1e-20)
    out = x
    for j in range(ids.shape[1]):
        both = torch.einsum("th,tnh->tn", a, up[ids[:, j]])
        h = torch.nn.functional.silu(both[:, :layer.inner]) * both[:, layer.inner:]
        out = out + w[:, j:j + 1] * torch.einsum("tn,thn->th", h, down[ids[:, j]])
    return out


@pytest.mark.parametrize("tokens", [1, 40])
def test_gradients(tokens):
    import decoder_layer as ex
    import fp8_block_scaled_05_amd as fb
    banner(f"example layer's gradients, {tokens} tokens")
    layer = ex.Layer(hidden=256, experts=8, top_k=3, inner=128)
    g = torch.Generator(device="cuda").manual_seed(5)
    layer.norm = 1 + 0.2 * torch.randn(256, device="cuda", generator=g)
    x = torch.randn(tokens, 256, device="cuda", generator=g).bfloat16()
    grad = torch.randn(tokens, 256, device="cuda", generator=g).bfloat16()
    out, saved = layer.experts_forward(x)
    got, dx = layer.gradients(grad, saved)

    def weight(w):
        return torch.stack([fb.fp8_dequant(w[0][e], w[1][e].contiguous(), "128x128") for e in range(layer.experts)]).double().cpu()

    leaves = {k: v.requires_grad_(True) for k, v in dict(x=x.double().cpu(), router=layer.router.double().cpu(), up=weight(layer.up),
                                                          down=weight(layer.down), norm=layer.norm.double().cpu()).items()}
    ids = saved["ids"].long().cpu()
    with torch.enable_grad():
        want = _plain(layer, leaves["x"], leaves["router"], leaves["up"], leaves["down"], leaves["norm"], ids)
        (want * grad.double().cpu()).sum().backward()
    assert (out.double().cpu() - want.detach()).norm() <= 0.25 * (want.detach() - leaves["x"].detach()).norm() + 2.0 ** -8 * want.detach().norm()
    for name in ("router", "up", "down", "norm"):
        ref = leaves[name].grad
        assert got[name].shape == ref.shape and got[name].dtype is torch.float32
        assert (got[name].double().cpu() - ref).norm() <= 0.25 * ref.norm(), name
    through = leaves["x"].grad - grad.double().cpu()                     # without the residual's own part
    assert (dx.double().cpu() - grad.double().cpu() - through).norm() <= 0.25 * through.norm() + 2.0 ** -8 * leaves["x"].grad.norm()
    used = torch.zeros(layer.experts, dtype=torch.bool)
    used[ids.flatten()] = True
    assert (got["up"][~used.cuda()] == 0).all() and (got["down"][~used.cuda()] == 0).all()


def test_the_example_runs(monkeypatch, capsys):
    import decoder_layer as ex
    banner("examples/decoder_layer.py")
    monkeypatch.setattr(sys, "argv", ["decoder_layer.py", "--prompts", "130", "7", "--steps", "2"])
    ex.main()
    assert "clipped 1.000" in capsys.readouterr().out
