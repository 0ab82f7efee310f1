"""The example layer: prompts fed at once, in chunks, and token by token give the same layer.

Chunking changes which attention kernel runs and when a page's scale grows.  A weight's rounding to bf16 (2^-8) and a
cached value's second rounding (half a step, 2^-4) are random over the elements of a row, and the residual stream they
are added to is exact: a relative difference of norms of 0.05 is far above them, and far below any wrong page, position
or expert, which changes rows outright."""
import os
import sys

import pytest

from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("chunk", [1, 7, 64, 100])
def test_chunks_give_the_same_layer(chunk):
    import decoder_layer as ex
    banner(f"example layer, chunks of {chunk}")
    layer = ex.Layer()
    g = torch.Generator(device="cuda").manual_seed(3)
    lengths = [130, 1, 77]
    inputs = [torch.randn(n, 1024, device="cuda", generator=g).bfloat16() for n in lengths]
    whole = ex.run(layer, inputs, max(lengths), *ex.new_cache(layer, lengths))
    parts = ex.run(layer, inputs, chunk, *ex.new_cache(layer, lengths))
    for a, b in zip(whole, parts):
        assert torch.isfinite(a).all() and torch.isfinite(b).all()
        assert (a.float() - b.float()).norm() <= 0.05 * a.float().norm()


def test_router_gradient_against_differences():
    """A step of the router's weights along their gradient changes the output as the gradient says, the choice and the
    experts' outputs being held: central differences in float64 of the same weights."""
    import decoder_layer as ex
    layer = ex.Layer(experts=16, top_k=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(9, 1024, device="cuda", generator=g).bfloat16()
    grad = torch.randn(9, 1024, device="cuda", generator=g)
    _, saved = layer.routed(x)
    a, _, ids, y = saved
    dw = layer.router_gradient(grad, saved).double()
    way = torch.randn(dw.shape, device="cuda", generator=g).double()

    def value(step):
        s = torch.sigmoid(a.double() @ (layer.router.double() + step * way).t()).gather(1, ids.long())
        w = s / (s.sum(1, keepdim=True) + 1e-20)
        return float((y.double() * w[..., None] * grad.double()[:, None]).sum())

    h = 1e-5
    want, got = (value(h) - value(-h)) / (2 * h), float((dw * way).sum())
    # float32 gradients of 9 tokens, summed over 16 x 1024 weights: 2^-16 of the terms' magnitudes
    assert abs(got - want) <= 2.0 ** -16 * float((dw * way).abs().sum()) + 1e-6 * abs(want)
