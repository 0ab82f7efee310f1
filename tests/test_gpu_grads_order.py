"""Outputs of the clipping whose elements lie in their gradients' order are taken, whatever the strides of dimensions of one
element or of empty tensors; others are refused."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def test_order_of_elements():
    g = torch.Generator(device="cuda").manual_seed(0)
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=g)   # noqa: E731
    grads = [r(1, 64).t(), r(64, 1), r(4, 1, 6).permute(2, 1, 0), r(2, 3, 1, 1).to(memory_format=torch.channels_last), r(6, 4).t(), r(0, 5).t()]
    z = lambda *shape: torch.zeros(*shape, device="cuda")   # noqa: E731
    outs = [z(64, 1), z(1, 64).t(), z(4, 6, 1).permute(1, 2, 0), z(2, 3, 1, 1), z(6, 4).t(), z(5, 0)]
    fb.fp8_grad_clip(grads, torch.full((1,), 4.0, device="cuda"), 1.0, outs=outs)
    for a, b in zip(grads, outs):
        assert torch.equal(a * 0.25, b)
    for a, b in ((grads[4], z(4, 6)), (grads[2], z(6, 1, 4))):
        with pytest.raises(ValueError, match="strides"):
            fb.fp8_grad_clip([a], torch.ones(1, device="cuda"), 1.0, outs=[b])
