"""What the binding of the training step's operators refuses of GPU tensors: types, shapes, pitches, overlaps of lists.
Nothing is launched."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

F32, BF16, U8, I32 = torch.float32, torch.bfloat16, torch.uint8, torch.int32


def z(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def refused(error, *calls):
    for i, call in enumerate(calls):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was not refused")


def test_norm():
    x = z(4, 256)
    refused(ValueError, lambda: fb.fp8_rmsnorm_quant(x[0]), lambda: fb.fp8_rmsnorm_quant(z(256, 4).t()), lambda: fb.fp8_rmsnorm_quant(x, z(255)),
            lambda: fb.fp8_rmsnorm_quant(x, z(512)[::2]), lambda: fb.fp8_rmsnorm_quant(x, residual=z(4, 128)),
            lambda: fb.fp8_rmsnorm_quant(x, residual_out=z(4, 256)), lambda: fb.fp8_rmsnorm_quant(x, q=z(4, 128, dtype=U8)),
            lambda: fb.fp8_rmsnorm_quant(x, scale=z(4, 4)[:, ::2]), lambda: fb.fp8_rmsnorm_quant(x, quantize=False, with_y=True, q=z(4, 256, dtype=U8)),
            lambda: fb.fp8_rmsnorm_quant(x, torch.zeros(256)), lambda: fb.fp8_rmsnorm_backward(x, z(3, 256)), lambda: fb.fp8_rmsnorm_backward(x, x, dweight=z(256)),
            lambda: fb.fp8_rmsnorm_backward(x, x, z(256), dweight=z(128)))
    refused(TypeError, lambda: fb.fp8_rmsnorm_quant(x.half()), lambda: fb.fp8_rmsnorm_quant(x, z(256).double()),
            lambda: fb.fp8_rmsnorm_quant(x, residual=z(4, 256, dtype=BF16)), lambda: fb.fp8_rmsnorm_quant(x, y=z(4, 256, dtype=BF16)),
            lambda: fb.fp8_rmsnorm_backward(z(4, 256, dtype=BF16), x))
    refused(fb.Fp8bsError, lambda: fb.fp8_rmsnorm_quant(z(4, 100)), lambda: fb.fp8_rmsnorm_quant(x, eps=0.0), lambda: fb.fp8_rmsnorm_quant(x, quantize=False),
            lambda: fb.fp8_rmsnorm_quant(z(4, 260)[:, 2:258]), lambda: fb.fp8_rmsnorm_quant(z(1, 256).expand(4, 256)),
            lambda: fb.fp8_rmsnorm_backward(z(4, 100), z(4, 100), z(100)), lambda: fb.fp8_rmsnorm_quant(z(1, 32896)))


def test_activation():
    g = z(4, 256)
    refused(ValueError, lambda: fb.fp8_swiglu_quant(g, z(4, 128)), lambda: fb.fp8_swiglu_quant(g, z(3, 256)), lambda: fb.fp8_swiglu_backward(z(4, 128), g, g),
            lambda: fb.fp8_swiglu_backward(g, g, g, d=z(4, 256)), lambda: fb.fp8_swiglu_backward(g, g, g, scale=z(4, 2)))
    refused(TypeError, lambda: fb.fp8_swiglu_quant(g, g.bfloat16()), lambda: fb.fp8_swiglu_backward(g.bfloat16(), g, g), lambda: fb.fp8_swiglu_quant(g.half(), g.half()))
    refused(fb.Fp8bsError, lambda: fb.fp8_swiglu_quant(z(4, 100), z(4, 100)), lambda: fb.fp8_swiglu_quant(g, g, quantize=False))


def test_tiles_and_weight_gradients():
    x, off = z(4, 64), z(3, dtype=I32)
    refused(ValueError, lambda: fb.fp8_quant_grouped_t(x, z(1, dtype=I32)), lambda: fb.fp8_quant_grouped_t(x, z(1026, dtype=I32)),
            lambda: fb.fp8_quant_grouped_t(x, z(6, dtype=I32)[::2]), lambda: fb.fp8_quant_grouped_t(x, off, order=z(2, 2, dtype=I32)),
            lambda: fb.fp8_quant_grouped_t(x, off, q=z(64, 128, dtype=U8)), lambda: fb.fp8_quant_grouped_t(x, off, q=z(64, 300, dtype=U8)),
            lambda: fb.fp8_quant_grouped_t(x, off, scale=z(64, 3)), lambda: fb.fp8_quant_grouped_t(x, off, padded=z(2, dtype=I32)))
    refused(TypeError, lambda: fb.fp8_quant_grouped_t(x, z(3)), lambda: fb.fp8_quant_grouped_t(x.half(), off), lambda: fb.fp8_quant_grouped_t(x, off, order=z(4)))
    refused(fb.Fp8bsError, lambda: fb.fp8_quant_grouped_t(x, off, top_k=2), lambda: fb.fp8_quant_grouped_t(z(4, 72), off),
            lambda: fb.fp8_quant_grouped_t(x, off, order=z(4, dtype=I32), top_k=0), lambda: fb.fp8_quant_grouped_t(x, off, padded=off))
    a, s = z(32, 256, dtype=U8), z(32, 2)
    w = fb.fp8_blockscaled_grouped_wgrad
    refused(ValueError, lambda: w(off, a, s, z(32, 128, dtype=U8), s), lambda: w(off, a, z(32, 1), a, s), lambda: w(off, a, s, a, s, accumulate=True),
            lambda: w(off, a, s, a, s, y=z(2, 32, 16)), lambda: w(off, a, s, a, s, y=z(2, 32, 64)[:, :, ::2]), lambda: w(z(1, dtype=I32), a, s, a, s))
    refused(TypeError, lambda: w(off, a, s, a, s, y=z(2, 32, 32, dtype=torch.float16)), lambda: w(off, a, s, a, s, out_dtype=BF16, y=z(2, 32, 32)),
            lambda: w(off.long(), a, s, a, s), lambda: w(off, a.to(torch.int8), s, a, s), lambda: w(off, a, s.double(), a, s))
    refused(fb.Fp8bsError, lambda: w(off, z(24, 256, dtype=U8), z(24, 2), a, s), lambda: w(off, z(32, 200, dtype=U8), z(32, 1), z(32, 200, dtype=U8), z(32, 1)))


def test_gradients():
    g, norm = z(10), z(1)
    refused(ValueError, lambda: fb.fp8_grad_norm([z(10)[::2]]), lambda: fb.fp8_grad_norm([z(1).expand(5)]), lambda: fb.fp8_grad_norm([g], norm=z(2)),
            lambda: fb.fp8_grad_clip([g], z(2), 1.0), lambda: fb.fp8_grad_clip([g], norm, 1.0, outs=[]), lambda: fb.fp8_grad_clip([g], norm, 1.0, outs=[z(9)]),
            lambda: fb.fp8_grad_clip([z(4, 6)], norm, 1.0, outs=[z(6, 4).t()]), lambda: fb.fp8_grad_norm([g, torch.zeros(3)]))
    refused(TypeError, lambda: fb.fp8_grad_norm([g.half()]), lambda: fb.fp8_grad_norm(g), lambda: fb.fp8_grad_clip([g], norm.double(), 1.0),
            lambda: fb.fp8_grad_clip([g], norm, 1.0, outs=[z(10, dtype=BF16)]))
    refused(fb.Fp8bsError, lambda: fb.fp8_grad_clip([g], norm, 0.0), lambda: fb.fp8_grad_clip([g], norm, float("nan")))
