"""Clipping by factors near and below float32's normal range, and norms at both of its ends, against float64.

Roundings: the factor, two products (2^-24 each; 2^-22 for all, with a factor two bits below the normal range at worst), the
type's own; results below the normal range are held to 2^-149, 2^-133 in bf16."""
import numpy as np
import pytest

from gpu_util import banner
from train_util import BF16, F32, HALF, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("norm", [3.4e38, 1e38, 3e37, 1e30, 1.0, 2.0 ** -20, 2.0 ** -126])
@pytest.mark.parametrize("max_norm", [1e3, 1.0, 0.01, 1e-6, 1e-20, 2.0 ** -125, 2.0 ** -149])
def test_factors_of_all_sizes(max_norm, norm, dtype):
    banner(f"clipping from {norm} to {max_norm}, {dtype}")
    g = torch.Generator(device="cuda").manual_seed(0)
    value = torch.rand(5003, device="cuda", generator=g, dtype=torch.float64) * 2 - 1
    size = torch.exp2(-torch.rand(5003, device="cuda", generator=g, dtype=torch.float64) * 30)
    grads = [(value * size * norm).to(dtype)[3:], (value * norm).to(dtype)[:1000], torch.full((7,), norm, device="cuda").to(dtype)]
    given = torch.full((1,), norm, device="cuda")
    c = min(1.0, float(np.float32(max_norm)) / float(given))
    outs = fb.fp8_grad_clip(grads, given, max_norm, outs=[torch.empty_like(t) for t in grads])
    place = fb.fp8_grad_clip([t.clone() for t in grads], given, max_norm)
    for t, out, same in zip(grads, outs, place):
        broken = ~t.isfinite().cpu().numpy()              # 3.4e38 is an infinity in bf16, an input that the header excludes
        assert not np.isfinite(f64(out)[broken]).any()
        want = np.where(broken, 0.0, f64(t)) * c
        off = np.where(broken, 0.0, np.abs(f64(out) - want))
        assert (off <= (2.0 ** -22 + HALF[dtype] * (1 + 2.0 ** -20)) * np.abs(want) + (2.0 ** -148 if dtype is F32 else 2.0 ** -133)).all()
        assert torch.equal(out.nan_to_num(), same.nan_to_num())


@pytest.mark.parametrize("size", [2.0 ** 126, 1e38, 1e-38, 2.0 ** -133, 2.0 ** -149])
def test_norms_of_all_sizes(size):
    banner(f"norm of values of {size}")
    grads = [torch.full((n,), size, device="cuda") for n in (1, 2, 5)]
    want = size * np.sqrt(8.0)
    got = float(fb.fp8_grad_norm(grads))
    assert abs(got - want) <= 2.0 ** -24 * want * (1 + 2.0 ** -20) + 2.0 ** -150 * (1 + 2.0 ** -20) if want < 2.0 ** 128 else got == np.inf
