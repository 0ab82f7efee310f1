"""Sizes that a training operator does not take are refused before memory is taken for its outputs."""
import pytest

from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

U8, I32 = torch.uint8, torch.int32


def _refused(call, match):
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    with pytest.raises(fb.Fp8bsError, match=match):
        call()
    assert torch.cuda.max_memory_allocated() == before


def test_norm():
    banner("norm of columns out of range")
    for cols in (100, 32896, 65536):
        x, w = torch.zeros(512, cols, device="cuda"), torch.ones(cols, device="cuda")
        _refused(lambda: fb.fp8_rmsnorm_quant(x, w, with_y=True), "cols")
        _refused(lambda: fb.fp8_rmsnorm_quant(x, residual=x), "cols")
        _refused(lambda: fb.fp8_rmsnorm_backward(x, x, w), "cols")
        _refused(lambda: fb.fp8_rmsnorm_backward(x, x), "cols")


def test_activation():
    banner("activation of columns out of range")
    x = torch.zeros(512, 200, device="cuda")
    _refused(lambda: fb.fp8_swiglu_quant(x, x, with_y=True), "cols")
    _refused(lambda: fb.fp8_swiglu_backward(x, x, x, with_d=True), "cols")


def test_transposed_tiles():
    banner("transposed tiles of too many rows")
    off = torch.zeros(3, dtype=I32, device="cuda")
    x, ragged = torch.zeros((1 << 22) + 1, 16, device="cuda"), torch.empty(1 << 16, 24, device="cuda")
    order = torch.zeros((1 << 22) + 1, dtype=I32, device="cuda")
    few = x[:1000]
    _refused(lambda: fb.fp8_quant_grouped_t(x, off), "columns")
    _refused(lambda: fb.fp8_quant_grouped_t(few, off, order=order), "columns")
    _refused(lambda: fb.fp8_quant_grouped_t(ragged, off), "cols")


def test_weight_gradient():
    banner("weight gradients of sizes out of range")
    padded = torch.zeros(257, dtype=I32, device="cuda")

    def operand(rows, columns=128):
        return torch.zeros(rows, columns, dtype=U8, device="cuda"), torch.ones(rows, columns // 128, device="cuda")

    good, odd = operand(4096), operand(4104)
    _refused(lambda: fb.fp8_blockscaled_grouped_wgrad(padded, *good, *odd), "multiples of 16")
    _refused(lambda: fb.fp8_blockscaled_grouped_wgrad(padded, *odd, *good), "multiples of 16")
    ragged = torch.zeros(4096, 200, dtype=U8, device="cuda"), torch.ones(4096, 1, device="cuda")
    _refused(lambda: fb.fp8_blockscaled_grouped_wgrad(padded, *ragged, *ragged), "columns")
    wide = operand(16, (1 << 22) + 128)
    _refused(lambda: fb.fp8_blockscaled_grouped_wgrad(padded, *wide, *wide), "exceed")


def test_nothing_to_do_is_not_refused():
    """No rows of one operand: an empty result, whatever the other sizes."""
    padded = torch.zeros(3, dtype=I32, device="cuda")
    columns = (1 << 22) + 128
    a, b = torch.zeros(0, columns, dtype=U8, device="cuda"), torch.zeros(16, columns, dtype=U8, device="cuda")
    sa, sb = torch.ones(0, columns // 128, device="cuda"), torch.ones(16, columns // 128, device="cuda")
    assert fb.fp8_blockscaled_grouped_wgrad(padded, a, sa, b, sb).shape == (2, 0, 16)
    assert fb.fp8_blockscaled_grouped_wgrad(padded, b, sb, a, sa).shape == (2, 16, 0)
