"""Outputs that are an input themselves, as the header allows, and operands side by side in one buffer: the same bits as
apart."""
import pytest

from gpu_util import banner
from train_util import BF16, F32, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _rows(*shape, dtype, seed=0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 128), (1500, 1024), (700, 7168), (300, 16384), (300, 32768)])
def test_norm(rows, cols, dtype):
    banner(f"norm in place, {rows}x{cols} {dtype}")
    x, res, w = _rows(rows, cols, dtype=dtype), _rows(rows, cols, dtype=dtype, seed=1), _rows(cols, dtype=F32, seed=2)
    want = fb.fp8_rmsnorm_quant(x, w, residual=res, with_y=True)
    for y_at, out_at in ((0, None), (1, None), (0, 1), (1, 0)):
        a = [x.clone(), res.clone()]
        got = fb.fp8_rmsnorm_quant(a[0], w, residual=a[1], y=a[y_at], residual_out=None if out_at is None else a[out_at])
        assert got[2] is a[y_at] and all(same_bits(u, v) for u, v in zip(got, want))
    want, a = fb.fp8_rmsnorm_quant(x, w, with_y=True), x.clone()
    got = fb.fp8_rmsnorm_quant(a, w, y=a)
    assert got[2] is a and all(same_bits(u, v) for u, v in zip(got[:3], want[:3]))
    both = fb.fp8_rmsnorm_quant(x, w, residual=x, with_y=True)              # one tensor as both inputs, and the sum over it
    a = x.clone()
    got = fb.fp8_rmsnorm_quant(a, w, residual=a, residual_out=a, with_y=True)
    assert all(same_bits(u, v) for u, v in zip(got, both))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,cols", [(1, 128), (3000, 384), (16385, 512)])
def test_activation(rows, cols, dtype):
    banner(f"activation in place, {rows}x{cols} {dtype}")
    both, dy = _rows(rows, 2 * cols, dtype=dtype), _rows(rows, cols, dtype=dtype, seed=1)
    want = fb.fp8_swiglu_quant(both[:, :cols], both[:, cols:], with_y=True)
    for half in (0, 1):
        a = both.clone()
        parts = a.split(cols, 1)
        got = fb.fp8_swiglu_quant(*parts, y=parts[half])
        assert same_bits(got[2].contiguous(), want[2]) and same_bits(got[0], want[0]) and same_bits(got[1], want[1])
        assert same_bits(parts[1 - half].contiguous(), both.split(cols, 1)[1 - half].contiguous())
    want = fb.fp8_swiglu_backward(dy, both[:, :cols], both[:, cols:], with_d=True)
    a = torch.cat([both[:, cols:], both[:, :cols]], 1)                      # up before gate, and d over both
    got = fb.fp8_swiglu_backward(dy, a[:, cols:], a[:, :cols], d=a)
    assert got[2] is a and all(same_bits(u, v) for u, v in zip(got, want))
    a = torch.cat([both[:, :cols], dy], 1)                                  # over gate and dy
    got = fb.fp8_swiglu_backward(a[:, cols:], a[:, :cols], both[:, cols:], d=a)
    assert all(same_bits(u, v) for u, v in zip(got, want))


def test_operands_side_by_side():
    """Columns of one buffer, rows of another: apart, though their ranges of addresses are not."""
    banner("operands of one buffer")
    rows, cols = 333, 256
    x, res, dy = (_rows(rows, cols, dtype=BF16, seed=s) for s in range(3))
    w = _rows(cols, dtype=F32, seed=3)
    wide = torch.zeros(rows, 5 * cols, dtype=BF16, device="cuda")
    part = wide.split(cols, 1)
    part[0].copy_(x), part[1].copy_(res)
    want = fb.fp8_rmsnorm_quant(x, w, residual=res, with_y=True)
    got = fb.fp8_rmsnorm_quant(part[0], w, residual=part[1], residual_out=part[2], y=part[3], q=part[4][:, :cols // 2].view(torch.uint8))
    assert all(same_bits(u.contiguous(), v) for u, v in zip(got, want))
    part[3].copy_(dy)
    want = fb.fp8_rmsnorm_backward(dy, x, w, dresidual=res)
    got = fb.fp8_rmsnorm_backward(part[3], part[0], w, dresidual=part[1], dx=part[4])
    assert all(same_bits(u.contiguous(), v) for u, v in zip(got, want))
    off = torch.tensor([0, 100, 333], dtype=torch.int32, device="cuda")
    q, scale, padded = fb.fp8_quant_grouped_t(x, off)
    columns = q.shape[1]
    buffer = torch.zeros(2 * cols, 2 * columns, dtype=torch.uint8, device="cuda")
    a = fb.fp8_quant_grouped_t(x, off, q=buffer[:cols, :columns])
    b = fb.fp8_quant_grouped_t(res, off, q=buffer[:cols, columns:])
    assert same_bits(a[0][:, :padded[-1]].contiguous(), q[:, :padded[-1]].contiguous())
    other = fb.fp8_quant_grouped_t(res, off)
    one = fb.fp8_blockscaled_grouped_wgrad(padded, q, scale, other[0], other[1])
    assert same_bits(fb.fp8_blockscaled_grouped_wgrad(padded, *a[:2], *b[:2]), one)


def test_overlaps_are_refused():
    """Nothing is launched."""
    x, w = _rows(8, 256, dtype=BF16), torch.ones(256, device="cuda")
    wide = _rows(9, 256, dtype=BF16)
    for call in (lambda: fb.fp8_rmsnorm_quant(x, residual=wide[:8], residual_out=wide[1:]), lambda: fb.fp8_rmsnorm_quant(wide[:8], y=wide[1:]),
                 lambda: fb.fp8_rmsnorm_quant(x, residual=wide[:8], residual_out=x, y=x), lambda: fb.fp8_rmsnorm_backward(x, wide[:8], w, dx=wide[1:]),
                 lambda: fb.fp8_rmsnorm_backward(x, x, w, dweight=w), lambda: fb.fp8_swiglu_quant(wide[:8], x, y=wide[1:]),
                 lambda: fb.fp8_swiglu_backward(x[:, :128], x[:, 128:], x[:, :128], d=wide[:8], q=wide[1:].view(torch.uint8)[:, :256])):
        with pytest.raises(fb.Fp8bsError, match="overlaps"):
            call()
