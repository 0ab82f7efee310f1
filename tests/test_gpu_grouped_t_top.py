"""Transposed tiles of the largest finite values: codes as the header says, all of them finite, and weight gradients of them
that are (a product with zeros is zero)."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import train
from train_util import BF16, F32, dev, on_gpu, rounded

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

MOST = {F32: float(np.finfo(np.float32).max), BF16: float(torch.finfo(BF16).max)}
STEPS = [1.0, 0.99, 0.97, 31 / 32, 0.9687, 0.95, 15 / 16, 0.9, 7 / 8, 0.87, 0.5, 2.0 ** -8, 2.0 ** -30, 0.0]      # of 2^128, below the type's largest


def _rows(dtype, rows, cols):
    x = np.resize(np.array([min(s * 2.0 ** 128, MOST[dtype]) for s in STEPS]), rows * cols).reshape(rows, cols)
    x *= np.where(np.arange(rows)[:, None] % 3 == 1, -1.0, 1.0)
    x[:, ::5] *= 0.4                                    # columns below the top next to those at it
    return rounded(x, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_codes(dtype):
    banner(f"transposed tiles of the largest {dtype} values")
    x, off = _rows(dtype, 301, 144), [0, 130, 130, 301]
    q, scale = np.zeros((144, 640), np.uint8), np.zeros((144, 5), np.float32)
    want = train.tiles(x, off, None, 1, q, scale)
    got = fb.fp8_quant_grouped_t(on_gpu(x, dtype), dev(np.asarray(off, np.int32)), q=dev(q), scale=dev(scale))
    for a, b in zip(got, want):
        assert np.array_equal(a.cpu().numpy().view(np.uint8), np.ascontiguousarray(b).view(np.uint8))
    assert (got[1] == 2.0 ** 120).any() and ((got[0] & 0x7f) == 0x77).any()
    back = fb.fp8_dequant(got[0], got[1])
    assert back.isfinite().all()
    value = torch.from_numpy(x).cuda().t()
    for lo, hi, at in ((0, 130, 0), (130, 301, 256)):
        # half a step, or what 240 * 2^120 lacks of the largest values: a sixteenth of 2^128
        assert (back[:, at:at + hi - lo].double() - value[:, lo:hi].double()).abs().le(2.0 ** 124 + 2.0 ** 110).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weight_gradient(dtype):
    banner(f"weight gradient of the largest {dtype} values")
    x, off = _rows(dtype, 200, 64), dev(np.array([0, 150, 200], np.int32))
    a, sa, padded = fb.fp8_quant_grouped_t(on_gpu(x, dtype), off)
    b, sb, _ = fb.fp8_quant_grouped_t(torch.zeros(200, 32, device="cuda"), off)
    assert (fb.fp8_blockscaled_grouped_wgrad(padded, a, sa, b, sb) == 0).all()
    assert (fb.fp8_blockscaled_grouped_wgrad(padded, b, sb, a, sa) == 0).all()
    tiny = torch.full((200, 32), 2.0 ** -20, device="cuda")
    b, sb, _ = fb.fp8_quant_grouped_t(tiny, off)
    y = fb.fp8_blockscaled_grouped_wgrad(padded, a, sa, b, sb)
    want, size, depth = train.wgrad(padded.cpu().numpy(), train.values(a.cpu().numpy(), sa.cpu().numpy()), train.values(b.cpu().numpy(), sb.cpu().numpy()))
    assert (np.abs(y.cpu().numpy() - want) <= np.array(depth)[:, None, None] * 2.0 ** -24 * size).all()
