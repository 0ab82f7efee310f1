"""Weight gradients at the ends of the range of scales, against float64 and the header's bound: depth * (2^-24 of the
products' magnitudes + 2^-126), half a step of the result's type."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import train
from train_util import BF16, F32, HALF, dev, f64

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _operand(rng, rows, columns, low, high):
    codes = rng.integers(0, 256, (rows, columns)).astype(np.uint8)
    codes = np.where(codes & 0x7f == 0x7f, 0x30, codes).astype(np.uint8)
    return codes, (2.0 ** rng.integers(low, high + 1, (rows, columns // 128))).astype(np.float32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("a_range,b_range", [((-100, -100), (-100, -100)), ((-100, -90), (-40, -20)), ((-70, -60), (-75, -55)), ((-100, 110), (-100, -98)),
                                             ((100, 119), (-100, -20))])
@pytest.mark.parametrize("n,k", [(48, 80), (272, 144)])
def test_small_and_large_scales(n, k, a_range, b_range, dtype):
    banner(f"weight gradient, scales 2^{a_range} and 2^{b_range}, {n}x{k}, {dtype}")
    rng = np.random.default_rng(n)
    padded = np.array([0, 256, 256, 640], np.int32)
    (a, sa), (b, sb) = _operand(rng, n, 640, *a_range), _operand(rng, k, 640, *b_range)
    for was in (None, 2.0 ** -110):
        given = None if was is None else torch.full((3, n, k), was, dtype=dtype, device="cuda")
        y = fb.fp8_blockscaled_grouped_wgrad(dev(padded), dev(a), dev(sa), dev(b), dev(sb), out_dtype=dtype, y=given, accumulate=was is not None)
        want, size, depth = train.wgrad(padded, train.values(a, sa), train.values(b, sb))
        slack = np.array(depth)[:, None, None] * (2.0 ** -24 * size + 2.0 ** -126)
        if was is not None:
            want, slack = want + was, slack + 2.0 ** -24 * np.abs(want + was)
        assert (np.abs(f64(y) - want) <= slack * (1 + 2 * HALF[dtype]) + HALF[dtype] * np.abs(want) + 2.0 ** -134).all()
