"""Inputs and checks of the training step's operators."""
import numpy as np
import torch

from decoder_util import bf16, dev
from gpu_util import host
from oracle import dequant_1x128, e4m3_half_ulp

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}          # half a step of the type, relative


def rounded(x, dtype):
    """float32 values that the type holds."""
    x = np.asarray(x, np.float32)
    return bf16(x) if dtype is BF16 else x


def on_gpu(x, dtype, pad=0):
    """A matrix on the GPU; pad > 0: as the left columns of a wider one."""
    t = dev(x).to(dtype)
    if not pad:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def check_near(got, want, slack, dtype, what=""):
    """Within `slack` (absolute, of float32 arithmetic) plus half a step of the type the result is held in."""
    off = np.abs(f64(got) - want)
    most = slack * (1 + 2 * HALF[dtype]) + HALF[dtype] * np.abs(want) + 2.0 ** -140
    bad = np.argwhere(~(off <= most))
    assert bad.size == 0, f"{what}: {len(bad)} values off, first at {bad[:3].tolist()}: {[(f64(got)[tuple(i)], want[tuple(i)], most[tuple(i)]) for i in bad[:3]]}"


def check_quantized(q, scale, want, slack, what=""):
    """Codes and scales of values that are within `slack` of `want`: a scale is amax / 448 of them, and a code's value is
    within half an E4M3 step of its value."""
    q, scale = q.cpu().numpy(), scale.cpu().numpy()
    rows, cols = want.shape
    amax, extra = np.abs(want).reshape(rows, -1, 128).max(2), slack.reshape(rows, -1, 128).max(2)
    ideal = amax / 448
    plain = ideal > 1.001e-10 + extra
    assert (np.abs(scale - ideal) <= extra / 448 + 2.0 ** -23 * ideal)[plain].all(), what
    s = np.repeat(scale.astype(np.float64), 128, 1)
    ratio = np.minimum(np.abs(want) / s, 448.0)
    off = np.abs(dequant_1x128(q, scale) - want)
    most = (e4m3_half_ulp(ratio * (1 + 2.0 ** -12)) * s) * (1 + 2.0 ** -12) + slack
    assert (off <= most).all(), (what, np.argwhere(off > most)[:3].tolist())


def same_bits(a, b):
    return np.array_equal(host(a).view(np.uint8), host(b).view(np.uint8))
