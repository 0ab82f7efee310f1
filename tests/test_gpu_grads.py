"""The norm of many tensors and their clipping.  The norm is a 64-bit sum: one float32 rounding (2^-24) and the sum's own
(2^-40).  A clipped value is two float32 roundings and the type's: bit-exact with those."""
import numpy as np
import pytest

from gpu_util import banner
from oracle import train
from train_util import BF16, F32, dev, same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

LENGTHS = [[1], [3, 0, 7], [16384], [16385, 1], [65536, 32768 + 5], [200001, 13, 4, 4096], [5] * 97, [1000] * 200, [0]]


def _tensors(lengths, dtype, seed=0, shift=0):
    """Tensors inside one buffer, the i-th starting i + shift elements behind a multiple of 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for i, n in enumerate(lengths):
        lead = (i + shift) % 9
        out.append(torch.randn(n + lead + 3, device="cuda", generator=g).to(dtype)[lead:lead + n])
    return out


def _near(norm, tensors):
    want = train.grad_norm([t.float().cpu().numpy() for t in tensors])
    assert norm.shape == (1,) and norm.dtype is F32
    assert abs(float(norm) - want) <= (2.0 ** -24 + 2.0 ** -40) * want


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths", LENGTHS, ids=lambda v: f"{len(v)}x{sum(v)}")
def test_norm_and_clip(lengths, dtype):
    banner(f"gradient norm of {len(lengths)} tensors, {sum(lengths)} elements, {dtype}")
    grads = _tensors(lengths, dtype)
    norm = fb.fp8_grad_norm(grads)
    _near(norm, grads)
    for max_norm in (float(norm) / 3 or 1.0, float(norm) * 2 or 1.0):
        clip = float(norm) > np.float32(max_norm)
        factor = torch.tensor(np.float32(max_norm) / np.float32(float(norm)) if clip else np.float32(1.0), device="cuda")
        want = [(t.float() * factor).to(dtype) for t in grads]
        outs = _tensors(lengths, dtype, seed=1, shift=2)
        got = fb.fp8_grad_clip(grads, norm, max_norm, outs=outs)
        assert got is outs and all(same_bits(a, b) for a, b in zip(got, want))
        place = [t.clone() for t in grads]
        got = fb.fp8_grad_clip(place, norm, max_norm)
        assert got is place and all(same_bits(a, b) for a, b in zip(got, want))
        assert all(same_bits(a, b) for a, b in zip(fb.fp8_grad_clip([t.clone() for t in grads], norm, max_norm,
                                                                     outs=[t.clone() for t in grads]), want))


def test_neighbours_stay():
    """Elements in front of and behind the tensors, which share their 16 bytes."""
    for dtype in (F32, BF16):
        buffer = torch.arange(1, 400, device="cuda").to(dtype)
        for lo, hi in ((1, 2), (3, 10), (5, 300), (8, 16), (7, 8), (9, 399)):
            t = buffer.clone()
            fb.fp8_grad_clip([t[lo:hi]], torch.full((1,), 4.0, device="cuda"), 1.0)
            want = buffer.clone()
            want[lo:hi] = (want[lo:hi].float() * 0.25).to(dtype)
            assert torch.equal(t, want), (dtype, lo, hi)
            other = torch.zeros_like(buffer)
            fb.fp8_grad_clip([buffer[lo:hi]], torch.full((1,), 4.0, device="cuda"), 1.0, outs=[other[400 - hi - 1:400 - lo - 1]])
            assert torch.equal(other[400 - hi - 1:400 - lo - 1], want[lo:hi]) and int((other != 0).sum()) == hi - lo


def test_types_shapes_and_orders_mix():
    g = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(33, 65, device="cuda", generator=g), torch.randn(4, 5, 6, device="cuda", generator=g).to(BF16),
             torch.randn(64, 48, device="cuda", generator=g).t(), torch.randn((), device="cuda", generator=g)]
    norm = fb.fp8_grad_norm(tuple(grads))
    _near(norm, grads)
    outs = [torch.empty_like(t) for t in grads]
    fb.fp8_grad_clip(grads, norm, 1.0, outs=outs)
    for a, b in zip(grads, outs):
        assert torch.equal((a.float() * (1.0 / norm)[0]).to(a.dtype), b)


def test_sizes_beyond_float32_squares():
    """Squares that overflow or vanish in float32."""
    for size in (1e30, 1e-30):
        grads = [torch.full((1000,), size, device="cuda"), torch.full((24,), -size, device="cuda")]
        norm = fb.fp8_grad_norm(grads)
        assert abs(float(norm) / (32 * np.float32(size)) - 1) <= 2.0 ** -23
        fb.fp8_grad_clip(grads, norm, size * 8)
        assert (grads[0] - size / 4).abs().max() <= 2.0 ** -22 * size
    assert float(fb.fp8_grad_norm([torch.full((16,), 3e38, device="cuda")])) == float("inf")
    assert float(fb.fp8_grad_norm([torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")])) == 0.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_broken_gradients_are_seen_and_left(bad):
    grads = [torch.ones(5000, device="cuda"), torch.ones(77, device="cuda", dtype=BF16)]
    grads[1][40] = bad
    norm = fb.fp8_grad_norm(grads)
    assert not torch.isfinite(norm).any()
    was = [t.clone() for t in grads]
    fb.fp8_grad_clip(grads, norm, 1.0)
    outs = fb.fp8_grad_clip(grads, norm, 1.0, outs=[torch.empty_like(t) for t in grads])
    for a, b, c in zip(grads, was, outs):
        assert same_bits(a, b)
        assert torch.equal(torch.nan_to_num(c.float()), torch.nan_to_num(a.float())) and torch.equal(c.isnan(), a.isnan())


def test_the_norm_of_ranks_parts():
    """Norms of parts join as the header says; the norm goes where it is asked to."""
    grads = _tensors([70000, 3, 12345, 9], F32, seed=4)
    whole = torch.empty(1, device="cuda")
    assert fb.fp8_grad_norm(grads, norm=whole) is whole
    parts = torch.cat([fb.fp8_grad_norm(grads[:2]), fb.fp8_grad_norm(grads[2:])])
    assert abs(float(parts.double().square().sum().sqrt()) / float(whole) - 1) <= 2.0 ** -22


def test_many_small_tensors():
    banner("gradient norm of 3000 tensors")
    grads = list(torch.randn(3000 * 40, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).split(40))
    norm = fb.fp8_grad_norm(grads)
    _near(norm, grads)
    want = [t * (0.5 / norm) for t in grads]
    fb.fp8_grad_clip(grads, norm, 0.5)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))


def test_beyond_4_gib():
    banner("gradient of more than 2^31 elements")
    n = (1 << 31) + 77
    t = torch.ones(n, dtype=BF16, device="cuda")
    t[-1] = 3.0
    norm = fb.fp8_grad_norm([t])
    assert abs(float(norm) / np.sqrt(n + 8.0) - 1) <= 2.0 ** -23
    fb.fp8_grad_clip([t], torch.full((1,), 2.0, device="cuda"), 1.0)
    assert float(t[-1]) == 1.5 and float(t[0]) == 0.5 and float(t[n // 2]) == 0.5 and float(t[-2]) == 0.5
    assert int((t[1 << 30:(1 << 30) + 100000] != 0.5).sum()) == 0


def test_shared_memory():
    """The same tensor twice counts twice in the norm and is refused by the clipping; neighbours, and outputs on their own
    inputs, are none of that."""
    t = torch.arange(1, 65, device="cuda").float()
    assert abs(float(fb.fp8_grad_norm([t, t])) / np.sqrt(2 * float(t.square().sum())) - 1) <= 2.0 ** -22
    norm = torch.full((1,), 2.0, device="cuda")
    for grads in ([t, t], [t[:33], t[32:]], [t, t[60:]]):
        with pytest.raises(fb.Fp8bsError, match="shares memory"):
            fb.fp8_grad_clip(grads, norm, 1.0)
    was = t.clone()
    fb.fp8_grad_clip([t[40:], t[:7], t[7:40]], norm, 1.0)
    assert torch.equal(t, was / 2)
    other = torch.empty(24, device="cuda")
    fb.fp8_grad_clip([t[:40], t[40:]], norm, 1.0, outs=[t[:40], other])
    assert torch.equal(t[:40], was[:40] / 4) and torch.equal(other, was[40:] / 4) and torch.equal(t[40:], was[40:] / 2)
