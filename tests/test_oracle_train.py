"""The oracle of the training step's operators against central differences, rational arithmetic and closed forms (no GPU)."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import e4m3_decode, quant_1x128, train

RNG = np.random.default_rng(0)


def differences(f, x, h=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        d[i] = (f(a) - f(b)) / (2 * h)
    return d


@pytest.mark.parametrize("weighted", [True, False])
def test_norm_gradient_is_the_difference(weighted):
    h, dy, w = RNG.standard_normal((3, 8)), RNG.standard_normal((3, 8)), RNG.standard_normal(8) if weighted else None
    dx, dw, _, _ = train.rmsnorm_grad(dy, h, w, 1e-3)
    assert np.allclose(dx, differences(lambda z: (train.rmsnorm(z, w, 1e-3) * dy).sum(), h), atol=1e-8)
    if weighted:
        assert np.allclose(dw, differences(lambda z: (train.rmsnorm(h, z, 1e-3) * dy).sum(), w), atol=1e-8)


def test_norm_closed_forms():
    """Equal values give 1 (without eps), and the gradient along h vanishes."""
    h = np.full((1, 128), -3.0)
    assert np.allclose(train.rmsnorm(h, None, 0.0), -1.0)
    dx, _, _, _ = train.rmsnorm_grad(h, h, None, 0.0)
    assert np.allclose(dx, 0.0)


def test_activation_gradient_is_the_difference():
    g, u, dy = RNG.standard_normal((3, 2, 6)) * 3
    d, _ = train.swiglu_grad(dy, g, u)
    assert np.allclose(d[:, :6], differences(lambda z: (train.swiglu(z, u) * dy).sum(), g), atol=1e-7)
    assert np.allclose(d[:, 6:], differences(lambda z: (train.swiglu(g, z) * dy).sum(), u), atol=1e-7)
    assert train.swiglu(np.array([[1e4, -1e4, 0.0]]), np.ones((1, 3))).tolist() == [[1e4, 0.0, 0.0]]


def test_exponents_in_rational_arithmetic():
    for amax in [2.0 ** -120, 448 * 2.0 ** -100, 1e-20, 447.9, 448.0, np.nextafter(np.float32(448), np.float32(1e9)), 449.0, 3e38]:
        e = train.exponent(float(amax))
        assert Fraction(float(amax)) <= 448 * Fraction(2) ** e
        assert e == train.MIN_EXP or Fraction(float(amax)) > 448 * Fraction(2) ** (e - 1)


def test_tiles_restart_at_every_expert():
    x = RNG.standard_normal((300, 4)).astype(np.float32)
    off = [0, 130, 130, 299]
    q, s, padded = train.tiles(x, off, None, 1, np.full((4, 640), 7, np.uint8), np.full((4, 5), 9, np.float32))
    assert padded.tolist() == [0, 256, 256, 512]
    for lo, hi, at in [(0, 128, 0), (128, 130, 1), (130, 258, 2), (258, 299, 3)]:
        v = e4m3_decode(q[:, 128 * at:128 * at + hi - lo]) * s[:, at:at + 1]
        assert np.abs(v - x[lo:hi].T).max() <= 2.0 ** -4 * np.abs(x[lo:hi]).max()
        assert (q[:, 128 * at + hi - lo:128 * at + 128] == 0).all()
    assert (q[:, 512:] == 7).all() and (s[:, 4:] == 9).all()
    # the same tile under 1x128 quantization: its scale is at most the power of two, and more than half of it
    _, plain = quant_1x128(np.ascontiguousarray(x[:128].T))
    assert (plain[:, 0] <= s[:, 0]).all() and (2 * plain[:, 0] > s[:, 0]).all()


def test_tiles_gather_by_order():
    x = RNG.standard_normal((5, 2)).astype(np.float32)
    order = np.array([9, 0, 3, -1, 10, 1])          # of 5 * 2 choices
    a, _, _ = train.tiles(x, [0, 6], order, 2, np.zeros((2, 128), np.uint8), np.zeros((2, 1), np.float32))
    zero = np.zeros(2)                                # a negative row times 0 would be -0, which has a code of its own
    rows = np.stack([x[4], x[0], x[1], zero, zero, x[0]])
    b, _, _ = train.tiles(rows, [0, 6], None, 1, np.zeros((2, 128), np.uint8), np.zeros((2, 1), np.float32))
    assert np.array_equal(a, b)


def test_offsets_that_fall_leave_disjoint_ranges():
    assert train.ranges([5, 3, 900, -2, 7], 10) == [(5, 5), (5, 10), (10, 10), (10, 10)]


def test_weight_gradient_brute_force():
    a, b = RNG.integers(-4, 5, (3, 384)).astype(float), RNG.integers(-4, 5, (2, 384)).astype(float)
    y, size, depth = train.wgrad([0, 128, 128, 384], a, b)
    assert depth == [128, 0, 256]
    for e, (lo, hi) in enumerate([(0, 128), (128, 128), (128, 384)]):
        for n in range(3):
            for k in range(2):
                assert y[e, n, k] == sum(a[n, p] * b[k, p] for p in range(lo, hi))
                assert size[e, n, k] == sum(abs(a[n, p] * b[k, p]) for p in range(lo, hi))


def test_gradient_norm():
    assert train.grad_norm([[3.0], [], [[4.0]]]) == 5.0
    assert train.grad_norm([np.full(4, 1e300 / 2 ** 510), np.zeros(2)]) > 0
