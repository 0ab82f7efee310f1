"""The operators of a training step: norm, gated activation and their gradients, transposed tiles of experts' rows, weight
gradients, gradient norm, in float64.  TEST INFRASTRUCTURE ONLY (see the package docstring)."""
import math

import numpy as np

from .e4m3 import e4m3_decode, e4m3_encode

MIN_EXP, TOP_EXP = -100, 120            # at the top codes end at 240: 256 * 2^120 is beyond float32


def rmsnorm(h, weight, eps):
    h = np.asarray(h, np.float64)
    y = h / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, np.float64)


def rmsnorm_grad(dy, h, weight, eps, dresidual=None):
    """(dx, dweight, and the sums of magnitudes behind each: what their rounding errors are measured against)."""
    h, dy = np.asarray(h, np.float64), np.asarray(dy, np.float64)
    g = dy if weight is None else dy * np.asarray(weight, np.float64)
    r = 1 / np.sqrt((h * h).mean(1, keepdims=True) + eps)
    dx = r * (g - h * r * r * (g * h).mean(1, keepdims=True))
    size = r * (np.abs(g) + np.abs(h) * r * r * np.abs(g * h).mean(1, keepdims=True))
    if dresidual is not None:
        dx = dx + dresidual
        size = size + np.abs(dresidual)
    return dx, (dy * h * r).sum(0), size, np.abs(dy * h * r).sum(0)


def sigmoid(x):
    """Without overflow on either side."""
    x = np.asarray(x, np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1 / (1 + e), e / (1 + e))


def swiglu(gate, up):
    return np.asarray(gate, np.float64) * sigmoid(gate) * np.asarray(up, np.float64)


def swiglu_grad(dy, gate, up):
    """(d gate | d up, and the magnitude of the terms behind each)."""
    g, u, dy = (np.asarray(v, np.float64) for v in (gate, up, dy))
    s, rest = sigmoid(g), sigmoid(-g)
    return (np.concatenate([dy * u * s * (1 + g * rest), dy * g * s], 1),
            np.concatenate([np.abs(dy * u) * s * (1 + np.abs(g) * rest), np.abs(dy * g) * s], 1))


def ranges(off, places):
    """Each expert's [lo, hi) of an offset table that may hold anything."""
    out, end = [], 0
    for e in range(len(off) - 1):
        lo = max(end, min(max(int(off[e]), 0), places))
        hi = max(lo, min(max(int(off[e + 1]), 0), places))
        out.append((lo, hi))
        end = hi
    return out


def exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    e = MIN_EXP
    while amax > math.ldexp(448.0, e):
        e += 1
    return e


def tiles(x, off, order, top_k, q, scale):
    """(q, scale, padded): copies of q [cols, columns] and scale [cols, columns / 128] with the experts' tiles written."""
    x, q, scale = np.asarray(x, np.float64), q.copy(), scale.copy()
    places = len(x) if order is None else len(order)
    padded = [0]
    for lo, hi in ranges(off, places):
        at = padded[-1]
        for p0 in range(lo, hi, 128):
            block = np.zeros((128, x.shape[1]))
            for i, p in enumerate(range(p0, min(p0 + 128, hi))):
                row = p if order is None else (int(order[p]) // top_k if order[p] >= 0 else -1)
                if 0 <= row < len(x):
                    block[i] = x[row]
            for c in range(x.shape[1]):
                amax = np.abs(block[:, c]).max()
                e = exponent(amax) if amax > 0 else 0
                most = 448 if e < TOP_EXP else 240
                q[c, at:at + 128] = e4m3_encode(np.clip(block[:, c] * 2.0 ** -e, -most, most).astype(np.float32))
                scale[c, at // 128] = 2.0 ** e
            at += 128
        padded.append(at)
    return q, scale, np.array(padded, np.int32)


def values(codes, scale):
    """Codes [rows, columns] times their 128-wide tiles' scales."""
    v = e4m3_decode(codes).astype(np.float64)
    return (v.reshape(len(codes), -1, 128) * np.asarray(scale, np.float64)[:, :, None]).reshape(codes.shape)


def wgrad(padded, a, b):
    """(y [experts, N, K], the sums of products' magnitudes, the depths) of operand values a [N, P], b [K, P]."""
    y, size, depth = [], [], []
    at = np.clip(np.asarray(padded, np.int64) // 128, 0, a.shape[1] // 128).tolist()
    for lo, hi in ((p, max(p, q)) for p, q in zip(at, at[1:])):
        u, v = a[:, 128 * lo:128 * hi], b[:, 128 * lo:128 * hi]
        y.append(u @ v.T)
        size.append(np.abs(u) @ np.abs(v).T)
        depth.append(128 * (hi - lo))
    return np.stack(y), np.stack(size), depth


def grad_norm(grads):
    return math.sqrt(math.fsum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
