"""The paged 8-bit key/value cache: append (norm, rotation, E4M3 store with one power-of-two scale per page
and head) and causal attention over it, in float64.  TEST INFRASTRUCTURE ONLY (see the package docstring).

Sequences: sequence b owns rows cu[b] .. cu[b+1]; its new token i has position lens[b] - new_b + i; position p
lives in page table[b][p // P] at offset p % P.
"""
import math

import numpy as np

from .e4m3 import e4m3_decode, e4m3_encode

MIN_EXP = -32


def norm(x, weight, eps):
    x = np.asarray(x, np.float64)
    if weight is None:
        return x
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rotate(x, angles, layout):
    """x [..., D], angles [..., rot] = cos | sin, broadcast over heads."""
    if angles is None:
        return x
    rot = angles.shape[-1]
    c, s = angles[..., :rot // 2].astype(np.float64), angles[..., rot // 2:].astype(np.float64)
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    y = x.copy()
    y[..., first] = x[..., first] * c - x[..., second] * s
    y[..., second] = x[..., second] * c + x[..., first] * s
    return y


def exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    e = MIN_EXP
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def rows_of(cu, lens):
    """(row, sequence, position) of every new token."""
    return [(cu[b] + i, b, int(lens[b]) - (cu[b + 1] - cu[b]) + i) for b in range(len(lens)) for i in range(cu[b + 1] - cu[b])]


def treat(x, weight, eps, rope, layout, cu, lens):
    """Normed and rotated rows [T, heads, D] in float64."""
    y = norm(x, weight, eps)
    if rope is None:
        return y
    for r, _, p in rows_of(cu, lens):
        y[r] = rotate(y[r], rope[p][None], layout)
    return y


def append(codes, scale, y, cu, lens, table, size):
    """Stores rows y [T, heads, D] into copies of codes [pages, heads, P, D] and scale [pages, heads]."""
    codes, scale = codes.copy(), scale.copy()
    for b in range(len(lens)):
        n = int(cu[b + 1] - cu[b])
        start = int(lens[b]) - n
        for p0 in [start] + list(range((start // size + 1) * size, int(lens[b]), size)) if n else []:
            p1 = min(int(lens[b]), (p0 // size + 1) * size)
            page, off = int(table[b][p0 // size]), p0 % size
            for h in range(codes.shape[1]):
                part = y[cu[b] + p0 - start:cu[b] + p1 - start, h]
                e = exponent(np.abs(part).max())
                if off:
                    old = int(math.log2(scale[page, h]))
                    if old >= e:
                        e = old
                    else:
                        codes[page, h, :off] = e4m3_encode((e4m3_decode(codes[page, h, :off]) * 2.0 ** (old - e)).astype(np.float32))
                scale[page, h] = np.float32(2.0) ** e
                codes[page, h, off:off + p1 - p0] = e4m3_encode((part * 2.0 ** -e).astype(np.float32))
    return codes, scale


def attention(q, k_codes, v_codes, k_scale, v_scale, cu, lens, table, size, window, softmax_scale):
    """(out [T, Hq, D], lse [T, Hq], weight of |v| [T, Hq, D], largest sum |q k| scale [T, Hq]) in float64."""
    t, hq, d = q.shape
    hk = k_codes.shape[1]
    out, lse = np.zeros((t, hq, d)), np.full((t, hq), -np.inf)
    absv, absz = np.zeros((t, hq, d)), np.zeros((t, hq))
    for r, b, p in rows_of(cu, lens):
        lo = max(0, p - window + 1) if window else 0
        at = np.arange(lo, p + 1)
        page, off = table[b][at // size], at % size
        for h in range(hq):
            g = h // (hq // hk)
            k = e4m3_decode(k_codes[page, g, off]).astype(np.float64) * k_scale[page, g][:, None]
            v = e4m3_decode(v_codes[page, g, off]).astype(np.float64) * v_scale[page, g][:, None]
            z = k @ q[r, h].astype(np.float64) * softmax_scale
            w = np.exp(z - z.max())
            lse[r, h] = z.max() + math.log(w.sum())
            w /= w.sum()
            out[r, h] = w @ v
            absv[r, h] = w @ np.abs(v)
            absz[r, h] = (np.abs(k) @ np.abs(q[r, h].astype(np.float64))).max() * abs(softmax_scale)
    return out, lse, absv, absz
