"""Mixture-of-experts routing: router, its gradient, dispatch, in float64.  TEST INFRASTRUCTURE ONLY (see the
package docstring)."""
import numpy as np

from .quantize import quant_1x128


def scores(x, kind):
    x = np.asarray(x, np.float64)
    if kind == "sigmoid":
        return 1 / (1 + np.exp(-x))
    e = np.exp(x - x.max(1, keepdims=True))
    return e / e.sum(1, keepdims=True)


def route(x, top_k, kind, bias, groups, top_groups, renorm, scale):
    """(ids, weights): the choice is made on float32 scores, ties to the lower index."""
    s = scores(x, kind)
    b = s.astype(np.float32)
    if bias is not None:
        b = b + bias.astype(np.float32)
    ids = np.empty((x.shape[0], top_k), np.int32)
    size = x.shape[1] // groups
    for t in range(x.shape[0]):
        marks = []
        for g in range(groups):
            two = sorted(b[t, g * size:(g + 1) * size], reverse=True)[:2]
            marks.append(np.float32(two[0] + two[1]) if size > 1 else two[0])
        keep = sorted(range(groups), key=lambda g: (-marks[g], g))[:top_groups]
        live = sorted((e for g in keep for e in range(g * size, (g + 1) * size)), key=lambda e: (-b[t, e], e))
        ids[t] = live[:top_k]
    w = np.take_along_axis(s, ids, 1)
    if renorm:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return ids, w * scale


def weights_at(x, ids, kind, renorm, scale):
    """The router's weights for a fixed choice: what the gradient is of."""
    w = np.take_along_axis(scores(x, kind), ids, 1)
    if renorm:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return w * scale


def route_grad(grad, x, ids, kind, renorm, scale):
    """Ids outside the experts have no weight; one that stands twice adds up."""
    s = scores(x, kind)
    d = np.zeros_like(s)
    for t in range(x.shape[0]):
        live = [(j, e) for j, e in enumerate(ids[t]) if 0 <= e < x.shape[1]]
        w = np.array([s[t, e] for _, e in live])
        g = np.array([grad[t, j] * scale for j, _ in live], np.float64)
        if renorm and len(live):
            total = w.sum() + 1e-20
            g = (g - (g * w / total).sum()) / total
        for (_, e), gi, wi in zip(live, g, w):
            d[t, e] += gi * wi * ((1 - wi) if kind == "sigmoid" else 1)
        if kind == "softmax":
            d[t] -= s[t] * (g * w).sum()
    return d


def dispatch(x, ids, experts):
    """(codes, scale, offsets, order, position) of float32 rows x."""
    t, k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    flat = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(flat, kind="stable").astype(np.int32)
    position = np.empty(t * k, np.int32)
    position[order] = np.arange(t * k)
    offsets = np.searchsorted(flat[order], np.arange(experts + 1)).astype(np.int32)
    codes, scale = quant_1x128(x)
    q, s = codes[order // k], scale[order // k]
    dead = flat[order] == experts
    q[dead], s[dead] = 0, 1.0
    return q, s, offsets, order, position.reshape(t, k)
