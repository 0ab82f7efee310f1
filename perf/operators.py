"""Cases of the operators around the FP8 GEMMs of one decoder layer: the 8-bit key/value cache (append and
attention) and the mixture-of-experts routing (router, its gradient, dispatch), with their plain forms.

Shared layout.  New tokens of all sequences are packed: sequence b owns rows cu[b] .. cu[b+1] of q, k and v.
seq_lens[b] counts the cached tokens including the new ones, so new token i of sequence b sits at position
seq_lens[b] - new_b + i.  Position p lives in page block_table[b, p // P] at offset p % P.  The cache holds E4M3
codes [pages, kv heads, P, head_dim] for keys and for values, and one power-of-two float32 scale per page and head.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
MIN_EXP = -32          # the smallest exponent of a cache scale
LOG2E = 1.4426950408889634


# --------------------------------------------------------------------------
# cases
def listed():
    return [
        # One token of each of 33 running sequences: the call that a decode step makes in every layer.
        dict(name="append_decode", op="append", batch=33, new=1, context=2000, q_heads=64, kv_heads=8, head_dim=128, page=64,
             rot=128, layout="half", norm=False),
        # Prompts of different lengths, packed: q and k normalised per head and rotated on the way.
        dict(name="append_prompts", op="append", batch=6, new=4096, context=6000, q_heads=64, kv_heads=8, head_dim=128, page=64,
             rot=128, layout="half", norm=True),
        # A single user's next token over a short history: nothing but latency.
        dict(name="attend_one", op="attend", batch=1, new=1, context=1025, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0),
        # A server's decode step: many sequences of different lengths.
        dict(name="attend_batch", op="attend", batch=64, new=1, context=8192, q_heads=64, kv_heads=8, head_dim=128, page=64, window=0),
        # One long document: the cache of a single sequence has to be split over the whole chip.
        dict(name="attend_long", op="attend", batch=1, new=1, context=100003, q_heads=64, kv_heads=8, head_dim=128, page=128, window=0),
        # Chunks of prompts over what earlier chunks left, with a sliding window and narrow heads.
        dict(name="attend_chunk", op="attend", batch=5, new=512, context=6000, q_heads=32, kv_heads=8, head_dim=64, page=16, window=4096),
        # Whole prompts, causal, packed.
        dict(name="attend_prompt", op="attend", batch=2, new=8192, context=8192, q_heads=32, kv_heads=8, head_dim=128, page=64, window=0),
        # The router in a decode step: sigmoid scores, balance bias, groups.
        dict(name="route_decode", op="route", tokens=32, experts=256, top_k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             renorm=True, scale=2.5, dtype="f32"),
        # The router over a training batch.
        dict(name="route_train", op="route", tokens=32768, experts=256, top_k=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             renorm=True, scale=2.5, dtype="f32"),
        # Its gradient, with softmax scores.
        dict(name="route_grad", op="route_grad", tokens=32768, experts=160, top_k=6, score="softmax", renorm=False, scale=1.0, dtype="bf16"),
        # A decode step's rows on their way to the experts.
        dict(name="dispatch_decode", op="dispatch", tokens=32, hidden=7168, experts=256, top_k=8),
        # A training batch's rows on their way to the experts.
        dict(name="dispatch_train", op="dispatch", tokens=8192, hidden=7168, experts=256, top_k=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 8e12 + w["flops"] / 2.5e15


def _draw(rng):
    op = rng.choice(["append", "append", "attend", "attend", "attend", "route", "route_grad", "dispatch"])
    if op in ("append", "attend"):
        dim, kv = rng.choice([64, 128]), rng.choice([1, 2, 4, 8])
        case = dict(op=op, batch=_log(rng, 1, 64), new=rng.choice([1, 1, rng.randint(2, 8), _log(rng, 9, 8192)]), context=0,
                    q_heads=kv * rng.choice([1, 2, 4, 5, 8, 16]), kv_heads=kv, head_dim=dim, page=rng.choice([16, 32, 64, 128]))
        case["context"] = max(case["new"], _log(rng, 1, 100003))
        if op == "append":
            case.update(rot=rng.choice([dim, dim, dim // 2, 0]), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.5)
        else:
            case["window"] = rng.choice([0, 0, 0, _log(rng, 16, 4096)])
        return case
    if op == "dispatch":
        return dict(op=op, tokens=_log(rng, 1, 8192), hidden=128 * _log(rng, 4, 64), experts=_log(rng, 4, 384), top_k=rng.randint(1, 8))
    groups = rng.choice([1, 1, 4, 8])
    experts = groups * _log(rng, 2, 384 // groups)
    top = rng.randint(1, groups)
    case = dict(op=op, tokens=_log(rng, 1, 32768), experts=experts, top_k=rng.randint(1, min(8, top * (experts // groups))),
                score=rng.choice(["sigmoid", "softmax"]), renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                dtype=rng.choice(["f32", "bf16"]))
    if op == "route":
        case.update(bias=rng.random() < 0.6, groups=groups, top_groups=top)
    else:
        case["top_k"] = min(8, experts, case["top_k"])
        case["renorm"] = case["renorm"] and case["top_k"] > 1      # one renormalised weight is 1: it has no gradient
    return case


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        case = _draw(rng)
        if case["op"] in ("append", "attend"):
            tokens = case["batch"] * case["context"] * case["kv_heads"] * case["head_dim"]
            scores = case["batch"] * case["new"] * case["context"] * case["q_heads"]
            if tokens > 64 * 8192 * 8 * 128 or (case["op"] == "attend" and scores > 2 * 8192 * 8192 * 32):
                continue
        if _cost(case) <= top[case["op"]]:
            return case


def _lengths(case):
    """New tokens and cached tokens (the new ones included) of each sequence: the first is the largest, the others vary,
    and in a larger batch one sequence has nothing new."""
    rng = random.Random("%(batch)d %(new)d %(context)d" % case)
    new, total = [case["new"]], [case["context"]]
    for b in range(1, case["batch"]):
        n = rng.randint(max(1, case["new"] // 4), case["new"])
        new.append(0 if b == 4 else n)
        total.append(rng.randint(max(n, case["context"] // 8), case["context"]))
    return new, total


def _visible(n, total, window):
    """Sum over the n last tokens of a sequence of `total` tokens of how many tokens each sees."""
    last = np.arange(total - n, total, dtype=np.int64) + 1
    return int(np.minimum(last, window).sum()) if window else int(last.sum())


def work(case):
    op = case["op"]
    if op in ("append", "attend"):
        new, total = _lengths(case)
        t, d, hq, hk = sum(new), case["head_dim"], case["q_heads"], case["kv_heads"]
        if op == "append":
            elems = t * d * (hq + 2 * hk)
            return {"bytes": 2 * elems + 2 * t * d * hq + 2 * t * d * hk + 4 * t * case["rot"] + 8 * hk * (t // case["page"] + 1),
                    "flops": 8 * elems}
        span = sum(min(L, case["window"] + n - 1) if case["window"] else L for n, L in zip(new, total) if n)
        return {"bytes": 2 * span * hk * d + 8 * hk * (span // case["page"]) + 4 * t * d * hq + 4 * t * hq,
                "flops": 4 * d * hq * sum(_visible(n, L, case["window"]) for n, L in zip(new, total))}
    t, k = case["tokens"], case["top_k"]
    if op == "dispatch":
        h = case["hidden"]
        return {"bytes": 2 * t * h + t * k * (h + h // 32 + 12), "flops": 4 * t * h}
    e, size = case["experts"], 4 if case["dtype"] == "f32" else 2
    if op == "route":
        return {"bytes": size * t * e + 8 * t * k, "flops": 16 * t * e}
    return {"bytes": size * t * e * (2 if case["score"] == "softmax" else 1) + 8 * t * k, "flops": 16 * t * e}


# --------------------------------------------------------------------------
# inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape, outliers=0.0):
    x = torch.randn(*shape, generator=g, device=DEV)
    if outliers:
        x *= torch.where(torch.rand(*shape, generator=g, device=DEV) < outliers, 20.0, 1.0)
    return x


def _angles(rows, rot):
    """cos | sin of position * 10000^(-2i/rot), taken in 64 bits."""
    if not rot:
        return None
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(rows, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _cache(case, g):
    new, total = _lengths(case)
    width = -(-max(total) // case["page"])
    used = [-(-x // case["page"]) for x in total]
    pages = sum(used) + 3
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32).cpu()
    table, at = torch.full((case["batch"], width), -1, dtype=torch.int32), 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    s = dict(case=case, table=table.to(DEV), max_new=max(new), max_len=max(total),
             cu=torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device=DEV),
             lens=torch.tensor(total, dtype=torch.int32, device=DEV))
    for name in ("k", "v"):
        s[name + "_cache"] = (torch.randn(*shape, generator=g, device=DEV) * 64).clamp_(-448, 448).to(E4M3).view(torch.uint8)
        s[name + "_scale"] = torch.exp2(torch.randint(-7, -4, shape[:2], generator=g, device=DEV).float())
    return s, sum(new)


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    if op in ("append", "attend"):
        s, t = _cache(case, g)
        hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
        if op == "attend":
            s["q"] = _normal(g, t, hq, d).bfloat16()
            return s
        # q, k and v are slices of one projection's output, as a fused linear layer leaves them
        qkv = _normal(g, t, (hq + 2 * hk) * d, outliers=0.001).bfloat16()
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["new_k"] = qkv[:, hq * d:(hq + hk) * d].unflatten(1, (hk, d))
        s["new_v"] = qkv[:, (hq + hk) * d:].unflatten(1, (hk, d))
        s["rope"] = _angles(s["table"].shape[1] * case["page"], case["rot"])
        for name in ("q_weight", "k_weight"):
            s[name] = (1 + 0.1 * _normal(g, d)).bfloat16() if case["norm"] else None
        return s
    t, k = case["tokens"], case["top_k"]
    s = dict(case=case)
    if op == "dispatch":
        # some experts are asked for far more often than others; one token in 50 is padding
        e = case["experts"]
        liking = 2.0 * torch.randn(1, e, generator=g, device=DEV) + torch.randn(t, e, generator=g, device=DEV)
        s["ids"] = liking.argsort(1, descending=True)[:, :k].to(torch.int32)
        if e < k:
            s["ids"] = torch.cat([s["ids"], torch.full((t, k - e), -1, dtype=torch.int32, device=DEV)], 1)
        s["ids"][torch.rand(t, generator=g, device=DEV) < 0.02] = -1
        s["ids"] = s["ids"].contiguous()
        s["x"] = _normal(g, t, case["hidden"], outliers=0.001).bfloat16()
        return s
    e = case["experts"]
    s["logits"] = 2.0 * _normal(g, t, e)
    if case["dtype"] == "bf16":
        s["logits"] = s["logits"].bfloat16()
    if op == "route":
        s["bias"] = 0.05 * _normal(g, e) if case["bias"] else None
    else:
        s["ids"] = (s["logits"].float() + _normal(g, t, e)).argsort(1, descending=True)[:, :k].to(torch.int32).contiguous()
        s["grad"] = _normal(g, t, k)
    return s


# --------------------------------------------------------------------------
# the framework's calls
def _run_own(s):
    import fp8_block_scaled_05_amd as fb
    c = s["case"]
    if c["op"] in ("append", "attend"):
        cache = fb.KVCache(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        if c["op"] == "attend":
            return fb.fp8_kv_attention(s["q"], cache, s["cu"], s["lens"], s["table"], s["max_new"], s["max_len"], window=c["window"],
                                       return_lse=True)
        q = fb.fp8_kv_append(s["q"], s["new_k"], s["new_v"], cache, s["cu"], s["lens"], s["table"], s["max_new"], rope=s["rope"],
                             rope_layout=c["layout"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=1e-6)
        return q, s["k_cache"].view(E4M3), s["v_cache"].view(E4M3), s["k_scale"], s["v_scale"]
    if c["op"] == "route":
        return fb.fp8_moe_route(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], groups=c["groups"], top_groups=c["top_groups"],
                                renormalize=c["renorm"], scale=c["scale"])
    if c["op"] == "route_grad":
        return fb.fp8_moe_route_backward(s["grad"], s["logits"], s["ids"], score=c["score"], renormalize=c["renorm"], scale=c["scale"])
    q, scale, offsets, order, position = fb.fp8_moe_dispatch(s["x"], s["ids"], c["experts"])
    return q.view(E4M3), scale, offsets, order, position


# --------------------------------------------------------------------------
# the plain forms
def _owner(s, tokens):
    """Sequence and position of each packed new token."""
    at = torch.arange(tokens, device=DEV)
    b = torch.searchsorted(s["cu"][1:].contiguous(), at.to(torch.int32), right=True)
    cu, lens = s["cu"].long(), s["lens"].long()
    return b, lens[b] - (cu[b + 1] - at)


def _normed(x, weight, eps):
    x = x.float()
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * weight.float()


def _rotated(x, angles, layout):
    if angles is None:
        return x
    r = angles.shape[1]
    c, s = angles[:, None, :r // 2], angles[:, None, r // 2:]
    if layout == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat([a * c - b * s, b * c + a * s, x[..., r:]], -1)
    a, b = x[..., :r:2], x[..., 1:r:2]
    return torch.cat([torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), x[..., r:]], -1)


def _exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), MIN_EXP).clamp(min=MIN_EXP)


def _store(codes, scale, y, page, off, first):
    """New rows y [tokens, heads, dim] into their pages, with the pages' scales grown where they have to."""
    pages, heads, size, _ = codes.shape
    amax = torch.zeros(pages, heads, device=DEV).scatter_reduce_(0, page[:, None].expand(-1, heads), y.abs().amax(-1), "amax")
    older = page[first]                                   # pages that hold older tokens before these
    held = torch.zeros(pages, dtype=torch.bool, device=DEV)
    held[older] = True
    touched = torch.zeros(pages, dtype=torch.bool, device=DEV)
    touched[page] = True
    e_old = torch.where(held[:, None], torch.frexp(scale)[1] - 1, MIN_EXP)
    e_new = torch.maximum(_exponent(amax), e_old)
    was = codes[older].view(E4M3).float() * torch.exp2((e_old - e_new)[older].float())[..., None, None]
    keep = torch.arange(size, device=DEV)[None, :] < off[first][:, None]
    codes[older] = torch.where(keep[:, None, :, None], was.to(E4M3).view(torch.uint8), codes[older])
    scale.copy_(torch.where(touched[:, None], torch.exp2(e_new.float()), scale))
    z = y * torch.exp2(-e_new[page].float())[..., None]
    codes[page, :, off] = z.to(E4M3).view(torch.uint8)


def _append(s):
    c = s["case"]
    t = s["q"].shape[0]
    b, pos = _owner(s, t)
    page, off = s["table"][b, pos // c["page"]].long(), pos % c["page"]
    angles = s["rope"][pos] if s["rope"] is not None else None
    q = _rotated(_normed(s["q"], s["q_weight"], 1e-6), angles, c["layout"])
    k = _rotated(_normed(s["new_k"], s["k_weight"], 1e-6), angles, c["layout"])
    first = ((torch.arange(t, device=DEV) == s["cu"].long()[b]) & (off > 0)).nonzero()[:, 0]
    _store(s["k_cache"], s["k_scale"], k, page, off, first)
    _store(s["v_cache"], s["v_scale"], s["new_v"].float(), page, off, first)
    return q.bfloat16(), s["k_cache"].view(E4M3), s["v_cache"].view(E4M3), s["k_scale"], s["v_scale"]


def _gathered(s, name):
    """A batch's keys or values as float32 [batch, kv heads, positions, dim]."""
    idx = s["table"].clamp(min=0).long()
    x = s[name + "_cache"][idx].view(E4M3).float() * s[name + "_scale"][idx][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attend(s):
    c = s["case"]
    t, hq, d = s["q"].shape
    hk, n = c["kv_heads"], s["max_new"]
    b, pos = _owner(s, t)
    row = torch.arange(t, device=DEV) - s["cu"].long()[b]
    q = torch.zeros(c["batch"], n, hq, d, device=DEV)
    q[b, row] = s["q"].float()
    last = torch.full((c["batch"], n), -1, dtype=torch.long, device=DEV)
    last[b, row] = pos
    q = q.unflatten(2, (hk, hq // hk)).permute(0, 2, 3, 1, 4).flatten(2, 3)              # [batch, kv heads, G * new, dim]
    k, v = _gathered(s, "k"), _gathered(s, "v")
    z = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(1 / math.sqrt(d)).unflatten(2, (hq // hk, n))
    at = torch.arange(k.shape[2], device=DEV)
    hidden = at > last[..., None]
    if c["window"]:
        hidden |= at <= last[..., None] - c["window"]
    z.masked_fill_(hidden[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-3e38)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (hq // hk, n)) / torch.where(l > 0, l, 1.0)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, row]
    lse = (m + l.log())[..., 0].permute(0, 3, 1, 2).flatten(2, 3)[b, row]
    return o.bfloat16(), lse


def _scores(x, kind):
    """Scores rounded once from 64 bits to 32, so that the order of experts does not hang on how an exponential is computed."""
    x = x.double()
    if kind == "sigmoid":
        return (1 / (1 + torch.exp(-x))).float()
    e = torch.exp(x - x.amax(1, keepdim=True))
    return (e / e.sum(1, keepdim=True)).float()


def _route(s):
    c, x = s["case"], s["logits"].float()
    score = _scores(x, c["score"])
    b = score + s["bias"] if s["bias"] is not None else score
    if c["groups"] > 1:
        by = b.unflatten(1, (c["groups"], -1))
        two = by.sort(2, descending=True)[0][..., :2].sum(2)
        best = two.sort(dim=1, descending=True, stable=True)[1][:, :c["top_groups"]]
        keep = torch.zeros_like(two, dtype=torch.bool).scatter_(1, best, True)
        b = by.masked_fill(~keep[..., None], -math.inf).flatten(1)
    ids = b.sort(dim=1, descending=True, stable=True)[1][:, :c["top_k"]]
    w = score.gather(1, ids)
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return ids.to(torch.int32), w * c["scale"]


def _route_grad(s):
    c, x, ids = s["case"], s["logits"].float(), s["ids"].long()
    score = x.sigmoid() if c["score"] == "sigmoid" else x.softmax(1)
    w, g = score.gather(1, ids), s["grad"] * c["scale"]
    if c["renorm"]:
        total = w.sum(1, keepdim=True) + 1e-20
        g = (g - (g * w / total).sum(1, keepdim=True)) / total
    if c["score"] == "sigmoid":
        d = torch.zeros_like(x).scatter_(1, ids, g * w * (1 - w))
    else:
        d = torch.zeros_like(x).scatter_(1, ids, g * w) - score * (g * w).sum(1, keepdim=True)
    return d.to(s["logits"].dtype)


def _dispatch(s):
    c, ids = s["case"], s["ids"].flatten()
    e, k = c["experts"], c["top_k"]
    key = torch.where((ids >= 0) & (ids < e), ids, e).long()
    order = key.sort(dim=0, stable=True)[1]
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=DEV)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.bincount(key, minlength=e + 1)[:e].cumsum(0)
    x = s["x"].float().unflatten(1, (-1, 128))
    scale = x.abs().amax(-1) / torch.full((1, 1), 448.0, device=DEV)
    scale = torch.where(scale > 1e-10, scale, 1.0)
    codes = (x / scale[..., None]).to(E4M3).flatten(1).view(torch.uint8)
    lives = key[order] < e
    codes = torch.where(lives[:, None], codes[order // k], 0)
    scale = torch.where(lives[:, None], scale[order // k], 1.0)
    return codes.view(E4M3), scale, offsets, order.to(torch.int32), position.to(torch.int32).unflatten(0, (-1, k))


def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "attend": _attend, "route": _route, "route_grad": _route_grad, "dispatch": _dispatch}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
def _to_e4m3(x):
    """The E4M3 value nearest to each 64-bit x, ties to even, largest 448."""
    e = (torch.frexp(x)[1] - 1).clamp(min=-6).double()
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(s):
    c = s["case"]
    new, total = _lengths(c)
    d, r, size = c["head_dim"], c["rot"], c["page"]
    q, k, v = s["q"].double(), s["new_k"].double(), s["new_v"].double()
    if c["norm"]:
        q = q / torch.sqrt((q * q).sum(-1, keepdim=True) / d + 1e-6) * s["q_weight"].double()
        k = k / torch.sqrt((k * k).sum(-1, keepdim=True) / d + 1e-6) * s["k_weight"].double()
    pos = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(new, total)])
    if r:
        z = torch.complex(s["rope"][pos, :r // 2].double(), s["rope"][pos, r // 2:].double())[:, None]
        pairs = (lambda x: (x[..., :r // 2], x[..., r // 2:r])) if c["layout"] == "half" else (lambda x: (x[..., 0:r:2], x[..., 1:r:2]))
        for x in (q, k):
            a, b = pairs(x)
            turned = torch.complex(a, b) * z
            re, im = turned.real.clone(), turned.imag.clone()
            a.copy_(re), b.copy_(im)
    out = [q]
    table, at = s["table"].cpu().tolist(), 0
    state = []
    for name, y in (("k", k), ("v", v)):
        value, scale = s[name + "_cache"].view(E4M3).double(), s[name + "_scale"].double()
        state.append((value, scale, y))
    for b, (n, L) in enumerate(zip(new, total)):
        p = L - n
        while p < L:
            stop = min(L, (p // size + 1) * size)
            page, o, m = table[b][p // size], p % size, stop - p
            for value, scale, y in state:
                part = y[at:at + m].transpose(0, 1)                                        # [heads, m, dim]
                e = torch.ceil(torch.log2(part.abs().amax((1, 2)) / 448.0)).clamp(min=MIN_EXP)
                e = torch.where(torch.exp2(e - 1) * 448.0 >= part.abs().amax((1, 2)), (e - 1).clamp(min=MIN_EXP), e)
                if o:
                    e = torch.maximum(e, torch.log2(scale[page]).round())
                    value[page, :, :o] = _to_e4m3(value[page, :, :o] * (scale[page] / torch.exp2(e))[:, None, None])
                scale[page] = torch.exp2(e)
                value[page, :, o:o + m] = _to_e4m3(part * torch.exp2(-e)[:, None, None])
            at, p = at + m, stop
    (kv, ks, _), (vv, vs, _) = state
    return out + [kv, vv, ks, vs]


def _exact_attend(s):
    c = s["case"]
    new, total = _lengths(c)
    hq, hk, d, size = c["q_heads"], c["kv_heads"], c["head_dim"], c["page"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full((s["q"].shape[0], hq), -math.inf, dtype=torch.float64, device=DEV)
    at = 0
    for b, (n, L) in enumerate(zip(new, total)):
        if not n:
            continue
        pages = s["table"][b, :-(-L // size)].long()
        kv = [(s[x + "_cache"][pages].view(E4M3).double() * s[x + "_scale"][pages].double()[..., None, None])
              .permute(1, 0, 2, 3).reshape(hk, -1, d)[:, :L] for x in ("k", "v")]
        seen = torch.arange(L, device=DEV)[None, :]
        mine = torch.arange(L - n, L, device=DEV)[:, None]
        ok = (seen <= mine) & ((mine - seen < c["window"]) if c["window"] else True)
        for h in range(hq):
            for lo in range(0, n, 2048):
                rows = slice(at + lo, at + min(n, lo + 2048))
                z = s["q"][rows, h].double() @ kv[0][h // (hq // hk)].t() / math.sqrt(d)
                z = torch.where(ok[lo:lo + 2048], z, -math.inf)
                lse[rows, h] = torch.logsumexp(z, 1)
                o[rows, h] = torch.exp(z - lse[rows, h][:, None]) @ kv[1][h // (hq // hk)]
        at += n
    return o, lse


def _exact_route(s):
    c = s["case"]
    x = s["logits"].double().cpu().numpy()
    if c["score"] == "sigmoid":
        score = 1 / (1 + np.exp(-x))
    else:
        score = np.exp(x - x.max(1, keepdims=True))
        score /= score.sum(1, keepdims=True)
    b = score.astype(np.float32)
    if s["bias"] is not None:
        b = b + s["bias"].cpu().numpy()
    t, e = b.shape
    if c["groups"] > 1:
        by = b.reshape(t, c["groups"], -1)
        two = np.sort(by, 2)[..., -2:]
        two = (two[..., 1] + two[..., 0]) if by.shape[2] > 1 else two[..., 0]
        rank = np.argsort(np.argsort(-two, 1, kind="stable"), 1, kind="stable")
        b = np.where((rank < c["top_groups"])[..., None], by, -np.inf).reshape(t, e)
    ids = np.argsort(-b, 1, kind="stable")[:, :c["top_k"]]
    w = np.take_along_axis(score, ids, 1)
    if c["renorm"]:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return None, torch.from_numpy(w * c["scale"])


def _exact_route_grad(s):
    c = s["case"]
    x = s["logits"].double().requires_grad_(True)
    with torch.enable_grad():
        score = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
        w = torch.gather(score, 1, s["ids"].long())
        if c["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        (w * c["scale"] * s["grad"].double()).sum().backward()
    return x.grad


def _exact_dispatch(s):
    c = s["case"]
    k, e = c["top_k"], c["experts"]
    ids = s["ids"].flatten().cpu().numpy()
    order = np.concatenate([np.flatnonzero(ids == j) for j in range(e)] + [np.flatnonzero((ids < 0) | (ids >= e))])
    lives = torch.from_numpy((ids[order] >= 0) & (ids[order] < e)).to(DEV)
    x = s["x"].double().unflatten(1, (-1, 128))
    scale = x.abs().amax(-1) / 448.0
    scale = torch.where(scale > 1e-10, scale, 1.0)
    codes = _to_e4m3((x / scale.float().double()[..., None]).float().double()).flatten(1)     # the quotient is defined in 32 bits
    token = torch.from_numpy(order // k).to(DEV)
    return codes[token].mul_(lives[:, None]), torch.where(lives[:, None], scale[token], 1.0), None, None, None


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"append": _exact_append, "attend": _exact_attend, "route": _exact_route, "route_grad": _exact_route_grad,
                "dispatch": _exact_dispatch}[case["op"]](s)
