"""Cases of the operators of a training step around the FP8 GEMMs of one mixture-of-experts layer, with their plain forms:
the norm in front of a GEMM and its gradient, the gated activation between an expert's two GEMMs and its gradient, the
experts' weight gradients over ragged numbers of tokens, and the norm of all gradients with their clipping.

Shared layout.  8-bit outputs are E4M3 codes.  1x128 tiles have the scale amax / 448 (1 where that is not above 1e-10).
The operands of the weight gradients are transposed and tiled 128x1 along each expert's own rows: expert e's rows start at
column padded[e] = 128 * sum over f < e of ceil(rows of f / 128), the rest of its last tile is zero, and a tile's scale is
the smallest power of two, 2^e with e >= -100, under which its largest value fits 448 (1 for a tile of zeros).
"""
import math
import random

import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
MIN_EXP = -100
EPS = 1e-6


# --------------------------------------------------------------------------
# cases
def listed():
    return [
        # A decode step's tokens in front of a projection: residual added, normalised, quantized.  Latency.
        dict(name="norm_decode", op="norm", rows=32, cols=7168, dtype="bf16", residual=True, weight="bf16", y=False, q=True),
        # A training batch in front of the router and the experts: the normalised rows in both types.
        dict(name="norm_train", op="norm", rows=16387, cols=7168, dtype="bf16", residual=True, weight="bf16", y=True, q=True),
        # Its gradient: what comes down the residual stream joins, the weight's gradient is summed over the rows.
        dict(name="norm_grad", op="norm_grad", rows=8195, cols=7168, dtype="bf16", residual=True, weight="bf16"),
        # The rows of a decode step between an expert's two GEMMs.
        dict(name="act_decode", op="act", rows=256, cols=2048, dtype="bf16", y=False, q=True),
        # A training batch's rows there.
        dict(name="act_train", op="act", rows=32768, cols=2048, dtype="bf16", y=True, q=True),
        # Their gradient, quantized for the next GEMM and in 16 bits for the weight gradient.
        dict(name="act_grad", op="act_grad", rows=32768, cols=2048, dtype="bf16", d=True, q=True),
        # Few rows over many experts, some without any: tiles that are mostly padding, float32 rows.
        dict(name="tiles_odd", op="tiles", rows=1001, cols=2048, groups=64, dtype="f32", top_k=0),
        # A training batch's tokens, gathered into the order of their experts on the way.
        dict(name="tiles_train", op="tiles", rows=32768, cols=7168, groups=16, dtype="bf16", top_k=8),
        # Weight gradients of small experts.
        dict(name="wgrad_odd", op="wgrad", rows=1001, groups=32, n=512, k=1040, dtype="bf16"),
        # Weight gradients of one training batch over the experts of a rank.
        dict(name="wgrad_train", op="wgrad", rows=32768, groups=16, n=4096, k=7168, dtype="f32"),
        # The gradients of many layers: matrices, vectors, odd lengths.
        dict(name="grads_norm", op="grads", tensors=400, largest=7168 * 2048, dtype="f32", clip=False),
        # Gradients that are too long: the norm, then their scaling.
        dict(name="grads_clip", op="grads", tensors=48, largest=7168 * 4096, dtype="bf16", clip=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return w["bytes"] / 8e12 + w["flops"] / 2.5e15


def _draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "act", "act_grad", "tiles", "wgrad", "wgrad", "grads"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("norm", "norm_grad"):
        case = dict(op=op, rows=_log(rng, 1, 32768), cols=128 * _log(rng, 1, 128), dtype=dtype, residual=rng.random() < 0.7,
                    weight=rng.choice(["bf16", "f32", "none"]))
        if op == "norm":
            case["y"], case["q"] = rng.choice([(False, True), (True, True), (True, False)])
        return case
    if op in ("act", "act_grad"):
        case = dict(op=op, rows=_log(rng, 1, 65536), cols=128 * _log(rng, 1, 144), dtype=dtype)
        case["y" if op == "act" else "d"], case["q"] = rng.choice([(False, True), (True, True), (True, False)])
        return case
    if op == "tiles":
        return dict(op=op, rows=_log(rng, 1, 65536), cols=128 * _log(rng, 1, 56), groups=_log(rng, 1, 256), dtype=dtype,
                    top_k=rng.choice([0, 0, 1, 2, 6, 8]))
    if op == "wgrad":
        return dict(op=op, rows=_log(rng, 1, 32768), groups=_log(rng, 1, 128), n=16 * _log(rng, 4, 448), k=16 * _log(rng, 4, 448),
                    dtype=rng.choice(["f32", "f32", "bf16"]))
    clip = rng.random() < 0.5
    return dict(op=op, tensors=_log(rng, 1, 48 if clip else 800), largest=_log(rng, 100, 7168 * 4096), dtype=dtype, clip=clip)


def draw(rng):
    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    while True:
        case = _draw(rng)
        if case["op"] == "wgrad" and case["groups"] * _longest(case) > 4 * (case["rows"] + 128 * case["groups"]):
            continue                  # the plain form's padding
        if _cost(case) <= top[case["op"]]:
            return case


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def _counts(case):
    """Rows of each group, as from a router: some groups have many, one in five none."""
    rng = random.Random("%(rows)d %(groups)d" % case)
    liking = [0.0 if e % 5 == 3 else math.exp(0.5 * rng.gauss(0, 1)) for e in range(case["groups"])]
    total, at, out = sum(liking), 0.0, []
    for v in liking:
        at += v
        out.append(round(case["rows"] * at / total) - sum(out))
    return out


def _blocks(case):
    return sum(-(-n // 128) for n in _counts(case))


def _longest(case):
    return 128 * max(-(-n // 128) for n in _counts(case))


def _lengths(case):
    """Elements of each tensor: the first is the largest, every third is a vector of odd length."""
    rng = random.Random("%(tensors)d %(largest)d" % case)
    out = [case["largest"]]
    for i in range(1, case["tensors"]):
        out.append(rng.randint(1, 16384) if i % 3 == 0 else _log(rng, max(1, case["largest"] // 64), case["largest"]))
    return out


def work(case):
    op = case["op"]
    if op == "norm":
        t, e, s = case["rows"] * case["cols"], case["rows"] * case["cols"] // 128, _size(case["dtype"])
        b = t * s * (1 + 2 * case["residual"] + case["y"]) + (t + 4 * e) * case["q"]
        return {"bytes": b + _weight_bytes(case), "flops": 8 * t}
    if op == "norm_grad":
        t, s = case["rows"] * case["cols"], _size(case["dtype"])
        return {"bytes": t * s * (3 + case["residual"]) + 2 * _weight_bytes(case), "flops": 12 * t}
    if op == "act":
        t, s = case["rows"] * case["cols"], _size(case["dtype"])
        return {"bytes": t * s * (2 + case["y"]) + (t + t // 32) * case["q"], "flops": 10 * t}
    if op == "act_grad":
        t, s = case["rows"] * case["cols"], _size(case["dtype"])
        return {"bytes": t * s * (3 + 2 * case["d"]) + 2 * (t + t // 32) * case["q"], "flops": 20 * t}
    if op == "tiles":
        rows = -(-case["rows"] // max(1, case["top_k"]))           # a token is read once, however many experts take it
        blocks = _blocks(case)
        return {"bytes": rows * case["cols"] * _size(case["dtype"]) + 132 * blocks * case["cols"] + 4 * case["rows"] * (case["top_k"] > 0),
                "flops": 4 * case["rows"] * case["cols"]}
    if op == "wgrad":
        n, k, depth = case["n"], case["k"], 128 * _blocks(case)
        return {"bytes": (n + k) * (depth + depth // 32) + case["groups"] * n * k * _size(case["dtype"]), "flops": 2 * n * k * case["rows"]}
    total = sum(_lengths(case))
    return {"bytes": total * _size(case["dtype"]) * (3 if case["clip"] else 1), "flops": total * (3 if case["clip"] else 2)}


def _weight_bytes(case):
    return 0 if case["weight"] == "none" else case["cols"] * _size(case["weight"])


# --------------------------------------------------------------------------
# inputs
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 104729 + 11)
    return g


def _type(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _normal(g, *shape, outliers=0.0, dtype="f32"):
    x = torch.randn(*shape, generator=g, device=DEV)
    if outliers:
        x *= torch.where(torch.rand(*shape, generator=g, device=DEV) < outliers, 20.0, 1.0)
    return x.to(_type(dtype))


def _operand(g, rows, blocks):
    """Codes [rows, 128 * blocks] and power-of-two scales [rows, blocks] of a weight gradient's operand."""
    codes = (torch.randn(rows, 128 * blocks, generator=g, device=DEV) * 80).clamp_(-448, 448).to(E4M3).view(torch.uint8)
    return codes, torch.exp2(torch.randint(-12, -7, (rows, blocks), generator=g, device=DEV).float())


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = dict(case=case)
    if op in ("norm", "norm_grad"):
        t, n, dt = case["rows"], case["cols"], case["dtype"]
        # the weight's values stand for a trained norm's: around 1
        s["weight"] = None if case["weight"] == "none" else (1 + 0.2 * _normal(g, n)).to(_type(case["weight"]))
        s["x"] = _normal(g, t, n, outliers=0.001, dtype=dt)
        if op == "norm":
            s["residual"] = _normal(g, t, n, outliers=0.001, dtype=dt) if case["residual"] else None
        else:
            s["dy"] = (1e-3 * _normal(g, t, n)).to(_type(dt))
            s["dresidual"] = (1e-3 * _normal(g, t, n)).to(_type(dt)) if case["residual"] else None
        return s
    if op in ("act", "act_grad"):
        t, n, dt = case["rows"], case["cols"], case["dtype"]
        both = _normal(g, t, 2 * n, outliers=0.001, dtype=dt)            # one GEMM's output: gate beside up
        s["gate"], s["up"] = both[:, :n], both[:, n:]
        if op == "act_grad":
            s["dy"] = (1e-3 * _normal(g, t, n)).to(_type(dt))
        return s
    if op in ("tiles", "wgrad"):
        counts, blocks = _counts(case), _blocks(case)
        offsets = torch.tensor([0] + counts).cumsum(0)
        padded = torch.tensor([0] + [128 * -(-n // 128) for n in counts]).cumsum(0)
        if op == "wgrad":
            s["padded"], s["longest"] = padded.to(torch.int32).to(DEV), _longest(case)
            s["a"], s["a_scale"] = _operand(g, case["n"], blocks)
            s["b"], s["b_scale"] = _operand(g, case["k"], blocks)
            return s
        k, rows = case["top_k"], case["rows"]
        s["offsets"] = offsets.to(torch.int32).to(DEV)
        # the buffers that a program keeps: their columns behind the last expert's stay as they are
        width = (rows + 127 * min(rows, case["groups"])) // 128 * 128
        s["q"] = torch.zeros(case["cols"], width, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.zeros(case["cols"], width // 128, device=DEV)
        s["x"] = _normal(g, -(-rows // max(1, k)), case["cols"], outliers=0.001, dtype=case["dtype"])
        s["order"] = None if k == 0 else torch.randperm(-(-rows // k) * k, generator=g, device=DEV)[:rows].to(torch.int32)
        return s
    s["grads"] = [(0.01 * _normal(g, n)).to(_type(case["dtype"])) for n in _lengths(case)]
    if case["clip"]:
        s["outs"] = [torch.empty_like(x) for x in s["grads"]]
        s["max_norm"] = 1.0 if case["tensors"] > 1 else 1e-3
    return s


# --------------------------------------------------------------------------
# the framework's calls
def _run_own(s):
    import fp8_block_scaled_05_amd as fb
    c = s["case"]
    if c["op"] == "norm":
        q, scale, y, residual = fb.fp8_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantize=c["q"], with_y=c["y"])
        return {"q": q.view(E4M3) if q is not None else None, "scale": scale, "y": y, "residual": residual}
    if c["op"] == "norm_grad":
        return fb.fp8_rmsnorm_backward(s["dy"], s["x"], s["weight"], dresidual=s["dresidual"], eps=EPS)
    if c["op"] == "act":
        q, scale, y = fb.fp8_swiglu_quant(s["gate"], s["up"], quantize=c["q"], with_y=c["y"])
        return {"q": q.view(E4M3) if q is not None else None, "scale": scale, "y": y}
    if c["op"] == "act_grad":
        q, scale, d = fb.fp8_swiglu_backward(s["dy"], s["gate"], s["up"], quantize=c["q"], with_d=c["d"])
        return {"q": q.view(E4M3) if q is not None else None, "scale": scale, "d": d}
    if c["op"] == "tiles":
        q, scale, padded = fb.fp8_quant_grouped_t(s["x"], s["offsets"], order=s["order"], top_k=max(1, c["top_k"]), q=s["q"], scale=s["scale"])
        return q.view(E4M3), scale, padded
    if c["op"] == "wgrad":
        return fb.fp8_blockscaled_grouped_wgrad(s["padded"], s["a"], s["a_scale"], s["b"], s["b_scale"], out_dtype=_type(c["dtype"]))
    norm = fb.fp8_grad_norm(s["grads"])
    if c["clip"]:
        return norm, fb.fp8_grad_clip(s["grads"], norm, s["max_norm"], outs=s["outs"])
    return norm


# --------------------------------------------------------------------------
# the plain forms
def _tiled(y):
    """Codes and scales of float32 rows y in 1x128 tiles."""
    t = y.unflatten(1, (-1, 128))
    scale = t.abs().amax(-1) / torch.full((1, 1), 448.0, device=DEV)
    scale = torch.where(scale > 1e-10, scale, 1.0)
    return (t / scale[..., None]).flatten(1).to(E4M3), scale


def _norm(s):
    c, x = s["case"], s["x"]
    h, out = x, None
    if s["residual"] is not None:
        h = out = (x.float() + s["residual"].float()).to(x.dtype)      # the norm is that of the stored sum
    h = h.float()
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    q, scale = _tiled(y) if c["q"] else (None, None)
    return {"q": q, "scale": scale, "y": y.to(x.dtype) if c["y"] else None, "residual": out}


def _norm_grad(s):
    h, g = s["x"].float(), s["dy"].float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + EPS)
    dweight = None
    if s["weight"] is not None:
        dweight = (g * h * r).sum(0)
        g = g * s["weight"].float()
    dx = r * (g - h * r.square() * (g * h).mean(1, keepdim=True))
    if s["dresidual"] is not None:
        dx = dx + s["dresidual"].float()
    return dx.to(s["x"].dtype), dweight


def _act(s):
    c, g = s["case"], s["gate"].float()
    y = g / (1 + torch.exp(-g)) * s["up"].float()
    q, scale = _tiled(y) if c["q"] else (None, None)
    return {"q": q, "scale": scale, "y": y.to(s["gate"].dtype) if c["y"] else None}


def _act_grad(s):
    c, g, u, dy = s["case"], s["gate"].float(), s["up"].float(), s["dy"].float()
    sig = 1 / (1 + torch.exp(-g))
    d = torch.cat([dy * u * sig * (1 + g * (1 - sig)), dy * g * sig], 1)
    q, scale = _tiled(d) if c["q"] else (None, None)
    return {"q": q, "scale": scale, "d": d.to(s["gate"].dtype) if c["d"] else None}


def _exponent(amax):
    """The smallest e >= MIN_EXP with amax <= 448 * 2^e; 0 for a tile of zeros."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, (e - 9 + (m > 0.875).to(e.dtype)).clamp(min=MIN_EXP), 0)


def _tiles(s):
    c, off = s["case"], s["offsets"].long()
    width, cols = s["q"].shape[1], c["cols"]
    length = (off[1:] - off[:-1] + 127) // 128 * 128
    padded = torch.cat([off[:1], length.cumsum(0)])
    place = torch.arange(c["rows"], device=DEV)
    group = torch.searchsorted(off[1:].contiguous(), place, right=True)
    source = place if s["order"] is None else s["order"].long() // c["top_k"]
    z = torch.zeros(width, cols, device=DEV)
    z[padded[group] + place - off[group]] = s["x"][source].float()
    z = z.unflatten(0, (-1, 128))
    e = _exponent(z.abs().amax(1))
    codes = (z * torch.exp2(-e.float())[:, None]).to(E4M3).flatten(0, 1).t().contiguous()
    used = torch.arange(width // 128, device=DEV)[:, None] * 128 < padded[-1]
    return codes, torch.where(used, torch.exp2(e.float()), 0.0).t().contiguous(), padded.to(torch.int32)


def _wgrad(s):
    c, at = s["case"], s["padded"].long()
    depth = torch.arange(s["longest"], device=DEV)
    place = at[:-1, None] + depth                                     # [groups, longest]
    live = place < at[1:, None]
    place = place.clamp(max=max(0, s["a"].shape[1] - 1))
    a = (s["a"].view(E4M3).float().unflatten(1, (-1, 128)) * s["a_scale"][..., None]).flatten(1)
    b = (s["b"].view(E4M3).float().unflatten(1, (-1, 128)) * s["b_scale"][..., None]).flatten(1)
    a = a[:, place].permute(1, 0, 2) * live[:, None]                    # [groups, n, longest]
    b = b.t().contiguous()[place] * live[..., None]                     # [groups, longest, k]
    return torch.bmm(a.contiguous(), b).to(_type(c["dtype"]))


def _grads(s):
    norm = torch.stack([x.double().square().sum() for x in s["grads"]]).sum().sqrt().float().reshape(1)
    if not s["case"]["clip"]:
        return norm
    factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    return norm, [(x.float() * factor).to(x.dtype) for x in s["grads"]]


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm, "norm_grad": _norm_grad, "act": _act, "act_grad": _act_grad, "tiles": _tiles, "wgrad": _wgrad,
            "grads": _grads}[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# the definitions in 64 bits
def _to_e4m3(x):
    """The E4M3 value nearest to each 64-bit x, ties to even, largest 448."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    step = torch.where(x.abs() >= 16 * step, 2 * step, torch.where(x.abs() < 8 * step, step / 2, step)).clamp(min=2.0 ** -9)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_tiled(y):
    out, scales = torch.empty_like(y), []
    for lo in range(0, y.shape[1], 128):
        part = y[:, lo:lo + 128]
        scale = part.abs().amax(1, keepdim=True) / 448
        scale[scale <= 1e-10] = 1.0
        out[:, lo:lo + 128] = _to_e4m3(part / scale)
        scales.append(scale)
    return out, torch.cat(scales, 1)


def _exact_norm(s):
    c, h = s["case"], s["x"].double()
    total = None
    if c["residual"]:
        total = h + s["residual"].double()
        h = total.to(s["x"].dtype).double()
    y = h / ((h * h).sum(1, keepdim=True) / c["cols"] + EPS).sqrt()
    if c["weight"] != "none":
        y *= s["weight"].double()
    q, scale = _exact_tiled(y) if c["q"] else (None, None)
    return {"q": q, "scale": scale, "y": y if c["y"] else None, "residual": total}


def _exact_norm_grad(s):
    """By the chain rule through the root: y_j = w_j h_j / R, R = sqrt(mean(h^2) + eps), dR/dh_i = h_i / (cols R)."""
    c, h, dy = s["case"], s["x"].double(), s["dy"].double()
    w = s["weight"].double() if c["weight"] != "none" else torch.ones(c["cols"], dtype=torch.float64, device=DEV)
    root = ((h * h).sum(1, keepdim=True) / c["cols"] + EPS).sqrt()
    along = (dy * w * h).sum(1, keepdim=True) / root ** 2              # - sum_j dy_j dy_j/dR
    dx = dy * w / root - along * h / (c["cols"] * root)
    if c["residual"]:
        dx += s["dresidual"].double()
    return dx, (dy * h / root).sum(0) if c["weight"] != "none" else None


def _exact_act(s):
    c, g = s["case"], s["gate"].double()
    y = g * torch.sigmoid(g) * s["up"].double()
    q, scale = _exact_tiled(y) if c["q"] else (None, None)
    return {"q": q, "scale": scale, "y": y if c["y"] else None}


def _exact_act_grad(s):
    c = s["case"]
    g, u, dy = s["gate"].double().requires_grad_(True), s["up"].double().requires_grad_(True), s["dy"].double()
    with torch.enable_grad():
        (g * torch.sigmoid(g) * u).backward(dy)
    d = torch.cat([g.grad, u.grad], 1)
    q, scale = _exact_tiled(d) if c["q"] else (None, None)
    return {"q": q, "scale": scale, "d": d if c["d"] else None}


def _exact_tiles(s):
    c, counts, at, p = s["case"], _counts(s["case"]), 0, 0
    q = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    scale = torch.zeros(s["scale"].shape, dtype=torch.float64, device=DEV)
    source = torch.arange(c["rows"], device=DEV) if c["top_k"] == 0 else s["order"].long().div(c["top_k"], rounding_mode="floor")
    for n in counts:
        for lo in range(0, n, 128):
            m = min(128, n - lo)
            x = s["x"][source[at + lo:at + lo + m]].double()
            amax = x.abs().amax(0)
            e = torch.ceil(torch.log2(amax / 448))
            e = torch.where(torch.exp2(e - 1) * 448 >= amax, e - 1, torch.where(torch.exp2(e) * 448 < amax, e + 1, e)).clamp(min=MIN_EXP)
            unit = torch.where(amax > 0, torch.exp2(e), 1.0)
            q[:, p:p + m], scale[:, p // 128] = _to_e4m3(x / unit).t(), unit
            p += 128
        at += n
    return q, scale, None


def _exact_wgrad(s):
    c, p = s["case"], 0
    a, b = [(s[x].view(E4M3).double().reshape(s[x].shape[0], -1, 128) * s[x + "_scale"].double()[:, :, None]).flatten(1) for x in "ab"]
    y = torch.zeros(c["groups"], c["n"], c["k"], dtype=torch.float64, device=DEV)
    for e, n in enumerate(_counts(c)):
        depth = 128 * -(-n // 128)
        y[e] = a[:, p:p + depth] @ b[:, p:p + depth].t()
        p += depth
    return y


def _exact_grads(s):
    parts = [torch.linalg.vector_norm(x, dtype=torch.float64) for x in s["grads"]]
    norm = torch.linalg.vector_norm(torch.stack(parts)).reshape(1)
    if not s["case"]["clip"]:
        return norm
    factor = min(1.0, s["max_norm"] / float(norm))
    return norm, [x.double() * factor for x in s["grads"]]


def exact(case, seed):
    s = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "act": _exact_act, "act_grad": _exact_act_grad, "tiles": _exact_tiles,
                "wgrad": _exact_wgrad, "grads": _exact_grads}[case["op"]](s)
