"""One mixture-of-experts decoder layer on the FP8 path: prompts in chunks, then single tokens.

Every matrix product runs on the block-scaled FP8 GEMMs, the keys and values live in the paged 8-bit cache, and
the routed rows reach the experts as FP8.  Random weights.

    python examples/decoder_layer.py --prompts 700 64 1300 --steps 16
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_block_scaled_05_amd as fb   # noqa: E402

PAGE = 64


def normed(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


def quantized(w):
    return fb.fp8_quant_w_128x128(w.bfloat16())[:2]


class Layer:
    def __init__(self, hidden=1024, q_heads=16, kv_heads=4, dim=64, experts=32, top_k=4, inner=256, positions=8192, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *shape: torch.randn(*shape, device="cuda", generator=g) * shape[-1] ** -0.5   # noqa: E731
        self.heads, self.dim, self.experts, self.top_k, self.inner = (q_heads, kv_heads), dim, experts, top_k, inner
        self.qkv, self.proj = quantized(r((q_heads + 2 * kv_heads) * dim, hidden)), quantized(r(hidden, q_heads * dim))
        up, down = [quantized(r(2 * inner, hidden)) for _ in range(experts)], [quantized(r(hidden, inner)) for _ in range(experts)]
        self.up, self.down = ([torch.stack(t) for t in zip(*w)] for w in (up, down))
        self.router, self.balance = r(experts, hidden), 0.02 * r(experts)
        self.q_weight = self.k_weight = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        inv = 10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
        a = torch.arange(positions, dtype=torch.float64, device="cuda")[:, None] * inv
        self.rope = torch.cat([a.cos(), a.sin()], 1).float()

    def attention(self, x, cache, cu, lens, table, max_new, max_len):
        (hq, hk), d = self.heads, self.dim
        qkv = fb.fp8_blockscaled_gemm(*fb.fp8_quant_act_1x128(normed(x)), *self.qkv, out_dtype=torch.bfloat16)
        q, k, v = qkv.unflatten(1, (hq + 2 * hk, d)).split([hq, hk, hk], 1)
        q = fb.fp8_kv_append(q, k, v, cache, cu, lens, table, max_new, rope=self.rope, q_weight=self.q_weight, k_weight=self.k_weight)
        o = fb.fp8_kv_attention(q, cache, cu, lens, table, max_new, max_len)
        return x + fb.fp8_blockscaled_gemm(*fb.fp8_quant_act_1x128(o.flatten(1)), *self.proj, out_dtype=torch.bfloat16)

    def routed(self, x):
        """The experts' output, and what the router's gradient needs."""
        a = normed(x)
        logits = a.float() @ self.router.t()
        ids, w = fb.fp8_moe_route(logits, self.top_k, bias=self.balance, groups=4, top_groups=2)
        q, scale, offsets, _, position = fb.fp8_moe_dispatch(a, ids, self.experts)
        gate, up = fb.fp8_blockscaled_grouped_gemm(offsets, q, scale, *self.up, out_dtype=torch.bfloat16).split(self.inner, 1)
        h = (torch.nn.functional.silu(gate.float()) * up.float()).bfloat16()
        y = fb.fp8_blockscaled_grouped_gemm(offsets, *fb.fp8_quant_act_1x128(h), *self.down)[position.long()]     # [T, top_k, hidden]
        return x + (y * w[..., None]).sum(1).bfloat16(), (a, logits, ids, y)

    def router_gradient(self, grad, saved):
        """Gradient of sum(grad * output) with respect to the router's weights."""
        a, logits, ids, y = saved
        dlogits = fb.fp8_moe_route_backward((y * grad.float()[:, None]).sum(-1), logits, ids)
        return dlogits.t() @ a.float()

    def __call__(self, x, cache, cu, lens, table, max_new, max_len):
        return self.routed(self.attention(x, cache, cu, lens, table, max_new, max_len))[0]


def run(layer, inputs, chunk, cache, table):
    """Feeds each sequence's inputs [length, hidden] in chunks of at most `chunk` tokens; the outputs, packed alike."""
    done, out = [0] * len(inputs), [[] for _ in inputs]
    i32 = dict(dtype=torch.int32, device="cuda")
    while any(d < len(x) for d, x in zip(done, inputs)):
        new = [min(chunk, len(x) - d) for d, x in zip(done, inputs)]
        x = torch.cat([x[d:d + n] for x, d, n in zip(inputs, done, new)])
        done = [d + n for d, n in zip(done, new)]
        cu = torch.tensor([0] + new, **i32).cumsum(0, dtype=torch.int32)
        y = layer(x, cache, cu, torch.tensor(done, **i32), table, max(new), max(done))
        for o, part in zip(out, y.split(new)):
            o.append(part)
    return [torch.cat(o) for o in out]


def new_cache(layer, lengths):
    used = [-(-n // PAGE) for n in lengths]
    table = torch.full((len(lengths), max(used)), -1, dtype=torch.int32)
    pages = torch.randperm(sum(used)).to(torch.int32).split(used)
    for row, p in zip(table, pages):
        row[:len(p)] = p
    return fb.KVCache.empty(sum(used), layer.heads[1], PAGE, layer.dim), table.cuda()


def main():
    p = argparse.ArgumentParser()
    p.add_argument("--prompts", type=int, nargs="+", default=[700, 64, 1300])
    p.add_argument("--chunk", type=int, default=512)
    p.add_argument("--steps", type=int, default=16)
    args = p.parse_args()
    layer = Layer()
    g = torch.Generator(device="cuda").manual_seed(1)
    lengths = [n + args.steps for n in args.prompts]
    inputs = [torch.randn(n, 1024, device="cuda", generator=g).bfloat16() for n in lengths]
    cache, table = new_cache(layer, lengths)
    run(layer, [x[:n] for x, n in zip(inputs, args.prompts)], args.chunk, cache, table)
    torch.cuda.synchronize()

    n, i32 = len(inputs), dict(dtype=torch.int32, device="cuda")
    cu, start = torch.arange(n + 1, **i32), time.perf_counter()
    for s in range(args.steps):
        lens = torch.tensor([m + s + 1 for m in args.prompts], **i32)
        x = torch.stack([t[m + s] for t, m in zip(inputs, args.prompts)])
        y = layer(x, cache, cu, lens, table, 1, max(args.prompts) + s + 1)
    torch.cuda.synchronize()
    print(f"{n} sequences of {args.prompts} tokens, then {args.steps} steps: {(time.perf_counter() - start) / max(args.steps, 1) * 1e6:.0f} us a step")
    _, saved = layer.routed(y)
    dw = layer.router_gradient(torch.ones_like(y), saved)
    print(f"output norm {y.float().norm():.3f}, router gradient norm {dw.norm():.3e}")


if __name__ == "__main__":
    main()
