"""Appends of uneven batches: one long prompt among single tokens, whose workgroups are numbered over all sequences.
Without norm and rotation codes, scales and queries are equal bit for bit to the definition; the large batches are
compared with calls that bring their prompt and their single tokens apart."""
import numpy as np
import pytest

import oracle.kv_cache as kv
from decoder_util import Batch, angles, bf16, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

BATCHES = {
    "prompt first": ([200] + [1] * 9, [200] + [17 + 9 * i for i in range(9)]),
    "prompt last": ([1] * 9 + [161], [64 * (i + 1) for i in range(9)] + [300]),
    "nothing new": ([0, 0, 90, 0, 1, 0], [5, 9, 95, 1, 33, 64]),
    "more than a wave": ([1] * 70 + [250] + [1] * 70 + [0, 33], [40 + 3 * i for i in range(143)][:70] + [250] + [20 + i for i in range(70)] + [7, 40]),
}


@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("name", BATCHES)
def test_uneven_batches(name, dim, page):
    banner(f"append {name} dim {dim} page {page}")
    new, total = BATCHES[name]
    b = Batch(110, new, total, 2, dim, page)
    q, k, v = (bf16(np.random.default_rng(111).standard_normal((b.tokens, h, dim)) * 4) for h in (6, 2, 2))
    cache, cu, lens, table = b.on_gpu()
    got = fb.fp8_kv_append(*[dev(x, torch.bfloat16) for x in (q, k, v)], cache, cu, lens, table, b.max_new)
    assert np.array_equal(got.float().cpu().numpy(), q)
    for i, (y, c, s) in enumerate(((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale))):
        wc, ws = kv.append(b.codes[i], b.scales[i], y.astype(np.float64), b.cu, b.lens, b.table, page)
        assert np.array_equal(s.cpu().numpy(), ws) and np.array_equal(c.cpu().numpy(), wc)


@pytest.mark.parametrize("batch,prompt,at", [(1024, 16384, 1023), (256, 8192, 0), (300, 5000, 77)])
def test_one_prompt_among_single_tokens(batch, prompt, at):
    """1024 sequences of which one brings 16384 tokens: 17407 tokens in all, however many the longest times the batch are."""
    banner(f"append {batch} sequences, one of {prompt} tokens")
    hq, hk, dim, page, old = 64, 8, 128, 64, 37
    new = [1] * batch
    new[at] = prompt
    rng = np.random.default_rng(112)
    lens = np.array([n + old for n in new], np.int32)
    used = [-(-int(n) // page) for n in lens]
    table = np.full((batch, max(used)), -1, np.int32)
    order, taken = rng.permutation(sum(used)), 0
    for s, n in enumerate(used):
        table[s, :n] = order[taken:taken + n]
        taken += n
    tokens = sum(new)
    g = torch.Generator(device="cuda").manual_seed(113)
    qkv = torch.randn(tokens, (hq + 2 * hk) * dim, device="cuda", generator=g).bfloat16()
    weight = (1 + 0.1 * torch.randn(dim, device="cuda", generator=g)).bfloat16()
    rope = dev(angles(prompt + old, dim))
    caches = [fb.KVCache.empty(sum(used), hk, page, dim) for _ in range(2)]

    def append(cache, seqs, rows):
        n = len(seqs)
        cu = np.concatenate([[0], np.cumsum([new[s] for s in seqs])]).astype(np.int32)
        x = qkv[rows]
        a, c = hq * dim, (hq + hk) * dim
        return fb.fp8_kv_append(x[:, :a].unflatten(1, (hq, dim)), x[:, a:c].unflatten(1, (hk, dim)), x[:, c:].unflatten(1, (hk, dim)), cache,
                                dev(cu), dev(lens[seqs]), dev(table[seqs]), max(new[s] for s in seqs), rope=rope, q_weight=weight, k_weight=weight), n

    whole, _ = append(caches[0], list(range(batch)), slice(None))
    first = sum(new[:at])
    row = torch.ones(tokens, dtype=torch.bool, device="cuda")
    row[first:first + prompt] = False
    singles, n = append(caches[1], [s for s in range(batch) if s != at], row)
    long, _ = append(caches[1], [at], slice(first, first + prompt))
    assert n == batch - 1 and torch.equal(whole[row], singles) and torch.equal(whole[~row], long)
    for x, y in zip(caches[0].args, caches[1].args):
        assert torch.equal(x, y)
    assert bool(caches[0].k.any()) and bool(caches[0].v.any())


@pytest.mark.parametrize("new", [[1] * 40, [1] * 39 + [500], [60, 60, 60, 60]])
def test_crooked_tables(new):
    """cu and seq_lens that hold anything: pages that no sequence has, and what lies before and behind the queries and
    the cache, keep their bytes."""
    banner(f"append crooked {len(new)} x {new[-1]}")
    b = Batch(114, new, [n + 100 for n in new], 2, 64, 32)
    rng = np.random.default_rng(115)
    x = [dev(bf16(rng.standard_normal((b.tokens, h, 64))), torch.bfloat16) for h in (6, 2, 2)]
    t, n = b.tokens, len(new)
    cus = [[0, t] * n, [t, 0] * n, [-7, t // 2, -(1 << 31), (1 << 31) - 1] * n, [(1 << 31) - 1] * (n + 1), [0] * (n + 1), list(range(t, t - n - 1, -1))]
    lens = [b.lens, np.full(n, -3), np.full(n, -(1 << 31)), np.full(n, (1 << 31) - 1), np.array([(1 << 30) + i for i in range(n)]), np.arange(n)]
    mine = np.zeros(b.pages + 2, bool)
    mine[1 + b.table[b.table >= 0]] = True
    for cu in [b.cu] + [np.array(c[:n + 1], np.int64) for c in cus]:
        for length in lens:
            # the cache lies between two pages that it does not have, the queries between two rows
            wide = [torch.full((b.pages + 2, *c.shape[1:]), 77, dtype=torch.uint8, device="cuda") for c in b.codes]
            scales = [torch.full((b.pages + 2, 2), 0.5, device="cuda") for _ in range(2)]
            cache = fb.KVCache(*[w[1:-1] for w in wide], *[s[1:-1] for s in scales])
            q_out = torch.full((t + 2, 6, 64), 5.0, dtype=torch.bfloat16, device="cuda")
            fb.fp8_kv_append(*x, cache, dev(cu.astype(np.int32)), dev(length.astype(np.int64).astype(np.int32)), dev(b.table), b.max_new, q_out=q_out[1:-1])
            torch.cuda.synchronize()
            assert bool((q_out[0] == 5).all()) and bool((q_out[-1] == 5).all())
            for w, s in zip(wide, scales):
                assert bool((w[dev(~mine)] == 77).all()) and bool((s[dev(~mine)] == 0.5).all())
