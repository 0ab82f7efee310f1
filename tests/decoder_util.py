"""Seeded batches over a paged cache, as numpy arrays and on the GPU."""
import numpy as np
import torch

from fp8_block_scaled_05_amd import synth


def bf16(x):
    """Values rounded to bf16, as float32."""
    return synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(np.asarray(x, np.float32)))


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


class Batch:
    """new and total tokens per sequence; every sequence's pages are a random draw; unused table entries are -1."""

    def __init__(self, seed, new, total, kv_heads, dim, page):
        rng = self.rng = np.random.default_rng(seed)
        self.new, self.lens, self.page, self.heads, self.dim = new, np.array(total, np.int32), page, kv_heads, dim
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.cu[-1])
        used = [-(-n // page) for n in total]
        self.pages = sum(used) + 2
        width = max(used + [1])
        order, at = rng.permutation(self.pages), 0
        self.table = np.full((len(new), width), -1, np.int32)
        for b, n in enumerate(used):
            self.table[b, :n] = order[at:at + n]
            at += n
        shape = (self.pages, kv_heads, page, dim)
        # any finite code: 0x7f and 0xff are NaN
        self.codes = [np.where(c & 0x7f == 0x7f, 0x30, c).astype(np.uint8) for c in rng.integers(0, 256, (2, *shape))]
        self.scales = [np.float32(2.0) ** rng.integers(-9, -5, shape[:2]).astype(np.float32) for _ in range(2)]

    def on_gpu(self):
        import fp8_block_scaled_05_amd as fb
        cache = fb.KVCache(dev(self.codes[0]), dev(self.codes[1]), dev(self.scales[0]), dev(self.scales[1]))
        return cache, dev(self.cu), dev(self.lens), dev(self.table)

    @property
    def max_new(self):
        return max(self.new)

    @property
    def max_len(self):
        return int(self.lens.max())


def angles(rows, rot, theta=10000.0):
    inv = theta ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(rows)[:, None] * inv
    return np.concatenate([np.cos(a), np.sin(a)], 1).astype(np.float32)
