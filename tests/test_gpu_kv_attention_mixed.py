"""Attention over uneven batches, and softmax scales that are negative or zero, against float64.  Tolerances as in
test_gpu_kv_attention.py."""
import numpy as np
import pytest

import test_gpu_kv_attention as one
from decoder_util import Batch, bf16
from gpu_util import banner
from test_gpu_kv_attention_many import _check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dim,window", [(128, 0), (64, 0), (64, 300)])
def test_one_chunk_among_single_tokens(dim, window):
    banner(f"attend 63 single tokens and a chunk of 512, dim {dim} window {window}")
    rng = np.random.default_rng(140)
    new = [1] * 63 + [512]
    total = [int(n) for n in rng.integers(1, 2500, 63)] + [2400]
    _check(Batch(141, new, total, 2, dim, 64), 8, window)


@pytest.mark.parametrize("window", [0, 700])
def test_one_long_sequence_among_many(window):
    banner(f"attend 63 sequences of 1000 and one of 60000, window {window}")
    _check(Batch(142, [1] * 64, [1000] * 30 + [60000] + [1000 - 7 * i for i in range(33)], 2, 64, 64), 8, window)


def test_chunks_of_very_different_lengths():
    banner("attend chunks over 3 to 30000 tokens")
    _check(Batch(143, [3, 300, 1, 0, 40, 64], [3, 300, 30000, 12, 700, 9000], 2, 128, 32), 8)


@pytest.mark.parametrize("scale", [-0.2, 0.0, -0.0, -1e-30])
@pytest.mark.parametrize("new,total,window", [([1, 1], [300, 1], 0), ([1], [4000], 0), ([5, 40], [90, 800], 33), ([300], [900], 0)])
def test_softmax_scales_not_above_zero(new, total, window, scale):
    banner(f"attend scale {scale} new {new}")
    b = Batch(144, new, total, 2, 64, 16)
    q = bf16(np.random.default_rng(145).standard_normal((b.tokens, 4, 64)))
    out, lse = one._attend(b, q, window, softmax_scale=scale)
    one._check(b, q, out, lse, window, scale)
