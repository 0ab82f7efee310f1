"""Router, its gradient and the dispatch against their float64 definitions.

Tolerances: the ids are equal.  A weight is one rounding from 64 bits, a sum of up to 32 terms, a quotient and a
product in float32: relative 2^-18 is generous.  A gradient is a handful of float32 operations; with renormalised
weights it is a difference of terms of size |g| / S, so its error is 2^-18 of the row's largest such term; a bf16
result adds its half step, 2^-8."""
import numpy as np
import pytest

import oracle.moe as moe
from decoder_util import bf16, dev
from gpu_util import banner
from oracle import dequant_1x128, quant_1x128

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

ROUTES = [
    # tokens, experts, top_k, score, bias, groups, top_groups, renorm, scale
    (33, 256, 8, "sigmoid", True, 8, 4, True, 2.5),
    (7, 160, 6, "softmax", False, 1, 1, False, 1.0),
    (5, 160, 6, "softmax", False, 8, 3, False, 16.0),
    (1, 2, 1, "sigmoid", False, 1, 1, True, 1.0),
    (9, 1, 1, "softmax", True, 1, 1, True, 1.0),
    (300, 64, 8, "softmax", True, 4, 2, True, 1.0),
    (13, 384, 8, "sigmoid", False, 1, 1, True, 2.5),
    (17, 72, 5, "sigmoid", True, 8, 2, False, 1.0),
    (6, 1024, 32, "softmax", True, 64, 8, True, 1.0),
    (6, 8, 4, "sigmoid", True, 8, 5, True, 1.0),
    (1030, 100, 7, "sigmoid", True, 4, 3, True, 1.0),
    (64, 512, 10, "softmax", True, 16, 16, False, 1.0),
    (513, 256, 8, "sigmoid", False, 4, 2, False, 1.0),
    (40, 248, 8, "sigmoid", True, 8, 8, True, 1.0),
]


def _logits(rng, tokens, experts, dtype):
    x = (2.0 * rng.standard_normal((tokens, experts))).astype(np.float32)
    return bf16(x) if dtype is torch.bfloat16 else x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,k,score,bias,groups,top,renorm,scale", ROUTES)
def test_route(tokens, experts, k, score, bias, groups, top, renorm, scale, dtype):
    banner(f"route {tokens}x{experts} k {k} {score} groups {groups}/{top} {dtype}")
    rng = np.random.default_rng(40)
    x = _logits(rng, tokens, experts, dtype)
    bi = (0.05 * rng.standard_normal(experts)).astype(np.float32) if bias else None
    ids, w = fb.fp8_moe_route(dev(x, dtype), k, score=score, bias=dev(bi) if bias else None, groups=groups, top_groups=top,
                              renormalize=renorm, scale=scale)
    want_ids, want = moe.route(x, k, score, bi, groups, top, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(w.cpu().numpy() - want) <= 2.0 ** -18 * want).all()


@pytest.mark.parametrize("tokens", [3, 700])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_ties_go_to_the_lower_index(score, tokens):
    """Equal logits, logits that saturate to equal scores, and equal marks of groups."""
    x = np.zeros((tokens, 64), np.float32)
    x[1::3, ::2] = 40.0
    x[2::3] = np.tile(np.array([1, 3, 2, 3], np.float32), 16)
    for groups, top in ((1, 1), (8, 3)):
        ids, w = fb.fp8_moe_route(dev(x), 6, score=score, groups=groups, top_groups=top)
        want_ids, want = moe.route(x, 6, score, None, groups, top, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert (np.abs(w.cpu().numpy() - want) <= 2.0 ** -18 * want).all()


@pytest.mark.parametrize("tokens", [2, 600])
def test_route_masked_experts(tokens):
    """Experts masked with -infinity or the type's lowest value, in the logits or by the bias, signed zeros, and a
    bias that makes every score negative."""
    rng = np.random.default_rng(41)
    x = _logits(rng, tokens, 64, torch.float32)
    x[:, 5:60] = -np.inf
    x[:, 2] = np.finfo(np.float32).min
    ids, w = fb.fp8_moe_route(dev(x), 8, score="softmax", groups=4, top_groups=2)
    want_ids, want = moe.route(x, 8, "softmax", None, 4, 2, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(w.cpu().numpy() - want) <= 2.0 ** -18 * want).all()
    bias = np.full(64, -3.0, np.float32)
    bias[10:] = -np.inf
    y = _logits(rng, tokens, 64, torch.float32)
    for k in (4, 12):                                  # 12: ties of -infinity
        ids, w = fb.fp8_moe_route(dev(y), k, bias=dev(bias))
        want_ids, want = moe.route(y, k, "sigmoid", bias, 1, 1, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert (np.abs(w.cpu().numpy() - want) <= 2.0 ** -18 * want).all()


@pytest.mark.parametrize("tokens", [2, 600])
def test_route_nan_is_chosen_last(tokens):
    x = np.tile(np.arange(16, dtype=np.float32), (tokens, 1))
    x[:, 7] = np.nan
    ids, w = fb.fp8_moe_route(dev(x), 16, renormalize=False)
    assert np.array_equal(ids.cpu().numpy()[0], [15, 14, 13, 12, 11, 10, 9, 8, 6, 5, 4, 3, 2, 1, 0, 7])
    assert torch.isnan(w[:, 15]).all() and not torch.isnan(w[:, :15]).any()


def test_route_pitched_logits():
    rng = np.random.default_rng(42)
    for tokens in (5, 800):
        x = _logits(rng, tokens, 200, torch.float32)
        ids, w = fb.fp8_moe_route(dev(x)[:, 3:131], 4, groups=4, top_groups=2)
        want_ids, _ = moe.route(x[:, 3:131], 4, "sigmoid", None, 4, 2, True, 1.0)
        assert np.array_equal(ids.cpu().numpy(), want_ids)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("tokens,experts,k,renorm,scale", [(9, 160, 6, False, 1.0), (300, 256, 8, True, 2.5), (1, 1, 1, False, 1.0),
                                                          (5, 1024, 32, True, 1.0), (41, 33, 3, True, 1.0), (700, 72, 8, True, 1.0)])
def test_route_gradient(tokens, experts, k, renorm, scale, score, dtype):
    banner(f"route grad {tokens}x{experts} k {k} {score} {dtype}")
    rng = np.random.default_rng(43)
    x = _logits(rng, tokens, experts, dtype)
    ids = np.argsort(rng.random((tokens, experts)), 1)[:, :k].astype(np.int32)
    g = rng.standard_normal((tokens, k)).astype(np.float32)
    d = fb.fp8_moe_route_backward(dev(g), dev(x, dtype), dev(ids), score=score, renormalize=renorm, scale=scale)
    assert d.dtype == dtype
    want = moe.route_grad(g, x, ids, score, renorm, scale)
    total = moe.weights_at(x, ids, score, False, 1.0).sum(1, keepdims=True) if renorm else 1.0
    size = np.abs(g).max(1, keepdims=True) * scale / total
    tol = 2.0 ** -18 * size + (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -20) * np.abs(want)
    assert (np.abs(d.float().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(score, renorm):
    """Central differences of the float64 weights at a fixed choice; h = 1e-4 leaves 1e-7 of truncation."""
    rng = np.random.default_rng(44)
    x = _logits(rng, 3, 12, torch.float32)
    ids = np.argsort(rng.random((3, 12)), 1)[:, :4].astype(np.int32)
    g = rng.standard_normal((3, 4)).astype(np.float32)
    d = fb.fp8_moe_route_backward(dev(g), dev(x), dev(ids), score=score, renormalize=renorm, scale=1.5).cpu().numpy()
    for e in range(12):
        hi, lo = x.astype(np.float64), x.astype(np.float64)
        hi[:, e] += 1e-4
        lo[:, e] -= 1e-4
        diff = ((moe.weights_at(hi, ids, score, renorm, 1.5) - moe.weights_at(lo, ids, score, renorm, 1.5)) * g).sum(1) / 2e-4
        assert np.abs(d[:, e] - diff).max() <= 1e-5


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_route_gradient_of_missing_and_repeated_ids(score):
    rng = np.random.default_rng(45)
    x = _logits(rng, 4, 20, torch.float32)
    ids = np.array([[1, 2, -1], [3, 3, 5], [20, 99, -4], [0, 19, 7]], np.int32)
    g = rng.standard_normal((4, 3)).astype(np.float32)
    d = fb.fp8_moe_route_backward(dev(g), dev(x), dev(ids), score=score, renormalize=True).cpu().numpy()
    want = moe.route_grad(g, x, ids, score, True, 1.0)
    assert np.abs(d - want).max() <= 1e-5 * max(1.0, np.abs(want).max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,cols,experts,k", [(1, 128, 1, 1), (32, 1024, 256, 8), (7, 384, 4, 2), (600, 256, 16, 8), (2500, 128, 384, 4),
                                                  (1025, 640, 9, 1), (100, 2176, 1024, 32), (300, 128, 3, 3), (4096, 128, 64, 8)])
def test_dispatch_is_bit_exact(tokens, cols, experts, k, dtype):
    banner(f"dispatch {tokens}x{cols} experts {experts} k {k} {dtype}")
    rng = np.random.default_rng(46)
    x = (rng.standard_normal((tokens, cols)) * 3).astype(np.float32)
    x[rng.random(x.shape) < 1e-3] *= 50
    x = bf16(x) if dtype is torch.bfloat16 else x
    ids = rng.integers(0, experts, (tokens, k)).astype(np.int32)
    ids[rng.random((tokens, k)) < 0.5] = min(1, experts - 1)                       # one expert is asked for by half
    ids[rng.random(tokens) < 0.05] = -1
    ids[rng.random((tokens, k)) < 0.02] = experts + 3
    got = fb.fp8_moe_dispatch(dev(x, dtype), dev(ids), experts)
    for name, a, w in zip(("q", "scale", "offsets", "order", "position"), got, moe.dispatch(x, ids, experts)):
        assert np.array_equal(a.cpu().numpy(), w), name


def test_dispatch_of_nothing():
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    q, s, offsets, order, position = fb.fp8_moe_dispatch(x, torch.empty(0, 4, dtype=torch.int32, device="cuda"), 7)
    assert q.shape == (0, 256) and order.numel() == 0 and position.shape == (0, 4)
    assert offsets.tolist() == [0] * 8


def test_dispatch_of_padding_only():
    x = torch.ones(5, 128, dtype=torch.bfloat16, device="cuda")
    q, s, offsets, order, position = fb.fp8_moe_dispatch(x, torch.full((5, 2), -1, dtype=torch.int32, device="cuda"), 3)
    assert not q.any() and (s == 1).all() and offsets.tolist() == [0] * 4 and order.tolist() == list(range(10))


def test_dispatch_feeds_the_grouped_gemm():
    """The experts' products of the dispatched rows, gathered back and weighted, are the routed layer's output."""
    rng = np.random.default_rng(47)
    t, h, n, e, k = 50, 256, 128, 8, 2
    x = bf16(rng.standard_normal((t, h)))
    w = bf16(rng.standard_normal((e, n, h)) * 0.05)
    logits = rng.standard_normal((t, e)).astype(np.float32)
    ids, weights = fb.fp8_moe_route(dev(logits), k)
    q, s, offsets, order, position = fb.fp8_moe_dispatch(dev(x, torch.bfloat16), ids, e)
    wq = [fb.fp8_quant_w_128x128(dev(w[i], torch.bfloat16)) for i in range(e)]
    y = fb.fp8_blockscaled_grouped_gemm(offsets, q, s, torch.stack([a[0] for a in wq]), torch.stack([a[1] for a in wq]))
    got = (y[position.long()] * weights[..., None]).sum(1).cpu().numpy()
    xd = dequant_1x128(*quant_1x128(x)).astype(np.float64)
    from oracle import dequant_128x128, quant_128x128
    wd = [dequant_128x128(*quant_128x128(w[i])).astype(np.float64) for i in range(e)]
    wi, ww = moe.route(logits, k, "sigmoid", None, 1, 1, True, 1.0)
    want = np.stack([sum(ww[i, j] * (xd[i] @ wd[wi[i, j]].T) for j in range(k)) for i in range(t)])
    bound = np.stack([sum(ww[i, j] * (np.abs(xd[i]) @ np.abs(wd[wi[i, j]]).T) for j in range(k)) for i in range(t)])
    assert (np.abs(got - want) <= 3e-5 * bound).all()
