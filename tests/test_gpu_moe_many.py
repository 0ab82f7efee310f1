"""The router over many tokens (16 lanes a token instead of 64), against its float64 definition.  Tolerances as in
test_gpu_moe.py."""
import numpy as np
import pytest

import oracle.moe as moe
from decoder_util import bf16, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

ROUTES = [
    # tokens, experts, top_k, score, bias, groups, top_groups, renorm, scale
    (5001, 256, 8, "sigmoid", True, 8, 4, True, 2.5),
    (4096, 160, 6, "softmax", False, 1, 1, False, 1.0),
    (4099, 100, 7, "sigmoid", True, 4, 3, True, 1.0),
    (4100, 33, 5, "softmax", True, 3, 2, True, 1.0),
    (4097, 64, 32, "sigmoid", False, 16, 8, True, 1.0),
    (4111, 1, 1, "softmax", True, 1, 1, True, 1.0),
    (4111, 8, 8, "softmax", False, 1, 1, True, 1.0),
    (4200, 128, 20, "softmax", True, 2, 1, True, 1.0),
    (4200, 130, 3, "sigmoid", True, 13, 5, False, 1.0),
    (4200, 384, 8, "sigmoid", True, 32, 5, True, 1.0),
    (4200, 384, 8, "softmax", True, 8, 3, True, 2.5),
    (4200, 301, 6, "sigmoid", True, 7, 2, False, 1.0),
    (70, 301, 6, "sigmoid", True, 7, 2, False, 1.0),
    (70, 500, 9, "softmax", False, 10, 3, True, 1.0),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tokens,experts,k,score,bias,groups,top,renorm,scale", ROUTES)
def test_route_and_gradient(tokens, experts, k, score, bias, groups, top, renorm, scale, dtype):
    banner(f"route {tokens}x{experts} k {k} {score} groups {groups}/{top} {dtype}")
    rng = np.random.default_rng(80)
    x = (2.0 * rng.standard_normal((tokens, experts))).astype(np.float32)
    x = bf16(x) if dtype is torch.bfloat16 else x
    bi = (0.05 * rng.standard_normal(experts)).astype(np.float32) if bias else None
    ids, w = fb.fp8_moe_route(dev(x, dtype), k, score=score, bias=dev(bi) if bias else None, groups=groups, top_groups=top,
                              renormalize=renorm, scale=scale)
    want_ids, want = moe.route(x, k, score, bi, groups, top, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    assert (np.abs(w.cpu().numpy() - want) <= 2.0 ** -18 * want).all()
    g = rng.standard_normal((tokens, k)).astype(np.float32)
    d = fb.fp8_moe_route_backward(dev(g), dev(x, dtype), ids, score=score, renormalize=renorm, scale=scale)
    want = moe.route_grad(g, x, want_ids, score, renorm, scale)
    total = moe.weights_at(x, want_ids, score, False, 1.0).sum(1, keepdims=True) if renorm else 1.0
    size = np.abs(g).max(1, keepdims=True) * scale / total
    tol = 2.0 ** -18 * size + (2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -20) * np.abs(want)
    assert (np.abs(d.float().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("tokens", [3, 4200])
def test_nan_in_a_group(tokens):
    """A NaN adds nothing to its group's mark and is chosen after every number."""
    x = np.tile(np.arange(32, dtype=np.float32) * 0.1, (tokens, 1))
    x[:, 31] = np.nan                                  # group 3: 30, 29 remain; group 2: 23, 22
    x[:, 16:23] = np.nan                               # group 2: only 23 remains, its mark is -infinity
    ids, _ = fb.fp8_moe_route(dev(x), 8, groups=4, top_groups=2, renormalize=False)
    assert (ids.cpu().numpy() == [30, 29, 28, 27, 26, 25, 24, 15]).all()
    ids, _ = fb.fp8_moe_route(dev(x), 9, groups=4, top_groups=3, renormalize=False)
    assert (ids.cpu().numpy() == [30, 29, 28, 27, 26, 25, 24, 15, 14]).all()


def test_rows_that_are_not_aligned():
    rng = np.random.default_rng(81)
    x = rng.standard_normal((4300, 200)).astype(np.float32)
    ids, w = fb.fp8_moe_route(dev(x)[:, 3:131], 4, groups=4, top_groups=2)
    want_ids, _ = moe.route(x[:, 3:131], 4, "sigmoid", None, 4, 2, True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    wide = torch.full((4300, 139), 7.0, device="cuda")
    g = rng.standard_normal((4300, 4)).astype(np.float32)
    d = fb.fp8_moe_route_backward(dev(g), dev(x)[:, 3:131], ids, dlogits=wide[:, 5:133])
    want = moe.route_grad(g, x[:, 3:131], want_ids, "sigmoid", True, 1.0)
    assert np.abs(d.cpu().numpy() - want).max() <= 2.0 ** -18 * np.abs(g).max() / 0.1
    assert bool((wide[:, :5] == 7).all()) and bool((wide[:, 133:] == 7).all())
