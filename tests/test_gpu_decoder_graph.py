"""The decoder layer's operators captured in a HIP graph and on a side stream.  A graph is replayed several times with
eager work and synchronization in between, on inputs changed in place, and every replay is checked against eager calls."""
import numpy as np
import pytest

from decoder_util import Batch, angles, dev
from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _layer(b, s, cache, lens):
    q = fb.fp8_kv_append(s["q"], s["k"], s["v"], cache, s["cu"], lens, s["table"], b.max_new, rope=s["rope"])
    out, lse = fb.fp8_kv_attention(q, cache, s["cu"], lens, s["table"], b.max_new, b.max_len, return_lse=True)
    ids, w = fb.fp8_moe_route(s["logits"], 4, bias=s["bias"], groups=4, top_groups=2)
    d = fb.fp8_moe_route_backward(s["grad"], s["logits"], ids)
    return (q, out, lse, ids, w, d, *fb.fp8_moe_dispatch(out.flatten(1), ids, 32))


def _state(b, tokens, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=g)   # noqa: E731
    return dict(q=r(tokens, 8, 64).bfloat16(), k=r(tokens, 2, 64).bfloat16(), v=r(tokens, 2, 64).bfloat16(), logits=r(tokens, 32),
                bias=0.1 * r(32), grad=r(tokens, 4))


@pytest.mark.parametrize("new,total", [([1, 1, 1], [3000, 40, 700]), ([300, 200], [300, 900])])
def test_graph_replays_match_eager(new, total):
    banner(f"graph: decoder layer new {new}")
    b = Batch(50, new, total, 2, 64, 32)
    _, cu, lens, table = b.on_gpu()
    base = dict(cu=cu, table=table, rope=dev(angles(4096, 64)))
    s = {**base, **_state(b, b.tokens, 0)}
    pristine = b.on_gpu()[0]
    cache = b.on_gpu()[0]

    def restore(c):
        for x, y in ((c.k, pristine.k), (c.v, pristine.v), (c.k_scale, pristine.k_scale), (c.v_scale, pristine.v_scale)):
            x.copy_(y)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(b, s, cache, lens)                      # warm-up outside the graph
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _layer(b, s, cache, lens)
    torch.cuda.synchronize()
    for r in range(4):
        fresh = _state(b, b.tokens, 10 + r)
        for k, v in fresh.items():
            s[k].copy_(v)
        restore(cache)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*captured, cache.k, cache.v, cache.k_scale, cache.v_scale)]
        other = b.on_gpu()[0]
        want = [*_layer(b, {**base, **fresh}, other, lens), other.k, other.v, other.k_scale, other.v_scale]
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), f"replay {r}: output {i} differs from the eager call"


def test_side_stream_orders_with_its_own_work():
    """Calls on a side stream use that stream: inputs written there just before are seen."""
    b = Batch(51, [1] * 9, [900 + 37 * i for i in range(9)], 2, 64, 64)
    cache, cu, lens, table = b.on_gpu()
    s = dict(cu=cu, table=table, rope=dev(angles(4096, 64)), **_state(b, 9, 1))
    want = _layer(b, s, cache, lens)
    torch.cuda.synchronize()
    cache2 = b.on_gpu()[0]
    held = {k: v.clone() for k, v in s.items()}
    for k in ("q", "k", "v", "logits"):
        s[k].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.ones(1 << 28, device="cuda")
        for _ in range(4):
            big.mul_(1.5)                              # the copies below wait behind this
        for k in ("q", "k", "v", "logits"):
            s[k].copy_(held[k])
        got = _layer(b, s, cache2, lens)
    side.synchronize()
    for i, (x, y) in enumerate(zip(got, want)):
        assert torch.equal(x, y), i
    assert np.isfinite(got[2].cpu().numpy()).all()
