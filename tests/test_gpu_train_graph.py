"""The training step's operators in a run, captured in a HIP graph, on a side stream, and two calls at once.  A graph is
replayed several times with eager work and synchronization in between, on inputs changed in place, and every replay is
checked against eager calls."""
import threading

import pytest

from gpu_util import banner
from train_util import same_bits

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")

EXPERTS, HIDDEN, INNER, TOP = 6, 384, 256, 2


def _state(tokens, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *shape: torch.randn(*shape, device="cuda", generator=g)   # noqa: E731
    return dict(x=r(tokens, HIDDEN).bfloat16(), residual=r(tokens, HIDDEN).bfloat16(), weight=r(HIDDEN), dy=r(tokens, HIDDEN).bfloat16(),
                ids=torch.randint(-1, EXPERTS, (tokens, TOP), device="cuda", generator=g).to(torch.int32),
                halves=r(tokens * TOP, 2 * INNER).bfloat16(), dh=r(tokens * TOP, INNER).bfloat16())


def _step(s):
    q, scale, y, h = fb.fp8_rmsnorm_quant(s["x"], s["weight"], residual=s["residual"], with_y=True)
    _, _, offsets, order, _ = fb.fp8_moe_dispatch(y, s["ids"], EXPERTS)
    gate, up = s["halves"].split(INNER, 1)
    act = fb.fp8_swiglu_quant(gate, up, with_y=True)
    back = fb.fp8_swiglu_backward(s["dh"], gate, up, with_d=True)
    a, sa, padded = fb.fp8_quant_grouped_t(back[2], offsets)
    b, sb, _ = fb.fp8_quant_grouped_t(y, offsets, order=order, top_k=TOP)
    dw = fb.fp8_blockscaled_grouped_wgrad(padded, a, sa, b, sb)
    dx, dweight = fb.fp8_rmsnorm_backward(s["dy"], h, s["weight"], dresidual=s["dy"])
    norm = fb.fp8_grad_norm([dw, dweight])
    clipped = fb.fp8_grad_clip([dw, dweight], norm, 1.0, outs=[torch.empty_like(dw), torch.empty_like(dweight)])
    return (q, scale, y, h, *act, *back, padded, dw, dx, dweight, norm, *clipped)


@pytest.mark.parametrize("tokens", [1, 5, 700])
def test_graph_replays_match_eager(tokens):
    banner(f"graph: training step of {tokens} tokens")
    s = _state(tokens, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _step(s)                                       # warm-up outside the graph
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = _step(s)
    torch.cuda.synchronize()
    for r in range(4):
        fresh = _state(tokens, 10 + r)
        for k, v in fresh.items():
            s[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in captured]
        want = _step(fresh)
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert same_bits(x, y), f"replay {r}: output {i} differs from the eager call"


def test_side_stream_orders_with_its_own_work():
    """Calls on a side stream use that stream: inputs written there just before are seen."""
    s = _state(300, 1)
    want = _step(s)
    torch.cuda.synchronize()
    held = {k: v.clone() for k, v in s.items()}
    for k in s:
        s[k].zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        big = torch.ones(1 << 28, device="cuda")
        for _ in range(4):
            big.mul_(1.5)                              # the copies below wait behind this
        for k in s:
            s[k].copy_(held[k])
        got = _step(s)
    side.synchronize()
    for i, (x, y) in enumerate(zip(got, want)):
        assert same_bits(x, y), i


def test_two_streams_at_once():
    """Workspaces are each call's own."""
    states = [_state(900, 20), _state(900, 21)]
    want = [_step(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(3):
        got = []
        for s, stream in zip(states, streams):
            with torch.cuda.stream(stream):
                got.append(_step(s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(same_bits(x, y) for x, y in zip(a, b))


def test_graphs_of_one_pool_in_turn():
    """Two captured steps whose workspaces share one pool's memory, replayed in turn."""
    banner("two graphs of one pool")
    states = [_state(500, 30), _state(700, 31)]
    want = [_step(s) for s in states]
    torch.cuda.synchronize()
    pool, graphs, got = torch.cuda.graph_pool_handle(), [], []
    for s in states:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            got.append(_step(s))
        graphs.append(graph)
    for turn in (0, 1, 1, 0, 1, 0):
        for x in got[turn]:
            x.zero_()
        graphs[turn].replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got[turn], want[turn])):
            assert same_bits(x, y), (turn, i)
        want[turn] = _step(states[turn])               # eager work between the replays
        torch.cuda.synchronize()


def test_calls_from_two_threads():
    banner("training step from two threads")
    states = [_state(400, 40), _state(64, 41)]
    want = [_step(s) for s in states]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(5):
                    with pytest.raises(fb.Fp8bsError, match=("eps", "max_norm")[i]):     # each thread's own message
                        if i == 0:
                            fb.fp8_rmsnorm_backward(states[0]["dy"], states[0]["dy"], eps=0.0)
                        else:
                            fb.fp8_grad_clip([want[1][0].float()], torch.ones(1, device="cuda"), -1.0)
                    got[i] = _step(states[i])
                torch.cuda.current_stream().synchronize()
        except BaseException as e:                     # noqa: BLE001 - shown by the main thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(same_bits(x, y) for x, y in zip(a, b))
