"""The router and the dispatch refuse sizes out of range with the library's status, before memory is allocated for them."""
import pytest

from gpu_util import banner

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
fb = pytest.importorskip("fp8_block_scaled_05_amd")


def _refused(call, text):
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    with pytest.raises(fb.Fp8bsError, match=text):
        call()
    assert torch.cuda.max_memory_allocated() - before <= 1 << 20


@pytest.mark.parametrize("top_k", [(1 << 31) - 1, 1 << 24, 65, 33, 0, -3])
def test_router(top_k):
    banner(f"route refuses top_k {top_k}")
    x = torch.zeros(1000, 64, device="cuda")
    _refused(lambda: fb.fp8_moe_route(x, top_k), "top_k")


@pytest.mark.parametrize("experts,k,text", [((1 << 31) - 1, 2, "experts"), (1025, 2, "experts"), (0, 2, "experts"), (-1, 2, "experts"), (8, 33, "top_k"), (8, 0, "top_k")])
def test_dispatch(experts, k, text):
    banner(f"dispatch refuses {experts} experts, top_k {k}")
    x, ids = torch.zeros(1000, 1024, device="cuda"), torch.zeros(1000, k, dtype=torch.int32, device="cuda")
    _refused(lambda: fb.fp8_moe_dispatch(x, ids, experts), text)
