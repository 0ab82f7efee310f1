"""The sort of the dispatch: every workgroup adds up the counts of all chunks, so their number may not grow with the choices
(no GPU: the workspace holds the counts)."""
import pytest

import fp8_block_scaled_05_amd as fb

MOST_CHUNKS = 256


@pytest.mark.parametrize("experts", [1, 256, 1024])
@pytest.mark.parametrize("top_k", [1, 8, 32])
def test_counts_are_bounded(experts, top_k):
    L = fb.lib()
    last = 0
    for tokens in (1, 4096, 8192, 32768, 65537, 1 << 20, 50_000_003, (1 << 31) // top_k - 1):
        need = L.fp8_moe_dispatch_workspace(tokens, experts, top_k)
        n = tokens * top_k
        if n <= 4096:
            assert need == 0
            continue
        chunks, rest = divmod(need, 4 * (experts + 1))
        assert rest == 0 and 1 <= chunks <= MOST_CHUNKS, (tokens, chunks)
        assert chunks >= min(MOST_CHUNKS // 2, -(-n // 2048)), (tokens, chunks)      # and there are enough to fill the chip's half
        last = max(last, chunks)
    assert last > MOST_CHUNKS // 2
