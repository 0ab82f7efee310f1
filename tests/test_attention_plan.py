"""How attention cuts up a call, read from its workspace (no GPU): splits * tokens * q_heads * (head_dim + 2) floats where
there is more than one split, else nothing."""
import struct

import pytest

import fp8_block_scaled_05_amd as fb

A = 0x10000            # a fake, 16-byte aligned "device" address; never dereferenced


def splits(batch, tokens, max_new, max_len, q_heads, kv_heads, dim, window=0):
    cache = struct.pack("4Q4q", A, A, A, A, 8, kv_heads, 16, dim)
    b = struct.pack("3Q6q", A, A, A, 1 << 17, 1 << 17, batch, tokens, max_new, max_len)
    need = fb.lib().fp8_kv_attention_workspace(cache, b, struct.pack("4Q5qd", A, A, A, 0, 0, q_heads * dim, dim, q_heads, window, 0.125))
    assert need >= 0 and need % (tokens * q_heads * (dim + 2) * 4) == 0
    return need // (tokens * q_heads * (dim + 2) * 4) or 1


@pytest.mark.parametrize("args,want", [
    # one token, 8 kv heads of 128: 8 waves of one workgroup up to 1280 tokens, then 128-key splits in rounds of 128
    ((1, 1, 1, 1280, 64, 8, 128), 1), ((1, 1, 1, 1281, 64, 8, 128), 6), ((1, 1, 1, 2000, 64, 8, 128), 8), ((1, 1, 1, 100003, 64, 8, 128), 87),
    # heads of 64: twice the tokens
    ((1, 1, 1, 2560, 64, 8, 64), 1), ((1, 1, 1, 2561, 64, 8, 64), 11),
    # 768 workgroups: 96 sequences of 8 heads fill them, 48 do in two splits
    ((64, 64, 1, 100003, 64, 8, 128), 1), ((48, 48, 1, 100003, 64, 8, 128), 2),
    # 2048 rows of one sequence: tiles of 16 rows up to 1536 tokens, unsplit; then 17 tiles of 128, three splits
    ((1, 512, 512, 1536, 32, 8, 64), 1), ((1, 512, 512, 1537, 32, 8, 64), 3),
    # a window bounds the keys: 100 (4096) + 16 + 64 of them; ceil(4176 / 256) splits
    ((1, 1, 1, 100003, 64, 8, 128, 100), 1), ((1, 1, 1, 100003, 64, 8, 128, 4096), 17),
    # more splits than the join takes are not made
    ((1, 1, 1, 1 << 20, 1, 1, 64), 512),
])
def test_splits(args, want):
    assert splits(*args) == want


def test_launches_are_bounded():
    """Splits never outnumber what the chip is filled with, nor 512, nor the steps in the keys."""
    many = 0
    for batch in (1, 3, 17, 64, 1000):
        for new in (1, 2, 8, 100, 4000):
            for max_len in (1, 100, 1300, 5000, 100000, 1 << 20):
                for q_heads, kv_heads in ((2, 2), (10, 2), (64, 8), (64, 1)):
                    for window in (0, 500):
                        n = splits(batch, batch * new, new, max_len, q_heads, kv_heads, 128, window)
                        group = q_heads // kv_heads
                        narrow = -(-new * group // 16) * batch * kv_heads
                        wide = (batch * new * group // 128 + batch) * kv_heads
                        assert 1 <= n <= 512 and n <= max(1, max_len // 128)
                        if n > 1:
                            many += 1
                            assert n * narrow <= 768 or n * wide <= 1024
                            assert new * group > 32 or n * narrow <= 768
    assert many > 50
