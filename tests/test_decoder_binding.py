"""What the native marshalling of the decoder layer's operators refuses, on CPU tensors: wrong shapes, types and layouts by
their own messages, and whatever is left because it is not on the GPU.  Nothing is launched."""
import types

import pytest

import fp8_block_scaled_05_amd as fb

torch = pytest.importorskip("torch")

A = 0x10000            # a fake, 16-byte aligned "device" address; never dereferenced
BF, I32 = torch.bfloat16, torch.int32


def _cache(heads=2, dim=64):
    from fp8_block_scaled_05_amd import decoder
    return types.SimpleNamespace(args=decoder._CACHE.pack(A, A, A, A, 8, heads, 16, dim))


def _batch(n=2, width=4):
    return torch.zeros(n + 1, dtype=I32), torch.ones(n, dtype=I32), torch.zeros(n, width, dtype=I32)


def _rows(heads, dim=64, tokens=5, dtype=BF):
    return torch.zeros(tokens, heads, dim, dtype=dtype)


def test_append_refusals():
    def call(q=_rows(4), k=_rows(2), v=_rows(2), cache=_cache(), batch=_batch(), **kw):
        fb.fp8_kv_append(q, k, v, cache, *batch, 4, **kw)
    for error, kw in [(TypeError, dict(k=_rows(2, dtype=torch.float32))), (ValueError, dict(k=_rows(3))), (ValueError, dict(v=_rows(2, tokens=4))),
                      (ValueError, dict(k=_rows(2)[0])), (TypeError, dict(k=None)), (TypeError, dict(v=3)), (ValueError, dict(k=_rows(2, dim=32))),
                      (TypeError, dict(cache=types.SimpleNamespace(args=b"short"))), (AttributeError, dict(cache=None)),
                      (KeyError, dict(rope_layout="third"))]:
        with pytest.raises(error):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):
        call()


def test_attention_refusals():
    def call(q=_rows(4), cache=_cache(), batch=_batch(), **kw):
        fb.fp8_kv_attention(q, cache, *batch, 4, 64, **kw)
    for error, kw in [(ValueError, dict(q=_rows(4, dim=128))), (TypeError, dict(q=_rows(4, dtype=torch.float16))), (ValueError, dict(q=_rows(4)[:, 0])),
                      (TypeError, dict(q=[1])), (AttributeError, dict(cache=3))]:
        with pytest.raises(error):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):
        call()


def test_router_refusals():
    x = torch.zeros(4, 64)
    for error, args, kw in [(ValueError, (x, 4), {}), (TypeError, (None, 4), {}), (KeyError, (x, 4), dict(score="tanh"))]:
        with pytest.raises(error):
            fb.fp8_moe_route(*args, **kw)
    g, ids = torch.zeros(4, 2), torch.zeros(4, 2, dtype=I32)
    for bad in [(None, x, ids), (g, x, None), (g, x, ids)]:
        with pytest.raises((TypeError, ValueError)):
            fb.fp8_moe_route_backward(*bad)


def test_dispatch_refusals():
    x, ids = torch.zeros(4, 128, dtype=BF), torch.zeros(4, 2, dtype=I32)
    for error, args in [(ValueError, (x, ids[:3], 8)), (ValueError, (x, ids.long(), 8)), (ValueError, (x, ids[:, 0], 8)), (ValueError, (x[0], ids, 8)),
                        (ValueError, (x.t(), torch.zeros(128, 2, dtype=I32), 8)), (ValueError, (x, ids.t().contiguous().t(), 8)), (TypeError, (x, 3, 8))]:
        with pytest.raises(error):
            fb.fp8_moe_dispatch(*args)
    with pytest.raises(ValueError, match="GPU"):
        fb.fp8_moe_dispatch(x, ids, 8)
