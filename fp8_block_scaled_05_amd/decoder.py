"""The operators between the FP8 GEMMs of a decoder layer (include/fp8bs_decoder.h): the paged 8-bit
key/value cache and the mixture-of-experts routing.

Like the rest of the binding this only marshals arguments onto the library's entry points of the same
names, on PyTorch's current stream.  A decode step makes these calls in every layer, so the tensors are
checked and their fields read by a native module (csrc/marshal.cpp), which the first call loads.
"""
import os
import struct

from . import _PKG, _check, _stream, _torch, lib

__all__ = ["KVCache", "fp8_kv_append", "fp8_kv_attention", "fp8_moe_route", "fp8_moe_route_backward", "fp8_moe_dispatch"]

ROPE = {"half": 0, "interleaved": 1}
SCORE = {"sigmoid": 0, "softmax": 1}

# The header's argument structs, for callers of the C entry points through lib().
_CACHE = struct.Struct("4Q4q")         # fp8bs_kv_cache
_BATCH = struct.Struct("3Q6q")         # fp8bs_kv_batch
_APPEND = struct.Struct("7Q10qd")      # fp8bs_kv_append_args
_ATTEND = struct.Struct("4Q5qd")       # fp8bs_kv_attention_args


MARSHAL_PATH = os.path.join(_PKG, "_marshal.so")


class _Unloaded:
    """Stands for the native module until a call asks for one of its functions."""

    def __getattr__(self, name):
        global _marshal
        lib(), _torch()                # the module is linked to both
        if not os.path.exists(MARSHAL_PATH):
            raise ImportError(f"{MARSHAL_PATH} is missing: build it with `python -m fp8_block_scaled_05_amd.build`")
        from . import _marshal as native
        _marshal = native
        return getattr(native, name)


_marshal = _Unloaded()


def _done(result):
    """The outputs of a call; its status raises."""
    if result.__class__ is int:
        _check(result)
    return result


class KVCache:
    """A paged cache: k, v uint8 [pages, kv_heads, page_size, head_dim] (E4M3 codes) and k_scale, v_scale
    float32 [pages, kv_heads] (powers of two), all contiguous.  The tensors stay the caller's, and are the cache's
    for good: other tensors take another KVCache.  Where a call finds their memory is read at that call."""
    __slots__ = ("args",)

    def __init__(self, k, v, k_scale, v_scale):
        object.__setattr__(self, "args", _marshal.cache(k, v, k_scale, v_scale))

    def __setattr__(self, name, value):
        raise AttributeError(f"{name}: a KVCache keeps its tensors; make another one for others")

    def __reduce__(self):              # copies are built anew, of copied tensors
        return KVCache, self.args

    k = property(lambda self: self.args[0])
    v = property(lambda self: self.args[1])
    k_scale = property(lambda self: self.args[2])
    v_scale = property(lambda self: self.args[3])

    @staticmethod
    def empty(pages, kv_heads, page_size, head_dim, device="cuda"):
        """An empty cache (zero codes, unit scales)."""
        torch = _torch()
        codes = [torch.zeros(pages, kv_heads, page_size, head_dim, dtype=torch.uint8, device=device) for _ in range(2)]
        return KVCache(*codes, *[torch.ones(pages, kv_heads, dtype=torch.float32, device=device) for _ in range(2)])


def fp8_kv_append(q, k, v, cache, cu, seq_lens, block_table, max_new, rope=None, rope_layout="half", q_weight=None, k_weight=None,
                  eps=1e-6, q_out=None):
    """Appends the new tokens' keys and values to the cache (in place) and returns the treated queries.

    q [T, Hq, D], k, v [T, Hk, D] bfloat16 (slices of one projection's output will do); per head: norm with
    q_weight / k_weight (bfloat16 [D] or None) and eps, rotation by rope (float32 [positions, rot], cos | sin of
    each position, or None) in the "half" or "interleaved" layout, then the E4M3 store with one power-of-two
    scale per page and head.  q None: only the cache is written and None is returned.
    cu int32 [B+1], seq_lens int32 [B] (the new tokens included), block_table int32 [B, width].
    """
    return _done(_marshal.kv_append(q, k, v, cache.args, cu, seq_lens, block_table, max_new, rope, ROPE[rope_layout], q_weight, k_weight,
                                    eps, q_out, _stream))


def fp8_kv_attention(q, cache, cu, seq_lens, block_table, max_new, max_len, window=0, softmax_scale=None, return_lse=False, out=None):
    """Causal attention of the new tokens (already appended) over the cache.

    q bfloat16 [T, Hq, D]; returns out bfloat16 [T, Hq, D], with return_lse also the float32 [T, Hq] log of each
    row's sum of exponentials.  window > 0: only the last `window` positions up to a token's own are seen.
    max_new and max_len bound the sequences' new tokens and lengths.  softmax_scale None: 1 / sqrt(D).
    """
    return _done(_marshal.kv_attention(q, cache.args, cu, seq_lens, block_table, max_new, max_len, window, softmax_scale, return_lse, out,
                                       _stream))


def fp8_moe_route(logits, top_k, score="sigmoid", bias=None, groups=1, top_groups=None, renormalize=True, scale=1.0, ids=None,
                  weights=None):
    """The top_k experts of each token and their weights: (ids int32 [T, top_k], weights float32 [T, top_k]).

    logits [T, E] float32 or bfloat16; score "sigmoid" or "softmax"; bias float32 [E] joins the scores for the
    choice only; groups / top_groups restrict it to the groups of experts with the best sums of their two best.
    """
    return _done(_marshal.moe_route(logits, top_k, SCORE[score], bias, groups, top_groups, renormalize, scale, ids, weights, _stream))


def fp8_moe_route_backward(grad, logits, ids, score="sigmoid", renormalize=True, scale=1.0, dlogits=None):
    """Gradient of fp8_moe_route's weights with respect to the logits, given grad float32 [T, top_k] of the weights:
    a tensor like logits."""
    return _done(_marshal.moe_route_backward(grad, logits, ids, SCORE[score], renormalize, scale, dlogits, _stream))


def fp8_moe_dispatch(x, ids, experts, q=None, scale=None):
    """The rows of x on their way to the experts: (q uint8 [T*top_k, H], scale float32 [T*top_k, H/128],
    offsets int32 [experts+1], order int32 [T*top_k], position int32 [T, top_k]).

    q, scale and offsets are the A operand of fp8_blockscaled_grouped_gemm; row p is token order[p] // top_k,
    and the result for choice (t, j) stands in row position[t, j].  Choices outside [0, experts) come last, as
    zero rows.
    """
    return _done(_marshal.moe_dispatch(x, ids, experts, q, scale, _stream))
