"""The operators between the FP8 GEMMs of a decoder layer (include/fp8bs_decoder.h): the paged 8-bit
key/value cache and the mixture-of-experts routing.

Like the rest of the binding this only marshals arguments onto the library's entry points of the same
names, on PyTorch's current stream.  A decode step makes these calls in every layer, so the checks are
written to cost little: argument structs (every field 8 bytes) are packed in one go.
"""
import struct

import torch

from . import _check, _dtype_code, _need, _on_gpu, _ptr, _stream, lib

__all__ = ["KVCache", "fp8_kv_append", "fp8_kv_attention", "fp8_moe_route", "fp8_moe_route_backward", "fp8_moe_dispatch"]

ROPE = {"half": 0, "interleaved": 1}
SCORE = {"sigmoid": 0, "softmax": 1}

_CACHE = struct.Struct("4Q4q")         # fp8bs_kv_cache
_BATCH = struct.Struct("3Q6q")         # fp8bs_kv_batch
_APPEND = struct.Struct("7Q10qd")      # fp8bs_kv_append_args
_ATTEND = struct.Struct("4Q5qd")       # fp8bs_kv_attention_args


class KVCache:
    """A paged cache: k, v uint8 [pages, kv_heads, page_size, head_dim] (E4M3 codes) and k_scale, v_scale
    float32 [pages, kv_heads] (powers of two), all contiguous.  The tensors stay the caller's."""
    __slots__ = ("k", "v", "k_scale", "v_scale", "device", "args")

    def __init__(self, k, v, k_scale, v_scale):
        shape = k.shape
        if len(shape) != 4:
            raise ValueError(f"k must be [pages, kv_heads, page_size, head_dim], got {tuple(shape)}")
        for t, want, dtype, name in ((k, shape, torch.uint8, "k"), (v, shape, torch.uint8, "v"),
                                     (k_scale, shape[:2], torch.float32, "k_scale"), (v_scale, shape[:2], torch.float32, "v_scale")):
            if t.shape != want or t.dtype != dtype:
                _need(t, want, dtype, name)
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        _on_gpu(k, v, k_scale, v_scale)
        self.k, self.v, self.k_scale, self.v_scale, self.device = k, v, k_scale, v_scale, k.device
        self.args = _CACHE.pack(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), *shape)

    @staticmethod
    def empty(pages, kv_heads, page_size, head_dim, device="cuda"):
        """An empty cache (zero codes, unit scales)."""
        codes = [torch.zeros(pages, kv_heads, page_size, head_dim, dtype=torch.uint8, device=device) for _ in range(2)]
        return KVCache(*codes, *[torch.ones(pages, kv_heads, dtype=torch.float32, device=device) for _ in range(2)])


def _batch(cu, seq_lens, block_table, tokens, max_new, max_len):
    i32 = torch.int32
    n = seq_lens.shape[0]
    if cu.dtype != i32 or seq_lens.dtype != i32 or block_table.dtype != i32:
        raise TypeError("cu, seq_lens and block_table must be int32")
    if cu.shape != (n + 1,) or seq_lens.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != n:
        raise ValueError(f"cu [B+1], seq_lens [B] and block_table [B, width] expected, got {tuple(cu.shape)}, "
                         f"{tuple(seq_lens.shape)}, {tuple(block_table.shape)}")
    width = block_table.shape[1]
    if not (cu.is_cuda and seq_lens.is_cuda and block_table.is_cuda):
        _on_gpu(cu, seq_lens, block_table)
    if not (cu.is_contiguous() and seq_lens.is_contiguous()) or (width > 1 and block_table.stride(1) != 1):
        raise ValueError("cu and seq_lens must be contiguous, block_table must have unit column stride")
    pitch = block_table.stride(0) if n > 1 else width
    return _BATCH.pack(cu.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(), pitch, width, n, tokens, max_new, max_len)


def _rows(t, heads, dim, tokens, name):
    """Pointer and pitches of a bfloat16 [tokens, heads, dim] tensor."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be bfloat16, got {t.dtype}")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, dim)}")
    if not t.is_cuda:
        _on_gpu(t)
    ld, hs, es = t.stride()
    if es != 1:
        raise ValueError(f"{name} must have unit stride within a head")
    return t.data_ptr(), (ld if tokens > 1 else heads * dim), (hs if heads > 1 else dim)


def fp8_kv_append(q, k, v, cache, cu, seq_lens, block_table, max_new, rope=None, rope_layout="half", q_weight=None, k_weight=None,
                  eps=1e-6, q_out=None):
    """Appends the new tokens' keys and values to the cache (in place) and returns the treated queries.

    q [T, Hq, D], k, v [T, Hk, D] bfloat16 (slices of one projection's output will do); per head: norm with
    q_weight / k_weight (bfloat16 [D] or None) and eps, rotation by rope (float32 [positions, rot], cos | sin of
    each position, or None) in the "half" or "interleaved" layout, then the E4M3 store with one power-of-two
    scale per page and head.  q None: only the cache is written and None is returned.
    cu int32 [B+1], seq_lens int32 [B] (the new tokens included), block_table int32 [B, width].
    """
    tokens, heads, dim = k.shape
    shape = cache.k.shape
    kp = _rows(k, shape[1], shape[3], tokens, "k")
    vp = _rows(v, shape[1], shape[3], tokens, "v")
    q_heads, qp, out = 0, (0, 0, 0), 0
    if q is not None:
        q_heads = q.shape[1]
        qp = _rows(q, q_heads, dim, tokens, "q")
        if q_out is None:
            q_out = torch.empty((tokens, q_heads, dim), dtype=torch.bfloat16, device=q.device)
        else:
            _on_gpu(q_out)
            _need(q_out, (tokens, q_heads, dim), torch.bfloat16, "q_out")
            if not q_out.is_contiguous():
                raise ValueError("q_out must be contiguous")
        out = q_out.data_ptr()
    rot = rows = rp = 0
    if rope is not None:
        if rope.dtype != torch.float32 or rope.dim() != 2 or not rope.is_contiguous():
            raise ValueError("rope must be a contiguous float32 [positions, rot] table")
        _on_gpu(rope)
        rows, rot = rope.shape
        rp = rope.data_ptr()
    wp = [0, 0]
    for i, (w, name) in enumerate(((q_weight, "q_weight"), (k_weight, "k_weight"))):
        if w is not None:
            _on_gpu(w)
            _need(w, (dim,), torch.bfloat16, name)
            if not w.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
            wp[i] = w.data_ptr()
    batch = _batch(cu, seq_lens, block_table, tokens, max_new, 1 << 30)
    args = _APPEND.pack(qp[0], kp[0], vp[0], out, rp, wp[0], wp[1], qp[1], qp[2], kp[1], kp[2], vp[1], vp[2], q_heads, rows, rot,
                        ROPE[rope_layout], eps)
    status = lib().fp8_kv_append(cache.args, batch, args, _stream())
    if status:
        _check(status)
    return q_out


def fp8_kv_attention(q, cache, cu, seq_lens, block_table, max_new, max_len, window=0, softmax_scale=None, return_lse=False, out=None):
    """Causal attention of the new tokens (already appended) over the cache.

    q bfloat16 [T, Hq, D]; returns out bfloat16 [T, Hq, D], with return_lse also the float32 [T, Hq] log of each
    row's sum of exponentials.  window > 0: only the last `window` positions up to a token's own are seen.
    max_new and max_len bound the sequences' new tokens and lengths.  softmax_scale None: 1 / sqrt(D).
    """
    tokens, heads, dim = q.shape
    if dim != cache.k.shape[3]:
        raise ValueError(f"q has head_dim {dim}, the cache {cache.k.shape[3]}")
    ptr, ld, hs = _rows(q, heads, dim, tokens, "q")
    if out is None:
        out = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=q.device)
    else:
        _on_gpu(out)
        _need(out, (tokens, heads, dim), torch.bfloat16, "out")
        if not out.is_contiguous():
            raise ValueError("out must be contiguous")
    lse = torch.empty((tokens, heads), dtype=torch.float32, device=q.device) if return_lse else None
    batch = _batch(cu, seq_lens, block_table, tokens, max_new, max_len)
    scale = dim ** -0.5 if softmax_scale is None else softmax_scale
    where = (ptr, out.data_ptr(), lse.data_ptr() if return_lse else 0)
    L = lib()
    args = _ATTEND.pack(*where, 0, 0, ld, hs, heads, window, scale)
    need = L.fp8_kv_attention_workspace(cache.args, batch, args)
    if need > 0:
        room = torch.empty(need, dtype=torch.uint8, device=q.device)
        args = _ATTEND.pack(*where, room.data_ptr(), need, ld, hs, heads, window, scale)
    status = L.fp8_kv_attention(cache.args, batch, args, _stream())
    if status:
        _check(status)
    return (out, lse) if return_lse else out


def _matrix(t, name):
    """Pitch of a 2-D tensor with unit column stride."""
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.stride(0) if rows > 1 else cols


def fp8_moe_route(logits, top_k, score="sigmoid", bias=None, groups=1, top_groups=None, renormalize=True, scale=1.0, ids=None,
                  weights=None):
    """The top_k experts of each token and their weights: (ids int32 [T, top_k], weights float32 [T, top_k]).

    logits [T, E] float32 or bfloat16; score "sigmoid" or "softmax"; bias float32 [E] joins the scores for the
    choice only; groups / top_groups restrict it to the groups of experts with the best sums of their two best.
    """
    tokens, experts = logits.shape
    _on_gpu(logits, bias, ids, weights)
    if bias is not None:
        _need(bias, (experts,), torch.float32, "bias")
        if not bias.is_contiguous():
            raise ValueError("bias must be contiguous")
    if ids is None:
        ids = torch.empty((tokens, top_k), dtype=torch.int32, device=logits.device)
    if weights is None:
        weights = torch.empty((tokens, top_k), dtype=torch.float32, device=logits.device)
    _need(ids, (tokens, top_k), torch.int32, "ids")
    _need(weights, (tokens, top_k), torch.float32, "weights")
    if not (ids.is_contiguous() and weights.is_contiguous()):
        raise ValueError("ids and weights must be contiguous")
    status = lib().fp8_moe_route(logits.data_ptr(), _dtype_code(logits, "logits"), tokens, experts, _matrix(logits, "logits"), SCORE[score],
                                 _ptr(bias), groups, groups if top_groups is None else top_groups, top_k, bool(renormalize), scale,
                                 ids.data_ptr(), weights.data_ptr(), _stream())
    if status:
        _check(status)
    return ids, weights


def fp8_moe_route_backward(grad, logits, ids, score="sigmoid", renormalize=True, scale=1.0, dlogits=None):
    """Gradient of fp8_moe_route's weights with respect to the logits, given grad float32 [T, top_k] of the weights:
    a tensor like logits."""
    tokens, experts = logits.shape
    top_k = ids.shape[1]
    _on_gpu(grad, logits, ids, dlogits)
    _need(ids, (tokens, top_k), torch.int32, "ids")
    _need(grad, (tokens, top_k), torch.float32, "grad")
    if not (ids.is_contiguous() and grad.is_contiguous()):
        raise ValueError("ids and grad must be contiguous")
    if dlogits is None:
        dlogits = torch.empty((tokens, experts), dtype=logits.dtype, device=logits.device)
    _need(dlogits, (tokens, experts), logits.dtype, "dlogits")
    status = lib().fp8_moe_route_backward(grad.data_ptr(), logits.data_ptr(), _dtype_code(logits, "logits"), tokens, experts,
                                          _matrix(logits, "logits"), ids.data_ptr(), top_k, SCORE[score], bool(renormalize), scale,
                                          dlogits.data_ptr(), _matrix(dlogits, "dlogits"), _stream())
    if status:
        _check(status)
    return dlogits


def fp8_moe_dispatch(x, ids, experts, q=None, scale=None):
    """The rows of x on their way to the experts: (q uint8 [T*top_k, H], scale float32 [T*top_k, H/128],
    offsets int32 [experts+1], order int32 [T*top_k], position int32 [T, top_k]).

    q, scale and offsets are the A operand of fp8_blockscaled_grouped_gemm; row p is token order[p] // top_k,
    and the result for choice (t, j) stands in row position[t, j].  Choices outside [0, experts) come last, as
    zero rows.
    """
    tokens, cols = x.shape
    if ids.dim() != 2 or ids.shape[0] != tokens or ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 [T, top_k] tensor")
    top_k = ids.shape[1]
    n, dev = tokens * top_k, x.device
    _on_gpu(x, ids, q, scale)
    if q is None:
        q = torch.empty((n, cols), dtype=torch.uint8, device=dev)
    if scale is None:
        scale = torch.empty((n, cols // 128), dtype=torch.float32, device=dev)
    _need(q, (n, cols), torch.uint8, "q")
    _need(scale, (n, cols // 128), torch.float32, "scale")
    if not (q.is_contiguous() and scale.is_contiguous()):
        raise ValueError("q and scale must be contiguous")
    offsets = torch.empty(max(experts, 0) + 1, dtype=torch.int32, device=dev)
    order = torch.empty(n, dtype=torch.int32, device=dev)
    position = torch.empty((tokens, top_k), dtype=torch.int32, device=dev)
    L = lib()
    need = L.fp8_moe_dispatch_workspace(tokens, experts, top_k)
    room = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    status = L.fp8_moe_dispatch(x.data_ptr(), _dtype_code(x, "x"), tokens, cols, _matrix(x, "x"), ids.data_ptr(), top_k, experts,
                                q.data_ptr(), scale.data_ptr(), offsets.data_ptr(), order.data_ptr(), position.data_ptr(),
                                _ptr(room), max(need, 0), _stream())
    if status:
        _check(status)
    return q, scale, offsets, order, position
