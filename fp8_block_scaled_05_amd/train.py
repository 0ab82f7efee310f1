"""The operators of a training step around the FP8 GEMMs of one layer (include/fp8bs_train.h): the norm in front of a
GEMM and the gated activation between two, quantized on the way out, their gradients, the experts' weight gradients,
and the norm of all gradients with their clipping.

Like the rest of the binding this only marshals arguments onto the library's entry points of the same names, through
the native module that decoder.py loads.  A call goes on the current stream of its tensors' device.
"""
from . import BF16, F32, _torch
from . import decoder as _decoder

__all__ = ["fp8_rmsnorm_quant", "fp8_rmsnorm_backward", "fp8_swiglu_quant", "fp8_swiglu_backward", "fp8_quant_grouped_t",
           "fp8_blockscaled_grouped_wgrad", "fp8_grad_norm", "fp8_grad_clip"]

_done = _decoder._done


def _stream_of(device):
    """A device's current stream's handle.  The first call puts torch's own function in this one's place: importing the
    package does not load torch."""
    global _stream_of
    _stream_of = _torch()._C._cuda_getCurrentRawStream
    return _stream_of(device)


def fp8_rmsnorm_quant(x, weight=None, residual=None, eps=1e-6, quantize=True, with_y=False, residual_out=None, y=None, q=None, scale=None):
    """h = x + residual (rounded to x's type), then y = h / sqrt(mean(h^2) + eps) * weight, quantized in 1x128 tiles:
    returns (q uint8 [T, H], scale f32 [T, H/128], y like x, residual_out like x).

    x, residual [T, H] bfloat16 or float32, weight [H] bfloat16 or float32.  q and scale are None without quantize, y
    without with_y, residual_out (which is h) without a residual.  q is quantized from the float32 y.  residual_out and y
    may each be residual or x itself; other outputs that share memory with an input or each other are refused, here and
    in the calls below.
    """
    return _done(_decoder._marshal.rmsnorm_quant(x, weight, residual, eps, quantize, with_y, residual_out, y, q, scale, _stream_of))


def fp8_rmsnorm_backward(dy, h, weight=None, dresidual=None, eps=1e-6, dx=None, dweight=None):
    """Gradient of fp8_rmsnorm_quant's y with respect to h (x or, with a residual, residual_out) and the weight:
    (dx like h, dweight f32 [H] or None without a weight).

    dresidual: what reaches residual_out from behind, added to dx, which is then the gradient of x and of residual alike.
    dx may be dy, h or dresidual itself.
    """
    return _done(_decoder._marshal.rmsnorm_backward(dy, h, weight, dresidual, eps, dx, dweight, _stream_of))


def fp8_swiglu_quant(gate, up, quantize=True, with_y=False, y=None, q=None, scale=None):
    """y = gate * sigmoid(gate) * up, quantized in 1x128 tiles: (q uint8 [T, F], scale f32 [T, F/128], y like gate).

    gate, up [T, F] bfloat16 or float32 (the halves of one GEMM's output will do).  q and scale are None without
    quantize, y without with_y.  y may be gate or up itself.
    """
    return _done(_decoder._marshal.swiglu_quant(gate, up, quantize, with_y, y, q, scale, _stream_of))


def fp8_swiglu_backward(dy, gate, up, quantize=True, with_d=False, d=None, q=None, scale=None):
    """Gradient of fp8_swiglu_quant's y, d = [d gate | d up] as one matrix: (q uint8 [T, 2F], scale f32 [T, 2F/128],
    d [T, 2F] like gate).  q and scale are None without quantize, d without with_d.  d may be the matrix whose halves
    gate and up are."""
    return _done(_decoder._marshal.swiglu_backward(dy, gate, up, quantize, with_d, d, q, scale, _stream_of))


def fp8_quant_grouped_t(x, offsets, order=None, top_k=1, q=None, scale=None, padded=None):
    """An operand of the experts' weight gradients: rows transposed and quantized in 128x1 tiles that start anew at
    every expert, with power-of-two scales: (q uint8 [H, P], scale f32 [H, P/128], padded int32 [experts+1]).

    x [T, H] bfloat16 or float32; offsets int32 [experts+1] as fp8_moe_dispatch gives them.  Place p is row p of x, or
    with order (int32 [places], fp8_moe_dispatch's) row order[p] // top_k: the rows need not be gathered first.  Expert
    e's places start at column padded[e].  P bounds what any offsets take; columns from padded[-1] on are not written.
    """
    return _done(_decoder._marshal.quant_grouped_t(x, offsets, order, top_k, q, scale, padded, _stream_of))


def fp8_blockscaled_grouped_wgrad(padded, a, a_scale, b, b_scale, out_dtype=None, y=None, accumulate=False):
    """The experts' weight gradients y[e] = A_e . B_e^T over each expert's own columns: [experts, N, K], float32 or
    bfloat16.  a [N, P] and b [K, P] with their scales as fp8_quant_grouped_t gives them, for the output's gradient and
    the input; padded from either.  accumulate: added to the given y."""
    torch = _torch()
    code = {None: -1, torch.bfloat16: BF16, torch.float32: F32}.get(out_dtype)
    if code is None:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {out_dtype}")
    return _done(_decoder._marshal.grouped_wgrad(padded, a, a_scale, b, b_scale, code, y, accumulate, _stream_of))


def fp8_grad_norm(grads, norm=None):
    """The 2-norm of all elements of a list of tensors (bfloat16 or float32, any shapes): float32 [1], summed in 64 bits.
    Over several ranks' parts: the root of the sum of their norms' squares."""
    return _done(_decoder._marshal.grad_norm(grads, norm, _stream_of))


def fp8_grad_clip(grads, norm, max_norm, outs=None):
    """Scales the tensors by max_norm / norm where norm (float32 [1], read on the GPU) is finite and above max_norm, in
    place or into outs; returns those.  No tensor that is written may share memory with another one (a gradient of shared
    weights belongs into the list once)."""
    return _done(_decoder._marshal.grad_clip(grads, norm, max_norm, outs, _stream_of))
