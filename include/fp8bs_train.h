/*
 * fp8bs_train.h - the operators around the FP8 GEMMs of one layer's training
 * step, part of libfp8bs.so (gfx950): the norm in front of a GEMM and its
 * gradient, the gated activation between an expert's two GEMMs and its
 * gradient, the experts' weight gradients over ragged numbers of tokens, and
 * the norm of all gradients with their clipping.
 *
 * The conventions of fp8bs.h hold: device pointers owned by the caller,
 * nothing allocated, no state between calls, no synchronization, work on the
 * caller's stream, synchronous validation with nothing enqueued when it
 * fails, 16-byte aligned rows (pointers and pitches), zero rows a no-op.
 * Every call may be captured in a HIP graph.  Argument structs and arrays of
 * descriptors are HOST memory, read during the call only.  For given
 * arguments no result changes from run to run.  Arithmetic is float32 (or
 * wider where it says so), each output is rounded once, to nearest even.
 * Inputs must be finite: a NaN or infinity leaves its own row's outputs
 * unspecified (its own column's too where an output is a sum over rows, its
 * tile's codes and scale for the transposed tiles) and every other one alone.
 * One exception: in h of the norm's gradient it leaves all of dweight
 * unspecified, of which every part has that row's root as a factor.
 */
#ifndef FP8BS_TRAIN_H
#define FP8BS_TRAIN_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Root-mean-square norm of rows, with the residual's addition in front and
 * the 1x128 quantization behind.  Per row:
 *   h = x + residual, rounded to dtype (h = x without a residual);
 *   y = h * rsqrt(mean(h^2) + eps) * weight     (weight 1 where it is NULL).
 * Outputs, each where its pointer is given:
 *   residual_out  h, what the next residual addition and the gradient read;
 *   y             rounded to dtype;
 *   q, scale      the float32 y quantized exactly as fp8_quant_act_1x128
 *                 quantizes a float32 input: codes, pitch ld_q, and
 *                 [rows, cols/128] scales.
 * residual_out needs a residual; at least one of y and q is asked for; q and
 * scale come together.  residual_out and y may each be x or residual itself (the
 * same pointer and pitch); otherwise no output may overlap an input or another
 * output (FP8BS_ERR_INVALID_ARG, here and below).
 *
 * x, residual, residual_out, y: [rows, cols] of dtype (bf16 or f32).
 * weight: [cols] of w_dtype, 16-byte aligned, or NULL.
 * cols: a multiple of 128, at most 32768.  eps: a positive normal float32.
 * |h| up to 2^60; a row whose squares' sum is beyond what is held (8 to 32 of
 * them in float32, those sums in 64 bits) comes out as NaN.
 */
typedef struct fp8bs_rmsnorm_args {
  const void* x;
  const void* residual;
  const void* weight;
  void* residual_out;
  void* y;
  uint8_t* q;
  float* scale;
  int64_t rows, cols;
  int64_t ld_x, ld_residual, ld_residual_out, ld_y, ld_q;
  int64_t dtype, w_dtype;     /* fp8bs_dtype */
  double eps;
} fp8bs_rmsnorm_args;

fp8bs_status fp8_rmsnorm_quant(const fp8bs_rmsnorm_args* args, hipStream_t stream);

/*
 * Gradient of the norm, through its y (a quantizer passes its gradient on
 * unchanged).  With r = rsqrt(mean(h^2) + eps), formed anew from h, and
 * g = dy * weight:
 *   dx      = r * (g - h * r^2 * mean(g * h)) + dresidual;
 *   dweight = sum over rows of dy * h * r.
 * dx is the gradient of x and of residual alike.
 *
 * dy, h, dresidual, dx: [rows, cols] of dtype; dresidual (what reaches
 * residual_out from behind) may be NULL.  dx may be dy, h or dresidual itself
 * (the same pointer and pitch).
 * |h|, |dy| and |dy * weight| up to 2^60.
 * dweight: float32 [cols], 16-byte aligned, written (zeros for zero rows), or
 * NULL.  No other output or workspace may overlap an input or another output.
 * workspace: at least fp8_rmsnorm_backward_workspace(rows, cols) bytes where
 * dweight is given, 16-byte aligned (NULL if that is 0); calls that may run at
 * the same time need their own.
 */
typedef struct fp8bs_rmsnorm_backward_args {
  const void* dy;
  const void* h;
  const void* weight;
  const void* dresidual;
  void* dx;
  float* dweight;
  void* workspace;
  int64_t workspace_bytes;
  int64_t rows, cols;
  int64_t ld_dy, ld_h, ld_dresidual, ld_dx;
  int64_t dtype, w_dtype;
  double eps;
} fp8bs_rmsnorm_backward_args;

fp8bs_status fp8_rmsnorm_backward(const fp8bs_rmsnorm_backward_args* args, hipStream_t stream);
/* Bytes of workspace for these sizes, or -1 if they are not valid. */
int64_t fp8_rmsnorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * Gated activation, quantized:  y = gate * sigmoid(gate) * up.
 * gate, up: [rows, cols] of dtype, each with its pitch (the two halves of one
 * GEMM's output, for example).  Outputs, each where its pointer is given, at
 * least one of them:
 *   y         [rows, cols] of dtype, rounded;
 *   q, scale  the float32 y quantized exactly as fp8_quant_act_1x128
 *             quantizes a float32 input.
 * cols % 128 == 0.  y may be gate or up itself (the same pointer and pitch);
 * otherwise no output may overlap an input or another output.
 * Inputs of any size: up multiplies gate * sigmoid(gate), which is no larger
 * than gate.  An exponential of a gate below -87 may count as 0, an error of
 * at most 2^-119 |up|.
 */
typedef struct fp8bs_swiglu_args {
  const void* gate;
  const void* up;
  void* y;
  uint8_t* q;
  float* scale;
  int64_t rows, cols;
  int64_t ld_gate, ld_up, ld_y, ld_q;
  int64_t dtype;
} fp8bs_swiglu_args;

fp8bs_status fp8_swiglu_quant(const fp8bs_swiglu_args* args, hipStream_t stream);

/*
 * Its gradient, as one matrix [rows, 2 cols], the layout of a GEMM output
 * whose halves are gate and up.  With s = sigmoid(gate):
 *   d[:, :cols] = dy * up * s * (1 + gate * (1 - s));
 *   d[:, cols:] = dy * gate * s.
 * Outputs, each where its pointer is given, at least one of them: d of dtype,
 * rounded; q [rows, 2 cols] and scale [rows, 2 cols / 128], the float32 values
 * quantized in 1x128 tiles.  Each half of d may be gate, up or dy itself (the same
 * pointer and pitch), so d the matrix that holds gate and up; no other overlap.
 * Inputs of any size, but |dy| up to 2^127: it multiplies the activation's
 * slope, at most 1.1, before up does.  Below gates of -87 as above: errors of
 * at most 2^-119 |dy up| and 2^-119 |dy|.
 */
typedef struct fp8bs_swiglu_backward_args {
  const void* dy;
  const void* gate;
  const void* up;
  void* d;
  uint8_t* q;
  float* scale;
  int64_t rows, cols;
  int64_t ld_dy, ld_gate, ld_up, ld_d, ld_q;
  int64_t dtype;
} fp8bs_swiglu_backward_args;

fp8bs_status fp8_swiglu_backward(const fp8bs_swiglu_backward_args* args, hipStream_t stream);

/*
 * Operands of the experts' weight gradients, whose products run over each
 * expert's own rows: the rows, transposed and quantized in 128x1 tiles that
 * start anew at every expert.
 *
 * Place p (0 <= p < places) is row p of x, or with `order` row
 * order[p] / top_k of x: fp8_moe_dispatch's order, so that the rows need not
 * be laid out by expert first.  An order outside [0, rows * top_k) stands for
 * a row of zeros.  Expert g owns places [off[g], off[g+1]); off is read as
 * fp8_blockscaled_grouped_gemm reads it (clamped into [0, places], each expert
 * starting no earlier than the previous one ends).
 *   padded[g]  128 * sum over f < g of ceil(places of f / 128), padded[G] the end;
 *   q          [cols, columns] codes: row c holds column c of x, expert g's
 *              places from column padded[g] on, then zeros up to padded[g+1];
 *   scale      [cols, columns / 128]: the smallest power of two 2^e, e >= -100,
 *              with amax <= 448 * 2^e over the tile, 1 for a tile of zeros;
 *              code = E4M3_RNE(x * 2^-e), at e = 120 (amax > 1.75 * 2^127) at
 *              most 240 in magnitude: 256 * 2^120 is beyond float32.
 * Columns from padded[G] on, of q and of scale, are left as they are.
 * The GEMM below applies a power of two while it widens the codes, exactly.
 * Values keep E4M3's relative precision; at its small end a tile loses up to an
 * octave of range, against a scale of amax / 448.
 *
 * x: [rows, cols] of x_dtype, pitch ld_x; cols % 16 == 0.
 * off: DEVICE int32 [G+1], 1 <= G <= 1024.  order: DEVICE int32 [places], or
 * NULL with places == rows and top_k == 1.  1 <= top_k <= 1024.
 * columns: at least fp8_quant_grouped_t_columns(places, G), a multiple of 128,
 * at most 2^22; ld_q >= columns.  padded: DEVICE int32 [G+1].
 * places == 0 writes padded alone (zeros).  No output may overlap an input or
 * another output.
 */
fp8bs_status fp8_quant_grouped_t(const void* x, int32_t x_dtype, int64_t rows, int64_t cols,
                                 int64_t ld_x, const int32_t* off, int32_t G,
                                 const int32_t* order, int64_t places, int32_t top_k,
                                 uint8_t* q, int64_t ld_q, float* scale, int64_t columns,
                                 int32_t* padded, hipStream_t stream);
/* 128 * the most tiles that `places` rows of G experts take, or -1 if the
 * sizes are not valid. */
int64_t fp8_quant_grouped_t_columns(int64_t places, int32_t G);

/*
 * The experts' weight gradients:
 *   y[g][n][k] (+)= sum over p in [padded[g], padded[g+1]) of
 *                   a[n,p] a_scale[n,p/128] * b[k,p] b_scale[k,p/128].
 * a: [N, columns] codes, pitch lda, and b: [K, columns], pitch ldb: the output
 * gradient's and the input's operands as fp8_quant_grouped_t writes them;
 * a_scale [N, columns/128], b_scale [K, columns/128] dense.
 * Scales must be powers of two from 2^-100 to 2^120, and a code times its scale
 * below 2^128, as that call writes them: the codes are widened to bf16 with the
 * scale applied (exactly), multiplied on the bf16 matrix cores and summed in
 * float32.  A scale that is no power of two or beyond that range makes the
 * results it belongs to NaN, and others of its expert; a value that is not
 * below 2^128 widens to infinity.
 * padded: DEVICE int32 [G+1], multiples of 128 (what a value exceeds one by is
 * dropped), read clamped into [0, columns]; an expert whose end lies before its
 * start has no rows.
 * y: [G, N, K] of y_dtype, dense, apart from the inputs.  accumulate 0: written, zeros for an expert
 * without rows; 1: added to (float32 sum, rounded once).
 * N % 16 == 0, K % 16 == 0, both at most 2^26, 1 <= G <= 1024, columns % 128
 * == 0 and at most 2^22 (lda and ldb too).
 * Accuracy, where no product and no sum passes float32's range: |y - exact| <=
 * depth * (2^-24 * sum |a b| + 2^-126), depth the expert's columns (+ half a
 * step of y_dtype; with accumulate the rounding of that sum).  2^-126: products
 * below float32's normal range, as of two operands with scales near 2^-100, may
 * count as zero.
 */
fp8bs_status fp8_blockscaled_grouped_wgrad(int64_t N, int64_t K, int64_t columns, int32_t G,
                                           const int32_t* padded, const uint8_t* a, int64_t lda,
                                           const float* a_scale, const uint8_t* b, int64_t ldb,
                                           const float* b_scale, void* y, int32_t y_dtype,
                                           int32_t accumulate, hipStream_t stream);

/*
 * The gradients of a step: n tensors of any lengths, each dense, of its own
 * type, aligned to its element.  p may be NULL where count is 0.
 */
typedef struct fp8bs_grad {
  void* p;
  int64_t count;
  int64_t dtype;              /* fp8bs_dtype */
} fp8bs_grad;

/*
 * norm[0] = sqrt(sum of all squares), summed in 64 bits, rounded once to
 * float32; 0 for no elements; NaN or infinity where a gradient is.  The norm
 * over several ranks' parts is the root of their squares' sum.
 * n: 0 .. 65536; norm: DEVICE float32[1].
 * workspace: at least fp8_grad_norm_workspace(grads, n) bytes, 16-byte
 * aligned (NULL if that is 0), apart from the tensors.
 */
fp8bs_status fp8_grad_norm(const fp8bs_grad* grads, int32_t n, float* norm, void* workspace,
                           int64_t workspace_bytes, hipStream_t stream);
int64_t fp8_grad_norm_workspace(const fp8bs_grad* grads, int32_t n);

/*
 * Clips: out = g * c, c = max_norm / norm[0] where norm[0] > max_norm and
 * norm[0] is finite, else 1 (a caller that skips steps of broken gradients
 * reads the norm).  norm is read on the device; the product is float32,
 * rounded to the tensor's type (c itself may lie below float32's range).  outs: n tensors of the same counts and types,
 * or NULL: in place, and where c is 1 nothing is touched.  outs[i] is
 * grads[i]'s own memory or overlaps no tensor of the call; a tensor that is
 * written overlaps no other one, and not norm (FP8BS_ERR_INVALID_ARG).
 * max_norm: finite, above 0 as a float32.
 */
fp8bs_status fp8_grad_clip(const fp8bs_grad* grads, const fp8bs_grad* outs, int32_t n,
                           const float* norm, double max_norm, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_TRAIN_H */
