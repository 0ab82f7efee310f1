/*
 * fp8bs_decoder.h - the operators that stand between the FP8 GEMMs of one
 * decoder layer, part of libfp8bs.so (gfx950): the 8-bit paged key/value
 * cache (append and attention) and the mixture-of-experts routing (router,
 * its gradient, dispatch of the rows to the experts as FP8 GEMM operands).
 *
 * The conventions of fp8bs.h hold: device pointers owned by the caller,
 * nothing allocated, no state between calls, no synchronization, work on the
 * caller's stream, synchronous validation with nothing enqueued when it
 * fails.  Every call may be captured in a HIP graph.  Argument structs are
 * HOST memory, read during the call only; every field is 8 bytes wide.
 *
 * The cache.  Position p of sequence b lives in page
 * block_table[b][p / page_size] at offset p % page_size.  k and v hold E4M3
 * codes [pages, kv_heads, page_size, head_dim] (dense, 16-byte aligned);
 * k_scale and v_scale hold one power of two per page and head,
 * [pages, kv_heads] float32: value = e4m3(code) * scale.
 *
 * The batch.  The new tokens of all sequences are packed: sequence b owns
 * rows [cu[b], cu[b+1]) of q, k, v.  seq_lens[b] counts its cached tokens
 * including the new ones, so new token i has position
 * seq_lens[b] - (cu[b+1] - cu[b]) + i.  cu, seq_lens and block_table are read
 * on the device only.  Whatever they hold, no access leaves the buffers that
 * the arguments describe: cu is clamped into [0, tokens], and cu[b+1] below
 * cu[b] counts as no new tokens; a position outside the block table's row, and
 * a page number outside [0, pages), is neither written nor seen.  Where cu
 * falls, sequences may claim the same rows: such rows of an output hold any of
 * their results or what they held, and tokens may not be stored.  At most
 * max_new tokens of a sequence and max_len positions are looked at.  Two sequences must not
 * have new tokens in the same page.
 */
#ifndef FP8BS_DECODER_H
#define FP8BS_DECODER_H

#include "fp8bs.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct fp8bs_kv_cache {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int64_t pages;
  int64_t kv_heads;
  int64_t page_size;          /* 16, 32, 64 or 128 */
  int64_t head_dim;           /* 64 or 128 */
} fp8bs_kv_cache;

typedef struct fp8bs_kv_batch {
  const int32_t* cu;          /* [batch + 1] */
  const int32_t* seq_lens;    /* [batch] */
  const int32_t* block_table; /* [batch, table_width], pitch ld_table */
  int64_t ld_table;
  int64_t table_width;
  int64_t batch;              /* 1 .. 65535 */
  int64_t tokens;             /* rows of q, k, v; at most 2^30 */
  int64_t max_new;            /* upper bound of cu[b+1] - cu[b] */
  int64_t max_len;            /* upper bound of seq_lens */
} fp8bs_kv_batch;

typedef enum fp8bs_rope_layout {
  FP8BS_ROPE_HALF = 0,        /* pairs (i, i + rot/2) */
  FP8BS_ROPE_INTERLEAVED = 1  /* pairs (2i, 2i + 1) */
} fp8bs_rope_layout;

/*
 * Append: per head, an optional norm of q and k, the position rotation, the
 * store of k and v into the cache.  For one row x of q or k (head_dim values,
 * float32 arithmetic):
 *   norm (weight given):  x = x * rsqrt(mean(x^2) + eps) * weight
 *   rotation (rot > 0):   pair (x1, x2) with angle i of its position p:
 *                         x1 c - x2 s, x2 c + x1 s, with
 *                         c = rope[p][i], s = rope[p][rot/2 + i]
 * q_out is the result rounded to bf16 (nearest even).  k (so treated) and v
 * (as it is) enter the cache.  For each page and head with new tokens the
 * scale's exponent is the smallest e >= -32 with amax(new) <= 448 * 2^e; where
 * the page already holds older tokens of the sequence (its first new token is
 * not at offset 0) e is at least the page's old exponent, and if it grew the
 * older codes are rounded to the new scale.  A code is
 * E4M3_RNE(value * 2^-e).  Bytes of the page past the last token keep what
 * they held.
 *
 * q, k, v:  bf16 [tokens, heads, head_dim] with unit element stride, 16-byte
 *           aligned, token pitch ld_* and head pitch hs_* in elements
 *           (multiples of 8): slices of one projection's output, for example.
 * q may be NULL with q_heads = 0 (cache only).  q_out is dense and may not
 * overlap an input.
 * rope:     float32 [rope_rows, rot], cos | sin; rot a multiple of 16 in
 *           0 .. head_dim; NULL with rot = 0.  A token whose position is
 *           outside [0, rope_rows) is not stored and its q_out row is zero.
 * q_weight, k_weight: bf16 [head_dim] or NULL (no norm of q / of k).
 * Inputs must be finite: a NaN or infinity gives unspecified codes and scale
 * for its page and head, and leaves every other page and head alone.
 * Limits: min(max_new, tokens) * q_heads < 2^31, and fewer than 2^24
 * workgroups, of which a call has at most
 *   3 (2 kv_heads (tokens / page_size + 2 batch) + tokens q_heads head_dim / 2^13 + batch).
 */
typedef struct fp8bs_kv_append_args {
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  const float* rope;
  const void* q_weight;
  const void* k_weight;
  int64_t ld_q, hs_q;
  int64_t ld_k, hs_k;
  int64_t ld_v, hs_v;
  int64_t q_heads;
  int64_t rope_rows;
  int64_t rot;
  int64_t rope_layout;        /* fp8bs_rope_layout */
  double eps;
} fp8bs_kv_append_args;

fp8bs_status fp8_kv_append(const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch,
                           const fp8bs_kv_append_args* args, hipStream_t stream);

/*
 * Attention of the new tokens over the cache (their own keys and values
 * already appended), causal, query heads grouped over kv heads
 * (head h reads kv head h / (q_heads / kv_heads)):
 *   z_j = softmax_scale * q . k_j  over positions j <= p, and p - j < window
 *         where window > 0;
 *   out = sum_j softmax(z)_j v_j;   lse = log sum_j exp(z_j).
 * A row that sees nothing gives out = 0 and lse = -infinity.  A row that sees
 * a key or value that is NaN becomes NaN; NaN in places that it does not see
 * (past the sequence's end, outside the window, in later tokens) does not
 * reach it.
 *
 * q:    bf16 [tokens, q_heads, head_dim], unit element stride, pitches ld_q,
 *       hs_q (multiples of 8), 16-byte aligned.
 * out:  bf16 [tokens, q_heads, head_dim], dense, 16-byte aligned.
 * lse:  float32 [tokens, q_heads], dense, or NULL.
 * workspace: device memory of at least
 *       fp8_kv_attention_workspace(cache, batch, args) bytes, 16-byte
 *       aligned (NULL if that is 0); its contents before and after the call
 *       mean nothing, and calls that may run at the same time need their own.
 * Products are of bf16 q and exactly widened cache values, summed in float32;
 * the softmax runs in float32; its weights are rounded to bf16 for the second
 * product.  For given arguments the result does not change from run to run.
 * Limits: min(max_new, tokens) * (q_heads / kv_heads) < 2^31, batch * kv_heads
 * < 2^23 and tokens * q_heads / 128 + batch * kv_heads < 2^23.
 */
typedef struct fp8bs_kv_attention_args {
  const void* q;
  void* out;
  float* lse;
  void* workspace;
  int64_t workspace_bytes;
  int64_t ld_q, hs_q;
  int64_t q_heads;
  int64_t window;             /* 0: no window */
  double softmax_scale;
} fp8bs_kv_attention_args;

fp8bs_status fp8_kv_attention(const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch,
                              const fp8bs_kv_attention_args* args, hipStream_t stream);

/* Bytes of workspace that fp8_kv_attention needs for these arguments (a
 * function of the sizes alone; the pointers are not looked at), or -1 if the
 * sizes are not valid. */
int64_t fp8_kv_attention_workspace(const fp8bs_kv_cache* cache, const fp8bs_kv_batch* batch,
                                   const fp8bs_kv_attention_args* args);

typedef enum fp8bs_score { FP8BS_SCORE_SIGMOID = 0, FP8BS_SCORE_SOFTMAX = 1 } fp8bs_score;

/*
 * Router.  Per token over `experts` logits:
 *   s = sigmoid(logit), or softmax over the experts, evaluated in 64 bits and
 *       rounded once to float32, so that the choice does not hang on how an
 *       exponential is computed;
 *   b = s + bias (float32; bias may be NULL), used for the choice only;
 *   groups > 1: the experts fall into `groups` equal runs; a group's mark is
 *       the float32 sum of its two largest b (its one b if it has one
 *       expert); the top_groups groups with the highest marks stay;
 *   ids = the top_k experts by b among those that stay, highest first;
 *   w = s[ids]; renormalize: w = w / (sum w + 1e-20); weights = w * scale.
 * Ties go to the lower index, for groups and experts.  A NaN counts as lower
 * than every number, so ids are always distinct and in range.
 *
 * logits: [tokens, experts] bf16 or f32, pitch ld >= experts, aligned to its
 *         element.  tokens < 2^26;  1 <= experts <= 1024; groups divides experts, groups <= 64;
 *         1 <= top_groups <= groups; 1 <= top_k <= min(32, top_groups *
 *         experts / groups).
 * ids:    int32 [tokens, top_k];  weights: float32 [tokens, top_k].
 */
fp8bs_status fp8_moe_route(const void* logits, int32_t dtype, int64_t tokens, int64_t experts,
                           int64_t ld, int32_t score, const float* bias, int32_t groups,
                           int32_t top_groups, int32_t top_k, int32_t renormalize, double scale,
                           int32_t* ids, float* weights, hipStream_t stream);

/*
 * Gradient of the router's weights with respect to the logits (the choice
 * itself and the bias have none).  With w the scores at ids and g = scale *
 * grad; renormalize: g = (g - sum(g w / S)) / S, S = sum w + 1e-20:
 *   sigmoid:  d[ids] = g w (1 - w), 0 elsewhere;
 *   softmax:  d = scattered(g w) - s * sum(g w).
 * An id outside [0, experts) has no weight and no gradient; an id that stands
 * twice adds up.
 *
 * grad: float32 [tokens, top_k];  ids: int32 [tokens, top_k], 1 <= top_k <= 32;
 * logits and dlogits: [tokens, experts] of dtype, pitches ld and ld_d.
 */
fp8bs_status fp8_moe_route_backward(const float* grad, const void* logits, int32_t dtype,
                                    int64_t tokens, int64_t experts, int64_t ld,
                                    const int32_t* ids, int32_t top_k, int32_t score,
                                    int32_t renormalize, double scale, void* dlogits,
                                    int64_t ld_d, hipStream_t stream);

/*
 * Dispatch: the rows of x on their way to the experts, as the A operand of
 * fp8_blockscaled_grouped_gemm.  The tokens * top_k choices (flat index
 * t * top_k + j) are ordered by expert, stably; choices outside
 * [0, experts) come last.
 *   order[p]       flat index of the choice at place p;
 *   position[t][j] place of choice (t, j): order inverted;
 *   offsets[e]     first place of expert e; offsets[experts] = number of live
 *                  choices;
 *   q[p], scale[p] row x[order[p] / top_k] quantized in 1x128 tiles exactly as
 *                  fp8_quant_act_1x128; places of dead choices get code 0 and
 *                  scale 1.
 * x: [tokens, cols] bf16 or f32, pitch ld_x, 16-byte aligned, cols % 128 == 0.
 * q: uint8 [tokens * top_k, cols] dense;  scale: float32
 * [tokens * top_k, cols / 128].  1 <= experts <= 1024, 1 <= top_k <= 32,
 * tokens * top_k < 2^31.
 * workspace: at least fp8_moe_dispatch_workspace(tokens, experts, top_k) bytes,
 * 4-byte aligned (NULL if that is 0).
 */
fp8bs_status fp8_moe_dispatch(const void* x, int32_t x_dtype, int64_t tokens, int64_t cols,
                              int64_t ld_x, const int32_t* ids, int32_t top_k, int32_t experts,
                              uint8_t* q, float* scale, int32_t* offsets, int32_t* order,
                              int32_t* position, void* workspace, int64_t workspace_bytes,
                              hipStream_t stream);
int64_t fp8_moe_dispatch_workspace(int64_t tokens, int32_t experts, int32_t top_k);

#ifdef __cplusplus
}
#endif

#endif /* FP8BS_DECODER_H */
