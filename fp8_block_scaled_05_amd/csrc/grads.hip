// Norm of many gradient tensors and their clipping, for gfx950.
//
//   norm = sqrt(sum of squares);   out = g min(1, max_norm / norm)
//
// Bound by memory.  The tensors of a launch come in a table among its
// arguments (a table in memory would have to be copied there first); each is
// cut into chunks of whole 16-byte pieces, and workgroups walk the chunks of
// all tensors, so that lengths do not matter.  Squares are summed in 64 bits:
// a float32's square neither overflows nor vanishes there, and the sum does
// not depend on how the tensors are cut beyond its own last bits.  The 64-bit
// instructions hide behind the reads.
#include <algorithm>
#include <memory>
#include <new>

#include "fp8bs_train.h"
#include "rows.hpp"

namespace fp8bs {
namespace {

// Tensors of one launch: the table stays below 4 KB of arguments.
constexpr int kSummed = 196, kClipped = 140;
constexpr int kPiece = 4;                     // 16-byte pieces of a thread and step
constexpr int64_t kChunkBytes = 256 * 16 * kPiece * 4;
constexpr int64_t kMostBlocks = 2048;
constexpr int32_t kMostTensors = 65536;
constexpr int64_t kMostElements = int64_t(1) << 44;

template <int kTensors, bool kOut>
struct Table {
  static constexpr int kMost = kTensors;
  const void* p[kTensors];
  void* out[kOut ? kTensors : 1];
  int64_t bytes[kTensors];                    // lowest bit set: bf16 (lengths are even)
  int32_t first[kTensors + 1];                // first chunk of each tensor
  int32_t n;
};
using SumTable = Table<kSummed, false>;
using ClipTable = Table<kClipped, true>;
static_assert(sizeof(SumTable) + 16 <= 4096 && sizeof(ClipTable) + 16 <= 4096, "arguments of one launch");

// One tensor's part in a chunk: `head` and `tail` are the elements in front of
// its first and behind its last whole 16-byte piece.
struct Chunk {
  const char* p;
  char* out;
  int64_t begin, end;                         // bytes of whole pieces
  int64_t bytes, body;                        // the tensor's; body: whole pieces end here
  int head;                                   // bytes
  bool bf16, first;
};
template <int kTensors, bool kOut>
__device__ __forceinline__ Chunk find(const Table<kTensors, kOut>& t, int chunk) {
  int lo = 0, hi = t.n - 1;                   // the last tensor whose first chunk is not behind
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  Chunk c;
  c.p = static_cast<const char*>(t.p[lo]);
  c.out = kOut ? static_cast<char*>(t.out[lo]) : nullptr;
  c.bf16 = t.bytes[lo] & 1;
  c.bytes = t.bytes[lo] & ~int64_t(1);
  c.head = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(c.p) & 15)) & 15);
  if (c.head > c.bytes) c.head = static_cast<int>(c.bytes);
  c.body = c.head + (c.bytes - c.head) / 16 * 16;
  c.first = chunk == t.first[lo];
  c.begin = c.head + (chunk - t.first[lo]) * kChunkBytes;
  c.end = min(c.begin + kChunkBytes, c.body);
  return c;
}
__device__ __forceinline__ float element(const char* p, bool bf16) {
  return bf16 ? __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(p)) << 16) : *reinterpret_cast<const float*>(p);
}
// Byte offset of this thread's element among the head's and the tail's of a
// tensor (at most 7 + 7 of them), or -1.
__device__ __forceinline__ int64_t edge(const Chunk& c) {
  const int elt = c.bf16 ? 2 : 4;
  const int64_t k = int64_t(threadIdx.x) * elt;
  if (!c.first) return -1;
  if (k < c.head) return k;
  const int64_t at = c.body + (k - c.head);
  return at < c.bytes ? at : -1;
}

template <bool kBf16>
__device__ __forceinline__ double squares(const u32x4& u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double a = kBf16 ? bf16_lo(w[i]) : __uint_as_float(w[i]);
    s = __builtin_fma(a, a, s);
    if constexpr (kBf16) {
      const double b = bf16_hi(w[i]);
      s = __builtin_fma(b, b, s);
    }
  }
  return s;
}

// Sum over a workgroup of kThreads.
template <int kThreads>
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) s += part[w];
  return s;
}

template <bool kBf16>
__device__ __forceinline__ double sum_pieces(const Chunk& c) {
  double s[kPiece] = {};
  for (int64_t at = c.begin + threadIdx.x * 16; at < c.end; at += 256 * 16 * kPiece) {
    u32x4 u[kPiece];
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      u[k] = u32x4{0, 0, 0, 0};
      if (at + k * 4096 < c.end) u[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c.p + at + k * 4096));
    }
#pragma unroll
    for (int k = 0; k < kPiece; ++k) s[k] += squares<kBf16>(u[k]);
  }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ __launch_bounds__(256) void grad_squares_kernel(const SumTable t, double* __restrict__ partial) {
  double s = 0.0;
  for (int chunk = blockIdx.x; chunk < t.first[t.n]; chunk += gridDim.x) {
    const Chunk c = find(t, chunk);
    s += c.bf16 ? sum_pieces<true>(c) : sum_pieces<false>(c);
    const int64_t at = edge(c);
    if (at >= 0) {
      const double v = element(c.p + at, c.bf16);
      s = __builtin_fma(v, v, s);
    }
  }
  s = block_sum<256>(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(1024) void grad_norm_kernel(const double* __restrict__ partial, int n, float* __restrict__ norm) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) s += partial[i];
  s = block_sum<1024>(s);
  if (threadIdx.x == 0) norm[0] = static_cast<float>(sqrt(s));
}

// max_norm / norm: f, or where that is below float32's normal range (norms of
// 10^38) f * 2^-126, which go to the values one after the other.
template <bool kTiny>
struct Factor {
  float f;
  __device__ __forceinline__ float times(float v) const { return kTiny ? v * 0x1p-126f * f : v * f; }
};

template <bool kBf16, bool kTiny>
__device__ __forceinline__ u32x4 scaled(const u32x4& u, Factor<kTiny> f) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = kBf16 ? round_bf16x2(f.times(bf16_lo(w[i])), f.times(bf16_hi(w[i]))) : __float_as_uint(f.times(__uint_as_float(w[i])));
  return u32x4{w[0], w[1], w[2], w[3]};
}

template <bool kBf16, bool kTiny>
__device__ __forceinline__ void scale_pieces(const Chunk& c, Factor<kTiny> f) {
  const bool aligned = ((reinterpret_cast<uintptr_t>(c.p) ^ reinterpret_cast<uintptr_t>(c.out)) & 15) == 0;
  for (int64_t at = c.begin + threadIdx.x * 16; at < c.end; at += 256 * 16 * kPiece) {
    u32x4 u[kPiece];
#pragma unroll
    for (int k = 0; k < kPiece; ++k)
      if (at + k * 4096 < c.end) u[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(c.p + at + k * 4096));
#pragma unroll
    for (int k = 0; k < kPiece; ++k) {
      if (at + k * 4096 >= c.end) break;
      const u32x4 v = scaled<kBf16, kTiny>(u[k], f);
      char* o = c.out + at + k * 4096;
      if (aligned) {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(o));
      } else {                                // the output starts elsewhere in its 16 bytes
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kBf16) {
            reinterpret_cast<uint16_t*>(o)[2 * i] = static_cast<uint16_t>(w[i]);
            reinterpret_cast<uint16_t*>(o)[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
          } else {
            reinterpret_cast<uint32_t*>(o)[i] = w[i];
          }
        }
      }
    }
  }
}

template <bool kTiny>
__device__ __forceinline__ void clip_chunks(const ClipTable& t, Factor<kTiny> f) {
  for (int chunk = blockIdx.x; chunk < t.first[t.n]; chunk += gridDim.x) {
    const Chunk c = find(t, chunk);
    if (c.bf16) scale_pieces<true, kTiny>(c, f);
    else scale_pieces<false, kTiny>(c, f);
    const int64_t at = edge(c);
    if (at >= 0) {
      const float v = f.times(element(c.p + at, c.bf16));
      if (c.bf16) *reinterpret_cast<uint16_t*>(c.out + at) = static_cast<uint16_t>(round_bf16x2(v, v));
      else *reinterpret_cast<float*>(c.out + at) = v;
    }
  }
}

__global__ __launch_bounds__(256) void grad_clip_kernel(const ClipTable t, const float* __restrict__ norm, float max_norm, int in_place) {
  const float n = *norm;
  const bool clip = n > max_norm && n < __builtin_inff();
  if (in_place && !clip) return;
  const float f = clip ? max_norm / n : 1.0f;
  if (f < 0x1p-126f) clip_chunks(t, Factor<true>{static_cast<float>(static_cast<double>(max_norm) / n * 0x1p126)});
  else clip_chunks(t, Factor<false>{f});
}

fp8bs_status check_grads(const char* fn, const fp8bs_grad* grads, int32_t n) {
  if (n < 0 || n > kMostTensors || (n > 0 && !grads)) return fail(FP8BS_ERR_INVALID_ARG, "%s: %d tensors", fn, n);
  int64_t total = 0;
  for (int32_t i = 0; i < n; ++i) {
    const fp8bs_grad& g = grads[i];
    if (g.dtype != FP8BS_BF16 && g.dtype != FP8BS_F32) return fail(FP8BS_ERR_INVALID_ARG, "%s: unknown type %lld of tensor %d", fn, (long long)g.dtype, i);
    if (g.count < 0 || g.count > kMostElements || (total += g.count) > kMostElements)
      return fail(FP8BS_ERR_INVALID_ARG, "%s: %lld elements in tensor %d", fn, (long long)g.count, i);
    if (g.count && !g.p) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (tensor %d)", fn, i);
    if (reinterpret_cast<uintptr_t>(g.p) % elem_size(static_cast<int32_t>(g.dtype)))
      return fail(FP8BS_ERR_ALIGNMENT, "%s: tensor %d is not aligned to its element", fn, i);
  }
  return FP8BS_OK;
}

// Whether every written tensor is apart from all others, from the norm and, but
// for its own input, from what is read: workgroups read and write at once.
struct Range {
  uintptr_t lo, hi;
  int32_t tensor;
  bool written;
};
fp8bs_status check_apart(const char* fn, const fp8bs_grad* grads, const fp8bs_grad* outs, int32_t n, const float* norm) {
  const int64_t most = 2 * int64_t(n) + 1;
  const std::unique_ptr<Range[]> r(new (std::nothrow) Range[most]);
  if (!r) return fail(FP8BS_ERR_INVALID_ARG, "%s: no memory to compare %d tensors", fn, n);
  int64_t k = 0;
  auto add = [&](const void* p, int64_t bytes, int32_t tensor, bool written) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    r[k++] = {lo, lo + bytes, tensor, written};
  };
  for (int32_t i = 0; i < n; ++i) {
    const int64_t bytes = grads[i].count * elem_size(static_cast<int32_t>(grads[i].dtype));
    if (!bytes) continue;
    if (outs && outs[i].p != grads[i].p) add(grads[i].p, bytes, i, false);
    add(outs ? outs[i].p : grads[i].p, bytes, i, true);
  }
  add(norm, 4, -1, false);
  auto before = [](const Range& a, const Range& b) { return a.lo < b.lo; };
  if (!std::is_sorted(r.get(), r.get() + k, before)) std::sort(r.get(), r.get() + k, before);
  // The furthest ends so far, of what is written and of everything.
  uintptr_t written = 0, all = 0;
  for (int64_t i = 0; i < k; ++i) {
    if (r[i].lo < written || (r[i].written && r[i].lo < all))
      return r[i].tensor < 0 ? fail(FP8BS_ERR_INVALID_ARG, "%s: norm shares memory with a tensor", fn)
                             : fail(FP8BS_ERR_INVALID_ARG, "%s: tensor %d shares memory with another one of the call", fn, r[i].tensor);
    all = std::max(all, r[i].hi);
    if (r[i].written) written = std::max(written, r[i].hi);
  }
  return FP8BS_OK;
}

// Calls f(table, blocks) for the tensors of each launch.  A chunk is a whole
// number of pieces; a launch ends with its table or when its chunks would not
// fit their count.
template <class T, class F>
void for_launches(const fp8bs_grad* grads, const fp8bs_grad* outs, int32_t n, F f) {
  T t;
  t.n = 0;
  int64_t chunks = 0;
  auto flush = [&] {
    if (!t.n) return;
    t.first[t.n] = static_cast<int32_t>(chunks);
    f(t, static_cast<uint32_t>(std::min(chunks, kMostBlocks)));
    t.n = 0;
    chunks = 0;
  };
  for (int32_t i = 0; i < n; ++i) {
    if (!grads[i].count) continue;
    const int64_t bytes = grads[i].count * elem_size(static_cast<int32_t>(grads[i].dtype));
    const int64_t own = (bytes + kChunkBytes - 1) / kChunkBytes;
    if (t.n == T::kMost || chunks + own > (int64_t(1) << 30)) flush();
    t.p[t.n] = grads[i].p;
    if constexpr (T::kMost == kClipped) t.out[t.n] = outs ? outs[i].p : grads[i].p;
    t.bytes[t.n] = bytes | (grads[i].dtype == FP8BS_BF16);
    t.first[t.n] = static_cast<int32_t>(chunks);
    ++t.n;
    chunks += own;
  }
  flush();
}

}  // namespace
}  // namespace fp8bs

using namespace fp8bs;

extern "C" int64_t fp8_grad_norm_workspace(const fp8bs_grad* grads, int32_t n) {
  if (check_grads("fp8_grad_norm_workspace", grads, n) != FP8BS_OK) return -1;
  int64_t blocks = 0;
  for_launches<SumTable>(grads, nullptr, n, [&](const SumTable&, uint32_t b) { blocks += b; });
  return blocks * 8;
}

extern "C" fp8bs_status fp8_grad_norm(const fp8bs_grad* grads, int32_t n, float* norm, void* workspace, int64_t workspace_bytes,
                                      hipStream_t stream) {
  const char* fn = "fp8_grad_norm";
  if (fp8bs_status st = check_grads(fn, grads, n)) return st;
  if (!norm) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (norm)", fn);
  if (!aligned4(norm)) return fail(FP8BS_ERR_ALIGNMENT, "%s: norm must be 4-byte aligned", fn);
  const int64_t need = fp8_grad_norm_workspace(grads, n);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(FP8BS_ERR_INVALID_ARG, "%s: workspace of %lld bytes needed", fn, (long long)need);
  if (need > 0 && !aligned16(workspace)) return fail(FP8BS_ERR_ALIGNMENT, "%s: workspace must be 16-byte aligned", fn);
  for (int32_t i = 0; i < n; ++i)
    if (overlap(line(workspace, need), line(grads[i].p, grads[i].count * elem_size(static_cast<int32_t>(grads[i].dtype)))))
      return fail(FP8BS_ERR_INVALID_ARG, "%s: workspace overlaps tensor %d", fn, i);
  begin_launch();
  double* partial = static_cast<double*>(workspace);
  int64_t at = 0;
  for_launches<SumTable>(grads, nullptr, n, [&](const SumTable& t, uint32_t blocks) {
    hipLaunchKernelGGL(grad_squares_kernel, dim3(blocks), dim3(256), 0, stream, t, partial + at);
    at += blocks;
  });
  hipLaunchKernelGGL(grad_norm_kernel, dim3(1), dim3(1024), 0, stream, partial, static_cast<int>(at), norm);
  return check_launch(fn);
}

extern "C" fp8bs_status fp8_grad_clip(const fp8bs_grad* grads, const fp8bs_grad* outs, int32_t n, const float* norm, double max_norm,
                                      hipStream_t stream) {
  const char* fn = "fp8_grad_clip";
  if (fp8bs_status st = check_grads(fn, grads, n)) return st;
  if (outs) {
    if (fp8bs_status st = check_grads(fn, outs, n)) return st;
    for (int32_t i = 0; i < n; ++i)
      if (outs[i].count != grads[i].count || outs[i].dtype != grads[i].dtype)
        return fail(FP8BS_ERR_INVALID_ARG, "%s: outs[%d] has another length or type", fn, i);
  }
  const float most = static_cast<float>(max_norm);
  if (!(most > 0.0f && most < __builtin_inff())) return fail(FP8BS_ERR_INVALID_ARG, "%s: max_norm must be finite and above 0", fn);
  if (!norm) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (norm)", fn);
  if (!aligned4(norm)) return fail(FP8BS_ERR_ALIGNMENT, "%s: norm must be 4-byte aligned", fn);
  if (fp8bs_status st = check_apart(fn, grads, outs, n, norm)) return st;
  if (std::all_of(grads, grads + n, [](const fp8bs_grad& g) { return g.count == 0; })) return FP8BS_OK;
  begin_launch();
  for_launches<ClipTable>(grads, outs, n, [&](const ClipTable& t, uint32_t blocks) {
    hipLaunchKernelGGL(grad_clip_kernel, dim3(blocks), dim3(256), 0, stream, t, norm, most, outs ? 0 : 1);
  });
  return check_launch(fn);
}
