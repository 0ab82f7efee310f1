// Rows of bf16 or float32 values in pieces of 8, and the 1x128 quantization of
// float32 values: shared by the kernels that work a row at a time between the
// GEMMs (norm.hip, swiglu.hip) and by the transposing quantizer.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>
#include <initializer_list>

#include "device.hpp"
#include "overlap.hpp"
#include "status.hpp"

namespace fp8bs {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// 8 consecutive values as they lie in memory.
template <bool kBf16>
struct Raw8 {
  u32x4 u[kBf16 ? 1 : 2];
};

// Column `col` of a row: the row's address may be uniform, the column's bytes
// stay a 32-bit offset to it (columns are below 2^29).
template <bool kBf16>
__device__ __forceinline__ const char* at(const void* p, int64_t row, int64_t ld, int col) {
  constexpr int kElt = kBf16 ? 2 : 4;
  return static_cast<const char*>(p) + row * ld * kElt + static_cast<uint32_t>(col) * kElt;
}
template <bool kBf16>
__device__ __forceinline__ char* at(void* p, int64_t row, int64_t ld, int col) {
  return const_cast<char*>(at<kBf16>(static_cast<const void*>(p), row, ld, col));
}

// kNT: read or written once by the kernel and not wanted in the caches.
template <bool kBf16, bool kNT = true>
__device__ __forceinline__ Raw8<kBf16> load8(const char* p) {
  Raw8<kBf16> r;
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
    const u32x4* v = reinterpret_cast<const u32x4*>(p) + i;
    r.u[i] = kNT ? __builtin_nontemporal_load(v) : *v;
  }
  return r;
}
template <bool kBf16, bool kNT = false>
__device__ __forceinline__ void store8(char* p, const Raw8<kBf16>& r) {
#pragma unroll
  for (int i = 0; i < (kBf16 ? 1 : 2); ++i) {
    u32x4* v = reinterpret_cast<u32x4*>(p) + i;
    if constexpr (kNT) __builtin_nontemporal_store(r.u[i], v);
    else *v = r.u[i];
  }
}

template <bool kBf16>
__device__ __forceinline__ void widen(const Raw8<kBf16>& r, float (&v)[8]) {
  if constexpr (kBf16) {
    const uint32_t u[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(u[i]);
      v[2 * i + 1] = bf16_hi(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[4 * i] = __uint_as_float(r.u[i].x);
      v[4 * i + 1] = __uint_as_float(r.u[i].y);
      v[4 * i + 2] = __uint_as_float(r.u[i].z);
      v[4 * i + 3] = __uint_as_float(r.u[i].w);
    }
  }
}

__device__ __forceinline__ uint32_t round_bf16x2(float a, float b) {
  const bf16x2 h = __builtin_convertvector(f32x2{a, b}, bf16x2);   // to nearest even
  return __builtin_bit_cast(uint32_t, h);
}
// Rounded to the type, once.
template <bool kBf16>
__device__ __forceinline__ Raw8<kBf16> narrow(const float (&v)[8]) {
  Raw8<kBf16> r;
  if constexpr (kBf16) {
    r.u[0] = u32x4{round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]), round_bf16x2(v[4], v[5]), round_bf16x2(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.u[i] = u32x4{__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]), __float_as_uint(v[4 * i + 3])};
  }
  return r;
}

// fl32(x / s), given r = fl32(1 / s) of an IEEE division.  x * r is within two
// units in the last place of the quotient, the first correction brings it
// within one, and from there Markstein's theorem (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34(1), 1990) gives the correctly rounded quotient.  It needs exact
// remainders: s is above 1e-10 and x at most 448 s, so a remainder is exact
// wherever the quotient is not far below the smallest code, and s = 1 leaves
// none.  The remainders have their signs flipped so that -0 stays -0.  Five
// instructions; an IEEE division takes about ten.
__device__ __forceinline__ float quotient(float x, float s, float r) {
  float q = x * r;
  q = __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
  return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
}

__device__ __forceinline__ float absmax8(const float (&v)[8]) {
  const float m0 = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fabsf(v[2]));
  const float m1 = fmaxf(fmaxf(fabsf(v[3]), fabsf(v[4])), fabsf(v[5]));
  return fmaxf(fmaxf(m0, m1), fmaxf(fabsf(v[6]), fabsf(v[7])));
}

// One 1x128 tile, 8 values in each of the 16 lanes of a DPP row: its scale
// (the same in every lane) and this lane's codes.
__device__ __forceinline__ uint2 quantize_tile(const float (&v)[8], float& s) {
  s = tile_scale(row16_max(absmax8(v)));
  const float r = 1.0f / s;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = quotient(v[i], s, r);
  return make_uint2(pack4_e4m3(q[0], q[1], q[2], q[3]), pack4_e4m3(q[4], q[5], q[6], q[7]));
}

// Sum over the 64 lanes of a wave, the same in every lane.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f<0x128>(v);
  v += dpp_f<0x124>(v);
  v += dpp_f<0x122>(v);
  v += dpp_f<0x121>(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Host check of one matrix of rows: its pointer, pitch and extent.
inline fp8bs_status check_matrix(const char* fn, const char* what, const void* p, int64_t rows, int64_t cols, int64_t ld, int elt) {
  if (!p) return fail(FP8BS_ERR_INVALID_ARG, "%s: null pointer (%s)", fn, what);
  if (ld < cols) return fail(FP8BS_ERR_INVALID_ARG, "%s: pitch of %s smaller than its row", fn, what);
  if (!sane_matrix(rows, ld, elt)) return fail(FP8BS_ERR_INVALID_ARG, "%s: size of %s exceeds any allocation", fn, what);
  if (!aligned16(p) || (ld * elt) % 16) return fail(FP8BS_ERR_ALIGNMENT, "%s: %s and its pitch must be 16-byte aligned", fn, what);
  return FP8BS_OK;
}

// Operands of a call, for the check that its outputs are apart from each other
// and from its inputs.  Workgroups read and write at once.  An output may be an
// input itself where the threads that write a place are those that have read
// it: `in_place` of both.
struct Operand {
  const char* name;
  Block block;
  bool in_place;
};
inline Block matrix_block(const void* p, int64_t rows, int64_t cols, int64_t ld, int elt) { return {p, rows, cols * elt, ld * elt}; }
inline fp8bs_status check_apart(const char* fn, std::initializer_list<Operand> outs, std::initializer_list<Operand> ins) {
  for (const Operand* o = outs.begin(); o != outs.end(); ++o) {
    for (const Operand* other = o + 1; other != outs.end(); ++other)
      if (overlap(o->block, other->block)) return fail(FP8BS_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, o->name, other->name);
    for (const Operand& in : ins)
      if (!(o->in_place && in.in_place && o->block == in.block) && overlap(o->block, in.block))
        return fail(FP8BS_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, o->name, in.name);
  }
  return FP8BS_OK;
}

}  // namespace fp8bs
