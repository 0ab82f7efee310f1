// Direct global-to-LDS loads and the LDS layout of matrix tiles whose rows
// hold 128 bytes.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace fp8bs {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Direct global->LDS buffer loads: lane i's 16 (or 4) bytes at
// voffset + soffset of the buffer land at LDS byte lds_addr + 16 i (4 i).
// Offsets outside the buffer read as zero.  Issued from inline asm so the
// compiler does not track them; the kernel orders them explicitly with
// s_waitcnt vmcnt + s_barrier before any wave reads the stage they fill.
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t lds_addr, int voffset, int soffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds_addr), "v"(voffset), "s"(rsrc), "s"(soffset) : "memory");
}
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t lds_addr, int voffset, int soffset) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, %3 offen lds"
               :: "s"(lds_addr), "v"(voffset), "s"(rsrc), "s"(soffset) : "memory");
}

// Buffer resource for `bytes` bytes at `base` (raw, stride 0).
__device__ __forceinline__ i32x4 make_rsrc(const void* base, uint64_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r.x = static_cast<int32_t>(static_cast<uint32_t>(a));
  r.y = static_cast<int32_t>(static_cast<uint32_t>(a >> 32) & 0xffffu);
  r.z = static_cast<int32_t>(bytes > 0xffffffffull ? 0xffffffffu : static_cast<uint32_t>(bytes));
  r.w = 0x00020000;
  return r;
}

// 32-bit LDS address of a __shared__ object.
template <typename T>
__device__ __forceinline__ uint32_t lds_addr(const T* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (const __attribute__((address_space(3))) T*)(p)));
}

// Wait until at most N of this wave's vector-memory operations are
// outstanding and all its LDS/scalar reads are done, then barrier.  The asm
// clobber keeps the compiler from moving memory operations across it.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (0 << 8));
  asm volatile("s_barrier" ::: "memory");
}

// 16-byte chunk swizzle of a 128-byte LDS row.
__device__ __forceinline__ int swz(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Byte offset of logical 16-byte chunk `chunk` of LDS row `row`.
__device__ __forceinline__ int lds_off(int row, int chunk) { return row * 128 + ((chunk ^ swz(row)) << 4); }

}  // namespace fp8bs
