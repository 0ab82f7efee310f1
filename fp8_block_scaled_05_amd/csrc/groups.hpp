// Experts' ranges in a device table of offsets that may hold anything.
#pragma once
#include <hip/hip_runtime.h>
#include <cstdint>

namespace fp8bs {

// Inclusive prefix sum and maximum over the 64 lanes of a wave.
__device__ __forceinline__ int prefix_sum(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(v, d);
    if (lane >= d) v += t;
  }
  return v;
}
__device__ __forceinline__ int prefix_max(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(v, d);
    if (lane >= d) v = max(v, t);
  }
  return v;
}

// Groups [g0, g0 + 64) of a table off[G+1], one per lane.  With c_g the
// offsets clamped into [0, most], group g owns [P_g, P_g+1), P_g = max(0, c_0
// .. c_g): the ranges never overlap, and for a valid table nothing changes.
// `run` is P at g0, and afterwards at g0 + 64.
struct GroupRange {
  int lo, hi;                                 // an empty range for a lane past the last group
};
__device__ __forceinline__ GroupRange group_ranges(const int32_t* off, int G, int most, int g0, int lane, int& run) {
  const int g = g0 + lane;
  const bool real = g < G;
  const int c = real ? min(max(off[g], 0), most) : 0;
  const int next = real ? min(max(off[g + 1], 0), most) : 0;
  GroupRange r;
  r.lo = max(run, prefix_max(c, lane));
  r.hi = real ? max(r.lo, next) : r.lo;
  run = __shfl(r.hi, 63);
  return r;
}

}  // namespace fp8bs
