// What the two kernels of the grouped products share: arguments, group offsets, epilogue values.
#pragma once

#include "common.cuh"
#include "grouped.h"

namespace msb {

constexpr int kGroupsMax = MSB_MAX_EXPERTS;

struct KArgs {
  const uint8_t* x;
  int64_t pitch;  // bytes between rows of x
  int32_t x_rows;
  const int32_t* rows;
  const int32_t* offsets;
  int32_t groups, out_rows, n, k, kbytes, mtiles;
  const uint8_t* w;  // and the weights' strides in bytes
  int64_t w_group, w_part, w_n, w_k;
  const float* x_scale;
  const float* w_scale;
  void* out;
  int64_t ldo;
  int wide;  // out may be written in 16-byte pieces
};

// First row of each group, by one warp: begin[0 .. groups] in shared memory.  Offsets outside
// [0, out_rows] or below an earlier one are raised or cut to it, so that no offsets lead
// outside the buffers.
__device__ inline void group_begins(const KArgs& a, int32_t* begin, int lane) {
  // eight loads in flight: one memory latency for up to 255 groups
  for (int b = 0; b <= a.groups; b += 256) {
    int o[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int e = b + q * 32 + lane;
      o[q] = e > a.groups ? 0 : a.offsets ? a.offsets[e] : e ? a.out_rows : 0;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int e = b + q * 32 + lane;
      if (e <= a.groups) begin[e] = min(max(o[q], 0), a.out_rows);
    }
  }
  __syncwarp();
  const int per = (a.groups + 32) >> 5;  // of groups + 1 offsets
  const int e0 = lane * per, e1 = min(e0 + per, a.groups + 1);
  int top = 0;
  for (int e = e0; e < e1; ++e) begin[e] = top = max(top, begin[e]);
  int above = top;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, above, o);
    if (lane >= o) above = max(above, v);
  }
  above = __shfl_up_sync(0xffffffffu, above, 1);
  if (lane == 0) above = 0;
  for (int e = e0; e < e1; ++e) begin[e] = max(begin[e], above);
  __syncwarp();
}

// The accumulator's value as a float; 8-bit: the integer sum times the two scales.
template <bool I8>
__device__ __forceinline__ float value(uint32_t v, float row_scale, float scale) {
  if constexpr (I8) return (float)(int32_t)v * row_scale * scale;
  return __uint_as_float(v);
}

// silu(g) * u, with the approximate exponential, off by up to (2 + 1.173 |g|) 2^-23, and quotient
// (2^-22): where g is negative silu is off by as much, 2^-18 at g = -20 and 2^-16 at -87, well below
// bf16's 2^-8.  Zero below g = -87.3, where silu is under 2e-36.  The exact quotient made the
// epilogue of a 256-row tile 10 us.
__device__ __forceinline__ float gated(float g, float u) { return __fdividef(g, 1.f + __expf(-g)) * u; }

inline KArgs kernel_args(const GroupedArgs& a) {
  const int es = a.i8 ? 1 : 2;
  KArgs k;
  k.x = static_cast<const uint8_t*>(a.x);
  k.pitch = a.ldx * es;
  k.x_rows = a.x_rows;
  k.rows = a.rows;
  k.offsets = a.offsets;
  k.groups = a.groups;
  k.out_rows = a.out_rows;
  k.n = a.n;
  k.k = a.k;
  k.kbytes = a.k * es;
  k.mtiles = a.swiglu ? (a.n + 127) / 128 : (a.n + 255) / 256;
  k.w = static_cast<const uint8_t*>(a.w);
  k.w_group = a.w_group * es, k.w_part = a.w_part * es, k.w_n = a.w_n * es, k.w_k = a.w_k * es;
  k.x_scale = a.x_scale;
  k.w_scale = a.w_scale;
  k.out = a.out;
  k.ldo = a.ldo;
  k.wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && (a.ldo % 8 == 0 || a.out_rows == 1);
  return k;
}

// Products of a few rows, on the CUDA cores (grouped_few.cu).
bool few_rows(const GroupedArgs& a);
int launch_few(const GroupedArgs& a, const KArgs& k, cudaStream_t st);

}  // namespace msb
