// Row-wise operators of the dense block: 8-bit quantisation, the weighted sum of a token's
// expert rows, and the norms around a block.  All are bound by memory: one block per row.
#include "common.cuh"
#include "dense.h"

namespace msb {
namespace {

constexpr int kNT = 256;

__device__ __forceinline__ float load(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_lo(static_cast<const uint16_t*>(p)[i]);
}

// Sum over the block, the same value in every thread.
__device__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) t += red[w];
  return t;
}

__global__ void __launch_bounds__(kNT) quantize_kernel(const void* x, bool f32, int64_t ldx, int k,
                                                       int8_t* q, int64_t ldq, float* scale) {
  __shared__ uint32_t red[kNT / 32];
  const int64_t row = blockIdx.x;
  // largest magnitude as bits: ascending with the value, infinities and NaN on top
  uint32_t big = 0;
  for (int i = threadIdx.x; i < k; i += kNT)
    big = max(big, __float_as_uint(load(x, f32, row * ldx + i)) & 0x7fffffffu);
  big = __reduce_max_sync(0xffffffffu, big);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = big;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kNT / 32; ++w) big = max(big, red[w]);
  const float most = __uint_as_float(big);
  const bool finite = big < 0x7f800000u, zero = most < 1.504632769e-36f;  // 2^-119
  const float inv = finite && !zero ? 127.f / most : 0.f;
  if (threadIdx.x == 0) scale[row] = !finite ? __uint_as_float(0x7fc00000u) : zero ? 0.f : most / 127.f;
  for (int i = threadIdx.x; i < k; i += kNT)
    q[row * ldq + i] = inv == 0.f ? 0 : (int8_t)__float2int_rn(load(x, f32, row * ldx + i) * inv);
}

__global__ void __launch_bounds__(kNT)
    combine_kernel(const void* y, bool f32, int64_t ldy, int y_rows, const int32_t* pos,
                   const float* weights, int top_e, int d, uint16_t* out, int64_t ldo) {
  const int64_t t = blockIdx.x;
  for (int i = threadIdx.x; i < d; i += kNT) {
    float acc = 0.f;
    for (int k = 0; k < top_e; ++k) {
      const int p = pos[t * top_e + k];
      if (p >= 0 && p < y_rows) acc = fmaf(weights[t * top_e + k], load(y, f32, p * ldy + i), acc);
    }
    out[t * ldo + i] = __bfloat16_as_ushort(__float2bfloat16_rn(acc));
  }
}

// b = [rms](y), h' = skip h + residual gate b, x = rms(h'); the row of h' waits in shared
// memory for its norm.
__global__ void __launch_bounds__(kNT) block_norm_kernel(const NormArgs a) {
  extern __shared__ float row[];
  __shared__ float red[kNT / 32];
  const int64_t t = blockIdx.x;
  float yscale = 1.f;
  if (a.y && a.post_norm) {
    float ss = 0.f;
    for (int i = threadIdx.x; i < a.d; i += kNT) {
      const float v = load(a.y, a.y_f32, t * a.ldy + i);
      ss = fmaf(v, v, ss);
    }
    yscale = 1.f / sqrtf(block_sum(ss, red) / (float)a.d + a.eps);
  }
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.d; i += kNT) {
    float v = a.skip * load(a.h, a.h_f32, t * a.ldh + i);
    if (a.y) {
      float b = load(a.y, a.y_f32, t * a.ldy + i) * yscale;
      if (a.post_norm && a.post) b *= load(a.post, a.w_f32, i);
      if (a.gate) b *= load(a.gate, a.gate_f32, t * a.gate_row + i * a.gate_col);
      v = fmaf(a.residual, b, v);
    }
    row[i] = v;
    ss = fmaf(v, v, ss);
    if (a.h_out) {
      if (a.h_f32) static_cast<float*>(a.h_out)[t * a.ldh_out + i] = v;
      else static_cast<uint16_t*>(a.h_out)[t * a.ldh_out + i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
  }
  if (!a.x) return;
  const float inv = 1.f / sqrtf(block_sum(ss, red) / (float)a.d + a.eps);
  for (int i = threadIdx.x; i < a.d; i += kNT) {
    float v = row[i] * inv;
    if (a.pre) v *= load(a.pre, a.w_f32, i);
    a.x[t * a.ldx + i] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

int done() { return cudaGetLastError() == cudaSuccess ? MSB_OK : MSB_ECUDA; }

}  // namespace

int launch_quantize(const void* x, bool f32, int64_t ldx, int rows, int k, int8_t* q, int64_t ldq,
                    float* scale, cudaStream_t st) {
  quantize_kernel<<<rows, kNT, 0, st>>>(x, f32, ldx, k, q, ldq, scale);
  return done();
}

int launch_combine(const void* y, bool f32, int64_t ldy, int y_rows, const int32_t* pos,
                   const float* weights, int tokens, int top_e, int d, uint16_t* out, int64_t ldo,
                   cudaStream_t st) {
  combine_kernel<<<tokens, kNT, 0, st>>>(y, f32, ldy, y_rows, pos, weights, top_e, d, out, ldo);
  return done();
}

int launch_block_norm(const NormArgs& a, int rows, cudaStream_t st) {
  const size_t smem = 4 * (size_t)a.d;
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(block_norm_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           4 * MSB_NORM_MAX_D) != cudaSuccess)
    return MSB_ECUDA;
  block_norm_kernel<<<rows, kNT, smem, st>>>(a);
  return done();
}

}  // namespace msb
