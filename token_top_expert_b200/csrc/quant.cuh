// Rounding of a row to 8-bit integers, for all kernels that do it alike.
#pragma once

#include "common.cuh"

namespace msb {

struct QuantScale {
  float scale, inv;
};
__device__ __forceinline__ QuantScale quant_scale(uint32_t big) {
  const float most = __uint_as_float(big);
  if (big >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.f};  // an infinity or NaN
  if (most < 1.504632769e-36f) return {0.f, 0.f};                      // below 2^-119
  return {most / 127.f, 127.f / most};
}
// The integer nearest to v * inv (at most 127 in magnitude), ties to even, in the low byte: adding
// 1.5 * 2^23 rounds the product to a whole number and leaves it in the low bits of the sum.
__device__ __forceinline__ uint32_t quant(float v, float inv) {
  return __float_as_uint(__fadd_rn(__fmul_rn(v, inv), 12582912.f));
}
__device__ __forceinline__ uint32_t quant4(const float* v, float inv) {
  return __byte_perm(__byte_perm(quant(v[0], inv), quant(v[1], inv), 0x0040),
                     __byte_perm(quant(v[2], inv), quant(v[3], inv), 0x0040), 0x5410);
}

}  // namespace msb
