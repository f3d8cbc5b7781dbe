// Host-side launch of the grouped product (internal to libmsb).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace msb {

// What one launch computes; strides in elements.  See include/msb_dense.h.
struct GroupedArgs {
  const void* x;             // activations [x_rows][ldx]
  int64_t ldx;
  int32_t x_rows;
  const int32_t* rows;       // row of x per output row, or null
  const int32_t* offsets;    // [groups + 1] on the device, or null (one group, all rows)
  int32_t groups, out_rows;
  const void* w;             // weights
  int64_t w_group, w_part, w_n, w_k;
  int32_t n, k;              // output columns, inner length
  const float* x_scale;      // 8-bit: scale of each row of x
  const float* w_scale;      // 8-bit: scale of each weight row, [groups][parts][n]
  void* out;
  int64_t ldo;
  bool i8, swiglu, out_f32;
};

int launch_grouped(const GroupedArgs& a, cudaStream_t st);

// x (bf16 or float, rows ldx elements apart) to 8 bits, then the product: a.x = q and a.x_scale =
// scale are scratch for it, unless one kernel does both.
int launch_linear(const GroupedArgs& a, const void* x, bool f32, int64_t ldx, int8_t* q, float* scale,
                  cudaStream_t st);

// Reads and clears the sticky error word of the current device (synchronises the stream).
int dense_check(cudaStream_t st);

}  // namespace msb
