// Host-side launches of the dense operators' small kernels (internal to libmsb).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "msb_dense.h"

namespace msb {

// Launch that may start while the kernel before it on the stream finishes; every kernel
// launched so waits for that (griddepcontrol.wait) before it touches memory.
template <typename... P, typename... A>
int launch_early(void (*kernel)(P...), int64_t blocks, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) == cudaSuccess) return MSB_OK;
  cudaGetLastError();  // reported here, not by the next call
  return MSB_ECUDA;
}

int route_blocks(int tokens, int experts);  // blocks of the routing kernels: rows of their histogram
int launch_route(const void* logits, bool bf16, int64_t ld, const uint8_t* mask, int tokens,
                 int experts, int top_e, bool renorm, int32_t* ids, float* weights,
                 int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t st);

int launch_quantize(const void* x, bool f32, int64_t ldx, int rows, int k, int8_t* q, int64_t ldq,
                    float* scale, cudaStream_t st);

int launch_combine(const void* y, bool f32, int64_t ldy, int y_rows, const int32_t* pos,
                   const float* weights, int tokens, int top_e, int d, uint16_t* out, int64_t ldo,
                   cudaStream_t st);

struct NormArgs {
  const void *h, *y, *pre, *post, *gate;
  void* h_out;
  uint16_t* x;
  int64_t ldh, ldy, ldh_out, ldx, gate_row, gate_col;
  int rows, d;
  bool h_f32, y_f32, w_f32, gate_f32, post_norm;
  float skip, residual, eps, inv_d;

  // Where element (t, i) of the gate lies, in elements.  Strides reach 2^28: a column's offset
  // alone passes 32 bits.
  __host__ __device__ int64_t gate_at(int64_t t, int64_t i) const { return t * gate_row + i * gate_col; }
};
int launch_block_norm(const NormArgs& a, cudaStream_t st);

}  // namespace msb
