// Row-wise operators of the dense block: 8-bit quantisation, the weighted sum of a token's
// expert rows, and the norms around a block.  All are bound by memory, so each element is read
// once, in 16-byte pieces (8 bf16), and waits in registers for its row's sum or maximum: a warp
// to a row of up to 1024 elements, else 256 or 512 threads.  Rows whose pitch, start or length
// is not a multiple of eight elements go element by element in the same way.
#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "dense.h"
#include "quant.cuh"

namespace msb {
namespace {

__device__ __forceinline__ float load(const void* p, bool f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_lo(static_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// W consecutive elements (8: the address is 16-byte aligned).
template <int W>
__device__ __forceinline__ void load_w(const void* p, bool f32, int64_t i, float (&v)[W]) {
  if constexpr (W == 1) {
    v[0] = load(p, f32, i);
  } else if (f32) {
    const float4 a = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    const float4 b = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
  }
}
template <int W>
__device__ __forceinline__ void store_w(void* p, bool f32, int64_t i, const float (&v)[W]) {
  if constexpr (W == 1) {
    if (f32) static_cast<float*>(p)[i] = v[0];
    else static_cast<uint16_t*>(p)[i] = bf16_bits(v[0]);
  } else if (f32) {
    float4* const o = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    o[0] = make_float4(v[0], v[1], v[2], v[3]);
    o[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
  }
}

// Sum (or maximum) over the NT threads of a row, the same value in each.  NT = 32: a warp, else
// the block; `red` is used once per call site.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = warp_sum(v);
  if constexpr (NT > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const float4* const r4 = reinterpret_cast<const float4*>(red);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < NT / 128; ++w) v += (r4[w].x + r4[w].y) + (r4[w].z + r4[w].w);
  }
  return v;
}
template <int NT>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* red) {
  v = __reduce_max_sync(0xffffffffu, v);
  if constexpr (NT > 32) {
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) v = max(v, red[w]);
  }
  return v;
}

__host__ __device__ constexpr int block_threads(int nt) { return nt == 32 ? 256 : nt; }

// Two neighbouring elements.  PAIR: one instruction works on both.
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
template <bool PAIR>
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  if constexpr (!PAIR) return make_float2(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y));
  float2 r;
  asm("{.reg .b64 a, b, c, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      "fma.rn.f32x2 r, a, b, c;\n mov.b64 {%0, %1}, r;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
template <bool PAIR>
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  if constexpr (!PAIR) return make_float2(a.x * b.x, a.y * b.y);
  float2 r;
  asm("{.reg .b64 a, b, r;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n"
      "mul.rn.f32x2 r, a, b;\n mov.b64 {%0, %1}, r;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Eight elements as they lie in memory.
template <bool F32>
struct Raw {
  uint4 a[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* const q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + i * (F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < (F32 ? 2 : 1); ++j) a[j] = q[j];
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    if constexpr (F32) {
      v[0] = __uint_as_float(a[0].x), v[1] = __uint_as_float(a[0].y), v[2] = __uint_as_float(a[0].z);
      v[3] = __uint_as_float(a[0].w), v[4] = __uint_as_float(a[1].x), v[5] = __uint_as_float(a[1].y);
      v[6] = __uint_as_float(a[1].z), v[7] = __uint_as_float(a[1].w);
    } else {
      v[0] = bf16_lo(a[0].x), v[1] = bf16_hi(a[0].x), v[2] = bf16_lo(a[0].y), v[3] = bf16_hi(a[0].y);
      v[4] = bf16_lo(a[0].z), v[5] = bf16_hi(a[0].z), v[6] = bf16_lo(a[0].w), v[7] = bf16_hi(a[0].w);
    }
  }
  __device__ __forceinline__ void get(float2 (&v)[4]) const {
    float f[8];
    get(f);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = make_float2(f[2 * c], f[2 * c + 1]);
  }
};
__device__ __forceinline__ void load_two(const void* p, bool f32, int64_t i, float2 (&v)[4]) {
  float f[8];
  load_w<8>(p, f32, i, f);
#pragma unroll
  for (int c = 0; c < 4; ++c) v[c] = make_float2(f[2 * c], f[2 * c + 1]);
}
__device__ __forceinline__ void store_two(void* p, bool f32, int64_t i, const float2 (&v)[4]) {
  float f[8];
#pragma unroll
  for (int c = 0; c < 4; ++c) f[2 * c] = v[c].x, f[2 * c + 1] = v[c].y;
  store_w<8>(p, f32, i, f);
}

// ------------------------------------------------------------------ 8-bit quantisation

// V pieces of W elements a thread.
template <int NT, int W, int V>
__global__ void __launch_bounds__(block_threads(NT))
    quantize_kernel(const void* x, bool f32, int64_t ldx, int rows, int k, int8_t* q, int64_t ldq, float* scale) {
  __shared__ uint32_t red[NT / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = (int64_t)blockIdx.x * (block_threads(NT) / NT) + threadIdx.x / NT;
  if (row >= rows) return;  // whole warps; larger rows have a block each
  const int tid = threadIdx.x % NT;
  float v[V][W];
  // largest magnitude as bits: ascending with the value, infinities and NaN on top
  uint32_t big = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = (j * NT + tid) * W;
    if (i < k) load_w<W>(x, f32, row * ldx + i, v[j]);
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if ((j * NT + tid) * W < k)
#pragma unroll
      for (int c = 0; c < W; ++c) big = max(big, __float_as_uint(v[j][c]) & 0x7fffffffu);
  const QuantScale qs = quant_scale(row_max<NT>(big, red));
  if (tid == 0) scale[row] = qs.scale;
  const bool zero = qs.inv == 0.f;  // nothing to scale, or not finite
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = (j * NT + tid) * W;
    if (i >= k) continue;
    int8_t* const o = q + row * ldq + i;
    if constexpr (W == 1) {
      *o = zero ? 0 : (int8_t)quant(v[j][0], qs.inv);
    } else {
      *reinterpret_cast<uint2*>(o) =
          zero ? make_uint2(0, 0) : make_uint2(quant4(&v[j][0], qs.inv), quant4(&v[j][4], qs.inv));
    }
  }
}

// Many rows: a warp to a row, V pieces of eight elements a lane, all on their way at once (8192 x
// 4096: 19.2 us, 5.2 TB/s, where a block per row takes 24).
template <int V, bool F32>
__global__ void __launch_bounds__(256) quantize_warp_kernel(const void* x, int64_t ldx, int rows, int k, int8_t* q,
                                                            int64_t ldq, float* scale) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int lane = threadIdx.x & 31;
  Raw<F32> r[V];
#pragma unroll
  for (int j = 0; j < V; ++j)
    if ((j * 32 + lane) * 8 < k) r[j].load(x, row * ldx + (j * 32 + lane) * 8);
  uint32_t big = 0;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if ((j * 32 + lane) * 8 < k) {
      float v[8];
      r[j].get(v);
#pragma unroll
      for (int c = 0; c < 8; ++c) big = max(big, __float_as_uint(v[c]) & 0x7fffffffu);
    }
  const QuantScale qs = quant_scale(__reduce_max_sync(0xffffffffu, big));
  if (lane == 0) scale[row] = qs.scale;
  const bool zero = qs.inv == 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = (j * 32 + lane) * 8;
    if (i >= k) continue;
    float v[8];
    r[j].get(v);
    *reinterpret_cast<uint2*>(q + row * ldq + i) =
        zero ? make_uint2(0, 0) : make_uint2(quant4(v, qs.inv), quant4(v + 4, qs.inv));
  }
}

// Rows of any length, read twice.
__global__ void __launch_bounds__(256)
    quantize_long_kernel(const void* x, bool f32, int64_t ldx, int k, int8_t* q, int64_t ldq, float* scale) {
  __shared__ uint32_t red[8];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = blockIdx.x;
  uint32_t big = 0;
  for (int i = threadIdx.x; i < k; i += 256) big = max(big, __float_as_uint(load(x, f32, row * ldx + i)) & 0x7fffffffu);
  const QuantScale qs = quant_scale(row_max<256>(big, red));
  if (threadIdx.x == 0) scale[row] = qs.scale;
  for (int i = threadIdx.x; i < k; i += 256)
    q[row * ldq + i] = qs.inv == 0.f ? 0 : (int8_t)quant(load(x, f32, row * ldx + i), qs.inv);
}

// ------------------------------------------------------------------ combine

constexpr int kCombineNT = 256;

// KP rows' pieces of a token in flight (top_e <= KP, or eight at a time).  The blocks stay and take
// one (token, run of 256 pieces) after another; where the next token's rows lie is read meanwhile.
// 8192 x 2048 bf16: top-8 46.6 us, 6.5 TB/s, top-2 17.3 us, 5.8 TB/s (29.2 with a block per item, whose
// loads of positions and rows follow one another).
template <bool F32, int KP>
__global__ void __launch_bounds__(kCombineNT)
    combine_kernel(const void* y, int64_t ldy, int y_rows, const int32_t* pos, const float* weights, uint32_t items,
                   int top_e, int d, uint32_t runs, uint16_t* out, int64_t ldo) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int32_t p[KP];
  const auto fetch = [&](uint32_t t, int k) {
#pragma unroll
    for (int j = 0; j < KP; ++j) p[j] = k + j < top_e ? pos[(int64_t)t * top_e + k + j] : -1;
  };
  uint32_t item = blockIdx.x;
  fetch(item / runs, 0);
  for (; item < items; item += gridDim.x) {
    const uint32_t t = item / runs, next = item + gridDim.x;
    const int i = ((int)(item - t * runs) * kCombineNT + threadIdx.x) * 8;
    float acc[8] = {};
    for (int k = 0; k < top_e; k += KP) {
      Raw<F32> r[KP];
      float w[KP];
      bool use[KP];
#pragma unroll
      for (int j = 0; j < KP; ++j) {
        use[j] = (uint32_t)p[j] < (uint32_t)y_rows && i < d;
        if (use[j]) r[j].load(y, p[j] * ldy + i);
      }
#pragma unroll
      for (int j = 0; j < KP; ++j) w[j] = use[j] ? weights[(int64_t)t * top_e + k + j] : 0.f;
      if (k + KP < top_e) fetch(t, k + KP);
      else if (next < items) fetch(next / runs, 0);
#pragma unroll
      for (int j = 0; j < KP; ++j)
        if (use[j]) {
          float v[8];
          r[j].get(v);
#pragma unroll
          for (int c = 0; c < 8; ++c) acc[c] = fmaf(w[j], v[c], acc[c]);
        }
    }
    if (i < d) store_w<8>(out, false, (int64_t)t * ldo + i, acc);
  }
}

// The same element by element.
__global__ void __launch_bounds__(kCombineNT)
    combine_any_kernel(const void* y, bool f32, int64_t ldy, int y_rows, const int32_t* pos, const float* weights,
                       int top_e, int d, int runs, uint16_t* out, int64_t ldo) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = blockIdx.x / runs;
  const int i = (int)(blockIdx.x % runs) * kCombineNT + threadIdx.x;
  if (i >= d) return;
  float acc = 0.f;
#pragma unroll 4
  for (int k = 0; k < top_e; ++k) {
    const int p = pos[t * top_e + k];
    if ((uint32_t)p < (uint32_t)y_rows) acc = fmaf(weights[t * top_e + k], load(y, f32, p * ldy + i), acc);
  }
  out[t * ldo + i] = bf16_bits(acc);
}

// ------------------------------------------------------------------ block norm

// Blocks of an SM that the registers are cut to: more keep more loads in flight, fewer do not
// spill (8192 x 4096, 4 and 3 blocks: bf16 48.5 and 51.4 us, float h 75.7 and 64.8).
template <int NT, int V, bool F32>
constexpr int kNormBlocks = (V == 4 ? 2 : V == 2 && F32 ? 3 : 4) * 256 / block_threads(NT);

// b = [rms](y), h' = skip h + residual gate b, x = rms(h'), rows in 16-byte pieces.  The blocks
// stay and take row after row: while a row's two sums cross the block, the next row's pieces
// are on their way.  bf16 rows are bound by the instructions (two thirds of the issue slots), so
// these work on two elements at a time (8192 x 4096: 46.8 us, 5.7 TB/s; 48.5 one by one, 77 with
// a block per row); float rows need the registers more (64.6 us, 6.2 TB/s; 66.8 in pairs).
template <int NT, int V, bool HF32, bool YF32>
__global__ void __launch_bounds__(block_threads(NT), kNormBlocks<NT, V, HF32 || YF32>) block_norm_kernel(const NormArgs a) {
  constexpr int kRows = block_threads(NT) / NT;
  constexpr bool PAIR = !HF32 && !YF32;
  alignas(16) __shared__ float red[2][2][NT / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int tid = threadIdx.x % NT;
  const int64_t step = (int64_t)gridDim.x * kRows;
  int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / NT;
  Raw<HF32> hn[V];
  Raw<YF32> yn[V];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = (j * NT + tid) * 8;
      if (row < a.rows && i < a.d) {
        if (a.y) yn[j].load(a.y, row * a.ldy + i);
        hn[j].load(a.h, row * a.ldh + i);
      }
    }
  };
  fetch(t);
  for (int turn = 0; t < a.rows; t += step, turn ^= 1) {  // a whole warp or block at a time
    Raw<HF32> hr[V];
    Raw<YF32> yr[V];
#pragma unroll
    for (int j = 0; j < V; ++j) hr[j] = hn[j], yr[j] = yn[j];
    fetch(t + step);
    float yscale = 1.f;
    if (a.post_norm) {
      float2 ss = two(0.f);
#pragma unroll
      for (int j = 0; j < V; ++j)
        if ((j * NT + tid) * 8 < a.d) {
          float2 y[4];
          yr[j].get(y);
#pragma unroll
          for (int c = 0; c < 4; ++c) ss = fma2<PAIR>(y[c], y[c], ss);
        }
      yscale = rsqrtf(fmaf(row_sum<NT>(ss.x + ss.y, red[turn][0]), a.inv_d, a.eps));
    }
    float2 h[V][4], ss = two(0.f);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = (j * NT + tid) * 8;
      if (i >= a.d) continue;
      hr[j].get(h[j]);
#pragma unroll
      for (int c = 0; c < 4; ++c) h[j][c] = mul2<PAIR>(h[j][c], two(a.skip));
      if (a.y) {
        float2 b[4], m[4];
        yr[j].get(b);
#pragma unroll
        for (int c = 0; c < 4; ++c) b[c] = mul2<PAIR>(b[c], two(yscale));
        if (a.post) {
          load_two(a.post, a.w_f32, i, m);
#pragma unroll
          for (int c = 0; c < 4; ++c) b[c] = mul2<PAIR>(b[c], m[c]);
        }
        if (a.gate) {
          if (a.gate_col == 0) {
            const float g = load(a.gate, a.gate_f32, t * a.gate_row);
#pragma unroll
            for (int c = 0; c < 4; ++c) m[c] = two(g);
          } else if (a.gate_col == 1) {
            load_two(a.gate, a.gate_f32, t * a.gate_row + i, m);
          } else {
            float g[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) g[c] = load(a.gate, a.gate_f32, t * a.gate_row + (i + c) * a.gate_col);
#pragma unroll
            for (int c = 0; c < 4; ++c) m[c] = make_float2(g[2 * c], g[2 * c + 1]);
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) b[c] = mul2<PAIR>(b[c], m[c]);
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) h[j][c] = fma2<PAIR>(two(a.residual), b[c], h[j][c]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) ss = fma2<PAIR>(h[j][c], h[j][c], ss);
      if (a.h_out) store_two(a.h_out, HF32, t * a.ldh_out + i, h[j]);
    }
    if (!a.x) continue;
    const float inv = rsqrtf(fmaf(row_sum<NT>(ss.x + ss.y, red[turn][1]), a.inv_d, a.eps));
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = (j * NT + tid) * 8;
      if (i >= a.d) continue;
#pragma unroll
      for (int c = 0; c < 4; ++c) h[j][c] = mul2<PAIR>(h[j][c], two(inv));
      if (a.pre) {
        float2 m[4];
        load_two(a.pre, a.w_f32, i, m);
#pragma unroll
        for (int c = 0; c < 4; ++c) h[j][c] = mul2<PAIR>(h[j][c], m[c]);
      }
      store_two(a.x, false, t * a.ldx + i, h[j]);
    }
  }
}

// An element of a row that starts at p, of either type.
__device__ __forceinline__ float at(const uint8_t* p, bool f32, int i) {
  return f32 ? reinterpret_cast<const float*>(p)[i] : bf16_lo(reinterpret_cast<const uint16_t*>(p)[i]);
}
__device__ __forceinline__ const uint8_t* from(const void* p, bool f32, int64_t i) {
  return p ? static_cast<const uint8_t*>(p) + i * (f32 ? 4 : 2) : nullptr;
}

// The same element by element, for rows that are not aligned in eights.
template <int NT, int V, bool HF32, bool YF32>
__global__ void __launch_bounds__(block_threads(NT)) block_norm_any_kernel(const NormArgs a) {
  alignas(16) __shared__ float red[2][NT / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t t = (int64_t)blockIdx.x * (block_threads(NT) / NT) + threadIdx.x / NT;
  if (t >= a.rows) return;  // whole warps; larger rows have a block each
  const int tid = threadIdx.x % NT, here = a.d - tid;  // elements j * NT < here are this thread's
  const uint8_t* const hp = from(a.h, HF32, t * a.ldh + tid);
  const uint8_t* const yp = from(a.y, YF32, t * a.ldy + tid);
  float h[V], y[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    y[j] = yp && j * NT < here ? at(yp, YF32, j * NT) : 0.f;
    h[j] = j * NT < here ? at(hp, HF32, j * NT) : 0.f;
  }
  if (yp) {
    if (a.post_norm) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) ss = fmaf(y[j], y[j], ss);
      const float yscale = rsqrtf(fmaf(row_sum<NT>(ss, red[0]), a.inv_d, a.eps));
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] *= yscale;
    }
    if (const uint8_t* const w = from(a.post, a.w_f32, tid)) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * NT < here) y[j] *= at(w, a.w_f32, j * NT);
    }
    if (a.gate && a.gate_col == 0) {
      const float g = load(a.gate, a.gate_f32, t * a.gate_row);
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] *= g;
    } else if (a.gate) {
      const uint8_t* const g = from(a.gate, a.gate_f32, a.gate_at(t, tid));
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (j * NT < here)
          y[j] *= a.gate_col == 1 ? at(g, a.gate_f32, j * NT) : load(g, a.gate_f32, a.gate_at(0, j * NT));
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    h[j] = fmaf(a.residual, y[j], a.skip * h[j]);
    ss = fmaf(h[j], h[j], ss);
  }
  if (a.h_out) {
    uint8_t* const o = const_cast<uint8_t*>(from(a.h_out, HF32, t * a.ldh_out + tid));
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * NT < here) {
        if constexpr (HF32) reinterpret_cast<float*>(o)[j * NT] = h[j];
        else reinterpret_cast<uint16_t*>(o)[j * NT] = bf16_bits(h[j]);
      }
  }
  if (!a.x) return;
  const float inv = rsqrtf(fmaf(row_sum<NT>(ss, red[1]), a.inv_d, a.eps));
#pragma unroll
  for (int j = 0; j < V; ++j) h[j] *= inv;
  if (const uint8_t* const w = from(a.pre, a.w_f32, tid)) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j * NT < here) h[j] *= at(w, a.w_f32, j * NT);
  }
  uint16_t* const o = a.x + t * a.ldx + tid;
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (j * NT < here) o[j * NT] = bf16_bits(h[j]);
}

// Blocks of a kernel that the current device holds at once.
template <auto kernel, int threads>
int resident() {
  static std::mutex mu;
  static int blocks[64] = {};
  int dev = 0, sms = 0, per = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  std::lock_guard<std::mutex> lock(mu);
  if (!blocks[dev]) {
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess &&
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) == cudaSuccess)
      blocks[dev] = sms * per;
    else
      cudaGetLastError();  // not kept: the next call asks again
  }
  return blocks[dev] > 0 ? blocks[dev] : 148;
}

template <bool F32, int KP>
int combine_wide(const void* y, int64_t ldy, int y_rows, const int32_t* pos, const float* weights, int tokens, int top_e,
                 int d, int runs, uint16_t* out, int64_t ldo, cudaStream_t st) {
  const uint32_t items = (uint32_t)tokens * runs;  // below 2^31: checked by the caller
  const int most = resident<combine_kernel<F32, KP>, kCombineNT>();
  return launch_early(combine_kernel<F32, KP>, std::min<uint32_t>(items, most), kCombineNT, 0, st, y, ldy, y_rows, pos,
                      weights, items, top_e, d, runs, out, ldo);
}

constexpr int kManyRows = 148 * 8;  // rows from which a warp per row fills the device

// Rows whose eights of elements are 16-byte aligned (a null pointer is).
bool by8(const void* p, int64_t pitch, int64_t rows) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (rows == 1 || pitch % 8 == 0);
}

template <int NT, int V, bool HF32, bool YF32>
int norm_wide(const NormArgs& a, cudaStream_t st) {
  constexpr int threads = block_threads(NT);
  const int64_t blocks = ((int64_t)a.rows * NT + threads - 1) / threads;
  const int most = resident<block_norm_kernel<NT, V, HF32, YF32>, threads>();
  return launch_early(block_norm_kernel<NT, V, HF32, YF32>, std::min<int64_t>(blocks, most), threads, 0, st, a);
}
template <int NT, int V>
int norm_wide_f32(const NormArgs& a, cudaStream_t st) {  // h, y or both in float
  if (!a.h_f32) return norm_wide<NT, V, false, true>(a, st);
  return a.y_f32 ? norm_wide<NT, V, true, true>(a, st) : norm_wide<NT, V, true, false>(a, st);
}
template <int NT, int W, int V>
int norm_rows(const NormArgs& a, cudaStream_t st) {
  constexpr int threads = block_threads(NT);
  if constexpr (W == 8) {
    return a.h_f32 || a.y_f32 ? norm_wide_f32<NT, V>(a, st) : norm_wide<NT, V, false, false>(a, st);
  } else {
    const auto kernel = a.h_f32 ? (a.y_f32 ? block_norm_any_kernel<NT, V, true, true> : block_norm_any_kernel<NT, V, true, false>)
                                : (a.y_f32 ? block_norm_any_kernel<NT, V, false, true>
                                           : block_norm_any_kernel<NT, V, false, false>);
    return launch_early(kernel, ((int64_t)a.rows * NT + threads - 1) / threads, threads, 0, st, a);
  }
}

// F(NT, W, V) for the smallest shape that holds k elements a row: in eights, one by one.
#define MSB_ROW_SHAPES_8(k, F)                  \
  if ((k) <= 256) return F(32, 8, 1);           \
  if ((k) <= 512) return F(32, 8, 2);           \
  if ((k) <= 1024) return F(32, 8, 4);          \
  if ((k) <= 2048) return F(256, 8, 1);         \
  if ((k) <= 4096) return F(256, 8, 2);         \
  if ((k) <= 8192) return F(512, 8, 2);         \
  if ((k) <= 16384) return F(512, 8, 4);
#define MSB_ROW_SHAPES_1(k, F)                  \
  if ((k) <= 128) return F(32, 1, 4);           \
  if ((k) <= 512) return F(32, 1, 16);          \
  if ((k) <= 1024) return F(256, 1, 4);         \
  if ((k) <= 4096) return F(256, 1, 16);        \
  if ((k) <= 16384) return F(512, 1, 32);

}  // namespace

int launch_quantize(const void* x, bool f32, int64_t ldx, int rows, int k, int8_t* q, int64_t ldq,
                    float* scale, cudaStream_t st) {
  const bool wide = k % 8 == 0 && by8(x, ldx, rows) && reinterpret_cast<uintptr_t>(q) % 8 == 0 &&
                    (rows == 1 || ldq % 8 == 0);
  if (wide && rows >= kManyRows && k > 1024 && k <= (f32 ? 2048 : 4096)) {
    const auto kernel = f32 ? quantize_warp_kernel<8, true>
                        : k <= 2048 ? quantize_warp_kernel<8, false> : quantize_warp_kernel<16, false>;
    return launch_early(kernel, ((int64_t)rows + 7) / 8, 256, 0, st, x, ldx, rows, k, q, ldq, scale);
  }
#define MSB_QUANT(NT, W, V)                                                                          \
  launch_early(quantize_kernel<NT, W, V>, ((int64_t)rows * NT + block_threads(NT) - 1) / block_threads(NT), \
         block_threads(NT), 0, st, x, f32, ldx, rows, k, q, ldq, scale)
  if (wide) {
    MSB_ROW_SHAPES_8(k, MSB_QUANT)
  } else {
    MSB_ROW_SHAPES_1(k, MSB_QUANT)
  }
#undef MSB_QUANT
  return launch_early(quantize_long_kernel, rows, 256, 0, st, x, f32, ldx, k, q, ldq, scale);
}

int launch_combine(const void* y, bool f32, int64_t ldy, int y_rows, const int32_t* pos,
                   const float* weights, int tokens, int top_e, int d, uint16_t* out, int64_t ldo,
                   cudaStream_t st) {
  const bool wide = d % 8 == 0 && by8(y, ldy, y_rows) && by8(out, ldo, tokens);
  const int runs = (d + kCombineNT * (wide ? 8 : 1) - 1) / (kCombineNT * (wide ? 8 : 1));
  const int64_t blocks = (int64_t)tokens * runs;
  if (blocks > 0x7fffffff) return MSB_EUNSUPPORTED;
  if (!wide)
    return launch_early(combine_any_kernel, blocks, kCombineNT, 0, st, y, f32, ldy, y_rows, pos, weights, top_e, d,
                        runs, out, ldo);
#define MSB_COMBINE(KP)                                                                                        \
  (f32 ? combine_wide<true, KP>(y, ldy, y_rows, pos, weights, tokens, top_e, d, runs, out, ldo, st)            \
       : combine_wide<false, KP>(y, ldy, y_rows, pos, weights, tokens, top_e, d, runs, out, ldo, st))
  return top_e > 4 ? MSB_COMBINE(8) : top_e > 2 ? MSB_COMBINE(4) : top_e > 1 ? MSB_COMBINE(2) : MSB_COMBINE(1);
#undef MSB_COMBINE
}

int launch_block_norm(const NormArgs& a, cudaStream_t st) {
  const int64_t rows = a.rows;
  bool wide = a.d % 8 == 0 && by8(a.h, a.ldh, rows) && by8(a.y, a.y ? a.ldy : 0, rows) &&
              by8(a.h_out, a.h_out ? a.ldh_out : 0, rows) && by8(a.x, a.x ? a.ldx : 0, rows) &&
              by8(a.pre, 0, 1) && by8(a.post, 0, 1);
  if (a.gate && a.gate_col == 1) wide = wide && by8(a.gate, a.gate_row, rows);
  const bool f32 = a.h_f32 || a.y_f32;
#define MSB_NORM(NT, W, V) norm_rows<NT, W, V>(a, st)
  if (!wide) {
    MSB_ROW_SHAPES_1(a.d, MSB_NORM)
  }
  // Rows in eights: threads and pieces a thread that keep the loads of about 64 KB in flight on
  // an SM where there are rows for it (8192 x 2048, 128 and 256 threads: bf16 24.9 and 29.6 us; 4
  // x 2048 2.6 and 2.1; float h, 8192 x 1024, 128 threads and a warp: 18.5 and 23.7).
  if (a.d <= 256) return MSB_NORM(32, 8, 1);
  if (a.d <= 512) return MSB_NORM(32, 8, 2);
  if (a.d <= 1024) return f32 ? norm_wide_f32<128, 1>(a, st) : norm_wide<32, 4, false, false>(a, st);
  if (a.d <= 2048) return rows >= kManyRows ? MSB_NORM(128, 8, 2) : MSB_NORM(256, 8, 1);
  if (a.d <= 4096) return MSB_NORM(256, 8, 2);
  if (a.d <= 8192) return MSB_NORM(512, 8, 2);
  if (a.d <= 16384) return MSB_NORM(512, 8, 4);
#undef MSB_NORM
  return MSB_EUNSUPPORTED;  // d <= MSB_NORM_MAX_D
}

}  // namespace msb
