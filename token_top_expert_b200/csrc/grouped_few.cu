// Grouped products of a few rows (decode), weights with k contiguous: each weight of the used
// experts is read once, from many warps at once, and multiplied on the CUDA cores; the matrix
// unit's tiles of 256 weight rows would put the stream of one token's eight experts on 96 of the
// 148 SMs, and one row's 4096 x 4096 product on 32.  Bound by the weights' bytes.  The warps
// stay and take two weight rows after another of the used groups, so that one warp's sums hide
// behind the others' loads; a group's rows are taken four, two and one at a time.
#include <algorithm>

#include "dense.h"
#include "grouped.cuh"
#include "quant.cuh"

namespace msb {
namespace {

// The groups that have rows, found by warp 0 of each block.
struct Used {
  int32_t begin[kGroupsMax + 1];
  int32_t group[kGroupsMax];
  int32_t count;
};
__device__ void find_used(const KArgs& a, Used& s) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    group_begins(a, s.begin, lane);
    int count = 0;
    for (int e0 = 0; e0 < a.groups; e0 += 32) {
      const int e = e0 + lane;
      const bool used = e < a.groups && s.begin[e + 1] > s.begin[e];
      const uint32_t m = __ballot_sync(0xffffffffu, used);
      if (used) s.group[count + __popc(m & ((1u << lane) - 1))] = e;
      count += __popc(m);
    }
    if (lane == 0) s.count = count;
  }
  __syncthreads();
}

__device__ __forceinline__ float x_scale(const KArgs& a, int p) {
  const int row = a.rows ? a.rows[p] : p;
  return (uint32_t)row < (uint32_t)a.x_rows ? a.x_scale[row] : 0.f;
}

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 16 bytes of the inner dimension: eight bf16 or sixteen 8-bit products.
__device__ __forceinline__ void dot16(const uint4& w, const uint4& x, float& acc) { acc = dot8(w, x, acc); }
__device__ __forceinline__ void dot16(const uint4& w, const uint4& x, int& acc) {
  acc = __dp4a((int)w.x, (int)x.x, acc);
  acc = __dp4a((int)w.y, (int)x.y, acc);
  acc = __dp4a((int)w.z, (int)x.z, acc);
  acc = __dp4a((int)w.w, (int)x.w, acc);
}
// The first `valid` bytes (below 16) of a piece, the rest zeros.
__device__ __forceinline__ uint4 load_part(const uint8_t* p, int valid) {
  uint32_t v[4] = {0, 0, 0, 0};
  for (int i = 0; i < valid; ++i) v[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

constexpr int kResident = 2;  // blocks of an SM

// P pieces of two weight rows, 32 pieces apart, times R rows of x.  The rows' indices may still be
// on their way: they are not looked at before the weights' loads are under way.
template <int P, int R, class Acc>
__device__ __forceinline__ void few_pieces(const KArgs& a, const uint8_t* w0, const uint8_t* w1, int (&row)[R],
                                           int64_t at, Acc (&acc)[2][R]) {
  uint4 v[2][P];
#pragma unroll
  for (int q = 0; q < P; ++q) v[0][q] = load_stream(w0 + at + q * 512);
#pragma unroll
  for (int q = 0; q < P; ++q) v[1][q] = load_stream(w1 + at + q * 512);
  const uint8_t* x[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    asm volatile("" : "+r"(row[r]));
    x[r] = a.x + (int64_t)((uint32_t)row[r] < (uint32_t)a.x_rows ? row[r] : 0) * a.pitch;
  }
#pragma unroll
  for (int q = 0; q < P; ++q)
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint4 xv = *reinterpret_cast<const uint4*>(x[r] + at + q * 512);
      dot16(v[0][q], xv, acc[0][r]);
      dot16(v[1][q], xv, acc[1][r]);
    }
}

// Two weight rows times R rows of x, output rows p0 .. p0 + R - 1: the warp's lanes take the
// pieces of k.  Lane 0 has the first channel, lane 1 the second; gated: lane 0 alone.
template <int R, bool I8, bool GATED, bool F32>
__device__ __forceinline__ void few_rows_of(const KArgs& a, const uint8_t* w0, const uint8_t* w1, int group, int ch,
                                            int p0, int lane) {
  using Acc = typename std::conditional<I8, int, float>::type;
  constexpr int P = R == 4 ? 4 : 8;
  const int whole = a.kbytes >> 4, tail = a.kbytes & 15;
  int row[R];  // of x; one outside gives zeros (and reads the first)
  Acc acc[2][R] = {};
#pragma unroll
  for (int r = 0; r < R; ++r) row[r] = a.rows ? a.rows[p0 + r] : p0 + r;
  int i = lane;
  for (; i + 32 * (P - 1) < whole; i += 32 * P) few_pieces<P>(a, w0, w1, row, (int64_t)i * 16, acc);
  if (P == 8 && i + 96 < whole) {
    few_pieces<4>(a, w0, w1, row, (int64_t)i * 16, acc);
    i += 128;
  }
  for (; i < whole; i += 32) few_pieces<1>(a, w0, w1, row, (int64_t)i * 16, acc);
  if (tail && lane == 0) {
    const uint4 v0 = load_part(w0 + (int64_t)whole * 16, tail), v1 = load_part(w1 + (int64_t)whole * 16, tail);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t at = (uint32_t)row[r] < (uint32_t)a.x_rows ? row[r] : 0;
      const uint4 xv = load_part(a.x + at * a.pitch + (int64_t)whole * 16, tail);
      dot16(v0, xv, acc[0][r]);
      dot16(v1, xv, acc[1][r]);
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      acc[0][r] += __shfl_xor_sync(0xffffffffu, acc[0][r], o);
      acc[1][r] += __shfl_xor_sync(0xffffffffu, acc[1][r], o);
    }
    if ((uint32_t)row[r] >= (uint32_t)a.x_rows) acc[0][r] = acc[1][r] = 0;
  }
  const int c = ch + (GATED ? 0 : lane);
  if (lane >= (GATED ? 1 : 2) || c >= a.n) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float v;
    if constexpr (I8) {
      const float xs = x_scale(a, p0 + r);
      const float* const ws = a.w_scale + (int64_t)group * (GATED ? 2 : 1) * a.n;
      v = GATED ? gated((float)acc[0][r] * xs * ws[ch], (float)acc[1][r] * xs * ws[a.n + ch])
                : (float)(lane == 0 ? acc[0][r] : acc[1][r]) * xs * ws[c];
    } else {
      v = GATED ? gated(acc[0][r], acc[1][r]) : lane == 0 ? acc[0][r] : acc[1][r];
    }
    const int64_t at = (int64_t)(p0 + r) * a.ldo + c;
    if constexpr (F32) static_cast<float*>(a.out)[at] = v;
    else static_cast<uint16_t*>(a.out)[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

// A warp takes two weight rows (gate and up of a channel, or two channels) at a time.
// SPREAD: `use` warps of a block do, else all eight (known to the compiler: it has no register left
// for reading it, 1 row by 4096 x 4096 7.8 and 8.3 us).
template <bool I8, bool GATED, bool F32, bool SPREAD>
__device__ __forceinline__ void few_items(const KArgs& a, const Used& s, int use) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int each = GATED ? a.n : (a.n + 1) / 2;  // pairs of weight rows of a group
  const int64_t items = (int64_t)s.count * each;
  if (SPREAD && warp >= use) return;
  const int warps = SPREAD ? use : 8;
  for (int64_t item = (int64_t)blockIdx.x * warps + warp; item < items; item += (int64_t)gridDim.x * warps) {
    const int slot = (int)(item / each), ch = (int)(item - (int64_t)slot * each) * (GATED ? 1 : 2);
    const int group = s.group[slot], end = s.begin[group + 1];
    const uint8_t* const w0 = a.w + (int64_t)group * a.w_group + (int64_t)ch * a.w_n;
    const uint8_t* const w1 = GATED ? w0 + a.w_part : ch + 1 < a.n ? w0 + a.w_n : w0;
    int p = s.begin[group];
    for (; p + 4 <= end; p += 4) few_rows_of<4, I8, GATED, F32>(a, w0, w1, group, ch, p, lane);
    if (p + 2 <= end) {
      few_rows_of<2, I8, GATED, F32>(a, w0, w1, group, ch, p, lane);
      p += 2;
    }
    if (p < end) few_rows_of<1, I8, GATED, F32>(a, w0, w1, group, ch, p, lane);
  }
}

template <bool I8, bool GATED, bool F32, bool SPREAD>
__global__ void __launch_bounds__(256, kResident) few_kernel(const KArgs a, int use) {
  __shared__ Used s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  find_used(a, s);
  few_items<I8, GATED, F32, SPREAD>(a, s, use);
}

// Rows of x before they are quantised.  by8: eights of elements are 16-byte aligned.
struct RawRows {
  const void* x;
  int64_t ldx;
  bool f32, by8;
};

// Elements i .. i + 7 of a row, zeros behind its end.
__device__ __forceinline__ void raw8(const RawRows& r, int64_t row, int i, int k, float (&v)[8]) {
  const int64_t at = row * r.ldx + i;
  if (r.by8 && i + 8 <= k) {
    if (r.f32) {
      const float4 lo = reinterpret_cast<const float4*>(static_cast<const float*>(r.x) + at)[0];
      const float4 hi = reinterpret_cast<const float4*>(static_cast<const float*>(r.x) + at)[1];
      v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w, v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(r.x) + at);
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
      v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
    return;
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    v[c] = i + c >= k ? 0.f
           : r.f32    ? static_cast<const float*>(r.x)[at + c]
                      : bf16_lo(static_cast<const uint16_t*>(r.x)[at + c]);
}

// Rows of x that one launch quantises on the way, and elements with them in sixteens.  One launch
// and two, cold weights: 1 x 4096, 4096 channels 6.6 and 6.6 us (a call of 14.5 us on the host
// against 16.1), 1 x 1024, 1024 channels 3.5 and 4.3, 8 x 512, 2048 channels 5.5 and 5.8, one
// token's 8-bit gate and up 8.8 and 9.4; but 2 x 4096 6.0 and 5.5, since every block rounds them all.
constexpr int kRawRows = 8, kRawElements = 4096;

// Quantising and the products in one launch: every block rounds the few rows of x for itself, into
// shared memory.  (Asking for the first weights ahead of that: 6.9 us instead of 6.6.)
template <bool GATED, bool F32>
__global__ void __launch_bounds__(256, kResident) few_linear_kernel(const KArgs args, const RawRows raw, int use) {
  constexpr int V = 4;  // pieces of eight of a thread: rows of 4096 / x_rows elements need at most that
  __shared__ uint4 xq[kRawElements / 16];  // [x_rows][pitch / 16]
  __shared__ Used s;
  __shared__ uint32_t big[kRawRows];
  __shared__ float scale[kRawRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x < kRawRows) big[threadIdx.x] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  KArgs a = args;
  a.x = reinterpret_cast<const uint8_t*>(xq);
  a.pitch = (a.k + 15) & ~15;
  a.x_scale = scale;
  // eight warps share the rows: one, two, four or eight to a row
  const int to = a.x_rows > 4 ? 1 : a.x_rows > 2 ? 2 : a.x_rows > 1 ? 4 : 8;
  const int row = warp / to, first = ((warp % to) * 32 + lane) * 8;
  const bool mine = row < a.x_rows;
  float v[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (mine && first + j * to * 256 < a.pitch) raw8(raw, row, first + j * to * 256, a.k, v[j]);
  find_used(a, s);  // a barrier at its end
  if (mine) {
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (first + j * to * 256 < a.pitch)
#pragma unroll
        for (int c = 0; c < 8; ++c) most = max(most, __float_as_uint(v[j][c]) & 0x7fffffffu);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) atomicMax(&big[row], most);
  }
  __syncthreads();
  if (mine) {
    const QuantScale qs = quant_scale(big[row]);
    if (warp % to == 0 && lane == 0) scale[row] = qs.scale;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = first + j * to * 256;
      if (i < a.pitch)
        *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(xq) + row * a.pitch + i) =
            qs.inv == 0.f ? make_uint2(0, 0) : make_uint2(quant4(v[j], qs.inv), quant4(v[j] + 4, qs.inv));
    }
  }
  __syncthreads();
  few_items<true, GATED, F32, true>(a, s, use);
}

// Blocks, and how many of a block's eight warps take items: all, but where the items would fill less
// than half the blocks that the device holds, only so many that every block has some (8 and
// fewer warps: 8 rows by 1024 x 1024 5.6 and 4.9 us, 4 rows by 2048 x 2048 6.2 and 5.6).
struct Shape {
  int blocks, use;
};
template <bool GATED>
Shape few_shape(const GroupedArgs& a) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return {0, 0};
  const int64_t items = (int64_t)std::min(a.groups, a.out_rows) * (GATED ? a.n : (a.n + 1) / 2);
  const int64_t most = (int64_t)kResident * sms, use = items <= 4 * most ? (items + most - 1) / most : 8;
  return {(int)std::min<int64_t>((items + use - 1) / use, most), (int)use};
}
template <bool I8, bool GATED, bool F32>
int launch(const GroupedArgs& a, const KArgs& k, cudaStream_t st) {
  const Shape s = few_shape<GATED>(a);
  if (!s.blocks) return MSB_ECUDA;
  return launch_early(s.use < 8 ? few_kernel<I8, GATED, F32, true> : few_kernel<I8, GATED, F32, false>, s.blocks, 256, 0,
                      st, k, s.use);
}
template <bool GATED, bool F32>
int launch_raw(const GroupedArgs& a, const KArgs& k, const RawRows& raw, cudaStream_t st) {
  const Shape s = few_shape<GATED>(a);
  return s.blocks ? launch_early(few_linear_kernel<GATED, F32>, s.blocks, 256, 0, st, k, raw, s.use) : MSB_ECUDA;
}

}  // namespace

// Up to 8 rows (4 of one weight that is large or has long rows), unless many weights have short rows,
// this kernel is the faster one (the matrix unit's time in brackets, cold weights): one token's gate
// and up, hidden 2048 x 768 channels x 128 experts top-8, 12.1 us (12.3), 8 bits 8.3 (8.8), but its
// 8-bit down product with k = 768 9.9 (6.3).  One bf16 weight n x k: 4096 x 4096, 1 row 7.8 us (11.4),
// 4 rows 10.6 (11.5), 8 rows 16.7 (11.6); 8 rows of 2048 x 2048 7.7 (8.1), 1024 x 1024 4.9 (6.3),
// but 512 x 4096 10.9 (8.5).  8 bits: 8 rows of 2048 x 2048 5.5 (6.7), 4096 x 4096 9.0 (8.9), 6 rows
// 7.9 (8.9).
bool few_rows(const GroupedArgs& a) {
  const int64_t kbytes = (int64_t)a.k * (a.i8 ? 1 : 2);
  const int64_t bytes = std::min(a.groups, a.out_rows) * (a.swiglu ? 2 : 1) * kbytes * a.n;
  const bool small = kbytes <= 4096 && bytes <= (a.i8 ? 16 : 8) << 20;
  if (a.w_k != 1 || a.out_rows > (a.groups > 1 || small ? 8 : 4)) return false;
  return kbytes >= 1024 || bytes <= 1 << 20;
}

int launch_few(const GroupedArgs& a, const KArgs& k, cudaStream_t st) {
  if (a.swiglu) return a.i8 ? launch<true, true, false>(a, k, st) : launch<false, true, false>(a, k, st);
  if (a.i8) return a.out_f32 ? launch<true, false, true>(a, k, st) : launch<true, false, false>(a, k, st);
  return a.out_f32 ? launch<false, false, true>(a, k, st) : launch<false, false, false>(a, k, st);
}

int launch_linear(const GroupedArgs& a, const void* x, bool f32, int64_t ldx, int8_t* q, float* scale,
                  cudaStream_t st) {
  const int64_t pitch = ((int64_t)a.k + 15) & ~15;
  if (few_rows(a) && a.x_rows > 0 && a.x_rows <= kRawRows && a.x_rows * pitch <= kRawElements) {
    const bool by8 = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (a.x_rows == 1 || ldx % 8 == 0);
    const RawRows raw = {x, ldx, f32, by8};
    const KArgs k = kernel_args(a);
    if (a.swiglu) return launch_raw<true, false>(a, k, raw, st);
    return a.out_f32 ? launch_raw<false, true>(a, k, raw, st) : launch_raw<false, false>(a, k, raw, st);
  }
  const int rc = a.x_rows > 0 ? launch_quantize(x, f32, ldx, a.x_rows, a.k, q, a.ldx, scale, st) : MSB_OK;
  return rc != MSB_OK ? rc : launch_grouped(a, st);
}

}  // namespace msb
