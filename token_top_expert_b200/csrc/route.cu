// Routing of any number of tokens: top-K experts, combine weights, and the plan of the grouped
// products (pairs sorted by expert and token), in at most two launches and without atomics on
// global memory, so that the plan is the same in every run.
//
// route_kernel: a block takes a run of consecutive tokens, a warp one token at a time: the
// experts' logits as order-preserving keys in registers, K rounds of a warp-wide maximum (two
// redux instructions: the key, then the lowest index that has it); the block counts its pairs
// per expert.  place_kernel: each block adds up the counts before its own (experts before, then
// blocks before), and places its pairs: a thread per (expert, run of the block's pairs) counts
// and then writes the pairs of its expert in order.  Up to kOneBlock tokens one block does both.
#include "common.cuh"
#include "dense.h"

namespace msb {
namespace {

constexpr int kNT = 1024;
constexpr int kOneBlock = 64;   // tokens up to which a single block routes and places
constexpr int kChunk = 4096;    // pairs placed at a time
constexpr int kMaxE = MSB_MAX_EXPERTS;

struct PlaceShared {
  int32_t ids[kChunk];
  int32_t part[kNT];
  int32_t part2[kNT];
  int32_t base[kMaxE];  // next row of each expert for this block's pairs
  int32_t warp[32];
  int32_t total;
};

// Key of a logit: ascending with the value, -0 = +0; 0 for NaN and -infinity (no candidate);
// +infinity as the largest finite float.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (!(v > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(fminf(v, 3.402823466e38f) + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

__device__ void place(const int32_t* ids, int32_t* rows, int32_t* pos, int32_t* offsets,
                      const int32_t* hist, int tokens, int experts, int top_e, int per,
                      PlaceShared& s) {
  const int b = blockIdx.x, nb = gridDim.x, tid = threadIdx.x;
  const int lane = tid & 31, warp = tid >> 5;
  const int epad = (experts + 31) & ~31;
  const int segs = min(16, kNT / epad);  // threads per expert
  const int seg = tid / epad, e = tid - seg * epad;
  const bool mine = seg < segs && e < experts;
  // counts of each expert in the blocks before this one, and in all
  int before = 0, all = 0;
  if (mine)
    for (int i = seg; i < nb; i += segs) {
      const int c = hist[(int64_t)i * experts + e];
      all += c;
      if (i < b) before += c;
    }
  s.part[tid] = all;
  s.part2[tid] = before;
  __syncthreads();
  all = before = 0;
  if (tid < experts)
    for (int i = 0; i < segs; ++i) all += s.part[i * epad + tid], before += s.part2[i * epad + tid];
  // rows of the experts before: exclusive scan of `all` over the threads (tid = expert)
  int inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) s.warp[warp] = inc;
  __syncthreads();
  int lead = 0;
  for (int w = 0; w < warp; ++w) lead += s.warp[w];
  const int off = lead + inc - all;
  if (tid < experts) {
    s.base[tid] = off + before;
    if (b == 0) offsets[tid] = off;
    if (tid == experts - 1) {
      s.total = off + all;
      if (b == 0) offsets[experts] = off + all;
    }
  }
  __syncthreads();
  const int64_t pairs = (int64_t)tokens * top_e;
  for (int64_t i = s.total + (int64_t)b * kNT + tid; i < pairs; i += (int64_t)nb * kNT) rows[i] = -1;
  // this block's pairs, a chunk at a time, in order
  const int64_t p0 = (int64_t)min(b * per, tokens) * top_e;
  const int64_t p1 = (int64_t)min((b + 1) * per, tokens) * top_e;
  for (int64_t c0 = p0; c0 < p1; c0 += kChunk) {
    const int n = (int)min((int64_t)kChunk, p1 - c0);
    for (int i = tid; i < n; i += kNT) s.ids[i] = ids[c0 + i];
    __syncthreads();
    const int run = (n + segs - 1) / segs;
    const int i0 = min(seg * run, n), i1 = min(i0 + run, n);
    int count = 0;
    if (mine)
      for (int i = i0; i < i1; ++i) count += s.ids[i] == e;
    s.part[tid] = count;
    __syncthreads();
    if (mine) {
      int at = s.base[e];
      for (int i = 0; i < seg; ++i) at += s.part[i * epad + e];
      if (count)
        for (int i = i0; i < i1; ++i)
          if (s.ids[i] == e) {
            rows[at] = (int32_t)((c0 + i) / top_e);
            pos[c0 + i] = at++;
          }
    }
    __syncthreads();
    if (tid < experts)
      for (int i = 0; i < segs; ++i) s.base[tid] += s.part[i * epad + tid];
    __syncthreads();
  }
}

// NV: values a lane holds (experts <= 32 NV).
template <int NV, bool BF16>
__global__ void __launch_bounds__(kNT, 1)
    route_kernel(const void* logits, int64_t ld, const uint8_t* mask, int tokens, int experts,
                 int top_e, int renorm, int32_t* ids, float* weights, int32_t* offsets,
                 int32_t* rows, int32_t* pos, int32_t* hist, int per) {
  __shared__ PlaceShared s;
  __shared__ int32_t count[kMaxE];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int e = tid; e < experts; e += kNT) count[e] = 0;
  __syncthreads();
  const int t1 = min((int)(blockIdx.x + 1) * per, tokens);
  for (int t = blockIdx.x * per + warp; t < t1; t += kNT / 32) {
    uint32_t key[NV];
    const bool use = !mask || mask[t] != 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = i * 32 + lane;
      float v = -INFINITY;
      if (use && e < experts) {
        if constexpr (BF16)
          v = bf16_lo(static_cast<const uint16_t*>(logits)[(int64_t)t * ld + e]);
        else
          v = static_cast<const float*>(logits)[(int64_t)t * ld + e];
      }
      key[i] = logit_key(v);
    }
    float top = 0.f, sum = 0.f, w = 0.f;
    int id = -1;
    for (int k = 0; k < top_e; ++k) {
      uint32_t best = 0;
      int at = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (key[i] > best) best = key[i], at = i * 32 + lane;
      const uint32_t most = __reduce_max_sync(0xffffffffu, best);
      if (most == 0) break;
      const int e = __reduce_min_sync(0xffffffffu, best == most ? (uint32_t)at : 0xffffffffu);
      const float v = key_logit(most);
      if (k == 0) {
        top = v;
        if (!renorm) {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (key[i]) sum += expf(key_logit(key[i]) - top);
          sum = warp_sum(sum);
        }
      }
      if (lane == k) id = e, w = expf(v - top);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * 32 + lane == e) key[i] = 0;
    }
    if (renorm) sum = warp_sum(w);
    if (lane < top_e) {
      const int64_t at = (int64_t)t * top_e + lane;
      ids[at] = id;
      weights[at] = id < 0 ? 0.f : w / sum;
      if (id < 0) pos[at] = -1;
      else atomicAdd(&count[id], 1);
    }
  }
  __syncthreads();
  for (int e = tid; e < experts; e += kNT) hist[(int64_t)blockIdx.x * experts + e] = count[e];
  if (gridDim.x == 1) {
    __syncthreads();
    place(ids, rows, pos, offsets, hist, tokens, experts, top_e, per, s);
  }
}

__global__ void __launch_bounds__(kNT, 1)
    place_kernel(const int32_t* ids, int32_t* rows, int32_t* pos, int32_t* offsets,
                 const int32_t* hist, int tokens, int experts, int top_e, int per) {
  __shared__ PlaceShared s;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  place(ids, rows, pos, offsets, hist, tokens, experts, top_e, per, s);
}

}  // namespace

int route_blocks(int tokens) {
  return tokens <= kOneBlock ? 1 : min(148, (tokens + 31) / 32);
}

int launch_route(const void* logits, bool bf16, int64_t ld, const uint8_t* mask, int tokens,
                 int experts, int top_e, bool renorm, int32_t* ids, float* weights,
                 int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t st) {
  const int nb = route_blocks(tokens), per = (tokens + nb - 1) / nb;
#define MSB_ROUTE(NV)                                                                               \
  launch_early(bf16 ? route_kernel<NV, true> : route_kernel<NV, false>, nb, kNT, 0, st, logits, ld, mask, \
               tokens, experts, top_e, renorm ? 1 : 0, ids, weights, offsets, rows, pos, hist, per)
  const int rc = experts <= 64    ? MSB_ROUTE(2)
                 : experts <= 128 ? MSB_ROUTE(4)
                 : experts <= 256 ? MSB_ROUTE(8)
                                  : MSB_ROUTE(16);
#undef MSB_ROUTE
  if (rc != MSB_OK || nb == 1) return rc;
  return launch_early(place_kernel, nb, kNT, 0, st, ids, rows, pos, offsets, hist, tokens, experts, top_e, per);
}

}  // namespace msb
