// Routing of any number of tokens: top-K experts, combine weights, and the plan of the grouped
// products (pairs sorted by expert and token), in at most two launches and without atomics on
// global memory, so that the plan is the same in every run.
//
// route_kernel: a block takes a run of consecutive tokens, a warp two tokens at a time: the
// experts' logits as order-preserving keys in registers, K rounds of a warp-wide maximum (two
// redux instructions: the key, then the lowest index that has it; the two tokens' chains
// overlap).  Every chunk of kChunk tokens leaves a bit per (expert, token) in shared memory:
// the bits below a pair's own are its rank among the block's pairs of that expert, and their
// number the expert's count.  place_kernel adds the counts of the experts and blocks before.
// Up to kOneBlock tokens one block does both.
//
// Bound by latency and issue: K rounds of about 50 instructions for two tokens, and the two
// launches.  128 experts top-8: 1 token 3.9 us, 64 tokens 8.3, 8192 tokens 13.7 (5.2 MB), 65536
// tokens 65.
#include "common.cuh"
#include "dense.h"

namespace msb {
namespace {

constexpr int kNT = 1024;
constexpr int kOneBlock = 64;  // tokens up to which a single block routes and places
constexpr int kChunk = 128;    // tokens whose bits are held at a time
constexpr int kMaxE = MSB_MAX_EXPERTS;

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

// The largest of N keys (N = 2 or 4) that lie 32 experts apart, and its expert; ties to the lower.
template <int N>
__device__ __forceinline__ void best_of(const uint32_t* key, int first, uint32_t& best, int& at) {
  const bool a = key[1] > key[0];
  best = a ? key[1] : key[0];
  at = a ? first + 32 : first;
  if constexpr (N == 4) {
    const bool b = key[3] > key[2];
    const uint32_t high = b ? key[3] : key[2];
    if (high > best) best = high, at = first + (b ? 96 : 64);
  }
}

// First row of each expert: exclusive scan of `all` (thread = expert) over the block.
__device__ __forceinline__ int rows_before(int all, int32_t* warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = all;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  int lead = lane < warp ? warps[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lead += __shfl_xor_sync(0xffffffffu, lead, o);
  return lead + inc - all;
}

// NV: values a lane holds (experts <= 32 NV).  One block: the whole plan.  More: pos holds each
// pair's rank among the block's, and hist the block's counts.
template <int NV, bool BF16>
__global__ void __launch_bounds__(kNT, 1)
    route_kernel(const void* logits, int64_t ld, const uint8_t* mask, int tokens, int experts,
                 int top_e, int renorm, int32_t* ids, float* weights, int32_t* offsets,
                 int32_t* rows, int32_t* pos, int32_t* hist, int per) {
  constexpr int kIn = NV < 4 ? NV : 4, kGroups = NV / kIn;
  __shared__ uint32_t bits[kChunk / 32][kMaxE];
  __shared__ int32_t count[kMaxE];  // pairs of each expert in the chunks before
  __shared__ int32_t chosen[kChunk * MSB_MAX_TOP_E];
  __shared__ int32_t warps[32];
  __shared__ int32_t total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = tid; i < kChunk / 32 * kMaxE; i += kNT) (&bits[0][0])[i] = 0;
  for (int e = tid; e < kMaxE; e += kNT) count[e] = 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  const int t1 = min((int)(blockIdx.x + 1) * per, tokens);
  for (int c0 = blockIdx.x * per; c0 < t1; c0 += kChunk) {
    const int n = min(kChunk, t1 - c0);  // tokens of the chunk
    for (int u = warp * 2; u < n; u += kNT / 16) {
      uint32_t key[2][NV];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int t = c0 + u + j;
        const bool use = u + j < n && (!mask || mask[t] != 0);
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
          key[j][i] = logit_key(v);
        }
      }
      float top[2] = {0.f, 0.f}, sum[2] = {0.f, 0.f}, w[2] = {0.f, 0.f};
      int id[2] = {-1, -1};
      // more than four values: the best of each four, so that only the four that lost one are looked
      // through again
      uint32_t gk[2][kGroups];
      int ga[2][kGroups];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < kGroups && kGroups > 1; ++g) best_of<kIn>(&key[j][g * kIn], g * kIn * 32 + lane, gk[j][g], ga[j][g]);
      for (int k = 0; k < top_e; ++k) {
        uint32_t best[2], most[2];
        int at[2], e[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if constexpr (kGroups == 1) best_of<kIn>(key[j], lane, gk[j][0], ga[j][0]);
          best[j] = gk[j][0];
          at[j] = ga[j][0];
#pragma unroll
          for (int g = 1; g < kGroups; ++g)
            if (gk[j][g] > best[j]) best[j] = gk[j][g], at[j] = ga[j][g];
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) most[j] = __reduce_max_sync(0xffffffffu, best[j]);
        if ((most[0] | most[1]) == 0) break;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          e[j] = __reduce_min_sync(0xffffffffu, best[j] == most[j] ? (uint32_t)at[j] : 0xffffffffu);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (most[j] == 0) continue;
          const float v = key_logit(most[j]);
          if (k == 0) {
            top[j] = v;
            if (!renorm) {
#pragma unroll
              for (int i = 0; i < NV; ++i)
                if (key[j][i]) sum[j] += expf(key_logit(key[j][i]) - v);
              sum[j] = warp_sum(sum[j]);
            }
          }
          if (lane == k) id[j] = e[j], w[j] = v;
          if constexpr (kGroups == 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (i * 32 + lane == e[j]) key[j][i] = 0;
            continue;
          }
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
            if (e[j] >> 5 >= g * kIn && e[j] >> 5 < (g + 1) * kIn) {  // the same for the warp
#pragma unroll
              for (int i = g * kIn; i < (g + 1) * kIn; ++i)
                if (i * 32 + lane == e[j]) key[j][i] = 0;
              best_of<kIn>(&key[j][g * kIn], g * kIn * 32 + lane, gk[j][g], ga[j][g]);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        w[j] = id[j] < 0 ? 0.f : expf(w[j] - top[j]);
        if (renorm) sum[j] = warp_sum(w[j]);
        const int t = u + j;
        if (t < n && lane < top_e) {
          const int64_t at = (int64_t)(c0 + t) * top_e + lane;
          ids[at] = id[j];
          weights[at] = id[j] < 0 ? 0.f : w[j] / sum[j];
          chosen[t * top_e + lane] = id[j];
          if (id[j] >= 0) atomicOr(&bits[t >> 5][id[j]], 1u << (t & 31));
        }
      }
    }
    __syncthreads();
    // rank of each pair among its expert's (and its row, where this block is all there is)
    if (gridDim.x == 1) {
      const int all = tid < experts ? __popc(bits[0][tid]) + __popc(bits[1][tid]) : 0;
      const int off = rows_before(all, warps);
      if (tid < experts) {
        offsets[tid] = off;
        count[tid] = off;
        if (tid == experts - 1) offsets[experts] = total = off + all;
      }
      __syncthreads();
    }
    for (int i = tid; i < n * top_e; i += kNT) {
      const int e = chosen[i], t = i / top_e;
      int rank = -1;
      if (e >= 0) {
        rank = count[e] + __popc(bits[t >> 5][e] & ((1u << (t & 31)) - 1));
        for (int q = 0; q < (t >> 5); ++q) rank += __popc(bits[q][e]);
        if (gridDim.x == 1) rows[rank] = t;
      }
      pos[(int64_t)c0 * top_e + i] = rank;
    }
    if (gridDim.x == 1) {
      for (int i = total + tid; i < n * top_e; i += kNT) rows[i] = -1;
      return;  // one chunk
    }
    __syncthreads();
    for (int e = tid; e < experts; e += kNT)
#pragma unroll
      for (int q = 0; q < kChunk / 32; ++q) {
        count[e] += __popc(bits[q][e]);
        bits[q][e] = 0;
      }
    __syncthreads();
  }
  if (gridDim.x == 1) {  // no tokens
    for (int e = tid; e <= experts; e += kNT) offsets[e] = 0;
    return;
  }
  for (int e = tid; e < experts; e += kNT) hist[(int64_t)blockIdx.x * experts + e] = count[e];
}

__global__ void __launch_bounds__(kNT, 1)
    place_kernel(const int32_t* ids, int32_t* rows, int32_t* pos, int32_t* offsets,
                 const int32_t* hist, int tokens, int experts, int top_e, int per) {
  __shared__ int32_t part[2][kNT];
  __shared__ int32_t base[kMaxE];
  __shared__ int32_t warps[32];
  __shared__ int32_t total;
  const int b = blockIdx.x, nb = gridDim.x, tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // counts of each expert in the blocks before this one, and in all: a thread per (expert,
  // every segs-th block)
  const int epad = (experts + 31) & ~31;
  const int segs = kNT / epad;
  const int seg = tid / epad, e = tid - seg * epad;
  int before = 0, all = 0;
  if (seg < segs && e < experts) {
#pragma unroll 10
    for (int i = seg; i < nb; i += segs) {
      const int c = hist[(int64_t)i * experts + e];
      all += c;
      before += i < b ? c : 0;
    }
  }
  part[0][tid] = all;
  part[1][tid] = before;
  __syncthreads();
  all = before = 0;
  if (tid < experts)
    for (int i = 0; i < segs; ++i) all += part[0][i * epad + tid], before += part[1][i * epad + tid];
  const int off = rows_before(all, warps);
  if (tid < experts) {
    base[tid] = off + before;
    if (b == 0) offsets[tid] = off;
    if (tid == experts - 1) {
      total = off + all;
      if (b == 0) offsets[experts] = off + all;
    }
  }
  __syncthreads();
  const int64_t pairs = (int64_t)tokens * top_e;
  for (int64_t i = total + (int64_t)b * kNT + tid; i < pairs; i += (int64_t)nb * kNT) rows[i] = -1;
  const int64_t p0 = (int64_t)min(b * per, tokens) * top_e;
  const int64_t p1 = (int64_t)min((b + 1) * per, tokens) * top_e;
  for (int64_t i = p0 + tid; i < p1; i += kNT) {
    const int id = ids[i];
    if (id < 0) continue;
    const int at = base[id] + pos[i];
    pos[i] = at;
    rows[at] = (int32_t)(i / top_e);
  }
}

}  // namespace

// Blocks of 16 tokens (8 of many experts), but one block up to kOneBlock tokens (16), which saves
// the second launch.  128 experts top-8, 256 tokens: 8.1 us (11.0 with 64 tokens a block).
int route_blocks(int tokens, int experts) {
  const int few = experts > 128 ? 2 : 1;
  if (tokens <= kOneBlock / (few * few)) return 1;
  return min(148, (tokens + 16 / few - 1) / (16 / few));
}

int launch_route(const void* logits, bool bf16, int64_t ld, const uint8_t* mask, int tokens,
                 int experts, int top_e, bool renorm, int32_t* ids, float* weights,
                 int32_t* offsets, int32_t* rows, int32_t* pos, int32_t* hist, cudaStream_t st) {
  const int nb = route_blocks(tokens, experts), per = (tokens + nb - 1) / nb;
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
