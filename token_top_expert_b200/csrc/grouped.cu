// Products of ragged groups of rows with their group's weight, bf16 or 8-bit integers:
//
//   out[p][n] = sum_k x[row(p)][k] * w[e][n][k]        offsets[e] <= p < offsets[e + 1]
//
// or, gated, out[p][j] = silu(g) * u with g, u the products with w[e][0][j] and w[e][1][j].
//
// The weights are the 256-row operand of the matrix unit and the rows of a group its N side,
// so that a group of any size fills the unit's rows: N runs over 32, 64, .. 256 in one kernel
// (a group of c rows is cut into ceil(c / 256) even pieces).  One row streams its experts'
// weights; a prompt runs at the matrix unit's rate.
//
// One CTA pair per tile (persistent, static order), 14 to 18 warps a CTA:
//   warps 0-3  epilogue: tensor memory -> registers -> scale / SwiGLU -> global
//   warp 4     issues the matrix instructions (even CTA) into one of two accumulators
//   warp 5     weights: one, two or eight tensor-map boxes per stage of 128 bytes of k
//   warps 6-   rows of x.  In order: boxes of 128, 64, 32 and 16 rows (warp 6).  Gathered: one or
//              two warps to a stage copy 16 bytes a thread, asynchronously, into the same
//              swizzle, wait for them and hand the stage over.  (A gathering tensor-map load,
//              four rows an instruction, took the copy unit 60 to 80 cycles for 512 bytes: gate
//              and up of 4096 tokens 497 us, where the rest of the kernel took 254.)  Row pointers and
//              swizzled places are kept per tile, rows behind the tile's last are left out, and only the
//              last stage and rows outside x have a size of their own: the kernel's instructions for
//              4096 tokens' gate and up went from 86 to 55 million (in order: 26), long runs at the
//              board's power limit from 262 to 250 us, 8-bit ones from 135 to 120.
//
// What bounds it: weights from memory while the groups are small (64 tokens' gate and up, hidden
// 2048 x 768 channels x 128 experts top-8, cold weights: 104 us for the 0.67 GB of the 106 experts in
// use, 6.4 TB/s).  4096 tokens' gate and up read 0.8 GB of weights and take 205 us in short runs; the
// same number of rows in equal groups of 256 180 us; in 8 groups, whose weights stay in L2, 139 (1.48
// PFLOP/s; with one weight 136).  So it is the weights' way from memory while the matrix unit works,
// then the uneven groups (1218 tiles of 171 rows on average, not 768 of 256; the busiest pair has
// 6 % more than the mean).  Gathering costs 3 us of it, the records' strides and SwiGLU nothing.  bf16
// 8192^3 takes 575 us (1.91 PFLOP/s) to 860 (1.28), by the clock that the board's power limit leaves;
// long runs of all of these are slower by up to a fifth.
#include <cuda.h>

#include <algorithm>
#include <cstddef>
#include <mutex>

#include "dense.h"
#include "grouped.cuh"
#include "grouped.h"
#include "tc.cuh"

namespace msb {

__device__ uint32_t g_dense_err;  // sticky error word, read by msb_dense_check

namespace {

constexpr int kTileM = 256;       // weight rows per CTA pair
constexpr int kStageBytes = 128;  // bytes of k per stage (one swizzle row)
constexpr int kABytes = 128 * kStageBytes;  // one CTA's weight rows of a stage

// bf16 products: the matrix unit cuts off each addition to its accumulator, an instruction's 16 k at
// a time, by less than 2^-23 of the sum so far and always towards zero: for values of one sign by up
// to 7.5e-9 of the sum per k (measured: 7e-9), for mixed signs far less (relative L2 1.5e-6 at k =
// 1536, 9e-6 at 8192).  Float outputs have an accumulator take kExactStages stages (256 k, 2e-7) at
// a time, bf16 ones kLongStages (32768 k: 2.4e-4 at most, a sixteenth of a bf16 rounding), and the
// epilogue sums these parts rounded to nearest, which 64-row tiles have registers for (bf16, 2048 rows
// by 1024 x 65536: 278 us, in one accumulator 198).  8-bit sums are exact.
constexpr int kExactStages = 4, kLongStages = 512;

// Stages summed in one accumulator; 0: all.  LONG: there are more than kLongStages.
template <bool I8, bool F32, bool LONG>
constexpr int kChunk = I8 ? 0 : F32 ? kExactStages : LONG ? kLongStages : 0;

// Bytes between the staged rows of an epilogue warp's 32 bf16 channels: 64 and 16 more, so that
// eight rows' 16-byte pieces fall into different banks.
constexpr int kOutPitch = 80;

// BN: most rows of x per tile.  256 for products bound by the matrix unit; 64 where the groups
// are small and the weights' bytes are all: the stages shrink, and more of them keep more
// weight bytes in flight (one SM's 96 KB against 160 KB).
template <int BN>
struct Cfg {
  static constexpr int kStages = BN == 256 ? 6 : BN == 128 ? 8 : 10;
  static constexpr int kBBytes = BN / 2 * kStageBytes;  // one CTA's rows of x of a stage
  static constexpr int kStage = kABytes + kBBytes;
  static constexpr int kSplit = BN == 256 ? 2 : 1;  // gathering warps of a stage
  static constexpr int kThreads = (6 + kSplit * kStages) * 32;
  static constexpr int kLaneRows = BN / 2 / kSplit / 4;  // rows of a gathering thread
  static constexpr int kBoxes = BN == 256 ? 4 : BN == 128 ? 3 : 2;       // x in order: boxes of 16 << i rows

  struct Shared {
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem, dead;
    int32_t first[kGroupsMax + 1];  // first piece of each group
    int32_t begin[kGroupsMax + 1];  // first row of each group
    alignas(16) float scale[4][BN];  // 8-bit: scales of the tile's rows of x, per epilogue warp
    alignas(16) uint8_t out[4][32 * kOutPitch];  // 32 rows of an epilogue warp's channels
  };
  static_assert(offsetof(Shared, scale) % 16 == 0 && offsetof(Shared, out) % 16 == 0 && kOutPitch % 16 == 0,
                "vector accesses");
  static constexpr size_t kSmemBytes = (size_t)kStages * kStage + 1024 + sizeof(Shared);
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

// Tensor maps of x in order: boxes of 16 << i rows.
struct RowMaps {
  CUtensorMap map[4];
};

// A bounded wait.  When it runs out, or another role of this CTA has given up, the caller
// stops waiting for good and leaves through the common exit.  A poll may sleep up to kNapNs (it
// ends with the phase all the same): with the default, far shorter one the waiting warps' polls
// took issue slots (256 x 4096 by 4096 x 4096 17.0 us, 15.0 with it; 64 tokens' gate and up 105 either way).
constexpr uint32_t kNapNs = 5000;
__device__ bool wait_slow(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1; i < kSpinLimit; ++i) {
    if (mbar_try_wait_sleep(bar, parity, kNapNs)) return true;
    if (*(volatile uint32_t*)dead) return false;
    if ((i & 15u) == 0 && globaltimer_ns() - t0 > kWaitLimitNs) break;
  }
  *(volatile uint32_t*)dead = 1;
  atomicOr(&g_dense_err, kErrTimeout);
  return false;
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  return mbar_try_wait_sleep(bar, parity, kNapNs) || wait_slow(bar, parity, dead);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* dead) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, dead));
}

struct Tile {
  int group, m, row0, rows;  // rows of x: [row0, row0 + rows), rows <= BN
};

// Rows and pieces before each group, by one warp: every lane takes a run of groups, scans over
// the lanes join them.
template <int BN>
__device__ void plan_groups(const KArgs& a, typename Cfg<BN>::Shared& s, int lane) {
  group_begins(a, s.begin, lane);
  const int per = (a.groups + 32) >> 5;  // of groups + 1 offsets
  const int e0 = lane * per, e1 = min(e0 + per, a.groups + 1);
  auto pieces = [&](int e) {
    return e < a.groups ? (s.begin[e + 1] - s.begin[e] + BN - 1) / BN : 0;
  };
  int sum = 0;
  for (int e = e0; e < e1; ++e) sum += pieces(e);
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += v;
  }
  before -= sum;
  for (int e = e0; e < e1; ++e) {
    s.first[e] = before;
    before += pieces(e);
  }
}

// The tile of index t (t < first[groups] * mtiles).  Inside a group eight weight tiles go
// over all its pieces before the next eight, so that the pairs at work share both operands.
template <class Shared>
__device__ __forceinline__ Tile tile_at(const KArgs& a, const Shared& s, int t) {
  int lo = 0, hi = a.groups;  // first[lo] * mtiles <= t < first[hi] * mtiles
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.first[mid] * a.mtiles <= t) lo = mid; else hi = mid;
  }
  const int pieces = s.first[lo + 1] - s.first[lo];
  const int r = t - s.first[lo] * a.mtiles;
  const int band = r / (8 * pieces);
  const int wide = min(8, a.mtiles - 8 * band);
  const int q = r - band * 8 * pieces;
  const int piece = q / wide;
  const int b = s.begin[lo], cnt = s.begin[lo + 1] - b;
  const int each = ((cnt + pieces - 1) / pieces + 31) & ~31;
  Tile tile;
  tile.group = lo;
  tile.m = 8 * band + q - piece * wide;
  tile.row0 = b + piece * each;
  tile.rows = min(each, cnt - piece * each);
  return tile;
}

// This warp has read all it wants of an accumulator.
template <class Shared>
__device__ __forceinline__ void release_acc(Shared& s, int buf, int lane) {
  tc_fence_before();
  __syncwarp();
  if (lane == 0) arrive_pair(map_to(smem_addr(&s.acc_empty[buf]), cluster_rank() & ~1u));
}

// Parts of a tile from the cluster's other pairs (SPLIT > 1: every pair takes a range of k).
// Each of their epilogue threads leaves its accumulator words in the stages of the first pair's
// CTA of the same weight rows, which has finished with them: word j of part p (1 ..) of warp w.
// All threads of the cluster meet twice, before the parts are written and before they are
// read; `met` counts.
__device__ __forceinline__ uint32_t part_offset(int part, int warp, int j, int lane) {
  return ((((part - 1) * 4 + warp) * 64 + j) * 32 + lane) * 4;
}
__device__ __forceinline__ void meet(int& met) {
  __syncwarp();
  cluster_sync();
  ++met;
}
template <bool I8>
__device__ __forceinline__ uint32_t add_part(uint32_t v, const uint8_t* stages, int part, int warp, int j, int lane) {
  const uint32_t w = *reinterpret_cast<const uint32_t*>(stages + part_offset(part, warp, j, lane));
  return I8 ? v + w : __float_as_uint(__uint_as_float(v) + __uint_as_float(w));
}

// One epilogue warp's 32 channels to float: a lane is a channel.  8-bit sums are exact; bf16
// products come in parts of kExactStages stages, which are summed here.
template <int BN, bool I8, int SPLIT>
__device__ __forceinline__ bool store_f32(const KArgs& a, typename Cfg<BN>::Shared& s, uint8_t* stages, const Tile& tile,
                                          uint32_t tmem, int& buf, uint32_t& phase, int nk, uint32_t rank, int part,
                                          int warp, int lane, int& met) {
  const int ch = tile.m * kTileM + (int)rank * 128 + warp * 32 + lane;
  float* const out = static_cast<float*>(a.out) + (int64_t)tile.row0 * a.ldo + ch;
  const uint32_t acc = tmem + ((uint32_t)(warp * 32) << 16);
  if constexpr (I8) {
    const float ws = ch < a.n ? a.w_scale[(int64_t)tile.group * a.n + ch] : 0.f;
    if (!wait_warp(&s.acc_full[buf], phase, &s.dead)) return false;
    tc_fence_after();
    if (SPLIT > 1) {
      meet(met);
      if (part == 0) meet(met);
    }
    for (int c0 = 0; c0 < tile.rows; c0 += 32) {
      uint32_t v[32];
      tmem_ld32(acc + buf * BN + c0, v);
      tmem_ld_wait();
      if (c0 + 32 >= tile.rows) release_acc(s, buf, lane);
      if (SPLIT > 1 && part > 0) {
        const uint32_t to = map_to(smem_addr(stages), rank);
#pragma unroll
        for (int c = 0; c < 32; ++c) store_cluster(to + part_offset(part, warp, c0 + c, lane), v[c]);
        continue;
      }
      if (SPLIT > 1)
        for (int q = 1; q < SPLIT; ++q)
#pragma unroll
          for (int c = 0; c < 32; ++c) v[c] = add_part<true>(v[c], stages, q, warp, c0 + c, lane);
      if (ch < a.n)
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c0 + c < tile.rows) out[(int64_t)(c0 + c) * a.ldo] = value<true>(v[c], s.scale[warp][c0 + c], ws);
    }
    if (++buf == 2) buf = 0, phase ^= 1;
  } else {
    static_assert(BN == 64, "the sums of a tile are held in registers");
    float sum[BN];
#pragma unroll
    for (int c = 0; c < BN; ++c) sum[c] = 0.f;
    for (int i = 0; i < nk; i += kExactStages) {
      if (!wait_warp(&s.acc_full[buf], phase, &s.dead)) return false;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32)
        if (c0 < tile.rows) {
          uint32_t v[32];
          tmem_ld32(acc + buf * BN + c0, v);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 32; ++c) sum[c0 + c] += __uint_as_float(v[c]);
        }
      release_acc(s, buf, lane);
      if (++buf == 2) buf = 0, phase ^= 1;
    }
    if (SPLIT > 1) {
      meet(met);
      if (part > 0) {
        const uint32_t to = map_to(smem_addr(stages), rank);
#pragma unroll
        for (int c = 0; c < BN; ++c) store_cluster(to + part_offset(part, warp, c, lane), __float_as_uint(sum[c]));
        return true;
      }
      meet(met);
      for (int q = 1; q < SPLIT; ++q)
#pragma unroll
        for (int c = 0; c < BN; ++c)
          sum[c] = __uint_as_float(add_part<false>(__float_as_uint(sum[c]), stages, q, warp, c, lane));
    }
    if (ch < a.n)
#pragma unroll
      for (int c = 0; c < BN; ++c)
        if (c < tile.rows) out[(int64_t)c * a.ldo] = sum[c];
  }
  return true;
}

// One epilogue warp's 32 accumulator rows to bf16: 32 channels, or 16 gated ones.  Channels lie
// along the lanes of tensor memory and contiguously in the output, so 32 columns (rows of out)
// at a time are turned through shared memory (transposing 8x8 stores) and leave as 16-byte
// pieces; element by element where out is not aligned for that or the channels end.
template <int BN, bool I8, bool GATED, bool LONG, int SPLIT>
__device__ __forceinline__ bool store_bf16(const KArgs& a, typename Cfg<BN>::Shared& s, uint8_t* stages,
                                           const Tile& tile, uint32_t tmem, int& buf, uint32_t& phase, int nk,
                                           uint32_t rank, int part, int warp, int lane, int& met) {
  constexpr int kCh = GATED ? 16 : 32;  // channels of this warp
  const int ch0 = GATED ? tile.m * 128 + (int)rank * 64 + warp * 16 : tile.m * kTileM + (int)rank * 128 + warp * 32;
  // scales of the accumulator rows lane / 4 + 8 i
  float ws[4] = {1.f, 1.f, 1.f, 1.f};
  if constexpr (I8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ch = ch0 + (GATED ? (i >> 1) * 8 : i * 8) + (lane >> 2);
      if (ch < a.n)
        ws[i] = GATED ? a.w_scale[((int64_t)tile.group * 2 + (i & 1)) * a.n + ch]
                      : a.w_scale[(int64_t)tile.group * a.n + ch];
    }
  }
  // 32 columns of the accumulator in use
  const auto columns = [&](int c0, uint32_t (&v)[2][16]) {
    const uint32_t acc = tmem + buf * BN + ((uint32_t)(warp * 32) << 16);
    tmem_ld16(acc + c0, v[0]);
    tmem_ld16(acc + (16u << 16) + c0, v[1]);
    tmem_ld_wait();
  };
  const auto next_acc = [&] {
    if (++buf == 2) buf = 0, phase ^= 1;
  };
  float sum[LONG ? BN / 32 : 1][2][16];
  if constexpr (LONG) {
    static_assert(BN == 64, "the sums of a tile are held in registers");
#pragma unroll
    for (int j = 0; j < BN; ++j) sum[j >> 5][j >> 4 & 1][j & 15] = 0.f;
    for (int i = 0; i < nk; i += kLongStages) {
      if (!wait_warp(&s.acc_full[buf], phase, &s.dead)) return false;
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32)
        if (c0 < tile.rows) {
          uint32_t v[2][16];
          columns(c0, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) sum[c0 >> 5][j >> 4][j & 15] += __uint_as_float(v[j >> 4][j & 15]);
        }
      release_acc(s, buf, lane);
      next_acc();
    }
  } else {
    if (!wait_warp(&s.acc_full[buf], phase, &s.dead)) return false;
    tc_fence_after();
  }
  if (SPLIT > 1) {
    meet(met);
    if (part == 0) meet(met);
  }
  uint8_t* const stage = s.out[warp];
  const int lim = a.n - ch0;  // channels of this warp that exist (may be <= 0)
  // 32 rows of out
  const auto store_rows = [&](int c0, uint32_t (&v)[2][16]) {
    if (SPLIT > 1 && part > 0) {
      const uint32_t to = map_to(smem_addr(stages), rank);
#pragma unroll
      for (int j = 0; j < 32; ++j) store_cluster(to + part_offset(part, warp, c0 + j, lane), v[j >> 4][j & 15]);
      return;
    }
    if (SPLIT > 1)
      for (int q = 1; q < SPLIT; ++q)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          v[j >> 4][j & 15] = add_part<I8>(v[j >> 4][j & 15], stages, q, warp, c0 + j, lane);
    __syncwarp();  // the last 32 rows have been read
    float2 rs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      rs[j] = I8 ? *reinterpret_cast<const float2*>(&s.scale[warp][c0 + 8 * j + 2 * (lane & 3)])
                 : make_float2(1.f, 1.f);
    // matrix j: columns 8 j .. 8 j + 7 of eight channels; its rows (columns) in shared memory
    const uint32_t dst = smem_addr(stage) + lane * kOutPitch;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t m[2][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo0 = value<I8>(v[i][4 * j], rs[j].x, ws[2 * i]);
        const float lo1 = value<I8>(v[i][4 * j + 1], rs[j].y, ws[2 * i]);
        const float hi0 = value<I8>(v[i][4 * j + 2], rs[j].x, ws[2 * i + 1]);
        const float hi1 = value<I8>(v[i][4 * j + 3], rs[j].y, ws[2 * i + 1]);
        if constexpr (GATED) {
          m[0][j] = pack_bf16(gated(lo0, hi0), gated(lo1, hi1));
        } else {
          m[0][j] = pack_bf16(lo0, lo1);
          m[1][j] = pack_bf16(hi0, hi1);
        }
      }
      if constexpr (GATED) {
        stsm_x4_trans(dst + i * 16, m[0][0], m[0][1], m[0][2], m[0][3]);
      } else {
        stsm_x4_trans(dst + i * 32, m[0][0], m[0][1], m[0][2], m[0][3]);
        stsm_x4_trans(dst + i * 32 + 16, m[1][0], m[1][1], m[1][2], m[1][3]);
      }
    }
    __syncwarp();
    uint16_t* const out = static_cast<uint16_t*>(a.out) + (int64_t)(tile.row0 + c0) * a.ldo + ch0;
    const int rows = min(32, tile.rows - c0);
    if (a.wide && lim >= kCh) {
      constexpr int kPieces = kCh / 8;  // 16-byte pieces of a row
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        const int at = q * 32 + lane, row = at / kPieces, piece = at % kPieces;
        if (row < rows)
          *reinterpret_cast<uint4*>(out + (int64_t)row * a.ldo + piece * 8) =
              *reinterpret_cast<const uint4*>(stage + row * kOutPitch + piece * 16);
      }
    } else {
      for (int at = lane; at < rows * kCh; at += 32) {
        const int row = at / kCh, c = at % kCh;
        if (c < lim) out[(int64_t)row * a.ldo + c] = *reinterpret_cast<const uint16_t*>(stage + row * kOutPitch + 2 * c);
      }
    }
  };
  if constexpr (LONG) {
#pragma unroll
    for (int c0 = 0; c0 < BN; c0 += 32)
      if (c0 < tile.rows) {
        uint32_t v[2][16];
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j >> 4][j & 15] = __float_as_uint(sum[c0 >> 5][j >> 4][j & 15]);
        store_rows(c0, v);
      }
  } else {
    for (int c0 = 0; c0 < tile.rows; c0 += 32) {
      uint32_t v[2][16];
      columns(c0, v);
      if (c0 + 32 >= tile.rows) release_acc(s, buf, lane);
      store_rows(c0, v);
    }
    next_acc();
  }
  return true;
}

// I8: 8-bit integers (else bf16).  MMAJOR: the weight's n runs contiguously (bf16 only).
// GATED: rows of the weight tile alternate in eights, gate and up.  F32: float output.  LONG: bf16
// sums of more than kLongStages stages (BN = 64).  SPLIT: pairs that share a tile's k (with one tile
// per cluster and BN = 64).
template <int BN, bool I8, bool MMAJOR, bool GATED, bool F32, bool LONG, int SPLIT>
__global__ void __cluster_dims__(2 * SPLIT, 1, 1) __launch_bounds__(Cfg<BN>::kThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ RowMaps xmaps,
                   const KArgs a) {
  using C = Cfg<BN>;
  constexpr int kStages = C::kStages, kSplit = C::kSplit;
  extern __shared__ uint8_t raw[];
  // stages on 1024-byte boundaries (the swizzle's period); same offset in both CTAs
  uint8_t* const stages = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  auto& s = *reinterpret_cast<typename C::Shared*>(stages + (size_t)kStages * C::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t leader = cluster_rank() & ~1u, rank = cluster_rank() & 1;  // of the pair, in the pair
  const int part = cluster_rank() >> 1;
  const int pair = blockIdx.x / (2 * SPLIT), pairs = gridDim.x / (2 * SPLIT);  // of clusters, if they are larger
  const int whole = (a.kbytes + kStageBytes - 1) / kStageBytes;
  const int kb = SPLIT > 1 ? whole * part / SPLIT : 0;  // first stage of k here, and how many
  const int nk = (SPLIT > 1 ? whole * (part + 1) / SPLIT : whole) - kb;
  int met = 0;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (warp == 0) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    plan_groups<BN>(a, s, lane);
  } else if (warp == 4) {
    tmem_alloc_pair(&s.tmem, 2 * BN);
  } else if (warp == 5 && lane == 0) {
    prefetch_map(&wmap);
    for (int i = 0; i < C::kBoxes && !a.rows; ++i) prefetch_map(&xmaps.map[i]);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], a.rows ? 1 + 2 * kSplit : 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.acc_full[i], 1);
      mbar_init(&s.acc_empty[i], 8);
    }
    s.dead = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = s.tmem;
  const int tiles = s.first[a.groups] * a.mtiles;
  bool ok = true;

  if (warp == 5) {
    // ------------------------------------------------ weights
    if (elect_one()) {
      const uint32_t base = smem_addr(stages), bars = map_to(smem_addr(&s.full[0]), leader);
      int st = 0;
      uint32_t phase = 0;
      for (int t = pair; ok && t < tiles; t += pairs) {
        const Tile tile = tile_at(a, s, t);
        const uint32_t bytes = 2 * kABytes + (a.rows ? 0 : ((tile.rows + 31) & ~31) * kStageBytes);
        int k0 = kb * (I8 ? kStageBytes : kStageBytes / 2);
        for (int i = 0; i < nk; ++i, k0 += I8 ? kStageBytes : kStageBytes / 2) {
          if (!(ok = wait_one(&s.empty[st], phase ^ 1, &s.dead))) break;
          const uint32_t bar = bars + st * 8, dst = base + st * C::kStage;
          if (rank == 0) mbar_arrive_expect_tx(&s.full[st], bytes);
          if constexpr (GATED) {
            // eight channels' gate rows, then their up rows: 16 rows of the tile
#pragma unroll
            for (int q = 0; q < 8; ++q)
              tma_load_4d(dst + q * 16 * kStageBytes, &wmap, k0, tile.m * 128 + (int)rank * 64 + q * 8, 0, tile.group,
                          bar);
          } else if constexpr (MMAJOR) {
#pragma unroll
            for (int q = 0; q < 2; ++q)
              tma_load_3d(dst + q * (kABytes / 2), &wmap, tile.m * kTileM + (int)rank * 128 + q * 64, k0, tile.group,
                          bar);
          } else {
            tma_load_3d(dst, &wmap, k0, tile.m * kTileM + (int)rank * 128, tile.group, bar);
          }
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
    }
  } else if (warp == 4 && rank == 0) {
    // ------------------------------------------------ matrix instructions of the pair
    if (elect_one()) {
      int st = 0, buf = 0;
      uint32_t phase = 0, acc_phase = 0;
      const int chunk = kChunk<I8, F32, LONG> ? kChunk<I8, F32, LONG> : nk;
      const uint32_t pa = smem_addr(stages);
      const uint64_t da0 = MMAJOR ? smem_desc(pa, kABytes / 2, 1024) : smem_desc(pa, 16, 1024);
      const uint64_t db0 = smem_desc(pa + kABytes, 16, 1024);
      for (int t = pair; ok && t < tiles; t += pairs) {
        const Tile tile = tile_at(a, s, t);
        const uint32_t idesc = instr_desc(I8 ? 2 : 1, MMAJOR, kTileM, (tile.rows + 31) & ~31);
        for (int i0 = 0; ok && i0 < nk; i0 += chunk) {
          if (!(ok = wait_one(&s.acc_empty[buf], acc_phase ^ 1, &s.dead))) break;
          tc_fence_after();
          const int i1 = min(i0 + chunk, nk);
          for (int i = i0; i < i1; ++i) {
            if (!(ok = wait_one(&s.full[st], phase, &s.dead))) break;
            tc_fence_after();
            const uint64_t da = da0 + st * (C::kStage >> 4), db = db0 + st * (C::kStage >> 4);
            // steps of 32 bytes of k; m-major: of 16 rows
#pragma unroll
            for (int q = 0; q < 4; ++q)
              mma_pair<I8>(tmem + buf * BN, da + q * (MMAJOR ? 2048 >> 4 : 32 >> 4), db + q * (32 >> 4), idesc,
                           i > i0 || q > 0);
            mma_commit_pair(&s.empty[st], 3u << leader);
            if (++st == kStages) st = 0, phase ^= 1;
          }
          if (!ok) break;
          mma_commit_pair(&s.acc_full[buf], 3u << leader);
          if (++buf == 2) buf = 0, acc_phase ^= 1;
        }
      }
    }
  } else if (warp >= 6 && a.rows) {
    // ------------------------------------------------ rows of x, gathered
    const int st = (warp - 6) / kSplit, part = (warp - 6) % kSplit;
    const int chunk = lane & 7, r0 = lane >> 3;  // 16-byte piece of 128, row of each four
    const uint32_t bar = map_to(smem_addr(&s.full[st]), leader);
    const uint32_t base = smem_addr(stages) + st * C::kStage + kABytes + r0 * kStageBytes;
    uint32_t phase = 0;
    int at = 0;  // stages before this tile, modulo the ring
    int next[C::kLaneRows], nmine = 0, nrows = 0;  // row indices are fetched a tile ahead
    const auto fetch = [&](int t) {
      if (t >= tiles) return;
      const Tile tile = tile_at(a, s, t);
      nmine = ((tile.rows + 31) & ~31) / (2 * kSplit);  // this warp's: 8, 16, .. C::kLaneRows * 4
      const int p0 = ((int)rank * kSplit + part) * nmine + r0;
      // and this lane's, four apart; what lies behind the tile's last row is not stored, nor copied
      nrows = min(nmine, tile.rows - p0);
#pragma unroll
      for (int q = 0; q < C::kLaneRows; ++q) next[q] = q * 4 < nrows ? a.rows[tile.row0 + p0 + q * 4] : 0;
    };
    fetch(pair);
    for (int t = pair; ok && t < tiles; t += pairs) {
      const int mine = nmine, rows = nrows;
      const uint8_t* src[C::kLaneRows];
      uint32_t there = 0;  // rows that exist
#pragma unroll
      for (int q = 0; q < C::kLaneRows; ++q) {
        const bool use = (uint32_t)next[q] < (uint32_t)a.x_rows;
        there |= (uint32_t)use << q;
        src[q] = a.x + (use ? (int64_t)next[q] * a.pitch + chunk * 16 : 0);
      }
      const bool all = __all_sync(0xffffffffu, there == ~0u >> (32 - C::kLaneRows));
      const uint32_t dst = base + part * mine * kStageBytes;
      fetch(t + pairs);
      int i = st - at;
      if (i < 0) i += kStages;
      at = (at + nk) % kStages;
      for (; i < nk; i += kStages) {
        if (!(ok = wait_warp(&s.empty[st], phase ^ 1, &s.dead))) break;
        phase ^= 1;
        const uint32_t k0 = (kb + i) * kStageBytes;
        const uint32_t even = dst + ((chunk ^ r0) << 4), odd = dst + ((chunk ^ (4 + r0)) << 4);
        if (all && (int)k0 + kStageBytes <= a.kbytes) {
#pragma unroll
          for (int q = 0; q < C::kLaneRows; ++q)
            if (q * 4 < rows) cp_async16((q & 1 ? odd : even) + q * 4 * kStageBytes, src[q] + k0);
        } else {  // zeros for rows outside x and behind the end of k
          const int left = a.kbytes - (int)k0 - chunk * 16;
          const uint32_t valid = left < 0 ? 0 : left > 16 ? 16 : left;
#pragma unroll
          for (int q = 0; q < C::kLaneRows; ++q)
            if (q * 4 < rows) {
              const uint32_t size = there >> q & 1 ? valid : 0;
              cp_async16((q & 1 ? odd : even) + q * 4 * kStageBytes, src[q] + (size ? k0 : 0), size);
            }
        }
        cp_async_wait_all();
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) arrive_pair(bar);
      }
    }
  } else if (warp == 6 && !a.rows) {
    // ------------------------------------------------ rows of x, as they lie
    if (elect_one()) {
      const uint32_t base = smem_addr(stages) + kABytes, bars = map_to(smem_addr(&s.full[0]), leader);
      int st = 0;
      uint32_t phase = 0;
      for (int t = pair; ok && t < tiles; t += pairs) {
        const Tile tile = tile_at(a, s, t);
        const int half = ((tile.rows + 31) & ~31) >> 1;
        const int row0 = tile.row0 + (int)rank * half;
        int k0 = kb * (I8 ? kStageBytes : kStageBytes / 2);
        for (int i = 0; i < nk; ++i, k0 += I8 ? kStageBytes : kStageBytes / 2) {
          if (!(ok = wait_one(&s.empty[st], phase ^ 1, &s.dead))) break;
          // rows behind the group's last belong to the next group: their columns of the
          // accumulator are not stored
#pragma unroll
          for (int b = C::kBoxes - 1; b >= 0; --b)
            if (half & (16 << b)) {
              const int done = half & ~((32 << b) - 1);
              tma_load_2d(base + st * C::kStage + done * kStageBytes, &xmaps.map[b], k0, row0 + done, bars + st * 8);
            }
          if (++st == kStages) st = 0, phase ^= 1;
        }
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------ epilogue
    int buf = 0;
    uint32_t acc_phase = 0;
    for (int t = pair; ok && t < tiles; t += pairs) {
      const Tile tile = tile_at(a, s, t);
      if constexpr (I8) {
        __syncwarp();  // the last tile's scales have been read
        for (int c = lane; c < tile.rows; c += 32) {
          const int row = a.rows ? a.rows[tile.row0 + c] : tile.row0 + c;
          s.scale[warp][c] = (uint32_t)row < (uint32_t)a.x_rows ? a.x_scale[row] : 0.f;
        }
        __syncwarp();
      }
      // the accumulator is handed back once it has been read, before the last stores
      if constexpr (F32) {
        ok = store_f32<BN, I8, SPLIT>(a, s, stages, tile, tmem, buf, acc_phase, nk, rank, part, warp, lane, met);
      } else {
        ok = store_bf16<BN, I8, GATED, LONG, SPLIT>(a, s, stages, tile, tmem, buf, acc_phase, nk, rank, part, warp, lane,
                                                    met);
      }
    }
  }
  __syncwarp();
  if (SPLIT > 1)
    while (met < 2) meet(met);
  // A role that gave up may leave copies or instructions in flight: they end within
  // microseconds; let them, so that none reaches an exited CTA or freed tensor memory.
  if (*(volatile uint32_t*)&s.dead) {
    const uint64_t t0 = globaltimer_ns();
    for (int i = 0; i < 4096 && globaltimer_ns() - t0 < 200000; ++i) __nanosleep(1000);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 4) {
    tc_fence_after();
    tmem_free_pair(tmem, 2 * BN);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = []() -> EncodeFn {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// Tensor map of the weights: {k, n, group} boxes of 128 bytes x 128 rows, {n, k, group} boxes
// of 64 n x 64 k where n runs contiguously, {k, n, part, group} boxes of 128 bytes x 8
// channels x 2 parts for the gated form.  Coordinates outside are filled with zeros.
bool weight_map(const GroupedArgs& a, CUtensorMap* map) {
  const EncodeFn encode = encode_fn();
  if (!encode) return false;
  const int es = a.i8 ? 1 : 2;
  const bool mmajor = a.w_k != 1;
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4], ones[4] = {1, 1, 1, 1};
  int rank = 3;
  if (a.swiglu) {
    rank = 4;
    dims[0] = a.k, dims[1] = a.n, dims[2] = 2, dims[3] = a.groups;
    strides[0] = a.w_n * es, strides[1] = a.w_part * es, strides[2] = a.w_group * es;
    box[0] = kStageBytes / es, box[1] = 8, box[2] = 2, box[3] = 1;
  } else if (mmajor) {
    dims[0] = a.n, dims[1] = a.k, dims[2] = a.groups;
    strides[0] = a.w_k * es, strides[1] = a.w_group * es;
    box[0] = 64, box[1] = 64, box[2] = 1;
  } else {
    dims[0] = a.k, dims[1] = a.n, dims[2] = a.groups;
    strides[0] = a.w_n * es, strides[1] = a.w_group * es;
    box[0] = kStageBytes / es, box[1] = 128, box[2] = 1;
  }
  return encode(map, a.i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                const_cast<void*>(a.w), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor maps of x: {k, row}, boxes of 128 bytes (none when the rows are gathered).
bool row_maps(const GroupedArgs& a, RowMaps* maps) {
  const int es = a.i8 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)a.k, (cuuint64_t)std::max(a.x_rows, 1)};
  const cuuint64_t strides[1] = {(cuuint64_t)(a.x_rows > 1 ? a.ldx * es : (a.k * es + 15) / 16 * 16)};
  for (int i = 0; i < 4 && !a.rows; ++i) {
    const cuuint32_t box[2] = {(cuuint32_t)(kStageBytes / es), 16u << i}, ones[2] = {1, 1};
    if (encode_fn()(&maps->map[i], a.i8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                    const_cast<void*>(a.x), dims, strides, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                    CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return false;
  }
  return true;
}

template <int BN, bool I8, bool MMAJOR, bool GATED, bool F32, int SPLIT = 1, bool LONG = false>
int launch(const CUtensorMap& map, const RowMaps& xmaps, const KArgs& k, cudaStream_t st) {
  const auto kernel = grouped_kernel<BN, I8, MMAJOR, GATED, F32, LONG, SPLIT>;
  static std::mutex mu;
  static int known[64] = {};  // SMs of each device whose kernel has its shared memory
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MSB_ECUDA;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!known[dev]) {  // a failure is reported, not kept: the next call tries again
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<BN>::kSmemBytes) !=
              cudaSuccess ||
          cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return MSB_ECUDA;
      }
      known[dev] = sms;
    }
    sms = known[dev];
  }
  // at most one pair (or cluster) per tile: pieces <= groups + rows / BN, and every piece has a row
  const int64_t most = ((int64_t)k.groups + k.out_rows / BN) * k.mtiles;
  const int64_t mine = (int64_t)k.out_rows * k.mtiles;
  const int64_t clusters = SPLIT > 1 ? (int64_t)(k.out_rows + BN - 1) / BN * k.mtiles
                                     : std::min<int64_t>(sms / 2, std::min(most, mine));
  return launch_early(kernel, 2 * SPLIT * clusters, Cfg<BN>::kThreads, Cfg<BN>::kSmemBytes, st, map, xmaps, k);
}

int stages_of(const KArgs& k) { return (k.kbytes + kStageBytes - 1) / kStageBytes; }

// bf16 outputs whose accumulators would take more than kLongStages stages, with `split` parts of k.
bool long_sums(const GroupedArgs& a, const KArgs& k, int split) {
  return !a.i8 && !a.out_f32 && (stages_of(k) + split - 1) / split > kLongStages;
}

template <int BN, int SPLIT = 1>
int launch_tile(const GroupedArgs& a, const CUtensorMap& map, const RowMaps& xmaps, const KArgs& k, cudaStream_t st) {
  if (a.i8) {
    if (a.swiglu) return launch<BN, true, false, true, false, SPLIT>(map, xmaps, k, st);
    return a.out_f32 ? launch<BN, true, false, false, true, SPLIT>(map, xmaps, k, st)
                     : launch<BN, true, false, false, false, SPLIT>(map, xmaps, k, st);
  }
  if constexpr (BN == 64) {
    if (long_sums(a, k, SPLIT))
      return a.swiglu     ? launch<BN, false, false, true, false, SPLIT, true>(map, xmaps, k, st)
             : a.w_k != 1 ? launch<BN, false, true, false, false, SPLIT, true>(map, xmaps, k, st)
                          : launch<BN, false, false, false, false, SPLIT, true>(map, xmaps, k, st);
    if (a.out_f32)
      return a.w_k != 1 ? launch<BN, false, true, false, true, SPLIT>(map, xmaps, k, st)
                        : launch<BN, false, false, false, true, SPLIT>(map, xmaps, k, st);
  }
  if (a.swiglu) return launch<BN, false, false, true, false, SPLIT>(map, xmaps, k, st);
  return a.w_k != 1 ? launch<BN, false, true, false, false, SPLIT>(map, xmaps, k, st)
                    : launch<BN, false, false, false, false, SPLIT>(map, xmaps, k, st);
}

constexpr int kPairs = 74;  // CTA pairs that the device holds

// Clusters of 2 * SPLIT CTAs that the current device holds at once (of any 64-row kernel: they
// take the same shared memory and threads).
template <int SPLIT>
int resident_clusters() {
  static std::mutex mu;
  static int known[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  std::lock_guard<std::mutex> lock(mu);
  if (known[dev] == 0) {
    const auto kernel = grouped_kernel<64, false, false, false, false, false, SPLIT>;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2 * SPLIT, attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * SPLIT * kPairs);
    cfg.blockDim = dim3(Cfg<64>::kThreads);
    cfg.dynamicSmemBytes = Cfg<64>::kSmemBytes;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg<64>::kSmemBytes) !=
            cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;  // not kept: the next call tries again
    }
    known[dev] = n > 0 ? n : -1;
  }
  return known[dev];
}

// Pairs that share the k of each tile of 64 rows: one group whose tiles are so few that the device
// holds all their clusters at once, and enough stages that the join (two meetings of the cluster and
// the parts' way through shared memory) pays.  Without and with it, 64 rows, cold bf16 weights n x k:
// four pairs, 512 x 2304 8.9 and 8.6 us, 2048 x 2560 (40 stages) 9.7 and 9.9, 2048 x 3584 11.9 and
// 10.6, 512 x 4096 12.4 and 9.6, 4096 x 4096 14.1 and 13.2, but 2048 x 2048 8.6 and 9.5, 1024 x 1024
// 6.5 and 8.2; two pairs, 5120 x 4096 (64 stages) 14.7 and 14.1, 8192 x 4096 17.6 and 17.5, 5120 x
// 8192 23.9 and 21.4, but 8192 x 3584 15.5 and 16.7; float outputs, 128 x 2048 (32 stages) 10.4 and
// 10.2; 8 bits, 1024 x 5120 (40 stages) 9.5 and 9.4, 1024 x 4096 8.5 and 9.1.
int split_k(const GroupedArgs& a, const KArgs& k) {
  const int64_t tiles = ((int64_t)a.out_rows + 63) / 64 * k.mtiles;
  const int stages = stages_of(k);
  if (a.groups != 1 || stages < (a.out_f32 && !a.i8 ? 32 : 40)) return 1;
  if (tiles <= resident_clusters<4>()) return 4;
  return stages >= 64 && tiles <= resident_clusters<2>() ? 2 : 1;
}

// Rows of the tile that serves a product.
int tile_rows(const GroupedArgs& a, const KArgs& k) {
  if ((a.out_f32 && !a.i8) || long_sums(a, k, 1)) return 64;  // sums in registers
  const int64_t rows = a.out_rows, groups = std::min<int64_t>(a.groups, rows);
  // Few tiles: the smallest that one round of the pairs holds (one 4096 x 4096 bf16 weight, 64-,
  // 128- and 256-row tiles: 256 rows 15.2, 17.5, 26.8 us; 512 rows 23.4, 18.1, 28.3; 1024 rows
  // 40.4, 29.9, 30.2).
  for (int bn = 64; bn <= 256; bn *= 2)
    if (k.mtiles * std::max(groups, (rows + bn - 1) / bn) <= kPairs) return bn;
  // Many: by the rows of a group, on average (gate and up of hidden 2048 x 768 channels x 128
  // experts, cold weights; bf16, 16 rows 124, 126, 132 us; 64 rows 140, 133, 139; 128 rows 188, 157,
  // 151; 8 bits, 16 rows 69, 68, 72; 64 rows 78, 73, 76; 128 rows 107, 89, 85).
  return rows <= 32 * groups ? 64 : rows <= 64 * groups ? 128 : 256;
}

}  // namespace

int launch_grouped(const GroupedArgs& a, cudaStream_t st) {
  const KArgs k = kernel_args(a);
  if (few_rows(a)) return launch_few(a, k, st);
  CUtensorMap map;
  RowMaps xmaps = {};
  if (!weight_map(a, &map) || !row_maps(a, &xmaps)) return MSB_ECUDA;
  switch (split_k(a, k)) {
    case 4: return launch_tile<64, 4>(a, map, xmaps, k, st);
    case 2: return launch_tile<64, 2>(a, map, xmaps, k, st);
  }
  switch (tile_rows(a, k)) {
    case 64: return launch_tile<64>(a, map, xmaps, k, st);
    case 128: return launch_tile<128>(a, map, xmaps, k, st);
    default: return launch_tile<256>(a, map, xmaps, k, st);
  }
}

int dense_check(cudaStream_t st) {
  uint32_t err = 0;
  const uint32_t zero = 0;
  if (cudaMemcpyFromSymbolAsync(&err, g_dense_err, 4, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return MSB_ECUDA;
  if (err != 0 && (cudaMemcpyToSymbolAsync(g_dense_err, &zero, 4, 0, cudaMemcpyHostToDevice, st) !=
                       cudaSuccess ||
                   cudaStreamSynchronize(st) != cudaSuccess))
    return MSB_ECUDA;
  return err & kErrTimeout ? MSB_ETIMEOUT : MSB_OK;
}

}  // namespace msb
