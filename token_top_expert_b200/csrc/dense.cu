// C ABI of the dense block and its operators (include/msb_dense.h): argument checks and the
// block's workspace and sequence of launches.
#include <cuda_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "common.cuh"
#include "dense.h"
#include "grouped.h"
#include "msb_dense.h"

namespace msb {
namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 39;  // bytes between neighbours a tensor map takes

bool aligned(const void* p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }
// Arrays of 4-byte elements (null ones pass).
bool aligned4(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (!aligned(p, 4)) return false;
  return true;
}
bool type_ok(int32_t t) { return t == MSB_BF16 || t == MSB_F32; }
int64_t size_of(int32_t t) { return t == MSB_F32 ? 4 : 2; }

// Bytes that `rows` rows of n elements, ld apart, reach over.
int64_t extent(int64_t rows, int64_t ld, int64_t n, int64_t size) {
  return rows > 0 ? ((rows - 1) * ld + n) * size : 0;
}
bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uint64_t)nb && y < x + (uint64_t)na;
}
// A row pitch in elements that the byte arithmetic of a call can take (2^31 rows, 4 bytes).
bool pitch_ok(int64_t ld) { return ld >= 0 && ld < (int64_t)1 << 28; }
// A row length (or experts of a token) that the kernels' 32-bit steps along it can take.
bool length_ok(int32_t n) { return n < 1 << 28; }

// Checks the arguments of a grouped product and completes `a`; MSB_OK with a.out_rows = 0 means
// that there is nothing to do.
int grouped_check(GroupedArgs& a, const msb_group_weights* w, int32_t out_type) {
  const int64_t es = a.i8 ? 1 : 2;
  if (!w || a.groups < 1 || a.n < 1 || a.k < 1 || a.out_rows < 0 || a.x_rows < 0 || !type_ok(out_type))
    return MSB_EINVAL;
  if (a.groups > MSB_MAX_EXPERTS || a.n > MSB_GROUPED_MAX_NK || a.k > MSB_GROUPED_MAX_NK ||
      a.out_rows > MSB_GROUPED_MAX_ROWS || (a.i8 && a.k > MSB_INT8_MAX_K)) return MSB_EUNSUPPORTED;
  if (!a.offsets && a.groups != 1) return MSB_EINVAL;
  if (!w->data || (a.i8 && !a.w_scale) || (a.out_rows > 0 && (!a.x || !a.out || (a.i8 && !a.x_scale))))
    return MSB_EINVAL;
  if (!aligned16(a.x) || !aligned16(w->data) || !pitch_ok(a.ldx) || !pitch_ok(a.ldo)) return MSB_EINVAL;
  if (!aligned4({a.rows, a.offsets, a.x_scale, a.w_scale}) || !aligned(a.out, size_of(out_type))) return MSB_EINVAL;
  if (a.x_rows > 1 && (a.ldx < 1 || a.ldx * es % 16)) return MSB_EINVAL;
  if (a.out_rows > 1 && a.ldo < a.n) return MSB_EINVAL;
  if (a.out_rows > 0 && a.x_rows < (a.rows ? 1 : a.out_rows)) return MSB_EINVAL;
  a.w = w->data;
  a.w_k = w->stride_k, a.w_n = w->stride_n, a.w_part = w->stride_part, a.w_group = w->stride_group;
  const int parts = a.swiglu ? 2 : 1;
  // a single k: n may be the contiguous one
  const bool m_major = a.w_k != 1 || (a.k == 1 && a.n > 1 && a.w_n == 1 && !a.swiglu && !a.i8);
  if (m_major && (a.w_n != 1 || a.swiglu)) return MSB_EINVAL;
  if (m_major && a.i8) return MSB_EUNSUPPORTED;
  // strides of dimensions of one element say nothing: any that a tensor map takes will do
  const int64_t unit = 16 / es;
  int64_t* const outer = m_major ? &a.w_k : &a.w_n;
  if ((m_major ? a.k : a.n) == 1) *outer = unit;
  if (parts == 1) a.w_part = unit;
  if (a.groups == 1) a.w_group = unit;
  for (int64_t s : {*outer, a.w_part, a.w_group})
    if (s <= 0 || s % unit || s * es >= kMaxStride) return MSB_EINVAL;
  const int64_t tiles = ((int64_t)a.groups + a.out_rows / 64) * (((int64_t)parts * a.n + 255) / 256);
  if (tiles >= (int64_t)1 << 30) return MSB_EUNSUPPORTED;
  const int64_t out_bytes = extent(a.out_rows, a.ldo, a.n, size_of(out_type));
  const int64_t w_bytes = ((a.groups - 1) * a.w_group + (parts - 1) * a.w_part +
                           (int64_t)(a.n - 1) * a.w_n + (int64_t)(a.k - 1) * a.w_k + 1) * es;
  if (overlaps(a.out, out_bytes, a.x, extent(a.x_rows, a.ldx, a.k, es)) ||
      overlaps(a.out, out_bytes, a.w, w_bytes))
    return MSB_EINVAL;
  a.out_f32 = out_type == MSB_F32;
  return MSB_OK;
}

int grouped(GroupedArgs a, const msb_group_weights* w, int32_t out_type, cudaStream_t st) {
  const int rc = grouped_check(a, w, out_type);
  return rc != MSB_OK || a.out_rows == 0 ? rc : launch_grouped(a, st);
}

GroupedArgs grouped_args(const void* x, int64_t ldx, int32_t x_rows, const int32_t* rows,
                         const int32_t* offsets, int32_t groups, int32_t out_rows, int32_t n,
                         int32_t k, void* out, int64_t ldo) {
  GroupedArgs a = {};
  a.x = x, a.ldx = ldx, a.x_rows = x_rows, a.rows = rows, a.offsets = offsets;
  a.groups = groups, a.out_rows = out_rows, a.n = n, a.k = k, a.out = out, a.ldo = ldo;
  return a;
}

// Workspace of a dense block; offsets in bytes.
struct DenseLayout {
  size_t logits, ids, weights, offsets, rows, pos, hist, q, q_scale, h, hq, h_scale, y, total;
  int64_t ldh;  // elements between rows of h (and bytes between rows of hq)
};

DenseLayout dense_layout(const msb_dims& m, int32_t tokens, bool int8) {
  DenseLayout L;
  size_t o = 0;
  const auto take = [&o](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) & ~(size_t)255;
    return at;
  };
  const size_t t = tokens, e = m.experts, r = t * m.top_e;
  L.ldh = (m.inter + 15) & ~15;
  L.logits = take(4 * t * e);
  L.ids = take(4 * r);
  L.weights = take(4 * r);
  L.offsets = take(4 * (e + 1));
  L.rows = take(4 * r);
  L.pos = take(4 * r);
  L.hist = take(msb_route_workspace_size(tokens, m.experts));
  L.q = take(int8 ? t * m.d : 0);
  L.q_scale = take(int8 ? 4 * t : 0);
  L.h = take(2 * r * L.ldh);
  L.hq = take(int8 ? r * L.ldh : 0);
  L.h_scale = take(int8 ? 4 * r : 0);
  L.y = take(2 * r * m.d);
  L.total = o;
  return L;
}

bool dense_dims_ok(const msb_dims* m, int* rc) {
  *rc = MSB_EINVAL;
  if (!m || m->d < 64 || m->d % 64 || m->inter < 1 || m->experts < 1 || m->top_e < 1 ||
      m->top_e > m->experts || (m->renorm != 0 && m->renorm != 1))
    return false;
  *rc = MSB_EUNSUPPORTED;
  return m->d <= MSB_MAX_D && m->inter <= MSB_MAX_INTER && m->experts <= MSB_MAX_EXPERTS &&
         m->top_e <= MSB_MAX_TOP_E;
}

// Gate/up and down weights: bf16 channel records, or 8 bits with scales.
struct DenseWeights {
  bool int8;
  const void *gate_up, *down;
  const float *gate_up_scale, *down_scale;
};

int dense_block(const void* x, int32_t tokens, const uint8_t* mask, const void* router_t,
                const DenseWeights& w, void* out, const msb_dims* dims, void* workspace,
                size_t workspace_bytes, cudaStream_t st) {
  int rc;
  if (!dense_dims_ok(dims, &rc)) return rc;
  if (tokens < 0) return MSB_EINVAL;
  if (tokens > MSB_DENSE_MAX_TOKENS) return MSB_EUNSUPPORTED;
  if (tokens == 0) return MSB_OK;
  if (!x || !router_t || !w.gate_up || !w.down || !out || !workspace) return MSB_EINVAL;
  if (w.int8 && (!w.gate_up_scale || !w.down_scale)) return MSB_EINVAL;
  if (!aligned4({w.gate_up_scale, w.down_scale}) || !aligned(out, 2)) return MSB_EINVAL;
  if (!aligned16(x) || !aligned16(router_t) || !aligned16(w.gate_up) || !aligned16(w.down) ||
      !aligned16(workspace))
    return MSB_EINVAL;
  const msb_dims& m = *dims;
  const int64_t d = m.d, act = (int64_t)tokens * d * 2;
  const DenseLayout L = dense_layout(m, tokens, w.int8);
  if (workspace_bytes < L.total) return MSB_EINVAL;
  if (overlaps(x, act, out, act) || overlaps(workspace, (int64_t)L.total, out, act) ||
      overlaps(workspace, (int64_t)L.total, x, act))
    return MSB_EINVAL;
  uint8_t* const ws = static_cast<uint8_t*>(workspace);
  const auto i32 = [ws](size_t at) { return reinterpret_cast<int32_t*>(ws + at); };
  const auto f32 = [ws](size_t at) { return reinterpret_cast<float*>(ws + at); };
  const int32_t r = tokens * m.top_e;
  const int64_t I = m.inter, ipad = L.ldh;

  msb_group_weights g = {router_t, 0, 0, d, 1};
  GroupedArgs a = grouped_args(x, d, tokens, nullptr, nullptr, 1, tokens, m.experts, m.d, ws + L.logits,
                               m.experts);
  rc = grouped(a, &g, MSB_F32, st);
  if (rc != MSB_OK) return rc;
  rc = launch_route(ws + L.logits, false, m.experts, mask, tokens, m.experts, m.top_e, m.renorm != 0,
                    i32(L.ids), f32(L.weights), i32(L.offsets), i32(L.rows), i32(L.pos), i32(L.hist), st);
  if (rc != MSB_OK) return rc;
  if (w.int8) {
    int8_t* const q = reinterpret_cast<int8_t*>(ws + L.q);
    int8_t* const hq = reinterpret_cast<int8_t*>(ws + L.hq);
    g = {w.gate_up, 2 * I * d, I * d, d, 1};
    a = grouped_args(q, d, tokens, i32(L.rows), i32(L.offsets), m.experts, r, m.inter, m.d, ws + L.h, ipad);
    a.i8 = a.swiglu = true, a.x_scale = f32(L.q_scale), a.w_scale = w.gate_up_scale;
    rc = grouped_check(a, &g, MSB_BF16);
    if (rc == MSB_OK) rc = launch_linear(a, x, false, d, q, f32(L.q_scale), st);
    if (rc != MSB_OK) return rc;
    g = {w.down, d * ipad, 0, ipad, 1};
    a = grouped_args(hq, ipad, r, nullptr, i32(L.offsets), m.experts, r, m.d, m.inter, ws + L.y, d);
    a.i8 = true, a.x_scale = f32(L.h_scale), a.w_scale = w.down_scale;
    rc = grouped_check(a, &g, MSB_BF16);
    if (rc == MSB_OK) rc = launch_linear(a, ws + L.h, false, ipad, hq, f32(L.h_scale), st);
  } else {
    g = {w.gate_up, 3 * d * I, d, 3 * d, 1};
    a = grouped_args(x, d, tokens, i32(L.rows), i32(L.offsets), m.experts, r, m.inter, m.d, ws + L.h, ipad);
    a.swiglu = true;
    rc = grouped(a, &g, MSB_BF16, st);
    if (rc != MSB_OK) return rc;
    g = {w.down, 3 * d * I, 0, 1, 3 * d};
    a = grouped_args(ws + L.h, ipad, r, nullptr, i32(L.offsets), m.experts, r, m.d, m.inter, ws + L.y, d);
    rc = grouped(a, &g, MSB_BF16, st);
  }
  if (rc != MSB_OK) return rc;
  return launch_combine(ws + L.y, false, d, r, i32(L.pos), f32(L.weights), tokens, m.top_e, m.d,
                        static_cast<uint16_t*>(out), d, st);
}

}  // namespace
}  // namespace msb

using namespace msb;

extern "C" {

int32_t msb_dense_check(void* stream) { return dense_check(static_cast<cudaStream_t>(stream)); }

size_t msb_route_workspace_size(int32_t tokens, int32_t experts) {
  if (tokens < 0 || tokens > MSB_DENSE_MAX_TOKENS || experts < 1 || experts > MSB_MAX_EXPERTS) return 0;
  return 4 * (size_t)route_blocks(tokens, experts) * experts;
}

int32_t msb_route(const void* logits, int32_t logits_type, int64_t ld, const uint8_t* mask,
                  int32_t tokens, int32_t experts, int32_t top_e, int32_t renorm, int32_t* ids,
                  float* weights, int32_t* offsets, int32_t* rows, int32_t* pos, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (tokens < 0 || experts < 1 || top_e < 1 || top_e > experts || (renorm != 0 && renorm != 1) ||
      !type_ok(logits_type) || !pitch_ok(ld) || (tokens > 1 && ld < experts))
    return MSB_EINVAL;
  if (tokens > MSB_DENSE_MAX_TOKENS || experts > MSB_MAX_EXPERTS || top_e > MSB_MAX_TOP_E)
    return MSB_EUNSUPPORTED;
  if (!offsets || !workspace || (tokens > 0 && (!logits || !ids || !weights || !rows || !pos)))
    return MSB_EINVAL;
  if (!aligned4({ids, weights, offsets, rows, pos, workspace}) || !aligned(logits, size_of(logits_type)))
    return MSB_EINVAL;
  if (workspace_bytes < msb_route_workspace_size(tokens, experts)) return MSB_EINVAL;
  return launch_route(logits, logits_type == MSB_BF16, ld, mask, tokens, experts, top_e, renorm != 0,
                      ids, weights, offsets, rows, pos, static_cast<int32_t*>(workspace),
                      static_cast<cudaStream_t>(stream));
}

int32_t msb_grouped_matmul(const void* x, int64_t ldx, int32_t x_rows, const int32_t* rows,
                           const int32_t* offsets, int32_t groups, int32_t out_rows,
                           const msb_group_weights* w, int32_t n, int32_t k, void* out,
                           int32_t out_type, int64_t ldo, void* stream) {
  const GroupedArgs a = grouped_args(x, ldx, x_rows, rows, offsets, groups, out_rows, n, k, out, ldo);
  return grouped(a, w, out_type, static_cast<cudaStream_t>(stream));
}

int32_t msb_grouped_swiglu(const void* x, int64_t ldx, int32_t x_rows, const int32_t* rows,
                           const int32_t* offsets, int32_t groups, int32_t out_rows,
                           const msb_group_weights* w, int32_t n, int32_t k, void* out,
                           int64_t ldo, void* stream) {
  GroupedArgs a = grouped_args(x, ldx, x_rows, rows, offsets, groups, out_rows, n, k, out, ldo);
  a.swiglu = true;
  return grouped(a, w, MSB_BF16, static_cast<cudaStream_t>(stream));
}

int32_t msb_int8_quantize(const void* x, int32_t x_type, int64_t ldx, int32_t rows, int32_t k,
                          int8_t* q, int64_t ldq, float* scale, void* stream) {
  if (rows < 0 || k < 1 || !type_ok(x_type) || !pitch_ok(ldx) || !pitch_ok(ldq) ||
      (rows > 1 && ldq < k) || (rows > 0 && (!x || !q || !scale)))
    return MSB_EINVAL;
  if (!length_ok(k)) return MSB_EUNSUPPORTED;
  if (!aligned(x, size_of(x_type)) || !aligned(scale, 4)) return MSB_EINVAL;
  if (overlaps(x, extent(rows, ldx, k, size_of(x_type)), q, extent(rows, ldq, k, 1)) ||
      overlaps(scale, 4 * (int64_t)rows, q, extent(rows, ldq, k, 1)) ||
      overlaps(scale, 4 * (int64_t)rows, x, extent(rows, ldx, k, size_of(x_type))))
    return MSB_EINVAL;
  if (rows == 0) return MSB_OK;
  return launch_quantize(x, x_type == MSB_F32, ldx, rows, k, q, ldq, scale,
                         static_cast<cudaStream_t>(stream));
}

int32_t msb_int8_matmul(const int8_t* q, int64_t ldq, const float* q_scale, int32_t x_rows,
                        const int32_t* rows, const int32_t* offsets, int32_t groups,
                        int32_t out_rows, const msb_group_weights* w, const float* w_scale,
                        int32_t n, int32_t k, void* out, int32_t out_type, int64_t ldo,
                        void* stream) {
  GroupedArgs a = grouped_args(q, ldq, x_rows, rows, offsets, groups, out_rows, n, k, out, ldo);
  a.i8 = true, a.x_scale = q_scale, a.w_scale = w_scale;
  return grouped(a, w, out_type, static_cast<cudaStream_t>(stream));
}

int32_t msb_int8_swiglu(const int8_t* q, int64_t ldq, const float* q_scale, int32_t x_rows,
                        const int32_t* rows, const int32_t* offsets, int32_t groups,
                        int32_t out_rows, const msb_group_weights* w, const float* w_scale,
                        int32_t n, int32_t k, void* out, int64_t ldo, void* stream) {
  GroupedArgs a = grouped_args(q, ldq, x_rows, rows, offsets, groups, out_rows, n, k, out, ldo);
  a.i8 = a.swiglu = true, a.x_scale = q_scale, a.w_scale = w_scale;
  return grouped(a, w, MSB_BF16, static_cast<cudaStream_t>(stream));
}

size_t msb_int8_linear_workspace_size(int32_t x_rows, int32_t k) {
  if (x_rows < 0 || k < 1 || k > MSB_INT8_MAX_K) return 0;
  const size_t pitch = ((size_t)k + 15) & ~(size_t)15;
  return std::max<size_t>((size_t)x_rows * (pitch + 4), 16);
}

int32_t msb_int8_linear(const void* x, int32_t x_type, int64_t ldx, int32_t x_rows,
                        const int32_t* rows, const int32_t* offsets, int32_t groups,
                        int32_t out_rows, const msb_group_weights* w, const float* w_scale,
                        int32_t n, int32_t k, int32_t swiglu, void* out, int32_t out_type,
                        int64_t ldo, void* workspace, size_t workspace_bytes, void* stream) {
  if (x_rows < 0 || k < 1 || !type_ok(x_type) || !pitch_ok(ldx) || (swiglu != 0 && swiglu != 1) ||
      (swiglu && out_type != MSB_BF16) || !workspace || !aligned16(workspace) || !aligned(x, size_of(x_type)) ||
      (x_rows > 0 && !x))
    return MSB_EINVAL;
  if (k > MSB_INT8_MAX_K) return MSB_EUNSUPPORTED;
  const int64_t need = (int64_t)msb_int8_linear_workspace_size(x_rows, k), pitch = ((int64_t)k + 15) & ~15;
  const int64_t xb = extent(x_rows, ldx, k, size_of(x_type)), ob = extent(out_rows, ldo, n, size_of(out_type));
  if (workspace_bytes < (size_t)need || overlaps(workspace, need, x, xb) || overlaps(out, ob, x, xb) ||
      overlaps(out, ob, workspace, need))
    return MSB_EINVAL;
  int8_t* const q = static_cast<int8_t*>(workspace);
  float* const scale = reinterpret_cast<float*>(q + x_rows * pitch);
  GroupedArgs a = grouped_args(q, pitch, x_rows, rows, offsets, groups, out_rows, n, k, out, ldo);
  a.i8 = true, a.swiglu = swiglu != 0, a.x_scale = scale, a.w_scale = w_scale;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int rc = grouped_check(a, w, out_type);
  if (rc != MSB_OK || out_rows == 0) return rc;
  return launch_linear(a, x, x_type == MSB_F32, ldx, q, scale, st);
}

int32_t msb_combine(const void* y, int32_t y_type, int64_t ldy, int32_t y_rows, const int32_t* pos,
                    const float* weights, int32_t tokens, int32_t top_e, int32_t d, void* out,
                    int64_t ldo, void* stream) {
  if (tokens < 0 || top_e < 1 || d < 1 || y_rows < 0 || !type_ok(y_type) || !pitch_ok(ldy) ||
      !pitch_ok(ldo) || (tokens > 1 && ldo < d))
    return MSB_EINVAL;
  if (!length_ok(d) || !length_ok(top_e)) return MSB_EUNSUPPORTED;
  if (tokens > 0 && (!pos || !weights || !out || (y_rows > 0 && !y))) return MSB_EINVAL;
  if (!aligned4({pos, weights}) || !aligned(y, size_of(y_type)) || !aligned(out, 2)) return MSB_EINVAL;
  if (overlaps(y, extent(y_rows, ldy, d, size_of(y_type)), out, extent(tokens, ldo, d, 2)))
    return MSB_EINVAL;
  if (tokens == 0) return MSB_OK;
  return launch_combine(y, y_type == MSB_F32, ldy, y_rows, pos, weights, tokens, top_e, d,
                        static_cast<uint16_t*>(out), ldo, static_cast<cudaStream_t>(stream));
}

int32_t msb_block_norm(const void* h, int32_t h_type, int64_t ldh, const void* y, int32_t y_type,
                       int64_t ldy, const void* pre_weight, const void* post_weight,
                       int32_t weight_type, int32_t post_norm, const void* gate,
                       int32_t gate_type, int64_t gate_row, int64_t gate_col, float skip_scale,
                       float residual_scale, float eps, void* h_out, int64_t ldh_out, void* x,
                       int64_t ldx, int32_t rows, int32_t d, void* stream) {
  if (rows < 0 || d < 1 || !type_ok(h_type) || (post_norm != 0 && post_norm != 1) || !(eps >= 0.f))
    return MSB_EINVAL;
  if ((y && !type_ok(y_type)) || (gate && !type_ok(gate_type)) ||
      ((pre_weight || post_weight) && !type_ok(weight_type)))
    return MSB_EINVAL;
  if (d > MSB_NORM_MAX_D) return MSB_EUNSUPPORTED;
  if (rows == 0) return MSB_OK;
  if ((!h_out && !x) || !h) return MSB_EINVAL;
  if (!y && (gate || post_norm || post_weight)) return MSB_EINVAL;
  if (!aligned(h, size_of(h_type)) || !aligned(h_out, size_of(h_type)) || !aligned(x, 2) ||
      (y && !aligned(y, size_of(y_type))) || (gate && !aligned(gate, size_of(gate_type))) ||
      !aligned(pre_weight, size_of(weight_type)) || !aligned(post_weight, size_of(weight_type)))
    return MSB_EINVAL;
  if (post_weight && !post_norm) return MSB_EINVAL;
  if (!pitch_ok(ldh) || !pitch_ok(ldy) || !pitch_ok(ldh_out) || !pitch_ok(ldx) || !pitch_ok(gate_row) ||
      !pitch_ok(gate_col) || (rows > 1 && ((h_out && ldh_out < d) || (x && ldx < d))))
    return MSB_EINVAL;
  const int64_t hb = extent(rows, ldh, d, size_of(h_type)), yb = extent(rows, ldy, d, size_of(y_type));
  const int64_t hob = extent(rows, ldh_out, d, size_of(h_type)), xb = extent(rows, ldx, d, 2);
  const int64_t gb = gate && rows > 0
                         ? ((rows - 1) * gate_row + (int64_t)(d - 1) * gate_col + 1) * size_of(gate_type)
                         : 0;
  const int64_t wb = size_of(weight_type) * d;
  if (h_out == h ? ldh_out != ldh : overlaps(h_out, hob, h, hb)) return MSB_EINVAL;
  if (overlaps(x, xb, h, hb) || overlaps(x, xb, h_out, hob)) return MSB_EINVAL;
  const void* outs[2] = {h_out, x};
  const int64_t sizes[2] = {hob, xb};
  for (int i = 0; i < 2; ++i)
    if (overlaps(outs[i], sizes[i], y, yb) || overlaps(outs[i], sizes[i], gate, gb) ||
        overlaps(outs[i], sizes[i], pre_weight, wb) || overlaps(outs[i], sizes[i], post_weight, wb))
      return MSB_EINVAL;
  NormArgs a;
  a.h = h, a.y = y, a.pre = pre_weight, a.post = post_weight, a.gate = gate, a.h_out = h_out;
  a.x = static_cast<uint16_t*>(x);
  a.ldh = ldh, a.ldy = ldy, a.ldh_out = ldh_out, a.ldx = ldx, a.gate_row = gate_row, a.gate_col = gate_col;
  a.rows = rows, a.d = d, a.h_f32 = h_type == MSB_F32, a.y_f32 = y_type == MSB_F32, a.w_f32 = weight_type == MSB_F32;
  a.gate_f32 = gate_type == MSB_F32, a.post_norm = post_norm != 0;
  a.skip = skip_scale, a.residual = residual_scale, a.eps = eps, a.inv_d = 1.f / (float)d;
  return launch_block_norm(a, static_cast<cudaStream_t>(stream));
}

size_t msb_dense_workspace_size(const msb_dims* dims, int32_t tokens, int32_t int8) {
  int rc;
  if (!dense_dims_ok(dims, &rc) || tokens < 0 || tokens > MSB_DENSE_MAX_TOKENS) return 0;
  return std::max<size_t>(dense_layout(*dims, tokens, int8 != 0).total, 256);
}

int32_t moe_dense_block(const void* x, int32_t tokens, const uint8_t* mask, const void* router_t,
                        const void* records, void* out, const msb_dims* dims, void* workspace,
                        size_t workspace_bytes, void* stream) {
  DenseWeights w = {false, records, nullptr, nullptr, nullptr};
  if (records && dims) w.down = static_cast<const uint16_t*>(records) + 2 * (int64_t)dims->d;
  return dense_block(x, tokens, mask, router_t, w, out, dims, workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

int32_t moe_dense_block_int8(const void* x, int32_t tokens, const uint8_t* mask,
                             const void* router_t, const int8_t* gate_up,
                             const float* gate_up_scale, const int8_t* down,
                             const float* down_scale, void* out, const msb_dims* dims,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const DenseWeights w = {true, gate_up, down, gate_up_scale, down_scale};
  return dense_block(x, tokens, mask, router_t, w, out, dims, workspace, workspace_bytes,
                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"
