// C ABI of the attention-layer calls: argument validation and launches (see
// include/pq1.h).  As in api.hip, everything is validated on the host before
// the HIP runtime is touched.
#include <math.h>

#include "api_checks.h"
#include "attn_internal.h"
#include "pq1.h"

namespace {

using pq1::aligned16;
using pq1::check_device;
using pq1::launched;
using pq1::overlaps;

constexpr int kMaxHeads = 1024, kMaxDim = 1024;
constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxRows = 0x7ff00000;  // of T * Hq: row numbers plus a tile stay in 31 bits
constexpr int64_t kMaxElems = int64_t{1} << 38;   // of one call's views
constexpr int64_t kMaxStride = int64_t{1} << 31;  // elements

int64_t elem_size(int32_t dtype) { return dtype == PQ1_F32 ? 4 : 2; }

bool known_type(int32_t dtype) {
  return dtype == PQ1_F32 || dtype == PQ1_BF16 || dtype == PQ1_F16;
}

bool two_byte_type(int32_t dtype) { return dtype == PQ1_BF16 || dtype == PQ1_F16; }

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Sizes shared by every view of a call.
pq1_status check_sizes(int64_t T, int64_t heads, int64_t D) {
  if (T < 0 || heads < 1 || D < 8 || D % 8 != 0) return PQ1_ERR_SHAPE;
  if (T >= kMaxTokens || heads > 4 * kMaxHeads || D > kMaxDim) return PQ1_ERR_SHAPE;
  if (T * heads * D > kMaxElems) return PQ1_ERR_SHAPE;
  return PQ1_OK;
}

pq1_status check_view(const pq1_heads& v) {
  if (v.data == nullptr) return PQ1_ERR_NULL;
  if (v.token_stride < 0 || v.head_stride < 0 || v.token_stride > kMaxStride ||
      v.head_stride > kMaxStride)
    return PQ1_ERR_SHAPE;
  const int64_t es = elem_size(v.dtype);
  if (!aligned16(v.data) || v.token_stride * es % 16 != 0 || v.head_stride * es % 16 != 0)
    return PQ1_ERR_ALIGN;
  return PQ1_OK;
}

// Bytes from a view's first to past its last element.
size_t span(const pq1_heads& v, int64_t T, int64_t heads, int64_t D) {
  return static_cast<size_t>((T - 1) * v.token_stride + (heads - 1) * v.head_stride + D) *
         static_cast<size_t>(elem_size(v.dtype));
}

// No two elements of an output share memory: heads inside a token, or tokens
// inside a head.
bool self_overlaps(const pq1_heads& v, int64_t T, int64_t heads, int64_t D) {
  const bool heads_inside = (heads == 1 || v.head_stride >= D) &&
                            (T == 1 || v.token_stride >= (heads - 1) * v.head_stride + D);
  const bool tokens_inside = (T == 1 || v.token_stride >= D) &&
                             (heads == 1 || v.head_stride >= (T - 1) * v.token_stride + D);
  return !heads_inside && !tokens_inside;
}

pq1_status check_spec(const pq1_rope_spec& s, int64_t D) {
  if (s.interleaved != 0 && s.interleaved != 1) return PQ1_ERR_ARG;
  if (s.inverse != 0 && s.inverse != 1) return PQ1_ERR_ARG;
  if (s.pairing != PQ1_ROPE_HALVES && s.pairing != PQ1_ROPE_ADJACENT) return PQ1_ERR_ARG;
  if (s.rot < 2 || s.rot % 2 != 0 || s.rot > D || s.axes < 1 || s.axes > 4) return PQ1_ERR_SHAPE;
  int64_t sum = 0;
  for (int a = 0; a < s.axes; ++a) {
    if (s.section[a] < 0 || s.section[a] > s.rot / 2) return PQ1_ERR_SHAPE;
    if (s.interleaved && a > 0 && s.section[a] > 0 &&
        a + s.axes * (s.section[a] - 1) >= s.rot / 2)
      return PQ1_ERR_SHAPE;
    sum += s.section[a];
  }
  return sum == s.rot / 2 ? PQ1_OK : PQ1_ERR_SHAPE;
}

pq1_status check_angles(const int32_t* positions, const double* freqs) {
  if (positions == nullptr || freqs == nullptr) return PQ1_ERR_NULL;
  if (misaligned(positions, 4) || misaligned(freqs, 8)) return PQ1_ERR_ALIGN;
  return PQ1_OK;
}

void set_spec(pq1::RopeArgs* a, const pq1_rope_spec& s, const int32_t* positions,
              const double* freqs) {
  a->positions = positions;
  a->freqs = freqs;
  a->rot = s.rot;
  a->axes = s.axes;
  for (int i = 0; i < s.axes; ++i) a->section[i] = s.section[i];
  a->interleaved = s.interleaved != 0;
  a->adjacent = s.pairing == PQ1_ROPE_ADJACENT;
  a->inverse = s.inverse != 0;
}

pq1_status check_cache(const pq1_kv_cache& c) {
  if (!two_byte_type(c.dtype)) return PQ1_ERR_ARG;
  if (c.pages < 1 || c.heads < 1 || c.heads > kMaxHeads || c.dim < 8 || c.dim % 8 != 0 ||
      c.dim > kMaxDim || c.page_size < 1 || c.page_size > 65536 ||
      (c.page_size & (c.page_size - 1)) != 0)
    return PQ1_ERR_SHAPE;
  if (c.pages > 0x7fffffff || c.pages * c.page_size * c.heads > (int64_t{1} << 40))
    return PQ1_ERR_SHAPE;
  if (c.k == nullptr || c.v == nullptr) return PQ1_ERR_NULL;
  if (!aligned16(c.k) || !aligned16(c.v)) return PQ1_ERR_ALIGN;
  return PQ1_OK;
}

size_t cache_bytes(const pq1_kv_cache& c) {
  return static_cast<size_t>(c.pages) * c.page_size * c.heads * c.dim * 2;
}

int log2_of(int32_t page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

pq1_status check_attention_sizes(int64_t B, int64_t T, int64_t Hq, int64_t heads, int64_t dim,
                                 int64_t max_q, int64_t max_kv) {
  if (dim != 64 && dim != 128 && dim != 256) return PQ1_ERR_SHAPE;
  if (heads < 1 || heads > kMaxHeads || Hq < heads || Hq > kMaxHeads || Hq % heads != 0)
    return PQ1_ERR_SHAPE;
  if (B < 0 || T < 0 || max_q < 0 || max_kv < 0) return PQ1_ERR_SHAPE;
  if (T >= kMaxTokens || T * Hq > kMaxRows || B >= kMaxTokens) return PQ1_ERR_SHAPE;
  return PQ1_OK;
}

}  // namespace

extern "C" {

pq1_status pq1_rope(const pq1_heads* x, const pq1_heads* y, const int32_t* positions,
                    const double* freqs, const pq1_rope_spec* spec, int64_t T, int32_t H,
                    int32_t D, void* stream) {
  if (x == nullptr || y == nullptr || spec == nullptr) return PQ1_ERR_NULL;
  if (!known_type(x->dtype) || !known_type(y->dtype)) return PQ1_ERR_ARG;
  if (H > kMaxHeads) return PQ1_ERR_SHAPE;
  if (pq1_status st = check_sizes(T, H, D); st != PQ1_OK) return st;
  if (pq1_status st = check_spec(*spec, D); st != PQ1_OK) return st;
  if (T == 0) return PQ1_OK;
  if (pq1_status st = check_view(*x); st != PQ1_OK) return st;
  if (pq1_status st = check_view(*y); st != PQ1_OK) return st;
  if (pq1_status st = check_angles(positions, freqs); st != PQ1_OK) return st;
  const size_t yb = span(*y, T, H, D);
  const bool in_place = x->data == y->data && x->dtype == y->dtype &&
                        x->token_stride == y->token_stride && x->head_stride == y->head_stride;
  if ((!in_place && overlaps(y->data, yb, x->data, span(*x, T, H, D))) ||
      self_overlaps(*y, T, H, D) ||
      overlaps(y->data, yb, positions, static_cast<size_t>(spec->axes) * T * 4) ||
      overlaps(y->data, yb, freqs, static_cast<size_t>(spec->rot) * 4))
    return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  pq1::RopeArgs a;
  a.x = x->data, a.x_ts = x->token_stride, a.x_hs = x->head_stride;
  a.y = y->data, a.y_ts = y->token_stride, a.y_hs = y->head_stride;
  a.T = T, a.Hx = H, a.D = D;
  set_spec(&a, *spec, positions, freqs);
  return launched(pq1::launch_rope(a, x->dtype, y->dtype, static_cast<hipStream_t>(stream)));
}

pq1_status pq1_kv_append(const pq1_heads* k, const pq1_heads* v, const int64_t* slots,
                         const pq1_heads* q, const pq1_heads* q_out, int32_t Hq,
                         const int32_t* positions, const double* freqs,
                         const pq1_rope_spec* spec, const pq1_kv_cache* cache, int64_t T,
                         void* stream) {
  if (k == nullptr || v == nullptr || cache == nullptr || (q != nullptr && q_out == nullptr))
    return PQ1_ERR_NULL;
  const int32_t hq = q != nullptr ? Hq : 0;
  if ((k->dtype != PQ1_F32 && k->dtype != cache->dtype) || v->dtype != k->dtype ||
      (q != nullptr && (q->dtype != k->dtype || q_out->dtype != cache->dtype)))
    return PQ1_ERR_ARG;
  if (pq1_status st = check_cache(*cache); st != PQ1_OK) return st;
  if ((q != nullptr && hq < 1) || hq > kMaxHeads) return PQ1_ERR_SHAPE;
  const int32_t H = cache->heads, D = cache->dim;
  if (pq1_status st = check_sizes(T, hq + 2 * H, D); st != PQ1_OK) return st;
  if (spec != nullptr) {
    if (pq1_status st = check_spec(*spec, D); st != PQ1_OK) return st;
  }
  if (T == 0) return PQ1_OK;
  if (slots == nullptr) return PQ1_ERR_NULL;
  if (pq1_status st = check_view(*k); st != PQ1_OK) return st;
  if (pq1_status st = check_view(*v); st != PQ1_OK) return st;
  if (q != nullptr) {
    if (pq1_status st = check_view(*q); st != PQ1_OK) return st;
    if (pq1_status st = check_view(*q_out); st != PQ1_OK) return st;
  }
  if (misaligned(slots, 8)) return PQ1_ERR_ALIGN;
  if (spec != nullptr) {
    if (pq1_status st = check_angles(positions, freqs); st != PQ1_OK) return st;
  }
  // every output against every input and every other output
  struct Range { const void* p; size_t n; };
  Range in[6] = {{k->data, span(*k, T, H, D)}, {v->data, span(*v, T, H, D)},
                 {slots, static_cast<size_t>(T) * 8}, {}, {}, {}};
  Range out[3] = {{cache->k, cache_bytes(*cache)}, {cache->v, cache_bytes(*cache)}, {}};
  int ni = 3, no = 2;
  if (q != nullptr) {
    in[ni++] = {q->data, span(*q, T, hq, D)};
    out[no++] = {q_out->data, span(*q_out, T, hq, D)};
  }
  if (spec != nullptr) {
    in[ni++] = {positions, static_cast<size_t>(spec->axes) * T * 4};
    in[ni++] = {freqs, static_cast<size_t>(spec->rot) * 4};
  }
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (overlaps(out[o].p, out[o].n, in[i].p, in[i].n)) return PQ1_ERR_ALIAS;
    for (int i = 0; i < o; ++i)
      if (overlaps(out[o].p, out[o].n, out[i].p, out[i].n)) return PQ1_ERR_ALIAS;
  }
  if (q != nullptr && self_overlaps(*q_out, T, hq, D)) return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  pq1::RopeArgs a;
  if (q != nullptr) {
    a.x = q->data, a.x_ts = q->token_stride, a.x_hs = q->head_stride;
    a.y = q_out->data, a.y_ts = q_out->token_stride, a.y_hs = q_out->head_stride;
  }
  a.k = k->data, a.k_ts = k->token_stride, a.k_hs = k->head_stride;
  a.v = v->data, a.v_ts = v->token_stride, a.v_hs = v->head_stride;
  a.slots = slots;
  a.k_cache = cache->k, a.v_cache = cache->v;
  a.slot_count = cache->pages * cache->page_size;
  a.page_shift = log2_of(cache->page_size);
  a.Hk = H, a.Hx = hq, a.D = D, a.T = T;
  if (spec != nullptr) set_spec(&a, *spec, positions, freqs);
  return launched(pq1::launch_rope(a, k->dtype, cache->dtype, static_cast<hipStream_t>(stream)));
}

size_t pq1_paged_attention_workspace_bytes(int64_t B, int64_t T, int32_t Hq, int32_t heads,
                                           int32_t dim, int64_t max_q, int64_t max_kv) {
  if (check_attention_sizes(B, T, Hq, heads, dim, max_q, max_kv) != PQ1_OK) return 0;
  if (B == 0 || T == 0) return 0;
  return pq1::plan_attention(B, T, Hq, heads, dim, max_q, max_kv).workspace_bytes;
}

pq1_status pq1_paged_attention(const pq1_heads* q, const pq1_heads* out,
                               const pq1_kv_cache* cache, const int32_t* page_table,
                               int64_t max_pages, const int32_t* cu_q, const int32_t* kv_len,
                               int64_t B, int64_t T, int32_t Hq, int64_t max_q, int64_t max_kv,
                               float scale, int32_t causal, int32_t window, void* workspace,
                               size_t workspace_bytes, void* stream) {
  if (q == nullptr || out == nullptr || cache == nullptr) return PQ1_ERR_NULL;
  if (!two_byte_type(cache->dtype) || q->dtype != cache->dtype ||
      (out->dtype != PQ1_F32 && out->dtype != cache->dtype))
    return PQ1_ERR_ARG;
  const float scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  if (!(scale > 0.0f) || !isfinite(scale_log2) || (causal != 0 && causal != 1) || window < 0 ||
      (window > 0 && causal == 0))
    return PQ1_ERR_ARG;
  if (pq1_status st = check_cache(*cache); st != PQ1_OK) return st;
  if (pq1_status st = check_attention_sizes(B, T, Hq, cache->heads, cache->dim, max_q, max_kv);
      st != PQ1_OK)
    return st;
  if (max_pages < 0 || max_pages > 0x7fffffff) return PQ1_ERR_SHAPE;
  if (B == 0 || T == 0) return PQ1_OK;
  const int32_t D = cache->dim;
  if (pq1_status st = check_sizes(T, Hq, D); st != PQ1_OK) return st;
  if (pq1_status st = check_view(*q); st != PQ1_OK) return st;
  if (pq1_status st = check_view(*out); st != PQ1_OK) return st;
  if (cu_q == nullptr || kv_len == nullptr || (page_table == nullptr && max_pages > 0))
    return PQ1_ERR_NULL;
  if (misaligned(page_table, 4) || misaligned(cu_q, 4) || misaligned(kv_len, 4))
    return PQ1_ERR_ALIGN;
  const pq1::AttnPlan plan =
      pq1::plan_attention(B, T, Hq, cache->heads, D, max_q, max_kv, window);
  if (!plan.fits) return PQ1_ERR_SHAPE;
  if (plan.workspace_bytes > 0) {
    if (workspace == nullptr) return PQ1_ERR_NULL;
    if (misaligned(workspace, 256)) return PQ1_ERR_ALIGN;
    if (workspace_bytes < plan.workspace_bytes) return PQ1_ERR_ARG;
  }
  struct Range { const void* p; size_t n; };
  const Range in[6] = {{q->data, span(*q, T, Hq, D)}, {cache->k, cache_bytes(*cache)},
                       {cache->v, cache_bytes(*cache)},
                       {page_table, static_cast<size_t>(B) * max_pages * 4},
                       {cu_q, static_cast<size_t>(B + 1) * 4},
                       {kv_len, static_cast<size_t>(B) * 4}};
  const size_t ob = span(*out, T, Hq, D);
  for (const Range& r : in)
    if (overlaps(out->data, ob, r.p, r.n) ||
        (plan.workspace_bytes > 0 && overlaps(workspace, plan.workspace_bytes, r.p, r.n)))
      return PQ1_ERR_ALIAS;
  if (self_overlaps(*out, T, Hq, D) ||
      (plan.workspace_bytes > 0 && overlaps(workspace, plan.workspace_bytes, out->data, ob)))
    return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  pq1::AttnArgs a;
  a.q = q->data, a.q_ts = q->token_stride, a.q_hs = q->head_stride;
  a.out = out->data, a.o_ts = out->token_stride, a.o_hs = out->head_stride;
  a.k_cache = cache->k, a.v_cache = cache->v;
  a.pages = static_cast<int>(cache->pages);
  a.page_shift = log2_of(cache->page_size);
  a.Hk = cache->heads, a.G = Hq / cache->heads, a.D = D;
  a.by_G = pq1::FastDiv(static_cast<uint32_t>(a.G));
  a.table = page_table, a.max_pages = static_cast<int>(max_pages);
  a.cu_q = cu_q, a.kv_len = kv_len, a.B = B, a.T = T;
  a.scale_log2 = scale_log2;
  a.causal = causal != 0;
  a.window = window;
  return launched(pq1::launch_attention(plan, a, cache->dtype, out->dtype, workspace,
                                        static_cast<hipStream_t>(stream)));
}

}  // extern "C"
