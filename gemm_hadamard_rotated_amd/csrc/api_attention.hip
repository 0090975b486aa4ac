// C ABI of the attention-layer calls: argument validation and launches (see
// include/pq1.h).  As in api.hip, everything is validated on the host before
// the HIP runtime is touched.
#include <math.h>

#include "attn_checks.h"

using namespace pq1;

namespace {

// What the three attention calls differ in.
struct AttnCall {
  CacheForm form;
  int32_t sinks = 0;
  const pq1_kv4_cache* cache4 = nullptr;  // kFourBit
};

size_t window_workspace_bytes(CacheForm form, int64_t B, int64_t T, int32_t Hq, int32_t heads, int32_t dim,
                              int64_t max_q, int64_t max_kv, int32_t window, int32_t sinks) {
  if (check_attention_sizes(B, T, Hq, heads, dim, max_q, max_kv) != PQ1_OK) return 0;
  if (B == 0 || T == 0 || window < 0 || sinks < 0 || (sinks > 0 && window == 0)) return 0;
  return plan_window(B, T, Hq, heads, dim, max_q, max_kv, window, sinks, form == kFourBit)
      .workspace_bytes;
}

pq1_status attend(const AttnCall& c, const pq1_heads* q, const pq1_heads* out,
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
      (window > 0 && causal == 0) || c.sinks < 0 || (c.sinks > 0 && window == 0))
    return PQ1_ERR_ARG;
  if (pq1_status st = c.form == kFourBit ? check_cache4(*c.cache4) : check_cache(*cache);
      st != PQ1_OK)
    return st;
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
  const AttnPlan plan =
      c.form == kTwoByte
          ? plan_attention(B, T, Hq, cache->heads, D, max_q, max_kv, window)
          : plan_window(B, T, Hq, cache->heads, D, max_q, max_kv, window, c.sinks,
                        c.form == kFourBit);
  if (!plan.fits) return PQ1_ERR_SHAPE;
  if (plan.workspace_bytes > 0) {
    if (workspace == nullptr) return PQ1_ERR_NULL;
    if (misaligned(workspace, 256)) return PQ1_ERR_ALIGN;
    if (workspace_bytes < plan.workspace_bytes) return PQ1_ERR_ARG;
  }
  Range in[8] = {{q->data, span(*q, T, Hq, D)},
                 {page_table, static_cast<size_t>(B) * max_pages * 4},
                 {cu_q, static_cast<size_t>(B + 1) * 4},
                 {kv_len, static_cast<size_t>(B) * 4}};
  if (c.form == kFourBit)
    ranges_of(*c.cache4, in + 4);
  else
    in[4] = {cache->k, cache_bytes(*cache)}, in[5] = {cache->v, cache_bytes(*cache)};
  const size_t ob = span(*out, T, Hq, D);
  for (const Range& r : in)
    if (overlaps(out->data, ob, r.p, r.n) ||
        (plan.workspace_bytes > 0 && overlaps(workspace, plan.workspace_bytes, r.p, r.n)))
      return PQ1_ERR_ALIAS;
  if (self_overlaps(*out, T, Hq, D) ||
      (plan.workspace_bytes > 0 && overlaps(workspace, plan.workspace_bytes, out->data, ob)))
    return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  AttnWindowArgs a;
  a.q = q->data, a.q_ts = q->token_stride, a.q_hs = q->head_stride;
  a.out = out->data, a.o_ts = out->token_stride, a.o_hs = out->head_stride;
  a.k_cache = cache->k, a.v_cache = cache->v;
  a.pages = static_cast<int>(cache->pages);
  a.page_shift = log2_of(cache->page_size);
  a.Hk = cache->heads, a.G = Hq / cache->heads, a.D = D;
  a.by_G = FastDiv(static_cast<uint32_t>(a.G));
  a.table = page_table, a.max_pages = static_cast<int>(max_pages);
  a.cu_q = cu_q, a.kv_len = kv_len, a.B = B, a.T = T;
  a.scale_log2 = scale_log2;
  a.causal = causal != 0;
  a.window = window;
  a.sinks = c.sinks;
  if (c.form == kFourBit) {
    a.k_scale = static_cast<const uint8_t*>(c.cache4->k_scale);
    a.v_scale = static_cast<const uint8_t*>(c.cache4->v_scale);
  }
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (c.form == kTwoByte)
    return launched(launch_attention(plan, a, cache->dtype, out->dtype, workspace, s));
  if (c.form == kTwoByteSinks)
    return launched(launch_sinks_attention(plan, a, cache->dtype, out->dtype, workspace, s));
  return launched(launch_kv4_attention(plan, a, cache->dtype, out->dtype, workspace, s));
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
  return attend({kTwoByte}, q, out, cache, page_table, max_pages, cu_q, kv_len, B, T, Hq, max_q,
                max_kv, scale, causal, window, workspace, workspace_bytes, stream);
}

size_t pq1_paged_attention_ex_workspace_bytes(int64_t B, int64_t T, int32_t Hq, int32_t heads,
                                              int32_t dim, int64_t max_q, int64_t max_kv,
                                              int32_t window, int32_t sinks) {
  return window_workspace_bytes(kTwoByteSinks, B, T, Hq, heads, dim, max_q, max_kv, window, sinks);
}

pq1_status pq1_paged_attention_ex(const pq1_heads* q, const pq1_heads* out,
                                  const pq1_kv_cache* cache, const int32_t* page_table,
                                  int64_t max_pages, const int32_t* cu_q, const int32_t* kv_len,
                                  int64_t B, int64_t T, int32_t Hq, int64_t max_q, int64_t max_kv,
                                  float scale, int32_t causal, int32_t window, int32_t sinks,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return attend({kTwoByteSinks, sinks}, q, out, cache, page_table, max_pages, cu_q, kv_len, B, T,
                Hq, max_q, max_kv, scale, causal, window, workspace, workspace_bytes, stream);
}

size_t pq1_kv4_attention_workspace_bytes(int64_t B, int64_t T, int32_t Hq, int32_t heads,
                                         int32_t dim, int64_t max_q, int64_t max_kv,
                                         int32_t window, int32_t sinks) {
  return window_workspace_bytes(kFourBit, B, T, Hq, heads, dim, max_q, max_kv, window, sinks);
}

pq1_status pq1_kv4_attention(const pq1_heads* q, const pq1_heads* out, const pq1_kv4_cache* cache,
                             const int32_t* page_table, int64_t max_pages, const int32_t* cu_q,
                             const int32_t* kv_len, int64_t B, int64_t T, int32_t Hq,
                             int64_t max_q, int64_t max_kv, float scale, int32_t causal,
                             int32_t window, int32_t sinks, void* workspace,
                             size_t workspace_bytes, void* stream) {
  if (cache == nullptr) return PQ1_ERR_NULL;
  const pq1_kv_cache sizes{cache->k,     cache->v,     cache->dtype, cache->page_size,
                           cache->pages, cache->heads, cache->dim};
  return attend({kFourBit, sinks, cache}, q, out, &sizes, page_table, max_pages, cu_q, kv_len, B, T,
                Hq, max_q, max_kv, scale, causal, window, workspace, workspace_bytes, stream);
}

}  // extern "C"
