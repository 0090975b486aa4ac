// C ABI of the calls around per-head norms and 4-bit caches: argument validation
// and launches (see include/pq1.h).  As in api.hip, everything is validated on the
// host before the HIP runtime is touched.
#include <math.h>

#include "attn_checks.h"

using namespace pq1;

namespace {

bool meets(const Range& a, const Range& b) { return overlaps(a.p, a.n, b.p, b.n); }

bool same_view(const pq1_heads& a, const pq1_heads& b) {
  return a.data == b.data && a.dtype == b.dtype && a.token_stride == b.token_stride &&
         a.head_stride == b.head_stride;
}

bool bad_eps(float eps) { return !(eps > 0.0f) || !isfinite(eps); }

pq1_status check_weight(const float* w) {
  if (w == nullptr) return PQ1_ERR_NULL;
  return aligned16(w) ? PQ1_OK : PQ1_ERR_ALIGN;
}

void add_angles(Range* in, int* n, const pq1_rope_spec* spec, const int32_t* positions,
                const double* freqs, int64_t T) {
  if (spec == nullptr) return;
  in[(*n)++] = {positions, static_cast<size_t>(spec->axes) * T * 4};
  in[(*n)++] = {freqs, static_cast<size_t>(spec->rot) * 4};
}

// What both appends check and pass on; `out` holds the cache's arrays.
pq1_status append(const pq1_heads* k, const pq1_heads* v, const int64_t* slots, const pq1_heads* q,
                  const pq1_heads* q_out, int32_t hq, const int32_t* positions,
                  const double* freqs, const pq1_rope_spec* spec, const pq1_head_norm* norm,
                  int32_t H, int32_t D, int32_t page_size, int64_t pages, int32_t dtype,
                  const Range* arrays, int count, bool cache4, NormArgs* a, int64_t T,
                  void* stream) {
  if ((k->dtype != PQ1_F32 && k->dtype != dtype) || v->dtype != k->dtype ||
      (q != nullptr && (q->dtype != k->dtype || q_out->dtype != dtype)))
    return PQ1_ERR_ARG;
  if (norm != nullptr && bad_eps(norm->eps)) return PQ1_ERR_ARG;
  if ((q != nullptr && hq < 1) || hq > kMaxHeads) return PQ1_ERR_SHAPE;
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
  const float* qw = norm != nullptr && q != nullptr ? norm->q_weight : nullptr;
  const float* kw = norm != nullptr ? norm->k_weight : nullptr;
  if ((qw != nullptr && !aligned16(qw)) || (kw != nullptr && !aligned16(kw))) return PQ1_ERR_ALIGN;
  // every output against every input and every other output
  Range in[8], out[5];
  int ni = 0, no = 0;
  in[ni++] = {k->data, span(*k, T, H, D)};
  in[ni++] = {v->data, span(*v, T, H, D)};
  in[ni++] = {slots, static_cast<size_t>(T) * 8};
  if (qw != nullptr) in[ni++] = {qw, static_cast<size_t>(D) * 4};
  if (kw != nullptr) in[ni++] = {kw, static_cast<size_t>(D) * 4};
  add_angles(in, &ni, spec, positions, freqs, T);
  while (no < count) out[no] = arrays[no], ++no;
  if (q != nullptr) {
    in[ni++] = {q->data, span(*q, T, hq, D)};
    out[no++] = {q_out->data, span(*q_out, T, hq, D)};
  }
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (meets(out[o], in[i])) return PQ1_ERR_ALIAS;
    for (int i = 0; i < o; ++i)
      if (meets(out[o], out[i])) return PQ1_ERR_ALIAS;
  }
  if (q != nullptr && self_overlaps(*q_out, T, hq, D)) return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  RopeArgs& r = a->rope;
  if (q != nullptr) {
    r.x = q->data, r.x_ts = q->token_stride, r.x_hs = q->head_stride;
    r.y = q_out->data, r.y_ts = q_out->token_stride, r.y_hs = q_out->head_stride;
  }
  r.k = k->data, r.k_ts = k->token_stride, r.k_hs = k->head_stride;
  r.v = v->data, r.v_ts = v->token_stride, r.v_hs = v->head_stride;
  r.slots = slots;
  r.slot_count = pages * page_size;
  r.page_shift = log2_of(page_size);
  r.Hk = H, r.Hx = hq, r.D = D, r.T = T;
  if (spec != nullptr) set_spec(&r, *spec, positions, freqs);
  a->x_weight = qw, a->k_weight = kw;
  a->eps = norm != nullptr ? norm->eps : 1.0;
  return launched(launch_norm_rope(*a, k->dtype, dtype, cache4, static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

pq1_status pq1_norm_rope(const pq1_heads* x, const pq1_heads* y, const float* weight, float eps,
                         const int32_t* positions, const double* freqs, const pq1_rope_spec* spec,
                         int64_t T, int32_t H, int32_t D, void* stream) {
  if (x == nullptr || y == nullptr) return PQ1_ERR_NULL;
  if (!known_type(x->dtype) || !known_type(y->dtype) || bad_eps(eps)) return PQ1_ERR_ARG;
  if (H > kMaxHeads) return PQ1_ERR_SHAPE;
  if (pq1_status st = check_sizes(T, H, D); st != PQ1_OK) return st;
  if (spec != nullptr) {
    if (pq1_status st = check_spec(*spec, D); st != PQ1_OK) return st;
  }
  if (T == 0) return PQ1_OK;
  if (pq1_status st = check_view(*x); st != PQ1_OK) return st;
  if (pq1_status st = check_view(*y); st != PQ1_OK) return st;
  if (pq1_status st = check_weight(weight); st != PQ1_OK) return st;
  if (spec != nullptr) {
    if (pq1_status st = check_angles(positions, freqs); st != PQ1_OK) return st;
  }
  const Range yr{y->data, span(*y, T, H, D)};
  Range in[4];
  int ni = 0;
  in[ni++] = {weight, static_cast<size_t>(D) * 4};
  add_angles(in, &ni, spec, positions, freqs, T);
  if (!same_view(*x, *y)) in[ni++] = {x->data, span(*x, T, H, D)};
  for (int i = 0; i < ni; ++i)
    if (meets(yr, in[i])) return PQ1_ERR_ALIAS;
  if (self_overlaps(*y, T, H, D)) return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  NormArgs a;
  RopeArgs& r = a.rope;
  r.x = x->data, r.x_ts = x->token_stride, r.x_hs = x->head_stride;
  r.y = y->data, r.y_ts = y->token_stride, r.y_hs = y->head_stride;
  r.T = T, r.Hx = H, r.D = D;
  if (spec != nullptr) set_spec(&r, *spec, positions, freqs);
  a.x_weight = weight, a.eps = eps;
  return launched(
      launch_norm_rope(a, x->dtype, y->dtype, false, static_cast<hipStream_t>(stream)));
}

size_t pq1_norm_rope_grad_workspace_bytes(int64_t T, int32_t D) {
  if (check_sizes(T, 1, D) != PQ1_OK) return 0;
  return static_cast<size_t>(norm_grad_parts(T)) * D * 4;
}

pq1_status pq1_norm_rope_grad(const pq1_heads* grad, const pq1_heads* x, const pq1_heads* dx,
                              const float* weight, float* dweight, float eps,
                              const int32_t* positions, const double* freqs,
                              const pq1_rope_spec* spec, int64_t T, int32_t H, int32_t D,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (grad == nullptr || x == nullptr || dx == nullptr) return PQ1_ERR_NULL;
  if (!known_type(grad->dtype) || !known_type(x->dtype) || dx->dtype != x->dtype || bad_eps(eps))
    return PQ1_ERR_ARG;
  if (H > kMaxHeads) return PQ1_ERR_SHAPE;
  if (pq1_status st = check_sizes(T, H, D); st != PQ1_OK) return st;
  if (spec != nullptr) {
    if (pq1_status st = check_spec(*spec, D); st != PQ1_OK) return st;
  }
  if (T == 0 && dweight == nullptr) return PQ1_OK;
  if (misaligned(dweight, 4)) return PQ1_ERR_ALIGN;
  const size_t need = dweight != nullptr ? pq1_norm_rope_grad_workspace_bytes(T, D) : 0;
  NormArgs a;
  if (T > 0) {
    if (pq1_status st = check_view(*grad); st != PQ1_OK) return st;
    if (pq1_status st = check_view(*x); st != PQ1_OK) return st;
    if (pq1_status st = check_view(*dx); st != PQ1_OK) return st;
    if (pq1_status st = check_weight(weight); st != PQ1_OK) return st;
    if (spec != nullptr) {
      if (pq1_status st = check_angles(positions, freqs); st != PQ1_OK) return st;
    }
    if (need > 0) {
      if (workspace == nullptr) return PQ1_ERR_NULL;
      if (misaligned(workspace, 256)) return PQ1_ERR_ALIGN;
      if (workspace_bytes < need) return PQ1_ERR_ARG;
    }
    // outputs against inputs and one another; dx may be either of its inputs
    const Range out[3] = {{dx->data, span(*dx, T, H, D)},
                          {dweight, static_cast<size_t>(D) * 4},
                          {workspace, need}};
    Range in[5];
    int ni = 0;
    in[ni++] = {grad->data, span(*grad, T, H, D)};
    in[ni++] = {x->data, span(*x, T, H, D)};
    in[ni++] = {weight, static_cast<size_t>(D) * 4};
    add_angles(in, &ni, spec, positions, freqs, T);
    const int outs = dweight == nullptr ? 1 : need > 0 ? 3 : 2;
    for (int o = 0; o < outs; ++o) {
      for (int i = 0; i < ni; ++i) {
        const bool itself = o == 0 && i < 2 && same_view(*dx, i == 0 ? *grad : *x);
        if (!itself && meets(out[o], in[i])) return PQ1_ERR_ALIAS;
      }
      for (int i = 0; i < o; ++i)
        if (meets(out[o], out[i])) return PQ1_ERR_ALIAS;
    }
    if (self_overlaps(*dx, T, H, D)) return PQ1_ERR_ALIAS;
    RopeArgs& r = a.rope;
    r.x = x->data, r.x_ts = x->token_stride, r.x_hs = x->head_stride;
    r.y = dx->data, r.y_ts = dx->token_stride, r.y_hs = dx->head_stride;
    a.grad = grad->data, a.g_ts = grad->token_stride, a.g_hs = grad->head_stride;
    if (spec != nullptr) set_spec(&r, *spec, positions, freqs);
  }
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  a.rope.T = T, a.rope.Hx = H, a.rope.D = D;
  a.x_weight = weight, a.eps = eps;
  return launched(launch_norm_rope_grad(a, grad->dtype, x->dtype, dweight,
                                        need > 0 ? static_cast<float*>(workspace) : nullptr,
                                        static_cast<hipStream_t>(stream)));
}

pq1_status pq1_kv_append_ex(const pq1_heads* k, const pq1_heads* v, const int64_t* slots,
                            const pq1_heads* q, const pq1_heads* q_out, int32_t Hq,
                            const int32_t* positions, const double* freqs,
                            const pq1_rope_spec* spec, const pq1_head_norm* norm,
                            const pq1_kv_cache* cache, int64_t T, void* stream) {
  if (norm == nullptr)
    return pq1_kv_append(k, v, slots, q, q_out, Hq, positions, freqs, spec, cache, T, stream);
  if (k == nullptr || v == nullptr || cache == nullptr || (q != nullptr && q_out == nullptr))
    return PQ1_ERR_NULL;
  if (pq1_status st = check_cache(*cache); st != PQ1_OK) return st;
  const Range arrays[2] = {{cache->k, cache_bytes(*cache)}, {cache->v, cache_bytes(*cache)}};
  NormArgs a;
  a.rope.k_cache = cache->k, a.rope.v_cache = cache->v;
  return append(k, v, slots, q, q_out, q != nullptr ? Hq : 0, positions, freqs, spec, norm,
                cache->heads, cache->dim, cache->page_size, cache->pages, cache->dtype, arrays, 2,
                false, &a, T, stream);
}

pq1_status pq1_kv4_append(const pq1_heads* k, const pq1_heads* v, const int64_t* slots,
                          const pq1_heads* q, const pq1_heads* q_out, int32_t Hq,
                          const int32_t* positions, const double* freqs,
                          const pq1_rope_spec* spec, const pq1_head_norm* norm,
                          const pq1_kv4_cache* cache, int64_t T, void* stream) {
  if (k == nullptr || v == nullptr || cache == nullptr || (q != nullptr && q_out == nullptr))
    return PQ1_ERR_NULL;
  if (pq1_status st = check_cache4(*cache); st != PQ1_OK) return st;
  Range arrays[4];
  ranges_of(*cache, arrays);
  NormArgs a;
  a.rope.k_cache = cache->k, a.rope.v_cache = cache->v;
  a.k_scale = static_cast<uint8_t*>(cache->k_scale);
  a.v_scale = static_cast<uint8_t*>(cache->v_scale);
  return append(k, v, slots, q, q_out, q != nullptr ? Hq : 0, positions, freqs, spec, norm,
                cache->heads, cache->dim, cache->page_size, cache->pages, cache->dtype, arrays, 4,
                true, &a, T, stream);
}

pq1_status pq1_kv4_read(const pq1_kv4_cache* cache, const int64_t* slots, const pq1_heads* k_out,
                        const pq1_heads* v_out, int64_t T, void* stream) {
  if (cache == nullptr || (k_out == nullptr && v_out == nullptr)) return PQ1_ERR_NULL;
  const pq1_heads* outs[2] = {k_out, v_out};
  for (const pq1_heads* o : outs)
    if (o != nullptr && (!known_type(o->dtype) || o->dtype != (k_out ? k_out : v_out)->dtype))
      return PQ1_ERR_ARG;
  if (pq1_status st = check_cache4(*cache); st != PQ1_OK) return st;
  const int32_t H = cache->heads, D = cache->dim;
  if (pq1_status st = check_sizes(T, 2 * H, D); st != PQ1_OK) return st;
  if (T == 0) return PQ1_OK;
  if (slots == nullptr) return PQ1_ERR_NULL;
  if (misaligned(slots, 8)) return PQ1_ERR_ALIGN;
  Range in[5], out[2];
  Range arrays[4];
  ranges_of(*cache, arrays);
  for (int i = 0; i < 4; ++i) in[i] = arrays[i];
  in[4] = {slots, static_cast<size_t>(T) * 8};
  int no = 0;
  for (const pq1_heads* o : outs) {
    if (o == nullptr) continue;
    if (pq1_status st = check_view(*o); st != PQ1_OK) return st;
    if (self_overlaps(*o, T, H, D)) return PQ1_ERR_ALIAS;
    out[no++] = {o->data, span(*o, T, H, D)};
  }
  for (int o = 0; o < no; ++o)
    for (const Range& r : in)
      if (meets(out[o], r)) return PQ1_ERR_ALIAS;
  if (no == 2 && meets(out[0], out[1])) return PQ1_ERR_ALIAS;
  if (pq1_status st = check_device(); st != PQ1_OK) return st;
  Read4Args a;
  a.k = static_cast<const uint8_t*>(cache->k);
  a.k_scale = static_cast<const uint8_t*>(cache->k_scale);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.v_scale = static_cast<const uint8_t*>(cache->v_scale);
  a.slots = slots;
  a.slot_count = cache->pages * cache->page_size;
  a.page_shift = log2_of(cache->page_size);
  if (k_out != nullptr)
    a.k_out = k_out->data, a.k_ts = k_out->token_stride, a.k_hs = k_out->head_stride;
  if (v_out != nullptr)
    a.v_out = v_out->data, a.v_ts = v_out->token_stride, a.v_hs = v_out->head_stride;
  a.T = T, a.H = H, a.D = D;
  return launched(launch_kv4_read(a, (k_out ? k_out : v_out)->dtype,
                                  static_cast<hipStream_t>(stream)));
}

}  // extern "C"
