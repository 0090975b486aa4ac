// Host-side checks shared by the attention-layer entry points
// (api_attention.hip, api_kv4.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "api_checks.h"
#include "attn_internal.h"
#include "pq1.h"

namespace pq1 {

constexpr int kMaxHeads = 1024, kMaxDim = 1024;
constexpr int64_t kMaxTokens = int64_t{1} << 30;
constexpr int64_t kMaxRows = 0x7ff00000;  // of T * Hq: row numbers plus a tile stay in 31 bits
constexpr int64_t kMaxElems = int64_t{1} << 38;   // of one call's views
constexpr int64_t kMaxStride = int64_t{1} << 31;  // elements

inline int64_t elem_size(int32_t dtype) { return dtype == PQ1_F32 ? 4 : 2; }

inline bool known_type(int32_t dtype) {
  return dtype == PQ1_F32 || dtype == PQ1_BF16 || dtype == PQ1_F16;
}

inline bool two_byte_type(int32_t dtype) { return dtype == PQ1_BF16 || dtype == PQ1_F16; }

inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Sizes shared by every view of a call.
inline pq1_status check_sizes(int64_t T, int64_t heads, int64_t D) {
  if (T < 0 || heads < 1 || D < 8 || D % 8 != 0) return PQ1_ERR_SHAPE;
  if (T >= kMaxTokens || heads > 4 * kMaxHeads || D > kMaxDim) return PQ1_ERR_SHAPE;
  if (T * heads * D > kMaxElems) return PQ1_ERR_SHAPE;
  return PQ1_OK;
}

inline pq1_status check_view(const pq1_heads& v) {
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
inline size_t span(const pq1_heads& v, int64_t T, int64_t heads, int64_t D) {
  return static_cast<size_t>((T - 1) * v.token_stride + (heads - 1) * v.head_stride + D) *
         static_cast<size_t>(elem_size(v.dtype));
}

// No two elements of an output share memory: heads inside a token, or tokens
// inside a head.
inline bool self_overlaps(const pq1_heads& v, int64_t T, int64_t heads, int64_t D) {
  const bool heads_inside = (heads == 1 || v.head_stride >= D) &&
                            (T == 1 || v.token_stride >= (heads - 1) * v.head_stride + D);
  const bool tokens_inside = (T == 1 || v.token_stride >= D) &&
                             (heads == 1 || v.head_stride >= (T - 1) * v.token_stride + D);
  return !heads_inside && !tokens_inside;
}

inline pq1_status check_spec(const pq1_rope_spec& s, int64_t D) {
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

inline pq1_status check_angles(const int32_t* positions, const double* freqs) {
  if (positions == nullptr || freqs == nullptr) return PQ1_ERR_NULL;
  if (misaligned(positions, 4) || misaligned(freqs, 8)) return PQ1_ERR_ALIGN;
  return PQ1_OK;
}

inline void set_spec(RopeArgs* a, const pq1_rope_spec& s, const int32_t* positions,
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

inline pq1_status check_cache(const pq1_kv_cache& c) {
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

inline size_t cache_bytes(const pq1_kv_cache& c) {
  return static_cast<size_t>(c.pages) * c.page_size * c.heads * c.dim * 2;
}

inline int log2_of(int32_t page_size) {
  int s = 0;
  while ((1 << s) < page_size) ++s;
  return s;
}

inline pq1_status check_attention_sizes(int64_t B, int64_t T, int64_t Hq, int64_t heads, int64_t dim,
                                 int64_t max_q, int64_t max_kv) {
  if (dim != 64 && dim != 128 && dim != 256) return PQ1_ERR_SHAPE;
  if (heads < 1 || heads > kMaxHeads || Hq < heads || Hq > kMaxHeads || Hq % heads != 0)
    return PQ1_ERR_SHAPE;
  if (B < 0 || T < 0 || max_q < 0 || max_kv < 0) return PQ1_ERR_SHAPE;
  if (T >= kMaxTokens || T * Hq > kMaxRows || B >= kMaxTokens) return PQ1_ERR_SHAPE;
  return PQ1_OK;
}

// Memory of an argument.
struct Range {
  const void* p;
  size_t n;
};

inline pq1_status check_cache4(const pq1_kv4_cache& c) {
  const pq1_kv_cache sizes{c.k, c.v, c.dtype, c.page_size, c.pages, c.heads, c.dim};
  if (pq1_status st = check_cache(sizes); st != PQ1_OK) return st;
  if (c.dim % 32 != 0) return PQ1_ERR_SHAPE;
  if (c.k_scale == nullptr || c.v_scale == nullptr) return PQ1_ERR_NULL;
  if (!aligned16(c.k_scale) || !aligned16(c.v_scale)) return PQ1_ERR_ALIGN;
  return PQ1_OK;
}

// The four arrays of a cache.
inline void ranges_of(const pq1_kv4_cache& c, Range* r) {
  const size_t rows = static_cast<size_t>(c.pages) * c.page_size * c.heads;
  r[0] = {c.k, rows * (c.dim / 2)};
  r[1] = {c.v, rows * (c.dim / 2)};
  r[2] = {c.k_scale, rows * (c.dim / 32)};
  r[3] = {c.v_scale, rows * (c.dim / 32)};
}

}  // namespace pq1
