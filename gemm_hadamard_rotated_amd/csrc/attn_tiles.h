// Device pieces shared by the attention kernels (paged_attention.hip: few rows;
// paged_attention_tiles.hip: tiles of many rows): which keys a row sees, how a
// row tile's keys are split, matrix-core products, probabilities as two-byte
// numbers, and the handling of infinities and NaN.
#pragma once

#include "attn_device.h"
#include "attn_internal.h"

namespace pq1 {

constexpr float kNegInf = -__builtin_inff();

// What a workgroup needs to know of its sequence.
struct Seq {
  int64_t q0;  // first row of q
  int n;       // new tokens
  int kv;      // keys
};

// The table and the lengths are read through the scalar cache.
using Const32 = const __attribute__((address_space(4))) int32_t;
__device__ __forceinline__ int32_t scalar_load(const int32_t* p, int64_t i) {
  return reinterpret_cast<Const32*>(reinterpret_cast<uintptr_t>(p))[i];
}

__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int64_t b) {
  int64_t q0 = scalar_load(a.cu_q, b), q1 = scalar_load(a.cu_q, b + 1);
  const int kv = scalar_load(a.kv_len, b);
  q0 = q0 < 0 ? 0 : q0 > a.T ? a.T : q0;
  q1 = q1 < q0 ? q0 : q1 > a.T ? a.T : q1;
  return {q0, static_cast<int>(q1 - q0), kv < 0 ? 0 : kv > kMaxKeys ? kMaxKeys : kv};
}

// Keys [lo, hi) that row i < n sees.
__device__ __forceinline__ void visible(const AttnArgs& a, const Seq& s, int i, int* lo, int* hi) {
  *lo = 0;
  *hi = s.kv;
  if (a.causal) {
    const int end = s.kv - (s.n - 1 - i);
    *hi = end < 0 ? 0 : end;
    if (a.window > 0 && *hi > a.window) *lo = *hi - a.window;
  }
}

// Rows of one (sequence, cache head) are numbered r = i * G + g over its new
// tokens i and the G query heads of the cache head, so that all of them share
// the keys and values a workgroup reads.  A tile of such rows sees keys
// [start, hi); they are cut into parts of `chunk` keys.
struct Parts {
  int start;  // rounded down to a multiple of 32
  int lo, hi;  // keys that some row sees
  int lo_max, hi_min;  // keys in [lo_max, hi_min) are seen by every row
  int chunk;
  __device__ __forceinline__ int count() const {
    const uint32_t keys = hi > start ? hi - start : 0;
    return static_cast<int>((keys + chunk - 1) / static_cast<uint32_t>(chunk));
  }
};

__device__ __forceinline__ Parts split_keys(const AttnArgs& a, const Seq& s, int r0, int rows,
                                            int chunk, int nsplit) {
  const int last = s.n * a.G - 1;
  const int i0 = a.by_G.div(r0), i1 = a.by_G.div(r0 + rows - 1 < last ? r0 + rows - 1 : last);
  Parts p;
  int lo0, hi0, lo1, hi1;
  visible(a, s, i0, &lo0, &hi0);
  visible(a, s, i1, &lo1, &hi1);
  p.start = lo0 & ~31;
  p.lo = lo0;
  p.hi = hi1;
  p.lo_max = lo1;
  p.hi_min = hi0;
  p.chunk = chunk;
  // A cache longer than the caller said stretches the parts, to whole key tiles
  // of either kernel as the plan's are: a part's last tile has no keys of the next.
  const int64_t room = static_cast<int64_t>(chunk) * nsplit;
  if (static_cast<int64_t>(p.hi) - p.start > room) {
    constexpr uint32_t step = kKeys * kWaves;
    const uint32_t need = (static_cast<uint32_t>(p.hi - p.start) + nsplit - 1) / nsplit;
    p.chunk = static_cast<int>((need + step - 1) / step * step);
  }
  return p;
}

// A tile of keys that not every row sees whole, or with a key on no page.
__device__ __forceinline__ bool is_edge(const Parts& pt, int j0, int keys, bool gone) {
  return j0 < pt.lo_max || j0 + keys > pt.hi_min || gone;
}

template <typename T>
using Vec8 = __attribute__((ext_vector_type(8))) T;
using F4 = __attribute__((ext_vector_type(4))) float;
using U4 = __attribute__((ext_vector_type(4))) uint32_t;
using U2 = __attribute__((ext_vector_type(2))) uint32_t;

__device__ __forceinline__ F4 mfma16(U4 a, U4 b, F4 c, bf16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(Vec8<bf16>, a),
                                                 __builtin_bit_cast(Vec8<bf16>, b), c, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma16(U4 a, U4 b, F4 c, f16) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(Vec8<f16>, a),
                                                __builtin_bit_cast(Vec8<f16>, b), c, 0, 0, 0);
}

// Maximum and sum over the lanes that share lane % 16.
__device__ __forceinline__ float max_groups(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_groups(float x) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Probabilities are carried times 2^kUp, which the division by their sum
// takes out again.  The running maximum may lag behind by kLag (fewer
// rescalings of the sums).
//   f16: up, so that it holds those down to 2^-22 of the largest in full;
//   2^(kUp + kLag) is within f16.
//   bf16: down, so that 2^(-kUp - kLag) values of any finite size, and any
//   number of values below 2^111, sum up within fp32.
template <typename T>
constexpr float kUp = __is_same(T, bf16) ? -20.0f : 8.0f;
constexpr float kLag = 6.0f;

// Scores (times scale_log2) past 2^24 are further apart than 1 from one float to
// the next, so a maximum that is rounded to one may be far from itself: its
// probability would be out of a two-byte number's range.  There the maximum is
// rounded down, and a score's distance from it, which one fused operation gives
// exactly, is held to the lag; that is within the rounding of such scores.
__device__ __forceinline__ bool is_far(float m) {
  const float a = __builtin_fabsf(m);
  return a >= 0x1p24f && a < __builtin_inff();
}
// raw * scale_log2, rounded down where it is far
__device__ __forceinline__ float scaled_max(float raw, float scale_log2) {
  const float top = raw * scale_log2;
  if (!is_far(top) || fmaf(raw, scale_log2, -top) >= 0.0f) return top;
  return __int_as_float(__float_as_int(top) + (top > 0.0f ? -1 : 1));
}
// a score whose distance from zero is that of sc from m
__device__ __forceinline__ float near_score(float sc, float scale_log2, float m) {
  const float d = fmaf(sc, scale_log2, -m);
  return (d > kLag ? kLag : d) * __builtin_amdgcn_rcpf(scale_log2);
}

// A probability as NP two-byte numbers whose sum it is: one where the result
// is rounded to that type anyway; for an fp32 result three bf16 or two f16,
// which hold all 24 or 22 bits.  An infinite value times each of them has to
// be an infinity, not NaN, so none of them is zero or negative.
//   bf16: each number is cut off, and what is left is kept above zero (by less
//   than 2^-100 of the largest probability).
//   f16: the first is cut from slightly less than the probability, so that
//   something is left for the second, which is rounded to nearest: together
//   they are the probability to 22 bits or, where it is small, to the nearest
//   2^-24 (2^-32 of the largest).  Below 1.75 of those the first is zero.
template <typename T, typename TO>
constexpr int kParts = sizeof(TO) == 2 ? 1 : __is_same(T, bf16) ? 3 : 2;

// The sum of the probabilities is that of the parts, except where these hold
// all of a probability.
template <typename T, int NP>
constexpr bool kSumParts = NP == 1 || __is_same(T, f16);

template <typename T, int NP>
__device__ __forceinline__ void split_probs(const float (&p)[8], U4 (&out)[NP]) {
  if constexpr (NP == 1) {
    Vec8<T> v;
#pragma unroll
    for (int t = 0; t < 8; ++t) v[t] = static_cast<T>(p[t]);
    out[0] = __builtin_bit_cast(U4, v);
  } else if constexpr (__is_same(T, f16)) {
    // p - c, exact, in one operation of mixed types (which the compiler does not
    // make of a difference: 8192 rows of 8 heads, 7168 keys, D = 64 254 -> 241 us)
    float minus = -1.0f;
    asm("" : "+s"(minus));
    Vec8<f16> rest;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float less[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) less[t] = fmaf(p[2 * w + t], 1.0f - 0x1p-23f, -0x1.8p-25f);
      const auto c = __builtin_amdgcn_cvt_pkrtz(less[0], less[1]);
      out[0][w] = __builtin_bit_cast(uint32_t, c);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        rest[2 * w + t] = static_cast<f16>(fmaf(static_cast<float>(c[t]), minus, p[2 * w + t]));
    }
    out[1] = __builtin_bit_cast(U4, rest);
  } else {
    constexpr float least = 0x1p-126f;
    float r[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) r[t] = p[t];
#pragma unroll
    for (int n = 0; n < NP; ++n)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        float& x = r[2 * w];
        float& y = r[2 * w + 1];
        const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
        out[n][w] = __builtin_amdgcn_perm(uy, ux, 0x07060302u);
        if (n + 1 < NP) {
          x = fmaxf(x - __uint_as_float(ux & 0xffff0000u), fminf(p[2 * w], least));
          y = fmaxf(y - __uint_as_float(uy & 0xffff0000u), fminf(p[2 * w + 1], least));
        }
      }
  }
}

// l + both probabilities of a pair: the sum of what the product takes, so that
// a rounding of the largest ones, or of many small ones, is divided out again.
template <typename T>
__device__ __forceinline__ float add_pair(uint32_t pair, float l) {
  if constexpr (__is_same(T, bf16)) {
    using B2 = __attribute__((ext_vector_type(2))) __bf16;
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(B2, pair),
                                           __builtin_bit_cast(B2, 0x3f803f80u), l, false);
  } else {
    using H2 = __attribute__((ext_vector_type(2))) _Float16;
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(H2, pair), __builtin_bit_cast(H2, 0x3c003c00u),
                                  l, false);
  }
}

// Bits 15 and 31 of the result say which of two elements is an infinity or NaN
// (an exponent of ones carries into its sign's place; the other bits are odds
// and ends).
constexpr uint32_t kOdd = 0x80008000u;
template <typename T>
__device__ __forceinline__ uint32_t odd_bits(uint32_t pair) {
  return __is_same(T, bf16) ? (pair & 0x7f807f80u) + 0x00800080u
                            : (pair & 0x7c007c00u) + 0x04000400u;
}
// The pair with zero in the place of those.
template <typename T>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t pair) {
  const uint32_t b = odd_bits<T>(pair) & kOdd;
  return pair & ~(b | (b - (b >> 15)));
}

// Where the values of a tile's edge are not finite, both kernels take them for
// zero, because times a probability of zero they would be NaN in the rows that
// do not see them.  Here the rows that do see them add them to their results:
// rows [r0, r0 + count) of one (sequence, cache head), keys [k0, k1) in tiles
// of `keys`.  Every thread of the workgroup calls it, after a barrier that
// follows the stores.
template <typename T, typename TO>
__device__ __forceinline__ void put_back(const AttnArgs& a, const Seq& s, const int32_t* table,
                                         int h, const Parts& pt, int k0, int k1, int keys,
                                         int64_t r0, int count, int threads, int split,
                                         bool partial, float* part_o) {
  const int lane = threadIdx.x & 63;
  const int Hq = a.Hk * a.G;
  for (int j0 = k0; j0 < k1; j0 += keys) {
    const int j = j0 + lane < k1 ? j0 + lane : k1 - 1;
    const int p = j >> a.page_shift;
    int page = p < a.max_pages ? table[p] : -1;
    if (page >= a.pages) page = -1;
    if (!is_edge(pt, j0, keys, __any(page < 0 && lane < keys))) continue;
    for (int key = 0; key < keys && j0 + key < k1; ++key) {
      const int pg = __shfl(page, key);
      if (pg < 0) continue;
      const T* src = static_cast<const T*>(a.v_cache) +
                     (((static_cast<int64_t>(pg) * a.Hk + h) << a.page_shift) +
                      ((j0 + key) & ((1 << a.page_shift) - 1))) * a.D;
      for (int e = threadIdx.x; e < count * a.D; e += threads) {
        const int64_t r = r0 + e / a.D;
        const int d = e % a.D;
        const float x = static_cast<float>(src[d]);
        if (r >= static_cast<int64_t>(s.n) * a.G || __builtin_isfinite(x)) continue;
        const int i = a.by_G.div(static_cast<uint32_t>(r));
        int lo, hi;
        visible(a, s, i, &lo, &hi);
        if (j0 + key < lo || j0 + key >= hi) continue;
        const int64_t row = s.q0 + i;
        const int hq = h * a.G + static_cast<int>(r) - i * a.G;
        if (partial) {
          part_o[((split * a.T + row) * Hq + hq) * a.D + d] += x;
        } else {
          TO* y = static_cast<TO*>(a.out) + row * a.o_ts + hq * a.o_hs + d;
          *y = static_cast<TO>(static_cast<float>(*y) + x);
        }
      }
    }
  }
}

}  // namespace pq1
