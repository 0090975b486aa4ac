// Norm of each head and rotation by positions in one pass, alone
// (pq1_norm_rope) or on the way into a cache of two-byte numbers
// (pq1_kv_append_ex) or of 4-bit ones (pq1_kv4_append).
//
//   y = R(p) (w * x * r),  r = (sum x^2 / D + eps)^(-1/2),
// R(p) the rotation of rope.hip.  A head lies in neighbouring lanes of one wave,
// eight elements a lane (two eights past 512), so its sum of squares is a few
// exchanges between lanes; the other halves of pairs come through LDS, which only
// the wave itself uses.  The (cos, sin) of a workgroup's tokens are put into LDS
// once for all heads.
//
// The sum of squares is in fp64 (whose products and sums gfx950 takes at the rate of
// fp32 ones), so that no finite head over- or underflows; r is fp32, where its square
// is far out of that range with x's exponent moved first.  Keys of a 4-bit cache stay
// in fp64 up to their code: there a rounding on the way would move values next to a border between
// two codes by a whole step.  They are narrowed to fp32 with their last bit set
// if that is inexact, so no value lands on a border that was not there.
//
// Bound: memory; next to it the fp64 sums and, into a 4-bit cache, the codes (vector
// instructions are 75 to 87 % of a busy CU's time).  8190 tokens of 24 heads of 256 in
// bf16: 43.7 us, 4.6 TB/s (a large copy reaches 5.1), the gradient 68 us, 4.4 TB/s; 4001
// tokens of 24 + 4 + 4 heads into a 4-bit cache 51 us; one token 3.3 us, where an empty
// kernel takes 3.  What paid: a workgroup walks over neighbouring heads with the next
// one's loads in flight (a workgroup for each few heads: 57 and 97 us, and the append
// 21 us more); two heads of a lane side by side took more registers and time (71 for 57
// us); constants of the fp64 series made where they are used, which leaves four waves to
// a SIMD (the append 6 us less).
#include "attn_device.h"
#include "attn_internal.h"
#include "kv4_format.h"

namespace pq1 {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 1024;  // most (cos, sin) pairs of a workgroup's LDS table

// Heads are numbered token by token; a workgroup takes `per` neighbouring ones,
// `chunk` at a time, whose tokens' table fits.
struct NormDims {
  double inv_D;       // 1 / D
  FastDiv per_token;  // heads of a token, of all streams
  FastDiv pairs;      // rot / 2 (1 without rotation)
  int lane_shift;     // log2 of the lanes of a head
  int chunk;
  int table;          // pairs of the table
  int64_t per, total;
};

enum Into { kPlain, kCache16, kCache4 };

__device__ __forceinline__ int axis_of(const RopeArgs& a, int p) {
  int ax = 0;
  if (a.interleaved) {
    const int r = p % a.axes;
    ax = p / a.axes < a.section[r] ? r : 0;
  } else {
    int end = a.section[0];
    while (ax + 1 < a.axes && p >= end) end += a.section[++ax];
  }
  return ax;
}

// (cos, sin) of an angle, by which a pair is turned.
__device__ __forceinline__ float2 turn_of(int32_t pos, double freq, bool inverse, float) {
  double turn = static_cast<double>(pos) * (freq * 0.15915494309189533577);
  turn -= rint(turn);
  float s, c;
  sincospif(2.0f * static_cast<float>(turn), &s, &c);
  return make_float2(c, inverse ? -s : s);
}
// A constant that is made where it is used (out of the loops around it, the
// series' constants would hold registers).
__device__ __forceinline__ double just(double c) {
  asm volatile("" : "+s"(c));
  return c;
}

// In fp64: the angle less the nearest multiple n of pi / 2 (taken as the sum of two
// numbers; the first difference is exact but for its last rounding, for n up to
// 2^31 the second's share is below 2^-24), then the power series up to x^17 and x^16,
// whose rest is below 2^-58 for |x| <= pi / 4.  From 2^48 on, where n itself begins to
// be rounded and an angle is off by more than 2^-5, its whole turns go first, as above.
__device__ __forceinline__ double2 turn_of(int32_t pos, double freq, bool inverse, double) {
  double angle = static_cast<double>(pos) * freq;
  if (!(fabs(angle) < just(0x1p48))) {
    // (the compiler may take the product into the difference, which then is its rounding,
    // of any size)
    double turn = static_cast<double>(pos) * (freq * just(0.15915494309189533577));
    turn -= rint(turn);
    angle = (turn - rint(turn)) * just(6.2831853071795864769);
  }
  const double n = rint(angle * 0.63661977236758134);
  const double x = fma(-n, 6.123233995736766e-17, fma(-n, 1.5707963267948966, angle));
  const double z = x * x;
  double s = just(1.0 / 355687428096000.0), c = just(1.0 / 20922789888000.0);
  s = fma(s, z, just(-1.0 / 1307674368000.0));
  c = fma(c, z, just(-1.0 / 87178291200.0));
  s = fma(s, z, just(1.0 / 6227020800.0));
  c = fma(c, z, just(1.0 / 479001600.0));
  s = fma(s, z, just(-1.0 / 39916800.0));
  c = fma(c, z, just(-1.0 / 3628800.0));
  s = fma(s, z, just(1.0 / 362880.0));
  c = fma(c, z, just(1.0 / 40320.0));
  s = fma(s, z, just(-1.0 / 5040.0));
  c = fma(c, z, just(-1.0 / 720.0));
  s = fma(s, z, just(1.0 / 120.0));
  c = fma(c, z, just(1.0 / 24.0));
  s = fma(s, z, just(-1.0 / 6.0));
  c = fma(c, z, just(-0.5));
  s = fma(s * z, x, x);
  c = fma(c, z, just(1.0));
  const int quarter = static_cast<int>(n - 4.0 * floor(0.25 * n));
  const double cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
  const bool minus_c = quarter == 1 || quarter == 2, minus_s = (quarter >= 2) != inverse;
  return make_double2(minus_c ? -cc : cc, minus_s ? -ss : ss);
}

// LDS that one wave writes and reads.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sum over the `lanes` (a power of two) neighbouring lanes of a head.
template <int CTRL>
__device__ __forceinline__ double add_dpp(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(u), CTRL, 0xf, 0xf, true);
  const uint32_t hi =
      __builtin_amdgcn_update_dpp(0u, static_cast<uint32_t>(u >> 32), CTRL, 0xf, 0xf, true);
  return v + __builtin_bit_cast(double, uint64_t{hi} << 32 | lo);
}
__device__ __forceinline__ double sum_lanes(double v, int lanes) {
  if (lanes > 1) v = add_dpp<0xb1>(v);    // neighbours
  if (lanes > 2) v = add_dpp<0x4e>(v);    // pairs
  if (lanes > 4) v = add_dpp<0x141>(v);   // fours (mirrored: a four's lanes are equal by now)
  if (lanes > 8) v = add_dpp<0x140>(v);   // eights
  if (lanes > 16) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t l = static_cast<uint32_t>(u), h = static_cast<uint32_t>(u >> 32);
    const auto lo = __builtin_amdgcn_permlane16_swap(l, l, false, false);
    const auto hi = __builtin_amdgcn_permlane16_swap(h, h, false, false);
    v = __builtin_bit_cast(double, uint64_t{hi[0]} << 32 | lo[0]) +
        __builtin_bit_cast(double, uint64_t{hi[1]} << 32 | lo[1]);
  }
  if (lanes > 32) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t l = static_cast<uint32_t>(u), h = static_cast<uint32_t>(u >> 32);
    const auto lo = __builtin_amdgcn_permlane32_swap(l, l, false, false);
    const auto hi = __builtin_amdgcn_permlane32_swap(h, h, false, false);
    v = __builtin_bit_cast(double, uint64_t{hi[0]} << 32 | lo[0]) +
        __builtin_bit_cast(double, uint64_t{hi[1]} << 32 | lo[1]);
  }
  return v;
}

// r of a head as an fp32 factor and a power of two for x: r = f 2^-ex, ex mostly 0.
struct Root {
  float f;
  int ex;
};
__device__ __forceinline__ Root root_of(double var) {
  if (var >= 0x1p-120 && var <= 0x1p120)
    return {__builtin_amdgcn_rsqf(static_cast<float>(var)), 0};
  int ex;  // var = m 2^(2 ex), m in [0.5, 2)
  frexp(var, &ex);
  ex >>= 1;
  return {__builtin_amdgcn_rsqf(static_cast<float>(ldexp(var, -2 * ex))), ex};
}
// x r but for the factor f
template <int NB>
__device__ __forceinline__ void shift_by(float (&x)[NB][8], int ex) {
  if (ex == 0) return;
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) x[i][j] = ldexpf(x[i][j], -ex);
}
// r in fp64: an estimate and two steps of Newton's method.
__device__ __forceinline__ double root64(double var) {
  double y = __builtin_amdgcn_rsq(var);
  const double half = 0.5 * var;
#pragma unroll
  for (int i = 0; i < 2; ++i) y = fma(y, fma(-half * y, y, 0.5), y);
  return var < __builtin_inf() ? y : var != var ? var : 0.0;
}

// Turns the pairs of a head, eight elements e[i] of it at 8 (l + lanes i); `head`
// and cs are 16-byte aligned where half is a multiple of eight.
template <typename Real, int NB, typename CS>
__device__ __forceinline__ void turn_head(Real (&e)[NB][8], const RopeArgs& a, const CS* cs, int l,
                                          int lanes, Real* head) {
  const int half = a.rot >> 1;
  if (a.adjacent) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int p = 4 * (l + lanes * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p + j >= half) continue;
        const Real c = cs[p + j].x, s = cs[p + j].y;
        const Real x0 = e[i][2 * j], x1 = e[i][2 * j + 1];
        e[i][2 * j] = x0 * c - x1 * s;
        e[i][2 * j + 1] = x1 * c + x0 * s;
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int d = 8 * (l + lanes * i);
    if (d < a.rot) {
      Pack<Real, 8> x;
#pragma unroll
      for (int j = 0; j < 8; ++j) x.e[j] = e[i][j];
      *reinterpret_cast<Pack<Real, 8>*>(head + d) = x;
    }
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int d = 8 * (l + lanes * i);
    if (half % 8 == 0) {
      if (d < a.rot) {
        const bool low = d < half;
        const Real* from = head + (low ? d + half : d - half);
        const CS* turns = cs + (low ? d : d - half);
        const Real sign = low ? Real(-1) : Real(1);
        // four at a time: all at once takes 48 registers in fp64
#pragma unroll
        for (int q = 0; q < 8; q += 4) {
          const Pack<Real, 4> other = *reinterpret_cast<const Pack<Real, 4>*>(from + q);
          const Pack<CS, 4> t = *reinterpret_cast<const Pack<CS, 4>*>(turns + q);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            e[i][q + j] = e[i][q + j] * t.e[j].x + sign * other.e[j] * t.e[j].y;
          if constexpr (sizeof(Real) == 8) __builtin_amdgcn_sched_barrier(0);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (d + j >= a.rot) continue;
        const bool low = d + j < half;
        const int p = low ? d + j : d + j - half;
        const Real x = head[low ? d + j + half : p];
        const Real c = cs[p].x, s = cs[p].y;
        e[i][j] = e[i][j] * c + (low ? -x : x) * s;
      }
    }
  }
  wave_fence();
}

// x as an fp32 number that compares with every number of 23 bits or less as x
// does: cut off, with the last bit set where something was.
__device__ __forceinline__ float narrow_odd(double x) {
  const float f = static_cast<float>(x);
  const double d = static_cast<double>(f);
  if (d == x) return f;
  uint32_t b = __float_as_uint(f);
  b -= fabs(d) > fabs(x);
  return __uint_as_float(b | 1u);
}

// Eights of a head, e[i] at 8 (l + lanes i), into a 4-bit cache's row.
template <typename T, int NB>
__device__ __forceinline__ void store4(const float (&e)[NB][8], uint8_t* codes, uint8_t* scales,
                                       int l, int lanes, int D) {
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int b = l + lanes * i;
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = __float_as_uint(e[i][j]) & 0x7fffffffu;
      top = top > u ? top : u;
    }
    // four neighbouring lanes are a group
    uint32_t u = __builtin_amdgcn_update_dpp(0u, top, 0xb1, 0xf, 0xf, true);
    top = top > u ? top : u;
    u = __builtin_amdgcn_update_dpp(0u, top, 0x4e, 0xf, 0xf, true);
    top = top > u ? top : u;
    const uint32_t byte = scale_for<T>(top);
    if (8 * b < D) {
      reinterpret_cast<uint32_t*>(codes)[b] = codes_of(e[i], byte);
      if (b % 4 == 0) scales[b / 4] = static_cast<uint8_t>(byte);
    }
  }
}

// What a workgroup has of one chunk: its first token, the place of its first head
// among that token's, its heads and tokens.
struct Chunk {
  int64_t t0;
  uint32_t off;
  int heads, tokens;
};
__device__ __forceinline__ Chunk chunk_at(const NormDims& dm, int64_t base, int64_t end) {
  Chunk c;
  c.t0 = dm.total >> 32 == 0 ? dm.per_token.div(static_cast<uint32_t>(base)) : base / dm.per_token.d;
  c.off = static_cast<uint32_t>(base - c.t0 * dm.per_token.d);
  c.heads = static_cast<int>(end - base < dm.chunk ? end - base : dm.chunk);
  c.tokens = dm.per_token.div(c.off + c.heads - 1) + 1;
  return c;
}

template <int NB>
__device__ __forceinline__ void load_weight(const float* weight, float (&w)[NB][8], int l,
                                            int lanes, int D) {
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int d = 8 * (l + lanes * i);
    if (weight != nullptr && d < D) {
      load_wide(weight + d, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
    }
  }
}

template <int NB>
__device__ __forceinline__ double square_sum(const float (&x)[NB][8]) {
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double z = x[i][j];
      sum = fma(z, z, sum);
    }
  return sum;
}

// LDS: the table, in fp32 and for a 4-bit cache in fp64 as well, then what a wave's
// lanes exchange.
template <Into INTO>
constexpr int kPairBytes = INTO == kCache4 ? 24 : 8;
template <Into INTO, int NB>
constexpr int kLaneBytes = 8 * NB * (INTO == kCache4 ? 8 : 4);
template <Into INTO>
__host__ __device__ __forceinline__ constexpr int table_bytes(int pairs) {
  return (kPairBytes<INTO> * pairs + 31) & ~15;
}

template <typename TI, typename TO, int NB, Into INTO>
__global__ __launch_bounds__(kThreads, INTO == kCache4 && NB == 1 ? 4 : 1) void norm_rope_kernel(
    NormArgs a, NormDims dm) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const RopeArgs& r = a.rope;
  const int half = r.rot >> 1;
  const int lanes = 1 << dm.lane_shift;
  const int l = threadIdx.x & (lanes - 1);
  const int item0 = threadIdx.x >> dm.lane_shift, items = kThreads >> dm.lane_shift;
  float2* const table = reinterpret_cast<float2*>(lds);
  double2* const table64 = reinterpret_cast<double2*>(lds + ((8 * dm.table + 15) & ~15));
  char* const head =
      lds + table_bytes<INTO>(dm.table) + (threadIdx.x - l) * kLaneBytes<INTO, NB>;

  float wx[NB][8];
  load_weight(a.x_weight, wx, l, lanes, r.D);

  const int64_t begin = blockIdx.x * dm.per;
  const int64_t end = begin + dm.per < dm.total ? begin + dm.per : dm.total;
  for (int64_t base = begin; base < end; base += dm.chunk) {
    const Chunk c = chunk_at(dm, base, end);
    // the next head on its way: kind 0 of x, 1 a key, 2 a value
    Pack<TI, 8> next[NB];
    int64_t slot = 0;
#pragma unroll
    for (int i = 0; i < NB; ++i) next[i] = {};
    auto place = [&](int n, int* tl, uint32_t* h, int* kind) {
      *tl = dm.per_token.div(c.off + n);
      *h = c.off + n - *tl * dm.per_token.d;
      *kind = 0;
      if (INTO != kPlain && *h >= static_cast<uint32_t>(r.Hx)) {
        *h -= r.Hx;
        *kind = *h >= static_cast<uint32_t>(r.Hk) ? 2 : 1;
        if (*kind == 2) *h -= r.Hk;
      }
    };
    auto fetch = [&](int n) {
      int tl, kind;
      uint32_t h;
      place(n, &tl, &h, &kind);
      const int64_t t = c.t0 + tl;
      const TI* src = static_cast<const TI*>(r.x) + t * r.x_ts + h * r.x_hs;
      if (INTO != kPlain && kind != 0) {
        src = kind == 2 ? static_cast<const TI*>(r.v) + t * r.v_ts + h * r.v_hs
                        : static_cast<const TI*>(r.k) + t * r.k_ts + h * r.k_hs;
        slot = r.slots[t];
      }
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
        if (d < r.D) next[i] = *reinterpret_cast<const Pack<TI, 8>*>(src + d);
      }
    };
    if (item0 < c.heads) fetch(item0);
    if (base != begin) __syncthreads();  // the table before is done with
    for (int i = threadIdx.x; i < c.tokens * half; i += kThreads) {
      const int t = static_cast<int>(dm.pairs.div(i));
      const int p = i - t * half;
      const int32_t pos = r.positions[axis_of(r, p) * r.T + c.t0 + t];
      if constexpr (INTO == kCache4) {
        const double2 cs = turn_of(pos, r.freqs[p], r.inverse, double{});
        table64[i] = cs;
        table[i] = make_float2(static_cast<float>(cs.x), static_cast<float>(cs.y));
      } else {
        table[i] = turn_of(pos, r.freqs[p], r.inverse, float{});
      }
    }
    __syncthreads();
    for (int n = item0; n < c.heads; n += items) {
      int tl, kind;
      uint32_t h;
      place(n, &tl, &h, &kind);
      float e[NB][8];
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) e[i][j] = static_cast<float>(next[i].e[j]);
      const int64_t row_slot = slot;
      // the next head's loads while this one is computed
      if (n + items < c.heads) fetch(n + items);
      void* dst;
      uint8_t* dst_scale = nullptr;
      if (INTO != kPlain && kind != 0) {
        if (row_slot < 0 || row_slot >= r.slot_count) continue;
        const int64_t page = row_slot >> r.page_shift;
        const int64_t row =
            ((page * r.Hk + h) << r.page_shift) + (row_slot - (page << r.page_shift));
        void* const cache = kind == 2 ? r.v_cache : r.k_cache;
        if constexpr (INTO == kCache4) {
          dst = static_cast<uint8_t*>(cache) + row * (r.D / 2);
          dst_scale = (kind == 2 ? a.v_scale : a.k_scale) + row * (r.D / kGroup4);
        } else {
          dst = static_cast<TO*>(cache) + row * r.D;
        }
      } else {
        dst = static_cast<TO*>(r.y) + (c.t0 + tl) * r.y_ts + h * r.y_hs;
      }
      const bool normed = (kind == 0 ? a.x_weight : kind == 1 ? a.k_weight : nullptr) != nullptr;
      const bool turned = half > 0 && kind != 2;
      double var = 0.0;
      if (normed) var = sum_lanes(square_sum(e), lanes) * dm.inv_D + a.eps;
      if (INTO == kCache4 && kind == 1 && (normed || turned)) {
        double z[NB][8];
        const double f = normed ? root64(var) : 1.0;
        float wk[NB][8];  // read again for each key: few heads are, and registers are short
        load_weight(a.k_weight, wk, l, lanes, r.D);
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) z[i][j] = normed ? e[i][j] * f * wk[i][j] : double{e[i][j]};
        if (turned)
          turn_head(z, r, table64 + tl * half, l, lanes, reinterpret_cast<double*>(head));
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) e[i][j] = narrow_odd(z[i][j]);
      } else {
        if (normed) {
          const Root f = root_of(var);
          shift_by(e, f.ex);
          float w[NB][8];
          if (INTO == kCache16 && kind == 1) load_weight(a.k_weight, w, l, lanes, r.D);
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              e[i][j] = e[i][j] * f.f * (INTO == kCache16 && kind == 1 ? w[i][j] : wx[i][j]);
        }
        if (turned) turn_head(e, r, table + tl * half, l, lanes, reinterpret_cast<float*>(head));
      }
      if (INTO == kCache4 && kind != 0) {
        store4<TO>(e, static_cast<uint8_t*>(dst), dst_scale, l, lanes, r.D);
      } else {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int d = 8 * (l + lanes * i);
          if (d < r.D) store_wide(static_cast<TO*>(dst) + d, e[i]);
        }
      }
    }
  }
}

// Heads of `streams` heads a token, cut for at most `most` workgroups of a kernel
// whose heads take 2^shift lanes at least; returns the workgroups.
int64_t cut_heads(NormDims* dm, const RopeArgs& r, int heads, int shift, int64_t most) {
  const int eights = r.D / 8 > 64 ? 2 : 1;  // of a lane
  const int half = r.rot / 2;
  dm->lane_shift = shift;
  while ((8 * eights << dm->lane_shift) < r.D) ++dm->lane_shift;
  dm->inv_D = 1.0 / r.D;
  dm->per_token = FastDiv(heads);
  dm->pairs = FastDiv(half > 0 ? half : 1);
  dm->total = r.T * heads;
  const int64_t items = kThreads >> dm->lane_shift;
  dm->per = ((dm->total + most - 1) / most + items - 1) / items * items;
  // n tokens' heads, wherever they begin, are of n + 1 tokens
  int64_t chunk = half > 0 ? int64_t{kTable / half - 1} * heads : int64_t{1} << 20;
  if (chunk > 1 << 20) chunk = 1 << 20;
  dm->chunk = static_cast<int>(chunk < dm->per ? chunk : dm->per);
  dm->table = static_cast<int>((heads - 1 + dm->chunk - 1) / heads + 1) * half;
  return (dm->total + dm->per - 1) / dm->per;
}

// whether lanes exchange halves of pairs
bool half_exchange(const RopeArgs& r) { return r.rot > 0 && !r.adjacent; }

template <typename TI, typename TO, Into INTO>
hipError_t launch_heads(const NormArgs& a, hipStream_t s) {
  const RopeArgs& r = a.rope;
  NormDims dm;
  const int heads = r.Hx + (INTO == kPlain ? 0 : 2 * r.Hk);
  // as many workgroups as the device holds at once, by registers; four lanes are a
  // group of a 4-bit cache
  const uint32_t blocks = static_cast<uint32_t>(
      cut_heads(&dm, r, heads, INTO == kCache4 ? 2 : 0, 1024));
  const bool two = r.D / 8 > 64;
  const int exchange = half_exchange(r) ? kThreads * (two ? kLaneBytes<INTO, 2> : kLaneBytes<INTO, 1>)
                                        : 0;
  const int lds = table_bytes<INTO>(dm.table) + exchange;
  if (two)
    norm_rope_kernel<TI, TO, 2, INTO><<<blocks, kThreads, lds, s>>>(a, dm);
  else
    norm_rope_kernel<TI, TO, 1, INTO><<<blocks, kThreads, lds, s>>>(a, dm);
  return hipGetLastError();
}

template <typename TI>
hipError_t launch_in(const NormArgs& a, int out_dtype, bool cache4, hipStream_t s) {
  const bool append = a.rope.slots != nullptr;
  switch (out_dtype) {
    case PQ1_BF16:
      if constexpr (!__is_same(TI, f16)) {
        if (append && cache4) return launch_heads<TI, bf16, kCache4>(a, s);
        if (append) return launch_heads<TI, bf16, kCache16>(a, s);
      }
      return launch_heads<TI, bf16, kPlain>(a, s);
    case PQ1_F16:
      if constexpr (!__is_same(TI, bf16)) {
        if (append && cache4) return launch_heads<TI, f16, kCache4>(a, s);
        if (append) return launch_heads<TI, f16, kCache16>(a, s);
      }
      return launch_heads<TI, f16, kPlain>(a, s);
    default:
      return launch_heads<TI, float, kPlain>(a, s);
  }
}

// ---------------------------------------------------------------------------
// Gradient: with u = R(p)^T g,
//   dw = sum over tokens and heads of u x r,
//   dx = r w u - x r^3 / D sum(w u x).
// Each lane keeps the sums of its eight elements of dw, a workgroup's go to the
// workspace, and a second kernel adds those in order, so that dw is the same from
// run to run.
// ---------------------------------------------------------------------------
template <typename TG, typename TX, int NB>
__global__ __launch_bounds__(kThreads) void norm_rope_grad_kernel(NormArgs a, NormDims dm,
                                                                  float* part_dw) {
  __shared__ __attribute__((aligned(16))) float2 table[kTable];
  __shared__ __attribute__((aligned(16))) float others[kThreads * 8 * NB];
  const RopeArgs& r = a.rope;
  const int half = r.rot >> 1;
  const int lanes = 1 << dm.lane_shift;
  const int l = threadIdx.x & (lanes - 1);
  float* const head = others + (threadIdx.x - l) * (8 * NB);
  const int item0 = threadIdx.x >> dm.lane_shift, items = kThreads >> dm.lane_shift;
  float w[NB][8], dw[NB][8];
  load_weight(a.x_weight, w, l, lanes, r.D);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  const int64_t begin = blockIdx.x * dm.per;
  const int64_t end = begin + dm.per < dm.total ? begin + dm.per : dm.total;
  for (int64_t base = begin; base < end; base += dm.chunk) {
    const Chunk c = chunk_at(dm, base, end);
    Pack<TG, 8> gn[NB];
    Pack<TX, 8> xn[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) gn[i] = {}, xn[i] = {};
    auto fetch = [&](int n) {
      const uint32_t tl = dm.per_token.div(c.off + n);
      const uint32_t h = c.off + n - tl * dm.per_token.d;
      const int64_t t = c.t0 + tl;
      const TG* gp = static_cast<const TG*>(a.grad) + t * a.g_ts + h * a.g_hs;
      const TX* xp = static_cast<const TX*>(r.x) + t * r.x_ts + h * r.x_hs;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
        if (d >= r.D) continue;
        gn[i] = *reinterpret_cast<const Pack<TG, 8>*>(gp + d);
        xn[i] = *reinterpret_cast<const Pack<TX, 8>*>(xp + d);
      }
    };
    if (item0 < c.heads) fetch(item0);
    if (base != begin) __syncthreads();
    for (int i = threadIdx.x; i < c.tokens * half; i += kThreads) {
      const int t = static_cast<int>(dm.pairs.div(i));
      const int p = i - t * half;
      const int32_t pos = r.positions[axis_of(r, p) * r.T + c.t0 + t];
      table[i] = turn_of(pos, r.freqs[p], !r.inverse, float{});
    }
    __syncthreads();
    for (int n = item0; n < c.heads; n += items) {
      const uint32_t tl = dm.per_token.div(c.off + n);
      const uint32_t h = c.off + n - tl * dm.per_token.d;
      float u[NB][8], x[NB][8];
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[i][j] = static_cast<float>(gn[i].e[j]), x[i][j] = static_cast<float>(xn[i].e[j]);
      // the next head's loads while this one is computed
      if (n + items < c.heads) fetch(n + items);
      const Root f = root_of(sum_lanes(square_sum(x), lanes) * dm.inv_D + a.eps);
      if (half > 0) turn_head(u, r, table + tl * half, l, lanes, head);
      // n = x r; dx = r (w u - n sum(w u n) / D)
      shift_by(x, f.ex);
      double along = 0.0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[i][j] *= f.f;
          dw[i][j] = fmaf(u[i][j], x[i][j], dw[i][j]);
          u[i][j] *= w[i][j];
          along = fma(static_cast<double>(u[i][j]), static_cast<double>(x[i][j]), along);
        }
      const float mean = static_cast<float>(sum_lanes(along, lanes) * dm.inv_D);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) u[i][j] = (u[i][j] - x[i][j] * mean) * f.f;
      shift_by(u, f.ex);
      TX* dp = static_cast<TX*>(r.y) + (c.t0 + tl) * r.y_ts + h * r.y_hs;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
        if (d < r.D) store_wide(dp + d, u[i]);
      }
    }
  }
  if (part_dw == nullptr) return;
  // the sums of the lanes that hold the same elements
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) head[8 * (l + lanes * i) + j] = dw[i][j];
  __syncthreads();
  for (int d = threadIdx.x; d < r.D; d += kThreads) {
    float sum = 0.0f;
    for (int i = 0; i < items; ++i) sum += others[i * (lanes * 8 * NB) + d];
    part_dw[static_cast<int64_t>(blockIdx.x) * r.D + d] = sum;
  }
}

// dw[d] = sum of the workgroups' sums: 16 elements a workgroup, a 64th of the sums a
// thread.
constexpr int kSumThreads = 1024, kSlices = kSumThreads / 16;
__global__ __launch_bounds__(kSumThreads) void sum_dw_kernel(const float* part_dw, int parts, int D,
                                                             float* dw) {
  __shared__ double sums[kSlices][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int d = blockIdx.x * 16 + c;
  double sum = 0.0;
  if (d < D) {
#pragma unroll 16
    for (int p = slice; p < parts; p += kSlices)
      sum += part_dw[static_cast<int64_t>(p) * D + d];
  }
  sums[slice][c] = sum;
  __syncthreads();
  if (slice == 0 && d < D) {
    sum = 0.0;
#pragma unroll 8
    for (int i = 0; i < kSlices; ++i) sum += sums[i][c];
    dw[d] = static_cast<float>(sum);
  }
}

template <typename TG, typename TX>
hipError_t launch_grad(const NormArgs& a, float* dw, float* part_dw, hipStream_t s) {
  const RopeArgs& r = a.rope;
  int parts = 0;
  if (r.T > 0) {
    NormDims dm;
    parts = static_cast<int>(cut_heads(&dm, r, r.Hx, 0, norm_grad_parts(r.T)));
    if (r.D / 8 > 64)
      norm_rope_grad_kernel<TG, TX, 2><<<parts, kThreads, 0, s>>>(a, dm, part_dw);
    else
      norm_rope_grad_kernel<TG, TX, 1><<<parts, kThreads, 0, s>>>(a, dm, part_dw);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (dw == nullptr) return hipSuccess;
  sum_dw_kernel<<<(r.D + 15) / 16, kSumThreads, 0, s>>>(part_dw, parts, r.D, dw);
  return hipGetLastError();
}

template <typename TG>
hipError_t launch_grad_in(const NormArgs& a, int x_dtype, float* dw, float* part, hipStream_t s) {
  switch (x_dtype) {
    case PQ1_BF16: return launch_grad<TG, bf16>(a, dw, part, s);
    case PQ1_F16: return launch_grad<TG, f16>(a, dw, part, s);
    default: return launch_grad<TG, float>(a, dw, part, s);
  }
}

}  // namespace

hipError_t launch_norm_rope(const NormArgs& a, int in_dtype, int out_dtype, bool cache4,
                            hipStream_t s) {
  switch (in_dtype) {
    case PQ1_BF16: return launch_in<bf16>(a, out_dtype, cache4, s);
    case PQ1_F16: return launch_in<f16>(a, out_dtype, cache4, s);
    default: return launch_in<float>(a, out_dtype, cache4, s);
  }
}

hipError_t launch_norm_rope_grad(const NormArgs& a, int g_dtype, int x_dtype, float* dw,
                                 float* part_dw, hipStream_t s) {
  switch (g_dtype) {
    case PQ1_BF16: return launch_grad_in<bf16>(a, x_dtype, dw, part_dw, s);
    case PQ1_F16: return launch_grad_in<f16>(a, x_dtype, dw, part_dw, s);
    default: return launch_grad_in<float>(a, x_dtype, dw, part_dw, s);
  }
}

}  // namespace pq1
