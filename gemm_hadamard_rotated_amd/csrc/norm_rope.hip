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
// The sum of squares and r are in fp64, so that no finite head over- or
// underflows; r is split into a power of two, which moves x's exponent, and an
// fp32 factor between 0.7 and 1.5.  Keys of a 4-bit cache stay in fp64 up to their
// code: there a rounding on the way would move values next to a border between
// two codes by a whole step.  They are narrowed to fp32 with their last bit set
// if that is inexact, so no value lands on a border that was not there.
#include <type_traits>

#include "attn_device.h"
#include "attn_internal.h"
#include "kv4_format.h"

namespace pq1 {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 1024;  // (cos, sin) pairs of a workgroup's LDS table

struct NormDims {
  FastDiv per_token;  // heads of a token, of all streams
  FastDiv parts;      // workgroups that share a token group
  FastDiv pairs;      // rot / 2 (1 without rotation)
  int lane_shift;     // log2 of the lanes of a head
  int tokens;         // tokens of a group
  int64_t first;      // group of this launch's first workgroup
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
__device__ __forceinline__ double2 turn_of(int32_t pos, double freq, bool inverse, double) {
  const double angle = static_cast<double>(pos) * freq;
  const double n = rint(angle * 0.15915494309189533577);
  double s, c;  // 2 pi as the sum of two numbers
  sincos(fma(-n, 2.4492935982947064e-16, fma(-n, 6.283185307179586477, angle)), &s, &c);
  return make_double2(c, inverse ? -s : s);
}

template <typename Real>
struct PairOf;
template <>
struct PairOf<float> { using type = float2; };
template <>
struct PairOf<double> { using type = double2; };

// LDS that one wave writes and reads.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ double sum_lanes(double v, int lanes) {
  for (int m = 1; m < lanes; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Turns the pairs of a head, eight elements e[i] of it at 8 (l + lanes i).
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
        const Real c = static_cast<Real>(cs[p + j].x), s = static_cast<Real>(cs[p + j].y);
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
#pragma unroll
      for (int j = 0; j < 8; ++j) head[d + j] = e[i][j];
    }
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int d = 8 * (l + lanes * i);
    if (half % 8 == 0) {
      if (d < a.rot) {
        const bool low = d < half;
        const Real* other = head + (low ? d + half : d - half);
        const CS* t = cs + (low ? d : d - half);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const Real c = static_cast<Real>(t[j].x), s = static_cast<Real>(t[j].y);
          e[i][j] = e[i][j] * c + (low ? -other[j] : other[j]) * s;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (d + j >= a.rot) continue;
        const bool low = d + j < half;
        const int p = low ? d + j : d + j - half;
        const Real x = head[low ? d + j + half : p];
        const Real c = static_cast<Real>(cs[p].x), s = static_cast<Real>(cs[p].y);
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
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
      const uint32_t u = __shfl_xor(top, m);
      top = top > u ? top : u;
    }
    const uint32_t byte = scale_for<T>(top);
    if (8 * b < D) {
      reinterpret_cast<uint32_t*>(codes)[b] = codes_of(e[i], byte);
      if (b % 4 == 0) scales[b / 4] = static_cast<uint8_t>(byte);
    }
  }
}

template <typename TI, typename TO, int NB, int U, Into INTO>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(NormArgs a, NormDims dm) {
  using Wide = typename std::conditional<INTO == kCache4, double, float>::type;
  using CS = typename PairOf<Wide>::type;
  __shared__ CS table[kTable];
  __shared__ __attribute__((aligned(16))) Wide others[kThreads * 8 * NB];
  const RopeArgs& r = a.rope;
  const uint32_t group = dm.parts.div(blockIdx.x);
  const uint32_t part = blockIdx.x - group * dm.parts.d;
  const int64_t t0 = (dm.first + group) * dm.tokens;
  const int nt = static_cast<int>(r.T - t0 < dm.tokens ? r.T - t0 : dm.tokens);
  const int half = r.rot >> 1;
  const uint32_t total = static_cast<uint32_t>(nt) * dm.per_token.d;
  const int lanes = 1 << dm.lane_shift;
  const int l = threadIdx.x & (lanes - 1);
  Wide* const head = others + (threadIdx.x - l) * (8 * NB);

  // kind: 0 of x, 1 a key, 2 a value
  int kind[U], token[U];
  void* dst[U];
  uint8_t* dst_scale[U];
  float e[U][NB][8];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    dst[k] = nullptr;
    dst_scale[k] = nullptr;
    const uint32_t u = ((part * U + k) * kThreads + threadIdx.x) >> dm.lane_shift;
    if (u >= total) continue;
    const uint32_t tl = dm.per_token.div(u);
    uint32_t h = u - tl * dm.per_token.d;
    const int64_t t = t0 + tl;
    token[k] = tl;
    kind[k] = 0;
    const TI* src;
    if (INTO != kPlain && h >= static_cast<uint32_t>(r.Hx)) {
      const int64_t slot = r.slots[t];
      if (slot < 0 || slot >= r.slot_count) continue;
      const int64_t page = slot >> r.page_shift;
      h -= r.Hx;
      kind[k] = h >= static_cast<uint32_t>(r.Hk) ? 2 : 1;
      if (kind[k] == 2) h -= r.Hk;
      src = kind[k] == 2 ? static_cast<const TI*>(r.v) + t * r.v_ts + h * r.v_hs
                         : static_cast<const TI*>(r.k) + t * r.k_ts + h * r.k_hs;
      const int64_t row = ((page * r.Hk + h) << r.page_shift) + (slot - (page << r.page_shift));
      void* const base = kind[k] == 2 ? r.v_cache : r.k_cache;
      if constexpr (INTO == kCache4) {
        dst[k] = static_cast<uint8_t*>(base) + row * (r.D / 2);
        dst_scale[k] = (kind[k] == 2 ? a.v_scale : a.k_scale) + row * (r.D / kGroup4);
      } else {
        dst[k] = static_cast<TO*>(base) + row * r.D;
      }
    } else {
      src = static_cast<const TI*>(r.x) + t * r.x_ts + h * r.x_hs;
      dst[k] = static_cast<TO*>(r.y) + t * r.y_ts + h * r.y_hs;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int d = 8 * (l + lanes * i);
      if (d < r.D) {
        load_wide(src + d, e[k][i]);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) e[k][i][j] = 0.0f;
      }
    }
  }

  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = static_cast<int>(dm.pairs.div(i));
    const int p = i - t * half;
    const int32_t pos = r.positions[axis_of(r, p) * r.T + t0 + t];
    table[i] = turn_of(pos, r.freqs[p], r.inverse, Wide{});
  }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (dst[k] == nullptr) continue;
    const float* weight = kind[k] == 0 ? a.x_weight : kind[k] == 1 ? a.k_weight : nullptr;
    const CS* cs = table + token[k] * half;
    const bool turned = half > 0 && kind[k] != 2;
    double var = 0.0;
    if (weight != nullptr) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double x = e[k][i][j];
          sum = fma(x, x, sum);
        }
      var = sum_lanes(sum, lanes) / r.D + a.eps;
    }
    if (INTO == kCache4 && kind[k] == 1 && (weight != nullptr || turned)) {
      Wide z[NB][8];
      const Wide f = weight != nullptr ? static_cast<Wide>(1.0 / sqrt(var)) : Wide(1);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
        float w[8];
        if (weight != nullptr && d < r.D) load_wide(weight + d, w);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          z[i][j] = weight != nullptr && d < r.D ? e[k][i][j] * f * w[j] : Wide(e[k][i][j]);
      }
      if (turned) turn_head(z, r, cs, l, lanes, head);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) e[k][i][j] = narrow_odd(z[i][j]);
    } else {
      if (weight != nullptr) {
        int ex;  // var = m 2^(2 ex), m in [0.5, 2)
        frexp(var, &ex);
        ex >>= 1;
        const float f = 1.0f / sqrtf(static_cast<float>(ldexp(var, -2 * ex)));
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int d = 8 * (l + lanes * i);
          if (d >= r.D) continue;
          float w[8];
          load_wide(weight + d, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) e[k][i][j] = ldexpf(e[k][i][j], -ex) * f * w[j];
        }
      }
      if (turned) turn_head(e[k], r, cs, l, lanes, reinterpret_cast<float*>(head));
    }
    if (INTO == kCache4 && kind[k] != 0) {
      store4<TO>(e[k], static_cast<uint8_t*>(dst[k]), dst_scale[k], l, lanes, r.D);
    } else {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
        if (d < r.D) store_wide(static_cast<TO*>(dst[k]) + d, e[k][i]);
      }
    }
  }
}

template <typename TI, typename TO, int NB, int U, Into INTO>
hipError_t launch_groups(const NormArgs& a, NormDims dm, hipStream_t s) {
  // A group's tokens fill its workgroup, or one token is shared by several;
  // the group's table has to fit.
  const int half = a.rope.rot / 2;
  const int64_t per_token = static_cast<int64_t>(dm.per_token.d) << dm.lane_shift;
  int64_t tokens = U * kThreads / per_token;
  if (tokens * half > kTable) tokens = kTable / half;
  if (tokens < 1) tokens = 1;
  dm.tokens = static_cast<int>(tokens);
  const int64_t parts = (tokens * per_token + U * kThreads - 1) / (U * kThreads);
  dm.parts = FastDiv(static_cast<uint32_t>(parts));
  const int64_t groups = (a.rope.T + tokens - 1) / tokens;
  // a launch holds less than 2^32 threads
  const int64_t most = ((int64_t{1} << 32) / kThreads - 1) / parts;
  for (dm.first = 0; dm.first < groups; dm.first += most) {
    const int64_t n = groups - dm.first < most ? groups - dm.first : most;
    norm_rope_kernel<TI, TO, NB, U, INTO>
        <<<dim3(static_cast<uint32_t>(n * parts)), kThreads, 0, s>>>(a, dm);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TI, typename TO, Into INTO>
hipError_t launch_heads(const NormArgs& a, hipStream_t s) {
  const RopeArgs& r = a.rope;
  NormDims dm;
  const int eights = r.D / 8 > 64 ? 2 : 1;  // of a lane
  dm.lane_shift = INTO == kCache4 ? 2 : 0;  // four lanes are a group of a 4-bit cache
  while ((8 * eights << dm.lane_shift) < r.D) ++dm.lane_shift;
  dm.per_token = FastDiv(r.Hx + (INTO == kPlain ? 0 : 2 * r.Hk));
  dm.pairs = FastDiv(r.rot > 0 ? r.rot / 2 : 1);
  if (eights == 2) return launch_groups<TI, TO, 2, 1, INTO>(a, dm, s);
  return launch_groups<TI, TO, 1, 1, INTO>(a, dm, s);
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
// Workgroups walk over groups of tokens; each lane keeps the sums of its eight
// elements of dw, a workgroup's go to the workspace, and a second kernel adds
// those in order, so that dw is the same from run to run.
// ---------------------------------------------------------------------------
constexpr int kGradTable = 2048;

template <typename TG, typename TX, int NB>
__global__ __launch_bounds__(kThreads) void norm_rope_grad_kernel(NormArgs a, NormDims dm,
                                                                  int64_t groups, float* part_dw) {
  __shared__ float2 table[kGradTable];
  __shared__ __attribute__((aligned(16))) float others[kThreads * 8 * NB];
  const RopeArgs& r = a.rope;
  const int half = r.rot >> 1;
  const int lanes = 1 << dm.lane_shift;
  const int l = threadIdx.x & (lanes - 1);
  float* const head = others + (threadIdx.x - l) * (8 * NB);
  const int item0 = threadIdx.x >> dm.lane_shift, items = kThreads >> dm.lane_shift;
  float w[NB][8], dw[NB][8];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int d = 8 * (l + lanes * i);
    if (d < r.D) {
      load_wide(a.x_weight + d, w[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[i][j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  for (int64_t grp = blockIdx.x; grp < groups; grp += gridDim.x) {
    const int64_t t0 = grp * dm.tokens;
    const int nt = static_cast<int>(r.T - t0 < dm.tokens ? r.T - t0 : dm.tokens);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = static_cast<int>(dm.pairs.div(i));
      const int p = i - t * half;
      const int32_t pos = r.positions[axis_of(r, p) * r.T + t0 + t];
      table[i] = turn_of(pos, r.freqs[p], !r.inverse, float{});
    }
    __syncthreads();
    const uint32_t total = static_cast<uint32_t>(nt) * dm.per_token.d;
    for (uint32_t it = item0; it < total; it += items) {
      const uint32_t tl = dm.per_token.div(it);
      const uint32_t h = it - tl * dm.per_token.d;
      const int64_t t = t0 + tl;
      const TG* gp = static_cast<const TG*>(a.grad) + t * a.g_ts + h * a.g_hs;
      const TX* xp = static_cast<const TX*>(r.x) + t * r.x_ts + h * r.x_hs;
      TX* dp = static_cast<TX*>(r.y) + t * r.y_ts + h * r.y_hs;
      float u[NB][8], x[NB][8];
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
        if (d < r.D) {
          load_wide(gp + d, u[i]);
          load_wide(xp + d, x[i]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) u[i][j] = x[i][j] = 0.0f;
        }
      }
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double z = x[i][j];
          sum = fma(z, z, sum);
        }
      const double var = sum_lanes(sum, lanes) / r.D + a.eps;
      int ex;
      frexp(var, &ex);
      ex >>= 1;
      const float f = 1.0f / sqrtf(static_cast<float>(ldexp(var, -2 * ex)));
      if (half > 0) turn_head(u, r, table + tl * half, l, lanes, head);
      // n = x r; dx = r (w u - n sum(w u n) / D)
      double along = 0.0;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[i][j] = ldexpf(x[i][j], -ex) * f;
          dw[i][j] = fmaf(u[i][j], x[i][j], dw[i][j]);
          u[i][j] *= w[i][j];
          along += static_cast<double>(u[i][j]) * x[i][j];
        }
      const float mean = static_cast<float>(sum_lanes(along, lanes) / r.D);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const int d = 8 * (l + lanes * i);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          u[i][j] = ldexpf((u[i][j] - x[i][j] * mean) * f, -ex);
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

// dw[d] = sum of the workgroups' sums: 16 elements a workgroup, a sixteenth of the
// workgroups a thread.
__global__ __launch_bounds__(256) void sum_dw_kernel(const float* part_dw, int parts, int D,
                                                     float* dw) {
  __shared__ double sums[16][17];
  const int c = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int d = blockIdx.x * 16 + c;
  double sum = 0.0;
  if (d < D)
    for (int p = slice; p < parts; p += 16) sum += part_dw[static_cast<int64_t>(p) * D + d];
  sums[slice][c] = sum;
  __syncthreads();
  if (slice == 0 && d < D) {
    for (int i = 1; i < 16; ++i) sum += sums[i][c];
    dw[d] = static_cast<float>(sum);
  }
}

NormDims grad_dims(const NormArgs& a, int64_t* groups) {
  const RopeArgs& r = a.rope;
  NormDims dm;
  const int eights = r.D / 8 > 64 ? 2 : 1;
  dm.lane_shift = 0;
  while ((8 * eights << dm.lane_shift) < r.D) ++dm.lane_shift;
  dm.per_token = FastDiv(r.Hx);
  dm.pairs = FastDiv(r.rot > 0 ? r.rot / 2 : 1);
  dm.parts = FastDiv(1);
  dm.first = 0;
  const int half = r.rot / 2;
  // eight heads for each place in the workgroup
  int64_t tokens = (8 * (kThreads >> dm.lane_shift) + r.Hx - 1) / r.Hx;
  if (tokens * half > kGradTable) tokens = kGradTable / half;
  dm.tokens = static_cast<int>(tokens);
  *groups = (r.T + tokens - 1) / tokens;
  return dm;
}

template <typename TG, typename TX>
hipError_t launch_grad(const NormArgs& a, float* dw, float* part_dw, hipStream_t s) {
  const int most = static_cast<int>(norm_grad_parts(a.rope.T));
  int parts = 0;
  if (a.rope.T > 0) {
    int64_t groups;
    const NormDims dm = grad_dims(a, &groups);
    parts = static_cast<int>(groups < most ? groups : most);
    if (a.rope.D / 8 > 64)
      norm_rope_grad_kernel<TG, TX, 2><<<parts, kThreads, 0, s>>>(a, dm, groups, part_dw);
    else
      norm_rope_grad_kernel<TG, TX, 1><<<parts, kThreads, 0, s>>>(a, dm, groups, part_dw);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  if (dw == nullptr) return hipSuccess;
  sum_dw_kernel<<<(a.rope.D + 15) / 16, 256, 0, s>>>(part_dw, parts, a.rope.D, dw);
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
