// Rotation by positions on one to four axes, alone (pq1_rope) or on the way
// into a paged cache (pq1_kv_append).
//
// Pair i of a head, (x0, x1), is turned by theta = p[a(i)] * freqs[i]:
//   y0 = x0 cos(theta) - x1 sin(theta),  y1 = x1 cos(theta) + x0 sin(theta).
// The angle depends on the token and the pair but not on the head, so a
// workgroup, with its loads in flight, puts (cos, sin) of its tokens' pairs into
// LDS, and all heads of those tokens use that table.  The angle is taken in
// turns in fp64 (p * f / 2 pi) and reduced there; only the reduced turn, at
// most half, is narrowed to fp32 for the sine and cosine.
//
// Bound: the memory traffic; a few tokens by the launch.  8190 tokens of 24
// heads of 256 bf16: 201 MB in 48 us, 4.2 TB/s (a large copy reaches 5.1);
// 4001 tokens of 24 + 4 + 4 heads, fp32 in, appended: 42 us, 4.7 TB/s; one token
// 3 us, as an empty kernel.
#include "attn_device.h"
#include "attn_internal.h"

namespace pq1 {

namespace {

constexpr int kThreads = 256;
constexpr int kTable = 2048;  // (cos, sin) pairs of a workgroup's LDS table

struct Dims {
  FastDiv per_token;   // units of a token
  FastDiv per_head;    // units of a rotated head
  FastDiv per_value;   // units of a value head
  FastDiv parts;       // workgroups that share a token group
  FastDiv pairs;       // rot / 2 (1 without rotation)
  int tokens;          // tokens of a group
  int64_t first;       // group of this launch's first workgroup
  int rot_units;       // units of a head that hold pairs; the rest are copies
  int tail;            // elements of a tail's unit
};

// A unit is some elements at each of two places of a head: the two halves of
// VEC pairs (or 2 VEC neighbours that are VEC pairs), 16 elements of a value,
// or a piece of a head's tail: 2 VEC elements where VEC is 4 or 8 (then every
// lane does the same); else 16, which begin at any pair of elements, or 2 of a
// tail of less than 8.  A last piece may overlap the one before or be one place
// twice.  A thread takes U units and has all their loads in flight before the
// workgroup makes its table.
template <int W, int ALIGN = 16, typename T>
__device__ __forceinline__ void load_first(const T* p, float (&o)[8]) {
  struct alignas(sizeof(T) * W < ALIGN ? sizeof(T) * W : ALIGN) Piece {
    T e[W];
  };
  const Piece x = *reinterpret_cast<const Piece*>(p);
#pragma unroll
  for (int i = 0; i < W; ++i) o[i] = static_cast<float>(x.e[i]);
}
template <int W, int ALIGN = 16, typename T>
__device__ __forceinline__ void store_first(T* p, const float (&v)[8]) {
  struct alignas(sizeof(T) * W < ALIGN ? sizeof(T) * W : ALIGN) Piece {
    T e[W];
  };
  Piece x;
#pragma unroll
  for (int i = 0; i < W; ++i) x.e[i] = static_cast<T>(v[i]);
  *reinterpret_cast<Piece*>(p) = x;
}
template <typename TI, typename TO, int VEC, int U, bool APPEND>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, Dims dm) {
  __shared__ float2 table[kTable];
  const uint32_t group = dm.parts.div(blockIdx.x);
  const uint32_t part = blockIdx.x - group * dm.parts.d;
  const int64_t t0 = (dm.first + group) * dm.tokens;
  const int nt = static_cast<int>(a.T - t0 < dm.tokens ? a.T - t0 : dm.tokens);
  const int half = a.rot >> 1;
  const uint32_t total = static_cast<uint32_t>(nt) * dm.per_token.d;

  TO* dst[U];
  // angle: of the unit's first pair; -1: a copy of a tail, -2: of a value
  int at0[U], at1[U], angle[U];
  float e[U][8], g[U][8];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    dst[k] = nullptr;
    const uint32_t u = (part * U + k) * kThreads + threadIdx.x;
    if (u >= total) continue;
    const uint32_t tl = dm.per_token.div(u);
    uint32_t w = u - tl * dm.per_token.d;
    const int64_t t = t0 + tl;
    const TI* src;
    bool value = false;
    const uint32_t nx = a.Hx * dm.per_head.d, nk = a.Hk * dm.per_head.d;
    if (APPEND && w >= nx) {
      const int64_t slot = a.slots[t];
      if (slot < 0 || slot >= a.slot_count) continue;
      const int64_t page = slot >> a.page_shift;
      const int64_t row = slot - (page << a.page_shift);
      w -= nx;
      value = w >= nk;
      if (value) w -= nk;
      const FastDiv& by = value ? dm.per_value : dm.per_head;
      const uint32_t h = by.div(w);
      w -= h * by.d;
      src = value ? static_cast<const TI*>(a.v) + t * a.v_ts + h * a.v_hs
                  : static_cast<const TI*>(a.k) + t * a.k_ts + h * a.k_hs;
      dst[k] = static_cast<TO*>(value ? a.v_cache : a.k_cache) +
               (((page * a.Hk + h) << a.page_shift) + row) * a.D;
    } else {
      const uint32_t h = dm.per_head.div(w);
      w -= h * dm.per_head.d;
      src = static_cast<const TI*>(a.x) + t * a.x_ts + h * a.x_hs;
      dst[k] = static_cast<TO*>(a.y) + t * a.y_ts + h * a.y_hs;
    }
    int step;
    if (value) {
      angle[k] = -2;
      at0[k] = 16 * w;
      step = 8;
    } else if (static_cast<int>(w) < dm.rot_units) {
      const int p0 = w * VEC;
      angle[k] = tl * half + p0;
      at0[k] = a.adjacent ? 2 * p0 : p0;
      step = a.adjacent ? VEC : half;
    } else {
      angle[k] = -1;
      at0[k] = a.rot + dm.tail * (static_cast<int>(w) - dm.rot_units);
      step = VEC >= 4 ? VEC : dm.tail == 16 ? 8 : 0;
    }
    at1[k] = at0[k] + step;
    if (VEC < 4 && angle[k] == -1 && dm.tail == 16) {
      at0[k] = at0[k] < a.D - 8 ? at0[k] : a.D - 8;
      at1[k] = at1[k] < a.D - 8 ? at1[k] : a.D - 8;
    }
    if (at1[k] >= a.D) at1[k] = at0[k];
    if (angle[k] >= 0 || (VEC >= 4 && angle[k] == -1) || VEC == 8) {
      load_first<VEC>(src + at0[k], e[k]);
      load_first<VEC>(src + at1[k], g[k]);
    } else if (APPEND && angle[k] == -2) {
      load_first<8>(src + at0[k], e[k]);
      load_first<8>(src + at1[k], g[k]);
    } else if (VEC < 4 && dm.tail == 16) {
      load_first<8, 2 * sizeof(TI)>(src + at0[k], e[k]);
      load_first<8, 2 * sizeof(TI)>(src + at1[k], g[k]);
    } else if (VEC < 4) {
      load_first<2>(src + at0[k], e[k]);
    }
  }

  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = static_cast<int>(dm.pairs.div(i));
    const int p = i - t * half;
    int ax = 0;
    if (a.interleaved) {
      const int r = p % a.axes;
      ax = p / a.axes < a.section[r] ? r : 0;
    } else {
      int end = a.section[0];
      while (ax + 1 < a.axes && p >= end) end += a.section[++ax];
    }
    const int32_t pos = a.positions[ax * a.T + t0 + t];
    double turn = static_cast<double>(pos) * (a.freqs[p] * 0.15915494309189533577);
    turn -= rint(turn);
    float s, c;
    sincospif(2.0f * static_cast<float>(turn), &s, &c);
    table[i] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();

#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (dst[k] == nullptr) continue;
    if (angle[k] >= 0) {
      const float2* cs = table + angle[k];
      if (a.adjacent) {
        float z[2 * VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[i] = e[k][i], z[VEC + i] = g[k][i];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float2 r = cs[i];
          const float x0 = z[2 * i], x1 = z[2 * i + 1];
          z[2 * i] = x0 * r.x - x1 * r.y;
          z[2 * i + 1] = x1 * r.x + x0 * r.y;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[k][i] = z[i], g[k][i] = z[VEC + i];
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float2 r = cs[i];
          const float x0 = e[k][i], x1 = g[k][i];
          e[k][i] = x0 * r.x - x1 * r.y;
          g[k][i] = x1 * r.x + x0 * r.y;
        }
      }
    }
    if (angle[k] >= 0 || (VEC >= 4 && angle[k] == -1) || VEC == 8) {
      store_first<VEC>(dst[k] + at0[k], e[k]);
      store_first<VEC>(dst[k] + at1[k], g[k]);
    } else if (APPEND && angle[k] == -2) {
      store_first<8>(dst[k] + at0[k], e[k]);
      store_first<8>(dst[k] + at1[k], g[k]);
    } else if (VEC < 4 && dm.tail == 16) {
      store_first<8, 2 * sizeof(TO)>(dst[k] + at0[k], e[k]);
      store_first<8, 2 * sizeof(TO)>(dst[k] + at1[k], g[k]);
    } else if (VEC < 4) {
      store_first<2>(dst[k] + at0[k], e[k]);
    }
  }
}

template <typename TI, typename TO, int VEC, int U, bool APPEND>
hipError_t launch_units(const RopeArgs& a, Dims dm, hipStream_t s) {
  // A group's tokens fill its workgroup, or one token is shared by several;
  // the group's table has to fit.
  const int half = a.rot / 2;
  const int64_t per_token = dm.per_token.d;
  int64_t tokens = U * kThreads / per_token;
  if (tokens * half > kTable) tokens = kTable / half;
  if (tokens < 1) tokens = 1;
  dm.tokens = static_cast<int>(tokens);
  const int64_t parts = (tokens * per_token + U * kThreads - 1) / (U * kThreads);
  dm.parts = FastDiv(static_cast<uint32_t>(parts));
  const int64_t groups = (a.T + tokens - 1) / tokens;
  // a launch holds less than 2^32 threads
  const int64_t most = ((int64_t{1} << 32) / kThreads - 1) / parts;
  for (dm.first = 0; dm.first < groups; dm.first += most) {
    const int64_t n = groups - dm.first < most ? groups - dm.first : most;
    rope_kernel<TI, TO, VEC, U, APPEND>
        <<<dim3(static_cast<uint32_t>(n * parts)), kThreads, 0, s>>>(a, dm);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TI, typename TO, int VEC, bool APPEND>
hipError_t launch_vec(const RopeArgs& a, hipStream_t s) {
  Dims dm;
  const int half = a.rot / 2;
  dm.rot_units = half / VEC;
  const int tail = a.D - a.rot;
  dm.tail = VEC >= 4 ? 2 * VEC : tail >= 8 ? 16 : 2;
  const int per_head = dm.rot_units + (tail + dm.tail - 1) / dm.tail;
  const int per_value = (a.D + 15) / 16;
  const int64_t per_token = static_cast<int64_t>(a.Hx + (APPEND ? a.Hk : 0)) * per_head +
                            (APPEND ? static_cast<int64_t>(a.Hk) * per_value : 0);
  dm.per_head = FastDiv(per_head);
  dm.per_value = FastDiv(per_value);
  dm.per_token = FastDiv(static_cast<uint32_t>(per_token));
  dm.pairs = FastDiv(half > 0 ? half : 1);
  // One unit a thread until those fill the device, then two (four: 50, eight:
  // 55, a loop over the units 66 us where two take 48).
  return a.T * per_token < 256 * 8 * kThreads ? launch_units<TI, TO, VEC, 1, APPEND>(a, dm, s)
                                              : launch_units<TI, TO, VEC, 2, APPEND>(a, dm, s);
}

template <typename TI, typename TO, bool APPEND>
hipError_t launch_types(const RopeArgs& a, hipStream_t s) {
  // 16-byte accesses (for two-byte types) where the pairs of a head come in
  // eights, shorter ones in fours, twos and ones (8000 tokens of 32 heads of 80,
  // 20 of them rotated: 28 us; pairs and tails all by single elements 39 us)
  const int half = a.rot / 2;
  if (half % 8 == 0) return launch_vec<TI, TO, 8, APPEND>(a, s);
  if (half % 4 == 0) return launch_vec<TI, TO, 4, APPEND>(a, s);
  if (half % 2 == 0) return launch_vec<TI, TO, 2, APPEND>(a, s);
  return launch_vec<TI, TO, 1, APPEND>(a, s);
}

template <typename TI>
hipError_t launch_in(const RopeArgs& a, int out_dtype, hipStream_t s) {
  const bool append = a.slots != nullptr;
  switch (out_dtype) {
    case PQ1_BF16:
      if constexpr (!__is_same(TI, f16))
        if (append) return launch_types<TI, bf16, true>(a, s);
      return launch_types<TI, bf16, false>(a, s);
    case PQ1_F16:
      if constexpr (!__is_same(TI, bf16))
        if (append) return launch_types<TI, f16, true>(a, s);
      return launch_types<TI, f16, false>(a, s);
    default:
      return launch_types<TI, float, false>(a, s);
  }
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int in_dtype, int out_dtype, hipStream_t s) {
  switch (in_dtype) {
    case PQ1_BF16: return launch_in<bf16>(a, out_dtype, s);
    case PQ1_F16: return launch_in<f16>(a, out_dtype, s);
    default: return launch_in<float>(a, out_dtype, s);
  }
}

}  // namespace pq1
