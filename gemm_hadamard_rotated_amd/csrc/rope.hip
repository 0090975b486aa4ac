// Rotation by positions on one to four axes, alone (pq1_rope) or on the way
// into a paged cache (pq1_kv_append).
//
// Pair i of a head, (x0, x1), is turned by theta = p[a(i)] * freqs[i]:
//   y0 = x0 cos(theta) - x1 sin(theta),  y1 = x1 cos(theta) + x0 sin(theta).
// The angle depends on the token and the pair but not on the head, so a
// workgroup first puts (cos, sin) of its tokens' pairs into LDS and then
// streams all heads of those tokens past the table.  The angle is taken in
// turns in fp64 (p * f / 2 pi) and reduced there; only the reduced turn, at
// most half, is narrowed to fp32 for the sine and cosine.
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
  int rot_units;       // units of a head that hold pairs; the rest are copies
};

// A unit is VEC pairs of a head (VEC elements from each of two places: VEC
// low and VEC high elements, or 2 VEC neighbours), VEC copied elements of a
// head's tail, or 8 elements of a value head.
template <typename TI, typename TO, int VEC, bool APPEND>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a, Dims dm) {
  __shared__ float2 table[kTable];
  const uint32_t group = dm.parts.div(blockIdx.x);
  const uint32_t part = blockIdx.x - group * dm.parts.d;
  const int64_t t0 = static_cast<int64_t>(group) * dm.tokens;
  const int nt = static_cast<int>(a.T - t0 < dm.tokens ? a.T - t0 : dm.tokens);
  const int half = a.rot >> 1;

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

  const uint32_t total = static_cast<uint32_t>(nt) * dm.per_token.d;
  for (uint32_t u = part * kThreads + threadIdx.x; u < total; u += dm.parts.d * kThreads) {
    const uint32_t tl = dm.per_token.div(u);
    uint32_t w = u - tl * dm.per_token.d;
    const int64_t t = t0 + tl;
    const TI* src;
    TO* dst;
    int64_t slot = 0;
    if (APPEND) {
      const uint32_t nx = a.Hx * dm.per_head.d, nk = a.Hk * dm.per_head.d;
      if (w >= nx) {
        slot = a.slots[t];
        if (slot < 0 || slot >= a.slot_count) continue;
        const int64_t page = slot >> a.page_shift;
        const int64_t row = slot - (page << a.page_shift);
        if (w >= nx + nk) {  // a value: 8 elements, rounded
          w -= nx + nk;
          const uint32_t h = dm.per_value.div(w), c = w - h * dm.per_value.d;
          float e[8];
          load_wide(static_cast<const TI*>(a.v) + t * a.v_ts + h * a.v_hs + 8 * c, e);
          store_wide(static_cast<TO*>(a.v_cache) +
                         (((page * a.Hk + h) << a.page_shift) + row) * a.D + 8 * c,
                     e);
          continue;
        }
        w -= nx;
        const uint32_t h = dm.per_head.div(w);
        w -= h * dm.per_head.d;
        src = static_cast<const TI*>(a.k) + t * a.k_ts + h * a.k_hs;
        dst = static_cast<TO*>(a.k_cache) + (((page * a.Hk + h) << a.page_shift) + row) * a.D;
      } else {
        const uint32_t h = dm.per_head.div(w);
        w -= h * dm.per_head.d;
        src = static_cast<const TI*>(a.x) + t * a.x_ts + h * a.x_hs;
        dst = static_cast<TO*>(a.y) + t * a.y_ts + h * a.y_hs;
      }
    } else {
      const uint32_t h = dm.per_head.div(w);
      w -= h * dm.per_head.d;
      src = static_cast<const TI*>(a.x) + t * a.x_ts + h * a.x_hs;
      dst = static_cast<TO*>(a.y) + t * a.y_ts + h * a.y_hs;
    }
    if (static_cast<int>(w) < dm.rot_units) {
      const int p0 = w * VEC;
      const float2* cs = table + tl * half + p0;
      const int at0 = a.adjacent ? 2 * p0 : p0;
      const int at1 = a.adjacent ? 2 * p0 + VEC : p0 + half;
      float e[VEC], g[VEC], y0[VEC], y1[VEC];
      load_wide(src + at0, e);
      load_wide(src + at1, g);
      if (a.adjacent) {
        float z[2 * VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) z[i] = e[i], z[VEC + i] = g[i];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float2 r = cs[i];
          const float x0 = z[2 * i], x1 = z[2 * i + 1];
          z[2 * i] = x0 * r.x - x1 * r.y;
          z[2 * i + 1] = x1 * r.x + x0 * r.y;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) y0[i] = z[i], y1[i] = z[VEC + i];
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float2 r = cs[i];
          y0[i] = e[i] * r.x - g[i] * r.y;
          y1[i] = g[i] * r.x + e[i] * r.y;
        }
      }
      store_wide(dst + at0, y0);
      store_wide(dst + at1, y1);
    } else {
      const int at = a.rot + (static_cast<int>(w) - dm.rot_units) * VEC;
      float e[VEC];
      load_wide(src + at, e);
      store_wide(dst + at, e);
    }
  }
}

template <typename TI, typename TO, int VEC, bool APPEND>
hipError_t launch_vec(const RopeArgs& a, hipStream_t s) {
  Dims dm;
  const int half = a.rot / 2;
  dm.rot_units = half / VEC;
  const int per_head = dm.rot_units + (a.D - a.rot) / VEC;
  const int per_value = a.D / 8;
  const int64_t per_token = static_cast<int64_t>(a.Hx + (APPEND ? a.Hk : 0)) * per_head +
                            (APPEND ? static_cast<int64_t>(a.Hk) * per_value : 0);
  dm.per_head = FastDiv(per_head);
  dm.per_value = FastDiv(per_value);
  dm.per_token = FastDiv(static_cast<uint32_t>(per_token));
  dm.pairs = FastDiv(half > 0 ? half : 1);
  // A few units for each thread where there are enough to fill the device,
  // one otherwise; a group's table has to fit.
  const int64_t total = a.T * per_token;
  const int64_t want = total / (256 * 8 * kThreads);  // units a thread would get
  const int64_t each = want < 1 ? 1 : want > 8 ? 8 : want;
  int64_t tokens = each * kThreads / per_token;
  if (tokens * half > kTable) tokens = kTable / half;
  if (tokens < 1) tokens = 1;
  dm.tokens = static_cast<int>(tokens);
  const int64_t per_group = tokens * per_token;
  const int64_t parts = (per_group + each * kThreads - 1) / (each * kThreads);
  dm.parts = FastDiv(static_cast<uint32_t>(parts));
  const int64_t groups = (a.T + tokens - 1) / tokens;
  rope_kernel<TI, TO, VEC, APPEND>
      <<<dim3(static_cast<uint32_t>(groups * parts)), kThreads, 0, s>>>(a, dm);
  return hipGetLastError();
}

template <typename TI, typename TO, bool APPEND>
hipError_t launch_types(const RopeArgs& a, hipStream_t s) {
  // 16-byte accesses where the pairs of a head come in eights, 8-byte ones
  // (for two-byte types) in fours, else single elements
  const int half = a.rot / 2;
  if (half % 8 == 0) return launch_vec<TI, TO, 8, APPEND>(a, s);
  if (half % 4 == 0) return launch_vec<TI, TO, 4, APPEND>(a, s);
  return launch_vec<TI, TO, 1, APPEND>(a, s);
}

template <typename TI>
hipError_t launch_in(const RopeArgs& a, int out_dtype, hipStream_t s) {
  const bool append = a.slots != nullptr;
  switch (out_dtype) {
    case PQ1_BF16:
      return append ? launch_types<TI, bf16, true>(a, s) : launch_types<TI, bf16, false>(a, s);
    case PQ1_F16:
      return append ? launch_types<TI, f16, true>(a, s) : launch_types<TI, f16, false>(a, s);
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
