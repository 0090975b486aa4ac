// Attention of new tokens over a paged key/value cache (pq1_paged_attention).
//
// Row (b, i, h) sees keys [lo, hi) of its sequence and computes
//   o = sum_j 2^(c q.k_j - m) v_j / sum_j 2^(c q.k_j - m),   c = scale log2(e),
// with a running maximum m over tiles of keys, so that one pass over the
// cache does: a tile with a larger maximum scales what was summed so far.
#include "attn_tiles.h"

namespace pq1 {

namespace {

// ---------------------------------------------------------------------------
// Few rows: 16 RB rows of one (sequence, cache head) and one part of its keys
// for a workgroup of four waves.
//
// Each wave takes every fourth tile of 32 keys straight into registers.  Both
// products are taken transposed: S^T = K Q^T leaves a lane the scores of one
// row (lane % 16) for keys 4g + i and 16 + 4g + i (g = lane / 16), and these
// are, as they stand, the operand of O^T = V^T P^T if V's rows are read in
// the same key order.  So the softmax is lane-local but for two exchanges,
// and neither P nor V goes through LDS: a lane reads 8 keys x 8 dimensions of
// V, and picking one dimension of the 8 keys is a byte permute of registers.
// ---------------------------------------------------------------------------
constexpr int kKeys = 32;   // keys of a tile
constexpr int kWaves = 4;

struct FewGrid {
  int row_tiles, nsplit, chunk;
};

// Rows of the cache that hold a tile's keys.  With pages of at least a tile
// (UNI) they are one run; else every lane keeps the page of one key.
struct TileAt {
  int64_t row;  // UNI: cache row of the first key
  int page;     // not UNI: page of key lane % 32
  bool bad;     // a key some row sees lies on no page of the cache
};

template <bool UNI>
__device__ __forceinline__ TileAt find_tile(const AttnArgs& a, const int32_t* table, int h, int j0,
                                            int hi, int lane) {
  TileAt t;
  const int mask = (1 << a.page_shift) - 1;
  if (UNI) {
    const int p = j0 >> a.page_shift;
    const int page = p < a.max_pages ? table[p] : -1;
    t.bad = page < 0 || page >= a.pages;
    t.row = ((static_cast<int64_t>(t.bad ? 0 : page) * a.Hk + h) << a.page_shift) + (j0 & mask);
    t.page = 0;
  } else {
    const int j = j0 + (lane & 31);
    const int p = j >> a.page_shift;
    int page = 0;
    bool bad = false;
    if (j < hi) {
      page = p < a.max_pages ? table[p] : -1;
      bad = page < 0 || page >= a.pages;
    }
    t.page = bad ? -1 : page;
    t.bad = __any(bad);
    t.row = 0;
  }
  return t;
}

template <typename T, typename TO, int D, int RB, bool UNI>
__global__ __launch_bounds__(64 * kWaves) void few_rows_kernel(AttnArgs a, FewGrid fg,
                                                               float* part_o, float2* part_ml) {
  constexpr int NP = kParts<T, TO>;
  constexpr int DV = D >= 128 ? 8 : 4;     // dimensions of V a lane reads at once
  constexpr int CH = D / (16 * DV);        // such pieces of a V row
  constexpr int NO = CH * DV;
  constexpr int ROWS = 16 * RB;
  using VReg = __attribute__((ext_vector_type(DV / 2))) uint32_t;
  __shared__ __attribute__((aligned(16))) float sum_o[kWaves][16][D + 4];
  __shared__ float sum_m[kWaves][16], sum_l[kWaves][16];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, g = lane >> 4;
  uint32_t id = blockIdx.x;
  const int split = id % fg.nsplit;
  id /= fg.nsplit;
  const int rt = id % fg.row_tiles;
  id /= fg.row_tiles;
  const int h = id % a.Hk;
  const int b = id / a.Hk;
  const Seq s = load_seq(a, b);
  const int32_t* table = a.table + b * a.max_pages;
  const int rows = s.n * a.G;
  const int Hq = a.Hk * a.G;

  for (int64_t r0 = static_cast<int64_t>(rt) * ROWS; r0 < rows;
       r0 += static_cast<int64_t>(fg.row_tiles) * ROWS) {
    const Parts pt = split_keys(a, s, static_cast<int>(r0), ROWS, fg.chunk, fg.nsplit);
    if (split > 0 && split >= pt.count) continue;
    const int k0 = pt.start + split * pt.chunk;
    const int k1 = pt.hi - k0 < pt.chunk ? pt.hi : k0 + pt.chunk;
    const bool one_token = r0 / a.G == ((r0 + ROWS < rows ? r0 + ROWS : rows) - 1) / a.G;

    int lo[RB], hi[RB];
    U4 q[RB][D / 32];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = static_cast<int>(r0) + 16 * rb + col;
      lo[rb] = hi[rb] = 0;
      const int i = r / a.G;
      if (r < rows) visible(a, s, i, &lo[rb], &hi[rb]);
      const T* src = static_cast<const T*>(a.q) + (s.q0 + i) * a.q_ts +
                     (h * a.G + r - i * a.G) * a.q_hs + 8 * g;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
        q[rb][d] = r < rows ? *reinterpret_cast<const U4*>(src + 32 * d) : U4{0, 0, 0, 0};
    }
    F4 o[RB][NO];
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      m[rb] = kNegInf;
      l[rb] = 0.0f;
#pragma unroll
      for (int n = 0; n < NO; ++n) o[rb][n] = F4{0, 0, 0, 0};
    }

    U4 kr[2][D / 32];
    VReg vr[8][CH];
    // Past the last tile nothing is fetched: a buffer of no records, or the
    // wave's last tile again.
    auto load_k = [&](const TileAt& t, int j0) {
      if constexpr (UNI) {
        const int left = j0 < k1 ? pt.hi - j0 : 0;
        const auto buf = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T*>(static_cast<const T*>(a.k_cache) + t.row * D), 0,
            (left < kKeys ? left : kKeys) * D * 2, 0x00027000);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int d = 0; d < D / 32; ++d)
            kr[e][d] = __builtin_amdgcn_raw_buffer_load_b128(
                buf, ((16 * e + col) * D + 8 * g + 32 * d) * 2, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = 16 * e + col;
          const int page = __shfl(t.page, key);
          const int64_t row =
              ((static_cast<int64_t>(page < 0 ? 0 : page) * a.Hk + h) << a.page_shift) +
              ((j0 + key) & ((1 << a.page_shift) - 1));
          const T* src = static_cast<const T*>(a.k_cache) + row * D + 8 * g;
#pragma unroll
          for (int d = 0; d < D / 32; ++d)
            kr[e][d] = *reinterpret_cast<const U4*>(src + 32 * d);
        }
      }
    };
    auto load_v = [&](const TileAt& t, int j0) {
      if constexpr (UNI) {
        const int left = pt.hi - j0;
        const auto buf = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T*>(static_cast<const T*>(a.v_cache) + t.row * D), 0,
            (left < kKeys ? left : kKeys) * D * 2, 0x00027000);
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int at = ((12 * (e >> 2) + e + 4 * g) * D + DV * col + 16 * DV * c) * 2;
            if constexpr (DV == 8)
              vr[e][c] = __builtin_amdgcn_raw_buffer_load_b128(buf, at, 0, 0);
            else
              vr[e][c] = __builtin_amdgcn_raw_buffer_load_b64(buf, at, 0, 0);
          }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = 12 * (e >> 2) + e + 4 * g;
          const int page = __shfl(t.page, key);
          const int64_t row =
              ((static_cast<int64_t>(page < 0 ? 0 : page) * a.Hk + h) << a.page_shift) +
              ((j0 + key) & ((1 << a.page_shift) - 1));
          const T* src = static_cast<const T*>(a.v_cache) + row * D + DV * col;
#pragma unroll
          for (int c = 0; c < CH; ++c)
            vr[e][c] = *reinterpret_cast<const VReg*>(src + 16 * DV * c);
        }
      }
    };

    int j0 = k0 + kKeys * wave;
    TileAt at{};
    if (j0 < k1) {
      at = find_tile<UNI>(a, table, h, j0, pt.hi, lane);
      load_k(at, j0);
    }
    for (; j0 < k1; j0 += kKeys * kWaves) {
      load_v(at, j0);
      const int jn = j0 + kKeys * kWaves;
      TileAt next = at;
      if (jn < k1) next = find_tile<UNI>(a, table, h, jn, pt.hi, lane);

      F4 sc[RB][2];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          sc[rb][e] = F4{0, 0, 0, 0};
#pragma unroll
          for (int d = 0; d < D / 32; ++d)
            sc[rb][e] = mfma16(kr[e][d], q[rb][d], sc[rb][e], T{});
        }
      load_k(next, jn < k1 ? jn : UNI ? k1 : j0);

      // A tile that not every row sees whole, or with a page missing
      const bool edge = j0 < pt.lo_max || j0 + kKeys > pt.hi_min || at.bad;
      bool patch = false;  // rows add this tile's infinities and NaN one by one
      if (edge) {
        bool odd = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = 12 * (e >> 2) + e + 4 * g;
          const bool gone = UNI ? at.bad : __shfl(at.page, key) < 0;
          const bool seen = j0 + key >= pt.lo && j0 + key < pt.hi && !gone;
#pragma unroll
          for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int w = 0; w < DV / 2; ++w) {
              vr[e][c][w] = seen ? vr[e][c][w] : 0u;
              odd |= not_finite<T>(vr[e][c][w]);
            }
        }
        patch = __any(odd) && !one_token;
        if (patch) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int w = 0; w < DV / 2; ++w) vr[e][c][w] = finite_or_zero<T>(vr[e][c][w]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 16 * e + 4 * g + i;
            const bool gone = UNI ? at.bad : __shfl(at.page, key) < 0;
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
              const bool seen = j0 + key >= lo[rb] && j0 + key < hi[rb];
              sc[rb][e][i] = !seen ? kNegInf : gone ? __builtin_nanf("") : sc[rb][e][i];
            }
          }
      }

      U4 pr[RB][NP];
#pragma unroll
      for (int rb = 0; rb < RB; ++rb) {
        float top = sc[rb][0][0];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[rb][e][i]);
        top = max_groups(top) * a.scale_log2;
        if (__any(top > m[rb] + kLag)) {
          const float up = fmaxf(m[rb], top);
          const float keep = m[rb] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[rb] - up);
          m[rb] = up;
          l[rb] *= keep;
#pragma unroll
          for (int n = 0; n < NO; ++n) o[rb][n] *= keep;
        }
        const float shift = m[rb] == kNegInf ? 0.0f : kUp - m[rb];
        float p[8];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[4 * e + i] = __builtin_amdgcn_exp2f(fmaf(sc[rb][e][i], a.scale_log2, shift));
            l[rb] += p[4 * e + i];
          }
        split_probs<T, NP>(p, pr[rb]);
      }
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int w = 0; w < DV / 2; ++w)
#pragma unroll
          for (int z = 0; z < 2; ++z) {  // dimension 2w + z of the lane's DV
            U4 f;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              f[e] = __builtin_amdgcn_perm(vr[2 * e + 1][c][w], vr[2 * e][c][w],
                                           z ? 0x07060302u : 0x05040100u);
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
#pragma unroll
              for (int n = NP - 1; n >= 0; --n)
                o[rb][c * DV + 2 * w + z] =
                    mfma16(f, pr[rb][n], o[rb][c * DV + 2 * w + z], T{});
          }
      if (patch) {
        for (int key = 0; key < kKeys; ++key) {
          const int page = UNI ? 0 : __shfl(at.page, key);
          const int64_t row =
              UNI ? at.row + key
                  : ((static_cast<int64_t>(page) * a.Hk + h) << a.page_shift) +
                        ((j0 + key) & ((1 << a.page_shift) - 1));
          if (j0 + key >= pt.hi || page < 0 || (UNI && at.bad)) continue;
          const T* src = static_cast<const T*>(a.v_cache) + row * D;
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            if (j0 + key >= lo[rb] && j0 + key < hi[rb]) {
#pragma unroll
              for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int z = 0; z < DV; ++z)
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float x = static_cast<float>(src[16 * DV * c + DV * (4 * g + i) + z]);
                    if (!__builtin_isfinite(x)) o[rb][c * DV + z][i] += x;
                  }
            }
        }
      }
      at = next;
    }

    // Join the four waves' sums, 16 rows at a time.
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const float ls = sum_groups(l[rb]);
      __syncthreads();
      if (g == 0) {
        sum_m[wave][col] = m[rb];
        sum_l[wave][col] = ls;
      }
      __syncthreads();
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sum_m[w][col]);
      const float keep = m[rb] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[rb] - top);
      // a wave without a finite score still hands on its NaN
      const float f = m[rb] == kNegInf ? 1.0f : keep;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int z = 0; z < DV; z += 4) {
            const int n = c * DV + z;
            *reinterpret_cast<F4*>(&sum_o[wave][col][16 * DV * c + DV * (4 * g + i) + z]) =
                F4{o[rb][n][i], o[rb][n + 1][i], o[rb][n + 2][i], o[rb][n + 3][i]} * f;
          }
      __syncthreads();
      for (int e = threadIdx.x; e < 16 * D / 4; e += 64 * kWaves) {
        const int row = e / (D / 4), d = 4 * (e - row * (D / 4));
        const int r = static_cast<int>(r0) + 16 * rb + row;
        if (r >= rows) continue;
        F4 x = F4{0, 0, 0, 0};
        float mx = kNegInf, lx = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) mx = fmaxf(mx, sum_m[w][row]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float mw = sum_m[w][row];
          lx += sum_l[w][row] * (mw == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(mw - mx));
          x += *reinterpret_cast<const F4*>(&sum_o[w][row][d]);
        }
        const int i = r / a.G;
        const int hq = h * a.G + r - i * a.G;
        if (fg.nsplit > 1) {
          const int64_t at_row = static_cast<int64_t>(split) * a.T * Hq + (s.q0 + i) * Hq + hq;
          *reinterpret_cast<F4*>(part_o + at_row * D + d) = x;
          if (d == 0) part_ml[at_row] = make_float2(mx, lx);
        } else {
          int rl, rh;
          visible(a, s, i, &rl, &rh);
          float y[4];
#pragma unroll
          for (int n = 0; n < 4; ++n) y[n] = rh > rl ? x[n] / lx : 0.0f;
          store_wide(static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs + d, y);
        }
      }
    }
    __syncthreads();
  }
}

// Joins the parts of every row: o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p.
// One wave per row, D / 64 dimensions a lane.
template <typename TO, int D>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, FewGrid fg, int tile_rows,
                                                   int tokens, const float* part_o,
                                                   const float2* part_ml) {
  constexpr int N = D / 64;
  const int lane = threadIdx.x & 63;
  const int Hq = a.Hk * a.G;
  const int heads4 = (Hq + 3) / 4;
  uint32_t id = blockIdx.x;
  const int hq = (id % heads4) * 4 + (threadIdx.x >> 6);
  id /= heads4;
  const int b = id / tokens;
  const Seq s = load_seq(a, b);
  if (hq >= Hq) return;
  const int64_t stride = a.T * Hq;
  for (int i = id % tokens; i < s.n; i += tokens) {
    const int r = i * a.G + hq % a.G;
    const Parts pt = split_keys(a, s, r / tile_rows * tile_rows, tile_rows, fg.chunk, fg.nsplit);
    int lo, hi;
    visible(a, s, i, &lo, &hi);
    const int64_t row = (s.q0 + i) * Hq + hq;
    float top = kNegInf;
    for (int p = lane; p < pt.count; p += 64) top = fmaxf(top, part_ml[p * stride + row].x);
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    float acc[N] = {}, l = 0.0f;
#pragma unroll 8
    for (int p = 0; p < pt.count; ++p) {
      const float2 ml = part_ml[p * stride + row];
      const float w = ml.x == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(ml.x - top);
      float x[N];
      load_wide(part_o + (p * stride + row) * D + N * lane, x);
      l += w * ml.y;
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] += w * x[n];
    }
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = hi > lo ? acc[n] / l : 0.0f;
    store_wide(static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs + N * lane, acc);
  }
}

template <typename T, typename TO, int D, int RB>
hipError_t launch_few(const AttnPlan& plan, const AttnArgs& a, void* workspace, hipStream_t s) {
  const FewGrid fg{static_cast<int>(plan.row_tiles), plan.nsplit, plan.chunk};
  float* part_o = static_cast<float*>(workspace);
  float2* part_ml =
      reinterpret_cast<float2*>(part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  const dim3 grid(static_cast<uint32_t>(a.B * a.Hk * plan.row_tiles * plan.nsplit));
  // pages of a whole key tile or more are read as one run
  if (a.page_shift >= 5)
    few_rows_kernel<T, TO, D, RB, true><<<grid, 64 * kWaves, 0, s>>>(a, fg, part_o, part_ml);
  else
    few_rows_kernel<T, TO, D, RB, false><<<grid, 64 * kWaves, 0, s>>>(a, fg, part_o, part_ml);
  return hipGetLastError();
}

template <typename TO, int D>
hipError_t launch_join(const AttnPlan& plan, const AttnArgs& a, void* workspace, hipStream_t s) {
  const FewGrid fg{static_cast<int>(plan.row_tiles), plan.nsplit, plan.chunk};
  const float* part_o = static_cast<const float*>(workspace);
  const float2* part_ml = reinterpret_cast<const float2*>(
      part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  const int64_t heads4 = (a.Hk * a.G + 3) / 4;
  const int64_t most = ((int64_t{1} << 24) - 1) / (a.B * heads4);  // below 2^32 threads
  const int64_t tokens = plan.tokens < most ? plan.tokens : most;
  join_kernel<TO, D><<<dim3(static_cast<uint32_t>(a.B * tokens * heads4)), 256, 0, s>>>(
      a, fg, plan.tile_rows, static_cast<int>(tokens), part_o, part_ml);
  return hipGetLastError();
}

template <typename T, typename TO, int D>
hipError_t launch_rows(const AttnPlan& plan, const AttnArgs& a, void* ws, hipStream_t s) {
  return plan.tile_rows == 16 ? launch_few<T, TO, D, 1>(plan, a, ws, s)
                              : launch_few<T, TO, D, 2>(plan, a, ws, s);
}

template <typename T, typename TO>
hipError_t launch_few_rows(const AttnPlan& plan, const AttnArgs& a, void* ws, hipStream_t s) {
  switch (a.D) {
    case 64: return launch_rows<T, TO, 64>(plan, a, ws, s);
    case 128: return launch_rows<T, TO, 128>(plan, a, ws, s);
    default: return launch_rows<T, TO, 256>(plan, a, ws, s);
  }
}

template <typename TO>
hipError_t join_parts(const AttnPlan& plan, const AttnArgs& a, void* ws, hipStream_t s) {
  switch (a.D) {
    case 64: return launch_join<TO, 64>(plan, a, ws, s);
    case 128: return launch_join<TO, 128>(plan, a, ws, s);
    default: return launch_join<TO, 256>(plan, a, ws, s);
  }
}

// A sequence's longest chunk has up to this many rows of a cache head in the
// few-rows kernel, more in the many-rows one.
constexpr int64_t kFewRows = 64;

}  // namespace

AttnPlan plan_attention(int64_t B, int64_t T, int Hq, int Hk, int D, int64_t max_q,
                        int64_t max_kv) {
  // A launch holds less than 2^32 threads.  Kernels walk on over rows that
  // their grid has no workgroup for, so a long chunk only costs balance.
  constexpr int64_t most = (int64_t{1} << 32) / (2 * kTileRows) - 1;
  constexpr int64_t cus = 256;
  AttnPlan p;
  if (B * Hk > most) return p;
  p.fits = true;
  p.tokens = max_q < 1 ? 1 : max_q < T ? max_q : T;
  const int64_t rows = p.tokens * (Hq / Hk);
  p.many = rows > kFewRows;
  p.tile_rows = p.many ? kTileRows : rows <= 16 ? 16 : 32;
  p.row_tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  if (p.row_tiles > most / (B * Hk)) p.row_tiles = most / (B * Hk);
  const int64_t kv = max_kv < 1 ? 1 : max_kv > 0x7fffffff ? 0x7fffffff : max_kv;
  const int64_t units = B * Hk * p.row_tiles;
  const int64_t step = kKeys * kWaves;
  int64_t parts = 1;
  if (p.many) {
    // One workgroup to a CU: as many parts as the device takes at once.  More,
    // to even out a last round, cost more than they give (192 workgroups of
    // 7168 keys: 396 us; in 4 parts, three full rounds: 407 us and 48 to join
    // them): idle CUs leave the others a higher clock.
    while (units * (parts + 1) <= cus && (parts + 1) * 256 <= kv) ++parts;
  } else if (units < 2 * cus) {
    // Enough workgroups for two on each CU, but no part shorter than one key
    // tile for each wave.
    parts = (2 * cus + units - 1) / units;
  }
  int64_t chunk = ((kv + parts - 1) / parts + step - 1) / step * step;
  p.chunk = chunk > 0x7fffff00 ? 0x7fffff00 : static_cast<int>(chunk);
  p.nsplit = static_cast<int>((kv + p.chunk - 1) / p.chunk);
  p.workspace_bytes = p.nsplit > 1 ? static_cast<size_t>(p.nsplit) * T * Hq * (D * 4 + 8) : 0;
  return p;
}

hipError_t launch_attention(const AttnPlan& plan, const AttnArgs& a, int dtype, int out_dtype,
                            void* workspace, hipStream_t s) {
  hipError_t e;
  if (plan.many)
    e = launch_many_rows(plan, a, dtype, out_dtype, workspace, s);
  else if (dtype == PQ1_BF16)
    e = out_dtype == PQ1_F32 ? launch_few_rows<bf16, float>(plan, a, workspace, s)
                             : launch_few_rows<bf16, bf16>(plan, a, workspace, s);
  else
    e = out_dtype == PQ1_F32 ? launch_few_rows<f16, float>(plan, a, workspace, s)
                             : launch_few_rows<f16, f16>(plan, a, workspace, s);
  if (e != hipSuccess || plan.nsplit == 1) return e;
  switch (out_dtype) {
    case PQ1_BF16: return join_parts<bf16>(plan, a, workspace, s);
    case PQ1_F16: return join_parts<f16>(plan, a, workspace, s);
    default: return join_parts<float>(plan, a, workspace, s);
  }
}

}  // namespace pq1
