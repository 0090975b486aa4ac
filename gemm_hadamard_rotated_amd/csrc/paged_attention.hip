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
//
// Bound: reading the cache; a call of one token by its fixed cost.  One token
// at 131071 keys (4 cache heads, D = 256): 98 us, 5.5 TB/s (a large copy
// reaches 5.1, a read alone 6.5); 64 tokens at 200 to 8000 keys: 231 us, 4.9
// TB/s; one token at 701 keys: 8 us for this kernel and 4.2 for the join, where
// an empty kernel takes 3.  What paid: as many workgroups as CUs (twice as
// many: 109 and 239 us), divisions by multiplication, lengths and page numbers
// through the scalar cache, runs of 16 keys as buffers whose end cuts off the
// keys past the last (31 KB of code became 13; one token 11.3 -> 8.0 us, drafts
// of 16 users in a window of 1024 keys 34 -> 22 us).  Two workgroups a CU where
// registers allow (D < 256; at 256 they spill: 240 -> 375 us).
// ---------------------------------------------------------------------------
struct FewGrid {
  int row_tiles, nsplit, chunk;
  FastDiv by_tiles, by_split, by_Hk;
};

// Where a tile's 32 keys are.  With pages of 16 keys or more (RUNS) they are
// two runs of 16 rows; else every lane keeps the page of one key.
struct TileAt {
  int64_t row[2];  // RUNS: cache rows of keys 0 and 16
  int keys[2];     // RUNS: keys there, none on a page that is not the cache's
  int page;        // not RUNS: page of key lane % 32, -1 for none
  uint32_t gone;   // visible keys on no page of the cache
};

template <bool RUNS>
__device__ __forceinline__ TileAt find_tile(const AttnArgs& a, const int32_t* table, int h, int j0,
                                            int hi, int lane) {
  TileAt t{};
  const int mask = (1 << a.page_shift) - 1;
  if constexpr (RUNS) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int j = j0 + 16 * e, p = j >> a.page_shift;
      int page = -1, keys = hi - j < 16 ? hi - j : 16;
      if (keys > 0 && p < a.max_pages) page = scalar_load(table, p);
      if (page < 0 || page >= a.pages) {
        if (keys > 0) t.gone |= (1u << keys) - 1 << 16 * e;
        page = keys = 0;
      }
      t.row[e] = ((static_cast<int64_t>(page) * a.Hk + h) << a.page_shift) + (j & mask);
      t.keys[e] = keys;
    }
  } else {
    const int j = j0 + (lane & 31);
    const int p = j >> a.page_shift;
    if (j < hi) {
      t.page = p < a.max_pages ? table[p] : -1;
      if (t.page >= a.pages) t.page = -1;
    }
    t.gone = static_cast<uint32_t>(__ballot(t.page < 0));
  }
  return t;
}

template <typename T, typename TO, int D, int RB, bool RUNS>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void few_rows_kernel(AttnArgs a, FewGrid fg,
                                                               float* part_o, float2* part_ml) {
  constexpr int NP = kParts<T, TO>;
  constexpr int DV = D >= 128 ? 8 : 4;     // dimensions of V a lane reads at once
  constexpr int CH = D / (16 * DV);        // such pieces of a V row
  constexpr int NO = CH * DV;
  constexpr int ROWS = 16 * RB;
  using VReg = __attribute__((ext_vector_type(DV / 2))) uint32_t;
  __shared__ __attribute__((aligned(16))) float sum_o[kWaves][16][D + 4];
  __shared__ float sum_m[kWaves][16], sum_l[kWaves][16];
  __shared__ int odd_of[kWaves];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const uint32_t id0 = fg.by_split.div(blockIdx.x), split = blockIdx.x - id0 * fg.by_split.d;
  const uint32_t id1 = fg.by_tiles.div(id0), rt = id0 - id1 * fg.by_tiles.d;
  const uint32_t b = fg.by_Hk.div(id1);
  const int h = id1 - b * fg.by_Hk.d;
  const Seq s = load_seq(a, b);
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int rows = s.n * a.G;
  const int Hq = a.Hk * a.G;

  for (int64_t r0 = static_cast<int64_t>(rt) * ROWS; r0 < rows;
       r0 += static_cast<int64_t>(fg.row_tiles) * ROWS) {
    const Parts pt = split_keys(a, s, static_cast<int>(r0), ROWS, fg.chunk, fg.nsplit);
    const int64_t from = pt.start + static_cast<int64_t>(split) * pt.chunk;
    if (split > 0 && from >= pt.hi) continue;
    const int k0 = static_cast<int>(from);
    const int k1 = pt.hi - k0 < pt.chunk ? pt.hi : k0 + pt.chunk;
    // rows of one token see the same keys
    const bool one_token = pt.lo == pt.lo_max && pt.hi == pt.hi_min;
    bool odd_values = false;  // infinities or NaN were taken out of V

    U4 q[RB][D / 32];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = static_cast<int>(r0) + 16 * rb + col;
      const int i = a.by_G.div(r);
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
    auto run_of = [&](const void* cache, const TileAt& t, int e) {
      return __builtin_amdgcn_make_buffer_rsrc(
          const_cast<T*>(static_cast<const T*>(cache) + t.row[e] * D), 0, t.keys[e] * D * 2,
          0x00020000);
    };
    auto row_of = [&](const TileAt& t, int j0, int key) {
      const int page = __shfl(t.page, key);
      return ((static_cast<int64_t>(page < 0 ? 0 : page) * a.Hk + h) << a.page_shift) +
             ((j0 + key) & ((1 << a.page_shift) - 1));
    };
    // Keys past the last read as zeros (RUNS) or as some row of the cache.
    auto load_k = [&](const TileAt& t, int j0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (RUNS) {
          const auto run = run_of(a.k_cache, t, e);
#pragma unroll
          for (int d = 0; d < D / 32; ++d)
            kr[e][d] =
                __builtin_amdgcn_raw_buffer_load_b128(run, (col * D + 8 * g + 32 * d) * 2, 0, 0);
        } else {
          const T* src = static_cast<const T*>(a.k_cache) + row_of(t, j0, 16 * e + col) * D + 8 * g;
#pragma unroll
          for (int d = 0; d < D / 32; ++d) kr[e][d] = *reinterpret_cast<const U4*>(src + 32 * d);
        }
      }
    };
    auto load_v = [&](const TileAt& t, int j0) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (RUNS) {
          const auto run = run_of(a.v_cache, t, e >> 2);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int at = (((e & 3) + 4 * g) * D + DV * col + 16 * DV * c) * 2;
            if constexpr (DV == 8)
              vr[e][c] = __builtin_amdgcn_raw_buffer_load_b128(run, at, 0, 0);
            else
              vr[e][c] = __builtin_amdgcn_raw_buffer_load_b64(run, at, 0, 0);
          }
        } else {
          const T* src = static_cast<const T*>(a.v_cache) +
                         row_of(t, j0, 12 * (e >> 2) + e + 4 * g) * D + DV * col;
#pragma unroll
          for (int c = 0; c < CH; ++c) vr[e][c] = *reinterpret_cast<const VReg*>(src + 16 * DV * c);
        }
      }
    };

    int j0 = k0 + kKeys * wave;
    TileAt at{};
    if (j0 < k1) {
      at = find_tile<RUNS>(a, table, h, j0, pt.hi, lane);
      load_k(at, j0);
    }
#pragma unroll 1
    for (; j0 < k1; j0 += kKeys * kWaves) {
      load_v(at, j0);
      // past the last tile nothing is fetched, or the same tile again
      const int jn = j0 + kKeys * kWaves;
      const TileAt next = find_tile<RUNS>(a, table, h, RUNS || jn < k1 ? jn : j0,
                                          RUNS ? k1 : pt.hi, lane);

      F4 sc[RB][2];
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
            sc[rb][e] = mfma16(kr[e][d], q[rb][d], d == 0 ? F4{0, 0, 0, 0} : sc[rb][e], T{});
      load_k(next, RUNS || jn < k1 ? jn : j0);

      if (is_edge(pt, j0, kKeys, at.gone != 0)) {
        // Values no row sees become zero, and where rows see different keys
        // infinities and NaN among the others too (put_back).
        if (!RUNS || !one_token || j0 < pt.lo) {
          const int lo = pt.lo - j0 - 4 * g, hi = pt.hi - j0 - 4 * g;
          const uint32_t gone = at.gone >> 4 * g;
          uint32_t odd = 0;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int key = 12 * (e >> 2) + e;
            const uint32_t seen =
                key >= lo && key < hi && (gone >> key & 1) == 0 ? 0xffffffffu : 0u;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int w = 0; w < DV / 2; ++w) {
                vr[e][c][w] &= seen;
                odd |= odd_bits<T>(vr[e][c][w]);
              }
          }
          if (!one_token && __any((odd & kOdd) != 0)) {
            odd_values = true;
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
              for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int w = 0; w < DV / 2; ++w) vr[e][c][w] = finite_or_zero<T>(vr[e][c][w]);
          }
        }
        const uint32_t gone = at.gone >> 4 * g;
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          const int r = static_cast<int>(r0) + 16 * rb + col;
          int lo = 0, hi = 0;
          if (r < rows) visible(a, s, a.by_G.div(r), &lo, &hi);
          lo -= j0 + 4 * g;
          hi -= j0 + 4 * g;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int key = 16 * e + i;
              sc[rb][e][i] = key < lo || key >= hi    ? kNegInf
                             : (gone >> key & 1) != 0 ? __builtin_nanf("")
                                                      : sc[rb][e][i];
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
        top = max_groups(top);
        if (__any(top * a.scale_log2 > m[rb] + kLag)) {
          const float up = fmaxf(m[rb], scaled_max(top, a.scale_log2));
          const float keep = m[rb] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[rb] - up);
          m[rb] = up;
          l[rb] *= keep;
#pragma unroll
          for (int n = 0; n < NO; ++n) o[rb][n] *= keep;
        }
        float shift = m[rb] == kNegInf ? 0.0f : kUp<T> - m[rb];
        if (__any(is_far(m[rb]))) {
          const bool far = is_far(m[rb]);
          shift = far ? kUp<T> : shift;
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sc[rb][e][i] =
                  far ? near_score(sc[rb][e][i], a.scale_log2, m[rb]) : sc[rb][e][i];
        }
        float p[8];
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[4 * e + i] = __builtin_amdgcn_exp2f(fmaf(sc[rb][e][i], a.scale_log2, shift));
            if constexpr (!kSumParts<T, NP>) l[rb] += p[4 * e + i];
          }
        split_probs<T, NP>(p, pr[rb]);
        if constexpr (kSumParts<T, NP>) {
#pragma unroll
          for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int w = 0; w < 4; ++w) l[rb] = add_pair<T>(pr[rb][n][w], l[rb]);
        }
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
      at = next;
    }

    // Join the four waves' sums, 16 rows at a time.
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const float ls = sum_groups(l[rb]);
      if (rb > 0) __syncthreads();
      if (g == 0) {
        sum_m[wave][col] = m[rb];
        sum_l[wave][col] = ls;
      }
      if (lane == 0) odd_of[wave] = odd_values;
      __syncthreads();
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, sum_m[w][col]);
      // a wave without a finite score still hands on its NaN
      const float f = m[rb] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(m[rb] - top);
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
        const int i = a.by_G.div(r);
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
    // Read before the barrier: past it the next rows' sums and flags are written.
    const bool put = !one_token && (odd_of[0] | odd_of[1] | odd_of[2] | odd_of[3]);
    __syncthreads();
    if (put) {
      put_back<T, TO>(a, s, table, h, pt, k0, k1, kKeys, r0, ROWS, 64 * kWaves, split,
                      fg.nsplit > 1, part_o);
      __syncthreads();
    }
  }
}

// Joins the parts of every row: o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// eight parts at a time with all their loads in flight, under a running
// maximum.  WPR waves share a row (each takes every WPR-th eight), D / 64
// dimensions a lane.
template <typename TO, int D, int WPR>
__global__ __launch_bounds__(256) void join_kernel(AttnArgs a, FewGrid fg, int tile_rows,
                                                   int tokens, const float* part_o,
                                                   const float2* part_ml) {
  constexpr int N = D / 64, RPW = 4 / WPR, BATCH = 8;
  __shared__ float sum_o[WPR > 1 ? 4 : 1][D];
  __shared__ float sum_m[4], sum_l[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int Hq = a.Hk * a.G;
  const uint32_t groups = (Hq + RPW - 1) / RPW;
  const uint32_t id = blockIdx.x / groups;
  const int hq = (blockIdx.x - id * groups) * RPW + wave / WPR;
  const uint32_t b = id / static_cast<uint32_t>(tokens);
  const Seq s = load_seq(a, b);
  if (hq >= Hq) return;  // (whole workgroups where waves share a row)
  const int64_t stride = a.T * Hq;
  const int hq_in = hq - static_cast<int>(a.by_G.div(hq)) * a.G;
  for (int i = id - b * tokens; i < s.n; i += tokens) {
    const int r = i * a.G + hq_in;
    // a tile's rows are a power of two
    const Parts pt = split_keys(a, s, r & -tile_rows, tile_rows, fg.chunk, fg.nsplit);
    const int count = pt.count();
    int lo, hi;
    visible(a, s, i, &lo, &hi);
    const int64_t row = (s.q0 + i) * Hq + hq;
    float acc[N] = {}, l = 0.0f, top = kNegInf;
    for (int p0 = wave % WPR * BATCH; p0 < count; p0 += WPR * BATCH) {
      float2 ml[BATCH];
      float x[BATCH][N], up = top;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        const int p = p0 + k < count ? p0 + k : count - 1;
        ml[k] = part_ml[p * stride + row];
        load_wide(part_o + (p * stride + row) * D + N * lane, x[k]);
      }
#pragma unroll
      for (int k = 1; k < BATCH; ++k) {  // past the last part: nothing
        const bool part = p0 + k < count;
        ml[k].x = part ? ml[k].x : kNegInf;
        ml[k].y = part ? ml[k].y : 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) x[k][n] = part ? x[k][n] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < BATCH; ++k) up = fmaxf(up, ml[k].x);
      const float keep = top == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(top - up);
      top = up;
      l *= keep;
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] *= keep;
#pragma unroll
      for (int k = 0; k < BATCH; ++k) {
        // a part without a finite score still hands on its NaN
        const float w = ml[k].x == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(ml[k].x - top);
        l += w * ml[k].y;
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] += w * x[k][n];
      }
    }
    if constexpr (WPR > 1) {
      if (lane == 0) sum_m[wave] = top, sum_l[wave] = l;
      store_wide(&sum_o[wave][N * lane], acc);
      __syncthreads();
      if (wave == 0) {
        top = kNegInf;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, sum_m[w]);
        l = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] = 0.0f;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float f = sum_m[w] == kNegInf ? 1.0f : __builtin_amdgcn_exp2f(sum_m[w] - top);
          float x[N];
          load_wide(&sum_o[w][N * lane], x);
          l += f * sum_l[w];
#pragma unroll
          for (int n = 0; n < N; ++n) acc[n] += f * x[n];
        }
      }
    }
    if (wave % WPR == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] = hi > lo ? acc[n] / l : 0.0f;
      store_wide(static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs + N * lane, acc);
    }
    if constexpr (WPR > 1) __syncthreads();
  }
}

FewGrid grid_of(const AttnPlan& plan, const AttnArgs& a) {
  return {static_cast<int>(plan.row_tiles), plan.nsplit, plan.chunk,
          FastDiv(static_cast<uint32_t>(plan.row_tiles)),
          FastDiv(static_cast<uint32_t>(plan.nsplit)), FastDiv(static_cast<uint32_t>(a.Hk))};
}

template <typename T, typename TO, int D, int RB>
hipError_t launch_few(const AttnPlan& plan, const AttnArgs& a, void* workspace, hipStream_t s) {
  const FewGrid fg = grid_of(plan, a);
  float* part_o = static_cast<float*>(workspace);
  float2* part_ml =
      reinterpret_cast<float2*>(part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  const dim3 grid(static_cast<uint32_t>(a.B * a.Hk * plan.row_tiles * plan.nsplit));
  // pages of half a key tile or more are read as runs
  if (a.page_shift >= 4)
    few_rows_kernel<T, TO, D, RB, true><<<grid, 64 * kWaves, 0, s>>>(a, fg, part_o, part_ml);
  else
    few_rows_kernel<T, TO, D, RB, false><<<grid, 64 * kWaves, 0, s>>>(a, fg, part_o, part_ml);
  return hipGetLastError();
}

template <typename TO, int D, int WPR>
hipError_t launch_join_waves(const AttnPlan& plan, const AttnArgs& a, void* workspace,
                             hipStream_t s) {
  const FewGrid fg = grid_of(plan, a);
  const float* part_o = static_cast<const float*>(workspace);
  const float2* part_ml = reinterpret_cast<const float2*>(
      part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  constexpr int RPW = 4 / WPR;
  const int64_t groups = (a.Hk * a.G + RPW - 1) / RPW;
  const int64_t most = ((int64_t{1} << 24) - 1) / (a.B * groups);  // below 2^32 threads
  const int64_t tokens = plan.tokens < most ? plan.tokens : most;
  join_kernel<TO, D, WPR><<<dim3(static_cast<uint32_t>(a.B * tokens * groups)), 256, 0, s>>>(
      a, fg, plan.tile_rows, static_cast<int>(tokens), part_o, part_ml);
  return hipGetLastError();
}

template <typename TO, int D>
hipError_t launch_join(const AttnPlan& plan, const AttnArgs& a, void* workspace, hipStream_t s) {
  // four waves to a row where there are several batches (64 parts: 9.1 -> 5.4 us)
  return plan.nsplit > 8 ? launch_join_waves<TO, D, 4>(plan, a, workspace, s)
                         : launch_join_waves<TO, D, 1>(plan, a, workspace, s);
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

}  // namespace

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
