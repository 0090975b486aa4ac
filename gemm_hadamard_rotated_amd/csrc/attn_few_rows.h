// Kernels of attention over a paged cache for few rows, and the join of a call's
// parts (paged_attention.hip, paged_attention_sinks.hip, kv4_attention.hip).
//
// Row (b, i, h) sees some keys of its sequence and computes
//   o = sum_j 2^(c q.k_j - m) v_j / sum_j 2^(c q.k_j - m),   c = scale log2(e),
// with a running maximum m over tiles of keys, so that one pass over the
// cache does: a tile with a larger maximum scales what was summed so far.
#pragma once

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

// Four-bit caches (F = kFourBit) go the same way.  A lane's 16 bytes of a K row are
// the 32 codes of one scale: they make four operands, for which the queries are
// read in the same order.  Of V a lane reads D / 16 codes of each of its 8 keys.
// Both become pairs of T by one instruction for two codes, each used once.  64 tokens at
// 200 to 8000 keys, 4 heads, D = 256: 66 us and 5 to join, 4.5 TB/s of the codes and
// scales, vector instructions 42 % of the time and matrix ones 13; one token at 131070
// keys 42 us.  Queries kept in LDS and V a tile ahead were slower (80 -> 91 us).
//
// This is one workgroup's part: rows r0 .. of a tile, places [k0, k1) of its walk.
template <typename T, typename TO, int D, int RB, bool RUNS, CacheForm F, typename Out>
__device__ __forceinline__ void few_rows_part(const Args<F>& a, const Seq& s, const int32_t* table,
                                              int h, int rows, int64_t r0, const Parts& pt, int k0,
                                              int k1, const Out& out) {
  constexpr bool FOUR = F == kFourBit;
  constexpr int NP = kParts<T, TO>;
  // dimensions of V a lane reads at once
  constexpr int DV = FOUR ? D / 16 : D >= 128 ? 8 : 4;
  constexpr int CH = D / (16 * DV);        // such pieces of a V row
  constexpr int NO = CH * DV;
  constexpr int ROWS = 16 * RB;
  using VReg = __attribute__((ext_vector_type(FOUR ? 1 : DV / 2))) uint32_t;
  // 4-bit K: KC pieces of a row a lane reads, of KW words (8 codes, one operand) each
  constexpr int KW = D >= 128 ? 4 : 2, KC = FOUR ? D / (32 * KW) : 1;
  constexpr int VW = D == 256 ? 2 : 1;     // words of V for a key
  __shared__ __attribute__((aligned(16))) float sum_o[kWaves][16][D + 4];
  __shared__ float sum_m[kWaves][16], sum_l[kWaves][16];
  __shared__ int odd_of[kWaves];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  // rows of one token see the same keys
  const bool one_token = pt.lo == pt.lo_max && pt.hi == pt.hi_min;
  bool odd_values = false;  // infinities or NaN were taken out of V

  U4 q[RB][D / 32];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb) {
    const int r = static_cast<int>(r0) + 16 * rb + col;
    const int i = a.by_G.div(r);
    const T* src = static_cast<const T*>(a.q) + (s.q0 + i) * a.q_ts +
                   (h * a.G + r - i * a.G) * a.q_hs + (FOUR ? 8 * KW : 8) * g;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const int at = FOUR ? 32 * KW * (d / KW) + 8 * (d % KW) : 32 * d;
      q[rb][d] = r < rows ? *reinterpret_cast<const U4*>(src + at) : U4{0, 0, 0, 0};
    }
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

  U4 kr[2][FOUR ? KC : D / 32];
  uint32_t ks[2][KC];  // scale bytes
  VReg vr[8][FOUR ? VW : CH];
  uint32_t vs[8];
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
  // Rows of n bytes of a 4-bit cache's array, from the tile's key 16 e on.
  auto run4_of = [&](const void* array, const TileAt& t, int e, int n) {
    return __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(static_cast<const uint8_t*>(array) + t.row[e] * n), 0, t.keys[e] * n,
        0x00020000);
  };
  // Keys past the last read as zeros (RUNS) or as some row of the cache.  (Pieces by the
  // scalar offset: what comes of adding them up may order the loads otherwise than
  // the products want them, 236 us for 232 in a decode of 64 at D = 256.)
  auto load_k = [&](const TileAt& t, int j0) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if constexpr (FOUR) {
        // byte of a lane's piece in a row, and of its scale
        const int at = 4 * KW * g, sat = KW * g / 4;
        if constexpr (RUNS) {
          const auto run = run4_of(a.k_cache, t, e, D / 2);
          const auto srun = run4_of(a.k_scale, t, e, D / 32);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            if constexpr (KW == 4) {
              kr[e][c] =
                  __builtin_amdgcn_raw_buffer_load_b128(run, col * (D / 2) + at + 64 * c, 0, 0);
            } else {
              const U2 x = __builtin_amdgcn_raw_buffer_load_b64(run, col * (D / 2) + at, 0, 0);
              kr[e][c] = U4{x[0], x[1], 0, 0};
            }
            ks[e][c] = __builtin_amdgcn_raw_buffer_load_b8(srun, col * (D / 32) + sat + 4 * c, 0, 0);
          }
        } else {
          const int64_t row = row_of(t, j0, 16 * e + col);
          const uint8_t* src = static_cast<const uint8_t*>(a.k_cache) + row * (D / 2) + at;
          const uint8_t* ssrc = a.k_scale + row * (D / 32) + sat;
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            if constexpr (KW == 4) {
              kr[e][c] = *reinterpret_cast<const U4*>(src + 64 * c);
            } else {
              const U2 x = *reinterpret_cast<const U2*>(src);
              kr[e][c] = U4{x[0], x[1], 0, 0};
            }
            ks[e][c] = ssrc[4 * c];
          }
        }
      } else if constexpr (RUNS) {
        const auto run = run_of(a.k_cache, t, e);
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
          kr[e][d] =
              __builtin_amdgcn_raw_buffer_load_b128(run, (col * D + 8 * g) * 2, 64 * d, 0);
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
      if constexpr (FOUR) {
        const int at = D / 32 * col, sat = col * D / 512;
        if constexpr (RUNS) {
          const auto run = run4_of(a.v_cache, t, e >> 2, D / 2);
          const auto srun = run4_of(a.v_scale, t, e >> 2, D / 32);
          const int key = (e & 3) + 4 * g;
          if constexpr (D == 256) {
            const U2 x = __builtin_amdgcn_raw_buffer_load_b64(run, key * (D / 2) + at, 0, 0);
            vr[e][0][0] = x[0];
            vr[e][VW - 1][0] = x[1];
          } else if constexpr (D == 128) {
            vr[e][0][0] = __builtin_amdgcn_raw_buffer_load_b32(run, key * (D / 2) + at, 0, 0);
          } else {
            vr[e][0][0] = __builtin_amdgcn_raw_buffer_load_b16(run, key * (D / 2) + at, 0, 0);
          }
          vs[e] = __builtin_amdgcn_raw_buffer_load_b8(srun, key * (D / 32) + sat, 0, 0);
        } else {
          const int64_t row = row_of(t, j0, 12 * (e >> 2) + e + 4 * g);
          const uint8_t* src = static_cast<const uint8_t*>(a.v_cache) + row * (D / 2) + at;
          if constexpr (D == 256) {
            const U2 x = *reinterpret_cast<const U2*>(src);
            vr[e][0][0] = x[0];
            vr[e][VW - 1][0] = x[1];
          } else if constexpr (D == 128) {
            vr[e][0][0] = *reinterpret_cast<const uint32_t*>(src);
          } else {
            vr[e][0][0] = *reinterpret_cast<const uint16_t*>(src);
          }
          vs[e] = a.v_scale[row * (D / 32) + sat];
        }
      } else if constexpr (RUNS) {
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

  // dimensions 2w and 2w + 1 of a lane's piece c of V, for its key e
  auto v_pair = [&](int e, int c, int w) {
    if constexpr (FOUR)
      return pair_at<T>(vr[e][w / 4][0], scale_of(vs[e]), w % 4);
    else
      return static_cast<uint32_t>(vr[e][c][w]);
  };

  int w0 = k0 + kKeys * wave;
  int j0 = pt.key_at<F>(w0);
  TileAt at{};
  if (w0 < k1) {
    at = find_tile<RUNS>(a, table, h, j0, pt.hi, lane);
    load_k(at, j0);
  }
#pragma unroll 1
  for (; w0 < k1; w0 += kKeys * kWaves) {
    load_v(at, j0);
    // past the last tile nothing is fetched, or the same tile again
    const int wn = w0 + kKeys * kWaves, jn = pt.key_at<F>(wn);
    const int end = F == kTwoByte ? k1 : wn < k1 ? pt.hi : 0;  // of the keys to fetch
    const TileAt next = find_tile<RUNS>(a, table, h, RUNS || wn < k1 ? jn : j0,
                                        RUNS ? end : pt.hi, lane);

    F4 sc[RB][2];
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          U4 kf;
          if constexpr (FOUR) {
            uint32_t pairs[4];
            pairs_of<T>(kr[e][d / KW][d % KW], scale_of(ks[e][d / KW]), pairs);
            kf = U4{pairs[0], pairs[1], pairs[2], pairs[3]};
          } else {
            kf = kr[e][d];
          }
          sc[rb][e] = mfma16(kf, q[rb][d], d == 0 ? F4{0, 0, 0, 0} : sc[rb][e], T{});
        }
    load_k(next, RUNS || wn < k1 ? jn : j0);

    if (is_edge<F>(a, pt, j0, kKeys, at.gone != 0)) {
      const int sinks = sinks_of<F>(a) - j0 - 4 * g;
      // Values no row sees become zero, and where rows see different keys
      // infinities and NaN among the others too (put_back).
      if (!RUNS || !one_token || j0 < pt.lo) {
        const int lo = pt.lo - j0 - 4 * g, hi = pt.hi - j0 - 4 * g;
        const uint32_t gone = at.gone >> 4 * g;
        uint32_t odd = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int key = 12 * (e >> 2) + e;
          const uint32_t seen = (key >= lo || (F != kTwoByte && key < sinks)) && key < hi &&
                                        (gone >> key & 1) == 0
                                    ? 0xffffffffu
                                    : 0u;
          if constexpr (FOUR) {
            // codes of zero, under a scale that is a number
            const bool take = seen != 0 && (one_token || vs[e] != kNanScale);
            odd |= seen != 0 && vs[e] > kMostExp<T> + 127 ? kOdd : 0u;
            vs[e] = take ? vs[e] : 127u;
#pragma unroll
            for (int w = 0; w < VW; ++w) vr[e][w][0] = take ? vr[e][w][0] : 0u;
            continue;
          }
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
          for (int e = 0; e < 8; ++e) {
            if constexpr (FOUR) {
              const bool far = vs[e] > kMostExp<T> + 127;
#pragma unroll
              for (int w = 0; w < VW; ++w)
                vr[e][w][0] &= far ? ~odd_codes<T>(vr[e][w][0], vs[e]) : 0xffffffffu;
              continue;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
              for (int w = 0; w < DV / 2; ++w) vr[e][c][w] = finite_or_zero<T>(vr[e][c][w]);
          }
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
            const bool before = key < lo && (F == kTwoByte || key >= sinks);
            sc[rb][e][i] = before || key >= hi      ? kNegInf
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
            f[e] = __builtin_amdgcn_perm(v_pair(2 * e + 1, c, w), v_pair(2 * e, c, w),
                                         z ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int rb = 0; rb < RB; ++rb)
#pragma unroll
            for (int n = NP - 1; n >= 0; --n)
              o[rb][c * DV + 2 * w + z] =
                  mfma16(f, pr[rb][n], o[rb][c * DV + 2 * w + z], T{});
        }
    at = next;
    j0 = jn;
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
      if (out.partial) {
        const int64_t at_row = out.at(16 * rb + row, s.q0 + i, hq);
        *reinterpret_cast<F4*>(out.o + at_row * D + d) = x;
        if (d == 0) out.ml[at_row] = make_float2(mx, lx);
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
    put_back_walk<T, TO, F>(a, s, table, h, pt, k0, k1, kKeys, r0, ROWS, 64 * kWaves, out);
    __syncthreads();
  }
}

template <typename T, typename TO, int D, int RB, bool RUNS>
__global__ __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) void few_rows_kernel(AttnArgs a,
                                                                                 FewGrid fg,
                                                                                 float* part_o,
                                                                                 float2* part_ml) {
  constexpr int ROWS = 16 * RB;
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
    const Parts pt = split_keys<kTwoByte>(a, s, static_cast<int>(r0), ROWS, fg.chunk, fg.nsplit);
    const int64_t from = pt.start + static_cast<int64_t>(split) * pt.chunk;
    if (split > 0 && from >= pt.end) continue;
    const int k0 = static_cast<int>(from);
    const int k1 = pt.end - k0 < pt.chunk ? pt.end : k0 + pt.chunk;
    const PartOut out{fg.nsplit > 1, static_cast<int64_t>(split) * a.T * Hq, Hq, part_o, part_ml};
    few_rows_part<T, TO, D, RB, RUNS, kTwoByte>(a, s, table, h, rows, r0, pt, k0, k1, out);
  }
}

// ---------------------------------------------------------------------------
// The further forms cut a tile's keys into steps of 128 and those in two ways.
//
// Parts: every (sequence, row tile, cache head) in as many parts as the plan says,
// of equal numbers of steps.
//
// Stretches, for batches whose lengths may differ: all tiles' steps, one tile after
// another (after kStart steps for each one's beginning, which costs as much), are a
// line, and each of as many workgroups as the device holds takes a stretch of the
// same length (64 tokens at 200 to 8000 keys, 4-bit, D = 256: 93 us with one
// workgroup for each, 83 in eight parts, 81 with kStart 0, 72 with 2; all at 4000
// keys: 55, 71, 62 and 64 us).  Every workgroup finds its stretch by itself, from
// the sequences' lengths.  Only the first and the last piece of a stretch can be
// parts of a tile's keys; they go to the stretch's two slots, and the workgroup
// with a tile's first piece notes for the join who has the others.
// ---------------------------------------------------------------------------
constexpr int kStep = kKeys * kWaves;
constexpr int kStart = 2;

struct Cut {
  int wgs;        // stretches; 0: parts
  int row_tiles;  // parts: of a (sequence, cache head), that have workgroups
  int nsplit;
  FastDiv by_split, by_tiles, by_Hk;
};

// Who has a tile's pieces: workgroups first .. first + count - 1.
struct Pieces {
  int first;
  int count2;  // 2 count, plus 1 if the first piece begins its stretch
};

// The same in all lanes, as the compiler may know.
__device__ __forceinline__ int64_t uniform(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(x >> 32));
  return static_cast<int64_t>(uint64_t{hi} << 32 | lo);
}

// Where stretches begin: about total w / wgs.  (In fp64, whose division is a tenth of
// a 64-bit one's code, and the code of a workgroup's only pass is what a short call
// waits for: any cut will do that all workgroups agree on and that leaves no stretch
// empty, as the join counts on every one between two others.  With total / wgs at
// least 1, and for 2^20 workgroups at most, the products are far enough from the
// integers below them.)
struct Cuts {
  int wgs;
  int64_t total;
  double each;
  __device__ __forceinline__ int64_t at(int w) const {
    return w == wgs ? total : uniform(static_cast<int64_t>(each * w));
  }
  // The stretch that a step is in.
  __device__ __forceinline__ int of(int64_t step) const {
    int w = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<double>(step) / each));
    w = w < wgs ? w : wgs - 1;
    if (at(w) > step) --w;
    if (at(w + 1) <= step) ++w;
    return w;
  }
};
__device__ __forceinline__ Cuts cuts_of(int wgs, int64_t total) {
  Cuts c;
  c.wgs = wgs < total ? wgs : static_cast<int>(total);
  c.total = total;
  c.each = static_cast<double>(total) / c.wgs;
  return c;
}

template <CacheForm F, int ROWS>
__device__ __forceinline__ Parts tile_walk(const Args<F>& a, const Seq& s, int64_t r0) {
  return split_keys<F>(a, s, static_cast<int>(r0), ROWS, kMaxKeys, 2);
}
__device__ __forceinline__ int64_t steps_of(const Parts& pt) {
  return pt.end <= 0 ? 1 : (static_cast<int64_t>(pt.end) + kStep - 1) / kStep;
}
// Parts of a tile's steps, and where one begins: the first ones have a step more.
__device__ __forceinline__ uint32_t parts_of_steps(uint32_t nsplit, uint32_t steps) {
  return nsplit < steps ? nsplit : steps;
}
__device__ __forceinline__ uint32_t first_step(uint32_t part, uint32_t parts, uint32_t steps) {
  const uint32_t each = steps / parts, more = steps - each * parts;
  return part * each + (part < more ? part : more);
}
// Steps of a sequence, all its heads.
template <CacheForm F, int ROWS>
__device__ __forceinline__ int64_t steps_of(const Args<F>& a, int64_t b) {
  const Seq s = load_seq(a, b);
  const int64_t rows = static_cast<int64_t>(s.n) * a.G;
  int64_t steps = 0;
  for (int64_t r0 = 0; r0 < rows; r0 += ROWS) steps += kStart + steps_of(tile_walk<F, ROWS>(a, s, r0));
  return steps * a.Hk;
}
// Where the notes of a sequence's row tiles begin: tiles of sequences before it are
// no more than this.
template <int ROWS>
__device__ __forceinline__ int64_t first_tile(const AttnArgs& a, const Seq& s, int64_t b) {
  return s.q0 * a.G / ROWS + b;
}

// Workgroups that a CU holds, by registers.
template <int D, int RB, CacheForm F>
constexpr int kFewPerCu = D == 256 && (F != kFourBit || RB == 2) ? 1 : 2;

template <typename T, typename TO, int D, int RB, bool RUNS, CacheForm F>
__global__ __launch_bounds__(64 * kWaves, (kFewPerCu<D, RB, F>)) void few_stretch_kernel(
    Args<F> a, Cut sg, float* part_o, float2* part_ml, Pieces* pieces) {
  constexpr int ROWS = 16 * RB;
  const int w = blockIdx.x;
  int64_t begin = 0, end = 0, at = 0;
  int64_t pos = 0;  // of the present tile's first step
  Cuts cuts{0, 0, 0};
  int b;
  int h = 0;
  int64_t r0 = 0;
  uint32_t split = 0;
  if (sg.wgs == 0) {
    // first parts first: a part's number must not decide the XCD
    split = sg.by_split.div(blockIdx.x);
    const uint32_t id0 = blockIdx.x - split * sg.by_split.d;
    const uint32_t id1 = sg.by_tiles.div(id0), rt = id0 - id1 * sg.by_tiles.d;
    b = sg.by_Hk.div(id1);
    h = id1 - b * sg.by_Hk.d;
    r0 = static_cast<int64_t>(rt) * ROWS;
  } else {
    // Every wave for itself: steps of a lane's sequences, summed up over the lanes.
    const int each = static_cast<int>((a.B + 63) / 64), lane = threadIdx.x & 63;
    const int b0 = lane * each, b1 = b0 + each < a.B ? b0 + each : static_cast<int>(a.B);
    int64_t mine = 0;
#pragma unroll 1
    for (int i = b0; i < b1; ++i) mine += steps_of<F, ROWS>(a, i);
    int64_t sum = mine;
#pragma unroll 1
    for (int m = 1; m < 64; m <<= 1) {
      const int64_t x = __shfl_up(sum, m);
      if (lane >= m) sum += x;
    }
    cuts = cuts_of(sg.wgs, uniform(__shfl(sum, 63)));
    if (w < cuts.wgs) {
      begin = cuts.at(w);
      end = cuts.at(w + 1);
      // the sequence, row tile and head that the first step is of
      const uint64_t past = __ballot(sum > begin);
      const int who = __builtin_ctzll(past);
      pos = uniform(__shfl(sum - mine, who));
      b = __builtin_amdgcn_readfirstlane(who * each);
#pragma unroll 1
      for (;; r0 += ROWS) {
        const Seq s = load_seq(a, b);
        if (r0 >= static_cast<int64_t>(s.n) * a.G) {
          ++b;
          r0 = -ROWS;
          continue;
        }
        const int64_t steps = kStart + steps_of(tile_walk<F, ROWS>(a, s, r0));
        if (pos + steps * a.Hk > begin) {
          while (pos + steps <= begin) pos += steps, ++h;
          break;
        }
        pos += steps * a.Hk;
      }
    }
    at = begin;
  }
  // One tile's piece after another.
  while (sg.wgs == 0 || at < end) {
    const Seq s = load_seq(a, b);
    const int64_t rows = static_cast<int64_t>(s.n) * a.G;
    if (r0 >= rows) {
      if (sg.wgs == 0) break;
      ++b;
      r0 = 0;
      continue;
    }
    const Parts pt = tile_walk<F, ROWS>(a, s, r0);
    int k0, k1;
    SlotOut out{false, sg.wgs > 0, 0, a.Hk * a.G, part_o, part_ml};
    const int64_t r = r0;
    const int head = h;
    if (sg.wgs == 0) {
      r0 += static_cast<int64_t>(sg.row_tiles) * ROWS;
      const uint32_t steps = static_cast<uint32_t>(steps_of(pt));
      const uint32_t parts = parts_of_steps(sg.nsplit, steps);
      if (split >= parts) continue;
      k0 = static_cast<int>(first_step(split, parts, steps)) * kStep;
      k1 = split + 1 < parts ? static_cast<int>(first_step(split + 1, parts, steps)) * kStep : pt.end;
      out.partial = parts > 1;
      out.first = static_cast<int64_t>(split) * a.T * out.Hq;
    } else {
      // places [off, off + n) of the tile's steps, of which the first kStart have no keys
      const int64_t steps = kStart + steps_of(pt), off = at - pos;
      const int64_t n = steps - off < end - at ? steps - off : end - at;
      const int64_t first = off > kStart ? off - kStart : 0, last = off + n - kStart;
      k0 = static_cast<int>(first * kStep);
      k1 = off + n < steps ? static_cast<int>(last * kStep) : pt.end;
      out.partial = first > 0 || off + n < steps;
      out.first = (int64_t{2} * w + (at == begin ? 0 : 1)) * ROWS;
      if (first == 0 && last > 0 && threadIdx.x == 0) {
        const int has_end = out.partial ? cuts.of(pos + steps - 1) : w;
        pieces[(first_tile<ROWS>(a, s, b) + r / ROWS) * a.Hk + head] =
            {w, 2 * (has_end - w + 1) + (at == begin)};
      }
      at += n;
      if (off + n == steps) {
        pos += steps;
        if (++h == a.Hk) h = 0, r0 += ROWS;
      }
      if (last <= 0) continue;  // the beginning alone: the next workgroup's
    }
    few_rows_part<T, TO, D, RB, RUNS, F>(a, s, a.table + static_cast<int64_t>(b) * a.max_pages,
                                         head, static_cast<int>(rows), r, pt, k0, k1, out);
  }
}

// Joins the parts of every row: o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// eight parts at a time with all their loads in flight, under a running
// maximum.  WPR waves share a row (each takes every WPR-th eight), D / 64
// dimensions a lane.
template <typename TO, int D, int WPR, typename At>
__device__ __forceinline__ void join_row(const AttnArgs& a, const float* part_o,
                                         const float2* part_ml, int count, bool sees,
                                         int64_t token, int hq, const At& at) {
  constexpr int N = D / 64, BATCH = 8;
  __shared__ float sum_o[WPR > 1 ? 4 : 1][D];
  __shared__ float sum_m[4], sum_l[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float acc[N] = {}, l = 0.0f, top = kNegInf;
  for (int p0 = wave % WPR * BATCH; p0 < count; p0 += WPR * BATCH) {
    float2 ml[BATCH];
    float x[BATCH][N], up = top;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int64_t row = at(p0 + k < count ? p0 + k : count - 1);
      ml[k] = part_ml[row];
      load_wide(part_o + row * D + N * lane, x[k]);
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
    for (int n = 0; n < N; ++n) acc[n] = sees ? acc[n] / l : 0.0f;
    store_wide(static_cast<TO*>(a.out) + token * a.o_ts + hq * a.o_hs + N * lane, acc);
  }
  if constexpr (WPR > 1) __syncthreads();
}

template <typename TO, int D, int WPR, bool SINKS>
__global__ __launch_bounds__(256) void join_kernel(Args<SINKS ? kTwoByteSinks : kTwoByte> a,
                                                   FewGrid fg, int tile_rows, int tokens,
                                                   const float* part_o, const float2* part_ml) {
  constexpr int RPW = 4 / WPR;
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
    const Parts pt = split_keys<SINKS ? kTwoByteSinks : kTwoByte, kTileKeys<D>>(
        a, s, r & -tile_rows, tile_rows, fg.chunk, fg.nsplit);
    const int count = pt.count();
    int lo, hi;
    visible(a, s, i, &lo, &hi);
    const int64_t row = (s.q0 + i) * Hq + hq;
    join_row<TO, D, WPR>(a, part_o, part_ml, count, hi > lo, s.q0 + i, hq,
                         [&](int p) -> int64_t { return p * stride + row; });
  }
}

// The same for the rows of few_stretch_kernel (ROWS in a tile).
template <typename TO, int D, int WPR, int ROWS, CacheForm F>
__global__ __launch_bounds__(256) void join_pieces_kernel(Args<F> a, Cut cut, int tokens,
                                                          const float* part_o,
                                                          const float2* part_ml,
                                                          const Pieces* pieces) {
  constexpr int RPW = 4 / WPR;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int Hq = a.Hk * a.G;
  const uint32_t groups = (Hq + RPW - 1) / RPW;
  const uint32_t id = blockIdx.x / groups;
  const int hq = (blockIdx.x - id * groups) * RPW + wave / WPR;
  const uint32_t b = id / static_cast<uint32_t>(tokens);
  const Seq s = load_seq(a, b);
  if (hq >= Hq) return;  // (whole workgroups where waves share a row)
  const int h = static_cast<int>(a.by_G.div(hq)), hq_in = hq - h * a.G;
  for (int i = id - b * tokens; i < s.n; i += tokens) {
    const int64_t r = static_cast<int64_t>(i) * a.G + hq_in, tile = r / ROWS;
    Pieces p{0, 0};
    int count;
    if (cut.wgs == 0) {
      const Parts pt = tile_walk<F, ROWS>(a, s, tile * ROWS);
      count = static_cast<int>(parts_of_steps(cut.nsplit, static_cast<uint32_t>(steps_of(pt))));
    } else {
      p = pieces[(first_tile<ROWS>(a, s, b) + tile) * a.Hk + h];
      count = p.count2 >> 1;
    }
    if (count <= 1) continue;  // the workgroup that had it all wrote the result
    int lo, hi;
    visible(a, s, i, &lo, &hi);
    const int row = static_cast<int>(r - tile * ROWS);
    join_row<TO, D, WPR>(
        a, part_o, part_ml, count, hi > lo, s.q0 + i, hq, [&](int part) -> int64_t {
          const int slot = 2 * (p.first + part) + (part == 0 && !(p.count2 & 1));
          return cut.wgs == 0 ? (part * a.T + s.q0 + i) * Hq + hq : int64_t{slot} * ROWS + row;
        });
  }
}

FewGrid grid_of(const AttnPlan& plan, const AttnArgs& a) {
  return {static_cast<int>(plan.row_tiles), plan.nsplit, plan.chunk,
          FastDiv(static_cast<uint32_t>(plan.row_tiles)),
          FastDiv(static_cast<uint32_t>(plan.nsplit)), FastDiv(static_cast<uint32_t>(a.Hk))};
}

Cut cut_of(const AttnPlan& plan, const AttnArgs& a) {
  return {plan.wgs,
          static_cast<int>(plan.row_tiles),
          plan.nsplit,
          FastDiv(static_cast<uint32_t>(a.B * a.Hk * plan.row_tiles)),
          FastDiv(static_cast<uint32_t>(plan.row_tiles)),
          FastDiv(static_cast<uint32_t>(a.Hk))};
}
// Rows of a cut's partial sums.
int64_t cut_rows(const AttnPlan& plan, const AttnArgs& a) {
  return plan.wgs > 0 ? int64_t{2} * plan.wgs * plan.tile_rows : plan.nsplit * a.T * a.Hk * a.G;
}

template <typename T, typename TO, int D, int RB, CacheForm F>
hipError_t launch_few(const AttnPlan& plan, const Args<F>& a, void* workspace, hipStream_t s) {
  float* part_o = static_cast<float*>(workspace);
  // pages of half a key tile or more are read as runs
  const bool runs = a.page_shift >= 4;
  if constexpr (F == kTwoByte) {
    const FewGrid fg = grid_of(plan, a);
    float2* part_ml = reinterpret_cast<float2*>(
        part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
    const dim3 grid(static_cast<uint32_t>(a.B * a.Hk * plan.row_tiles * plan.nsplit));
    if (runs)
      few_rows_kernel<T, TO, D, RB, true><<<grid, 64 * kWaves, 0, s>>>(a, fg, part_o, part_ml);
    else
      few_rows_kernel<T, TO, D, RB, false><<<grid, 64 * kWaves, 0, s>>>(a, fg, part_o, part_ml);
  } else {
    const Cut cut = cut_of(plan, a);
    float2* part_ml = reinterpret_cast<float2*>(part_o + cut_rows(plan, a) * D);
    Pieces* pieces = reinterpret_cast<Pieces*>(part_ml + cut_rows(plan, a));
    const dim3 grid(static_cast<uint32_t>(
        plan.wgs > 0 ? plan.wgs : a.B * a.Hk * plan.row_tiles * plan.nsplit));
    if (runs)
      few_stretch_kernel<T, TO, D, RB, true, F>
          <<<grid, 64 * kWaves, 0, s>>>(a, cut, part_o, part_ml, pieces);
    else
      few_stretch_kernel<T, TO, D, RB, false, F>
          <<<grid, 64 * kWaves, 0, s>>>(a, cut, part_o, part_ml, pieces);
  }
  return hipGetLastError();
}

template <typename TO, int D, int WPR>
hipError_t launch_pieces(const AttnPlan& plan, const AttnWindowArgs& a, void* workspace,
                         hipStream_t s) {
  const float* part_o = static_cast<const float*>(workspace);
  const float2* part_ml = reinterpret_cast<const float2*>(part_o + cut_rows(plan, a) * D);
  const Pieces* pieces = reinterpret_cast<const Pieces*>(part_ml + cut_rows(plan, a));
  constexpr int RPW = 4 / WPR;
  const int64_t groups = (a.Hk * a.G + RPW - 1) / RPW;
  const int64_t most = ((int64_t{1} << 24) - 1) / (a.B * groups);  // below 2^32 threads
  const int64_t tokens = plan.tokens < most ? plan.tokens : most;
  const dim3 grid(static_cast<uint32_t>(a.B * tokens * groups));
  const Cut cut = cut_of(plan, a);
  const int n = static_cast<int>(tokens);
  if (plan.tile_rows == 16)
    join_pieces_kernel<TO, D, WPR, 16, kTwoByteSinks>
        <<<grid, 256, 0, s>>>(a, cut, n, part_o, part_ml, pieces);
  else
    join_pieces_kernel<TO, D, WPR, 32, kTwoByteSinks>
        <<<grid, 256, 0, s>>>(a, cut, n, part_o, part_ml, pieces);
  return hipGetLastError();
}

template <bool SINKS>
using JoinArgs = Args<SINKS ? kTwoByteSinks : kTwoByte>;

template <typename TO, int D, int WPR, bool SINKS>
hipError_t launch_join_waves(const AttnPlan& plan, const JoinArgs<SINKS>& a, void* workspace,
                             hipStream_t s) {
  const FewGrid fg = grid_of(plan, a);
  const float* part_o = static_cast<const float*>(workspace);
  const float2* part_ml = reinterpret_cast<const float2*>(
      part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  constexpr int RPW = 4 / WPR;
  const int64_t groups = (a.Hk * a.G + RPW - 1) / RPW;
  const int64_t most = ((int64_t{1} << 24) - 1) / (a.B * groups);  // below 2^32 threads
  const int64_t tokens = plan.tokens < most ? plan.tokens : most;
  join_kernel<TO, D, WPR, SINKS><<<dim3(static_cast<uint32_t>(a.B * tokens * groups)), 256, 0, s>>>(
      a, fg, plan.tile_rows, static_cast<int>(tokens), part_o, part_ml);
  return hipGetLastError();
}

template <typename TO, int D, bool SINKS>
hipError_t launch_join(const AttnPlan& plan, const JoinArgs<SINKS>& a, void* workspace, hipStream_t s) {
  if constexpr (SINKS) {
    // as below, by the pieces of a tile where there are few
    if (!plan.many)
      return plan.nsplit > 8 || plan.wgs > 8 * a.B * a.Hk * plan.row_tiles
                 ? launch_pieces<TO, D, 4>(plan, a, workspace, s)
                 : launch_pieces<TO, D, 1>(plan, a, workspace, s);
  }
  // four waves to a row where there are several batches (64 parts: 9.1 -> 5.4 us)
  return plan.nsplit > 8 ? launch_join_waves<TO, D, 4, SINKS>(plan, a, workspace, s)
                         : launch_join_waves<TO, D, 1, SINKS>(plan, a, workspace, s);
}

template <typename T, typename TO, int D, CacheForm F>
hipError_t launch_rows(const AttnPlan& plan, const Args<F>& a, void* ws, hipStream_t s) {
  return plan.tile_rows == 16 ? launch_few<T, TO, D, 1, F>(plan, a, ws, s)
                              : launch_few<T, TO, D, 2, F>(plan, a, ws, s);
}

template <typename T, typename TO, CacheForm F>
hipError_t launch_dims(const AttnPlan& plan, const Args<F>& a, void* ws, hipStream_t s) {
  switch (a.D) {
    case 64: return launch_rows<T, TO, 64, F>(plan, a, ws, s);
    case 128: return launch_rows<T, TO, 128, F>(plan, a, ws, s);
    default: return launch_rows<T, TO, 256, F>(plan, a, ws, s);
  }
}

template <CacheForm F>
hipError_t launch_few_rows(const AttnPlan& plan, const Args<F>& a, int dtype, int out_dtype,
                           void* ws, hipStream_t s) {
  if (dtype == PQ1_BF16)
    return out_dtype == PQ1_F32 ? launch_dims<bf16, float, F>(plan, a, ws, s)
                                : launch_dims<bf16, bf16, F>(plan, a, ws, s);
  return out_dtype == PQ1_F32 ? launch_dims<f16, float, F>(plan, a, ws, s)
                              : launch_dims<f16, f16, F>(plan, a, ws, s);
}

template <typename TO, bool SINKS>
hipError_t join_dims(const AttnPlan& plan, const JoinArgs<SINKS>& a, void* ws, hipStream_t s) {
  switch (a.D) {
    case 64: return launch_join<TO, 64, SINKS>(plan, a, ws, s);
    case 128: return launch_join<TO, 128, SINKS>(plan, a, ws, s);
    default: return launch_join<TO, 256, SINKS>(plan, a, ws, s);
  }
}

template <bool SINKS>
hipError_t join_parts(const AttnPlan& plan, const JoinArgs<SINKS>& a, int out_dtype, void* ws,
                      hipStream_t s) {
  switch (out_dtype) {
    case PQ1_BF16: return join_dims<bf16, SINKS>(plan, a, ws, s);
    case PQ1_F16: return join_dims<f16, SINKS>(plan, a, ws, s);
    default: return join_dims<float, SINKS>(plan, a, ws, s);
  }
}

}  // namespace

}  // namespace pq1
