// Attention over a paged cache for many rows: prompts and chunks of prompts.
//
// A workgroup takes 32 RB rows for each of its waves, of one (sequence, cache
// head), and walks tiles of 64 keys.  A tile's K and V rows are copied one
// tile ahead straight from the cache into LDS (a lane gives the address of
// its 16 bytes, so a tile's pages may lie anywhere); every wave reads them all.
//
// Both products are taken transposed on 32x32x16 matrix instructions:
// S^T = K Q^T leaves lane l the scores of row l % 32 for keys 8 (i / 4) + 4 g
// + i % 4 (g = l / 32, i < 16), and eight of these are, as they stand, an
// operand of O^T = V^T P^T if V is read with the same key order, which LDS
// reads that transpose 4 keys x 16 dimensions do.  So P never leaves its lane, and a row's
// maximum and sum need one exchange between the two halves of a wave.
//
// 16-byte pieces of a row are stored XORed with bits of the row number, so
// that the rows read together lie in distinct banks (k_bits, v_bits).
#include "attn_tiles.h"

namespace pq1 {

namespace {

constexpr int kTileKeys = 64;

using F16 = __attribute__((ext_vector_type(16))) float;
using S4 = __attribute__((ext_vector_type(4))) short;
using LdsS4 = __attribute__((address_space(3))) S4;
using LdsVoid = __attribute__((address_space(3))) void;
using GlobalVoid = const __attribute__((address_space(1))) void;

__device__ __forceinline__ F16 mfma32(U4 a, U4 b, F16 c, bf16) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(Vec8<bf16>, a),
                                                 __builtin_bit_cast(Vec8<bf16>, b), c, 0, 0, 0);
}
__device__ __forceinline__ F16 mfma32(U4 a, U4 b, F16 c, f16) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(Vec8<f16>, a),
                                                __builtin_bit_cast(Vec8<f16>, b), c, 0, 0, 0);
}

// Piece c of row r lies in place c ^ k_bits(r) or c ^ v_bits(r) of its LDS
// row.  K: 16 neighbouring rows are read at one piece; V: four neighbouring
// rows at four pieces.  256 bytes are one round of the banks: two rows where
// D is 64.  Both are linear over XOR, so that a place is one XOR with a
// constant away from another.
template <int D>
__device__ __forceinline__ constexpr int k_bits(int r) {
  return D >= 128 ? r & 15 : r >> 1 & 7;
}
template <int D>
__device__ __forceinline__ constexpr int v_bits(int r) {
  return D >= 128 ? (r & 3) << 2 : (r & 2) << 1;
}

// Keeps what is computed from x out of the loop's registers: it is computed
// where it is used.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

struct TileGrid {
  int row_tiles, nsplit, chunk;
};

template <typename T, typename TO, int D, int NW, int RB>
__global__ __launch_bounds__(64 * NW) void many_rows_kernel(AttnArgs a, TileGrid tg,
                                                            float* part_o, float2* part_ml) {
  constexpr int NP = kParts<T, TO>;
  constexpr int ROWB = 2 * D;                   // bytes of a cache row
  constexpr int TILE = kTileKeys * ROWB;
  constexpr int PIECES = D / 8;                 // 16-byte pieces of a row
  constexpr int CROWS = 64 / PIECES;            // rows one copy of a wave fills
  constexpr int COPIES = kTileKeys / (CROWS * NW);
  constexpr int ROWS = 32 * RB * NW;
  constexpr int NB = D / 32;                    // blocks of 32 dimensions
  constexpr int EB = D * RB >= 256 ? 1 : 2;     // blocks of 32 keys whose scores are held
  __shared__ __attribute__((aligned(1024))) char k0_lds[TILE], v0_lds[TILE];
  __shared__ __attribute__((aligned(1024))) char k1_lds[TILE], v1_lds[TILE];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, g = lane >> 5;
  // Tiles with the most keys first; the cache heads of a tile next to one
  // another, so that where there are eight of them each L2 serves one.
  uint32_t id = blockIdx.x;
  const int h = id % a.Hk;
  id /= a.Hk;
  const int split = id % tg.nsplit;
  id /= tg.nsplit;
  const int b = id % a.B;
  const int rt = tg.row_tiles - 1 - static_cast<int>(id / a.B);
  const Seq s = load_seq(a, b);
  const int32_t* table = a.table + b * a.max_pages;
  const int rows = s.n * a.G;
  const int Hq = a.Hk * a.G;
  const int page_mask = (1 << a.page_shift) - 1;

  for (int64_t r0 = static_cast<int64_t>(rt) * ROWS; r0 < rows;
       r0 += static_cast<int64_t>(tg.row_tiles) * ROWS) {
    const Parts pt = split_keys(a, s, static_cast<int>(r0), ROWS, tg.chunk, tg.nsplit);
    if (split > 0 && split >= pt.count) continue;
    const int k0 = pt.start + split * pt.chunk;
    const int k1 = pt.hi - k0 < pt.chunk ? pt.hi : k0 + pt.chunk;

    // this wave's rows, and the keys that some of them sees
    const int wr0 = static_cast<int>(r0) + 32 * RB * wave;
    int wlo = 0, whi = 0;
    if (wr0 < rows) {
      int t;
      const int last = (wr0 + 32 * RB < rows ? wr0 + 32 * RB : rows) - 1;
      visible(a, s, wr0 / a.G, &wlo, &t);
      visible(a, s, last / a.G, &t, &whi);
    }
    int hi[RB];  // row col of a block sees keys [low(hi), hi)
    const auto low = [&](int end) { return a.window > 0 && end > a.window ? end - a.window : 0; };
    U4 q[RB][D / 16];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int r = wr0 + 32 * rb + col;
      hi[rb] = 0;
      const int i = r / a.G;
      int t;
      if (r < rows) visible(a, s, i, &t, &hi[rb]);
      const T* src = static_cast<const T*>(a.q) + (s.q0 + i) * a.q_ts +
                     (h * a.G + r - i * a.G) * a.q_hs + 8 * g;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
        q[rb][d] = r < rows ? *reinterpret_cast<const U4*>(src + 16 * d) : U4{0, 0, 0, 0};
    }
    F16 o[RB][NB];
    float m[RB], l[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      m[rb] = kNegInf;
      l[rb] = 0.0f;
#pragma unroll
      for (int n = 0; n < NB; ++n) o[rb][n] = F16{};
    }

    bool odd_values = false;  // infinities or NaN were taken out of V

    // Page of key j0 + lane; keys past the last take its page, so that every
    // address lies in the cache.  -1: no page of the cache.
    auto find_page = [&](int j0) {
      const int j = j0 + lane < pt.hi ? j0 + lane : pt.hi - 1;
      const int p = j >> a.page_shift;
      const int page = p < a.max_pages ? table[p] : -1;
      return page < 0 || page >= a.pages ? -1 : page;
    };
    auto row_of = [&](int page, int j) {
      return ((static_cast<int64_t>(page < 0 ? 0 : page) * a.Hk + h) << a.page_shift) +
             (j & page_mask);
    };
    auto copy = [&](int page, int j0, char* kb, char* vb) {
      const int j = j0 + lane < pt.hi ? j0 + lane : pt.hi - 1;
      const int64_t mine = row_of(page, j) * ROWB;
      const int mlo = static_cast<int>(mine), mhi = static_cast<int>(mine >> 32);
      const int ln = here(lane);
      const int r = wave * (COPIES * CROWS) + ln / PIECES;  // the row of copy 0
      const int kp = 16 * (ln % PIECES ^ k_bits<D>(r)), vp = 16 * (ln % PIECES ^ v_bits<D>(r));
#pragma unroll
      for (int c = 0; c < COPIES; ++c) {
        const int64_t at = (static_cast<int64_t>(__shfl(mhi, r + c * CROWS)) << 32) |
                           static_cast<uint32_t>(__shfl(mlo, r + c * CROWS));
        const int to = (wave * COPIES + c) * 1024;
        __builtin_amdgcn_global_load_lds(
            (GlobalVoid*)(static_cast<const char*>(a.k_cache) + at +
                          (kp ^ 16 * k_bits<D>(c * CROWS))),
            (LdsVoid*)(kb + to), 16, 0, 0);
        __builtin_amdgcn_global_load_lds(
            (GlobalVoid*)(static_cast<const char*>(a.v_cache) + at +
                          (vp ^ 16 * v_bits<D>(c * CROWS))),
            (LdsVoid*)(vb + to), 16, 0, 0);
      }
    };

    const int vrow = 4 * g + ((lane & 15) >> 2);           // V row of a transposing read
    const int vpiece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int kat = col * ROWB + 16 * (g ^ k_bits<D>(col));
    const int vat = vrow * ROWB + 16 * (vpiece ^ v_bits<D>(vrow)) + 8 * (lane & 1);

    auto tile = [&](const char* kb, char* vb, int j0, int page) {
      const uint64_t gone = __ballot(page < 0);  // keys on no page of the cache
      const bool edge = j0 < pt.lo_max || j0 + kTileKeys > pt.hi_min || gone != 0;
      if (edge) {
        // Values no row sees become zero, and where there are infinities or
        // NaN among the others these too: times a probability of zero they
        // would be NaN in the rows that do not see them.
        bool odd = false;
        constexpr int EACH = TILE / 16 / (64 * NW);
#pragma unroll
        for (int e = 0; e < EACH; ++e) {
          const int at = 64 * NW * e + here(threadIdx.x);
          const int r = at / PIECES;
          U4* v = reinterpret_cast<U4*>(vb + 16 * at);
          U4 x = *v;
          const bool seen = j0 + r >= pt.lo && j0 + r < pt.hi && !(gone >> r & 1);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            x[w] = seen ? x[w] : 0u;
            odd |= not_finite<T>(x[w]);
            x[w] = finite_or_zero<T>(x[w]);
          }
          *v = x;
        }
        odd_values |= __syncthreads_or(odd) != 0;
      }
      if (j0 >= whi || j0 + kTileKeys <= wlo) return;  // this wave's rows see none of it

#pragma unroll
      for (int e0 = 0; e0 < 2; e0 += EB) {
        const int kx = here(kat), vx = here(vat);
        F16 sc[RB][EB];
#pragma unroll
        for (int e = 0; e < EB; ++e)
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            const U4 f = *reinterpret_cast<const U4*>(
                kb + 32 * (e0 + e) * ROWB + (kx ^ 32 * (d & 7)) + 256 * (d >> 3));
#pragma unroll
            for (int rb = 0; rb < RB; ++rb)
              sc[rb][e] = mfma32(f, q[rb][d], d == 0 ? F16{} : sc[rb][e], T{});
          }
        if (edge) {
          // key numbers relative to the lane's first: compile-time constants
          const int at = j0 + 32 * e0 + 4 * g;
          const uint64_t lost = gone >> (32 * e0 + 4 * g);
#pragma unroll
          for (int e = 0; e < EB; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int key = 32 * e + 8 * (i >> 2) + (i & 3);
#pragma unroll
              for (int rb = 0; rb < RB; ++rb) {
                const bool seen = key >= low(hi[rb]) - at && key < hi[rb] - at;
                sc[rb][e][i] =
                    !seen ? kNegInf : lost >> key & 1 ? __builtin_nanf("") : sc[rb][e][i];
              }
            }
        }
        U4 pr[RB][EB][2][NP];
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
          float top = sc[rb][0][0];
#pragma unroll
          for (int e = 0; e < EB; ++e)
#pragma unroll
            for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[rb][e][i]);
          const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(top),
                                                           __float_as_uint(top), false, false);
          top = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1])) * a.scale_log2;
          if (__any(top > m[rb] + kLag)) {
            const float up = fmaxf(m[rb], top);
            const float keep = m[rb] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m[rb] - up);
            m[rb] = up;
            l[rb] *= keep;
#pragma unroll
            for (int n = 0; n < NB; ++n) o[rb][n] *= keep;
          }
          const float shift = m[rb] == kNegInf ? 0.0f : kUp - m[rb];
#pragma unroll
          for (int e = 0; e < EB; ++e)
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              float p[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(fmaf(sc[rb][e][8 * st + i], a.scale_log2, shift));
                l[rb] += p[i];
              }
              split_probs<T, NP>(p, pr[rb][e][st]);
            }
        }
#pragma unroll
        for (int e = 0; e < EB; ++e)
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              const char* src = vb + (32 * (e0 + e) + 16 * st) * ROWB + (vx ^ 64 * (n & 3)) +
                                256 * (n >> 2);
              const U2 x = __builtin_bit_cast(
                  U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4*)src));
              const U2 y = __builtin_bit_cast(
                  U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4*)(src + 8 * ROWB)));
              const U4 f = {x[0], x[1], y[0], y[1]};
#pragma unroll
              for (int rb = 0; rb < RB; ++rb)
#pragma unroll
                for (int z = NP - 1; z >= 0; --z)
                  o[rb][n] = mfma32(f, pr[rb][e][st][z], o[rb][n], T{});
            }
        if (e0 + EB < 2) __builtin_amdgcn_sched_barrier(0);
      }
    };

    // Tile t is computed while t + 1 is copied into the other buffers; a wave
    // waits for its own copies before the barrier that ends a tile.
    if (k0 < k1) {
      int page = find_page(k0);
      copy(page, k0, k0_lds, v0_lds);
      int next = find_page(k0 + kTileKeys);
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vector memory 0
      __syncthreads();
      for (int j0 = k0;;) {
        if (j0 + kTileKeys < k1) copy(next, j0 + kTileKeys, k1_lds, v1_lds);
        int then = find_page(j0 + 2 * kTileKeys);
        tile(k0_lds, v0_lds, j0, page);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        page = next;
        next = then;
        if ((j0 += kTileKeys) >= k1) break;
        if (j0 + kTileKeys < k1) copy(next, j0 + kTileKeys, k0_lds, v0_lds);
        then = find_page(j0 + 2 * kTileKeys);
        tile(k1_lds, v1_lds, j0, page);
        __builtin_amdgcn_s_waitcnt(0x0F70);
        __syncthreads();
        page = next;
        next = then;
        if ((j0 += kTileKeys) >= k1) break;
      }
    }

#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l[rb]),
                                                       __float_as_uint(l[rb]), false, false);
      const float sum = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
      const int r = wr0 + 32 * rb + col;
      if (r >= rows) continue;
      const int i = r / a.G;
      const int hq = h * a.G + r - i * a.G;
      const int64_t at_row = static_cast<int64_t>(split) * a.T * Hq + (s.q0 + i) * Hq + hq;
      if (tg.nsplit > 1) {
        if (g == 0) part_ml[at_row] = make_float2(m[rb], sum);
      }
      const float inv = 1.0f / sum;
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int i4 = 0; i4 < 4; ++i4) {
          const int d = 32 * n + 8 * i4 + 4 * g;
          float y[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) y[c] = o[rb][n][4 * i4 + c];
          if (tg.nsplit > 1) {
            store_wide(part_o + at_row * D + d, y);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = hi[rb] > 0 ? y[c] * inv : 0.0f;
            store_wide(static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs + d, y);
          }
        }
    }

    // Put back what the tiles' edges took out: rows that see an infinity or
    // NaN add it to their result.
    if (odd_values) {
      __syncthreads();
      for (int j0 = k0; j0 < k1; j0 += kTileKeys) {
        const int page = find_page(j0);
        const bool bad = __any(page < 0);
        if (j0 >= pt.lo_max && j0 + kTileKeys <= pt.hi_min && !bad) continue;
        for (int key = 0; key < kTileKeys && j0 + key < k1; ++key) {
          const int pg = __shfl(page, key);
          if (pg < 0) continue;
          const T* src = static_cast<const T*>(a.v_cache) + row_of(pg, j0 + key) * D;
          for (int e = threadIdx.x; e < ROWS * D; e += 64 * NW) {
            const int64_t r = r0 + e / D;
            const int d = e % D;
            const float x = static_cast<float>(src[d]);
            if (r >= rows || __builtin_isfinite(x)) continue;
            const int i = static_cast<int>(r) / a.G;
            int rlo, rhi;
            visible(a, s, i, &rlo, &rhi);
            if (j0 + key < rlo || j0 + key >= rhi) continue;
            const int hq = h * a.G + static_cast<int>(r) - i * a.G;
            if (tg.nsplit > 1) {
              part_o[(static_cast<int64_t>(split) * a.T * Hq + (s.q0 + i) * Hq + hq) * D + d] += x;
            } else {
              TO* y = static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs + d;
              *y = static_cast<TO>(static_cast<float>(*y) + x);
            }
          }
        }
      }
    }
  }
}

template <typename T, typename TO, int D>
hipError_t launch_tiles(const AttnPlan& plan, const AttnArgs& a, void* workspace, hipStream_t s) {
  const TileGrid tg{static_cast<int>(plan.row_tiles), plan.nsplit, plan.chunk};
  float* part_o = static_cast<float*>(workspace);
  float2* part_ml =
      reinterpret_cast<float2*>(part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  const dim3 grid(static_cast<uint32_t>(a.B * a.Hk * plan.row_tiles * plan.nsplit));
  constexpr int RB = 1, NW = kTileRows / (32 * RB);
  many_rows_kernel<T, TO, D, NW, RB><<<grid, 64 * NW, 0, s>>>(a, tg, part_o, part_ml);
  return hipGetLastError();
}

template <typename T, typename TO>
hipError_t launch_dim(const AttnPlan& plan, const AttnArgs& a, void* ws, hipStream_t s) {
  switch (a.D) {
    case 64: return launch_tiles<T, TO, 64>(plan, a, ws, s);
    case 128: return launch_tiles<T, TO, 128>(plan, a, ws, s);
    default: return launch_tiles<T, TO, 256>(plan, a, ws, s);
  }
}

}  // namespace

hipError_t launch_many_rows(const AttnPlan& plan, const AttnArgs& a, int dtype, int out_dtype,
                            void* workspace, hipStream_t s) {
  if (dtype == PQ1_BF16)
    return out_dtype == PQ1_F32 ? launch_dim<bf16, float>(plan, a, workspace, s)
                                : launch_dim<bf16, bf16>(plan, a, workspace, s);
  return out_dtype == PQ1_F32 ? launch_dim<f16, float>(plan, a, workspace, s)
                              : launch_dim<f16, f16>(plan, a, workspace, s);
}

}  // namespace pq1
