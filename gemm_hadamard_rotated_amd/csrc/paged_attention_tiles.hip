// Attention over a paged cache for many rows: prompts and chunks of prompts.
//
// A workgroup takes 256 rows of one (sequence, cache head), 32 for each of its
// eight waves, and walks tiles of keys (64; 32 where D is 256).  A tile's K
// and V rows are copied two tiles ahead straight from the cache into LDS (a
// lane gives the address of its 16 bytes, so a tile's pages may lie anywhere);
// every wave reads them all.
//
// Both products are taken transposed on 32x32x16 matrix instructions:
// S^T = K Q^T leaves lane l the scores of row l % 32 for keys 8 (i / 4) + 4 g
// + i % 4 (g = l / 32, i < 16), and eight of these are, as they stand, an
// operand of O^T = V^T P^T if V is read with the same key order, which LDS
// reads that transpose 4 keys x 16 dimensions do.  So P never leaves its lane,
// and a row's maximum and sum need one exchange between the halves of a wave.
//
// Bound: the matrix instructions and, for small D, the softmax between them.
// 8192 rows of 8 cache heads against 7168 keys take 445 to 454 us at D = 256
// (1061 to 1082 TFLOP/s), 255 to 261 us at 128 (921 to 945) and 186 to 188 us at
// 64 (641 to 646); a large library product reaches 1263 TFLOP/s on the same card.
// An fp32 result takes the second product three times for bf16 caches, 769 to
// 792, 429 to 440 and 318 to 324 us, and twice for f16, 658 to 681, 362 to 376
// and 238 to 241 us.
// What was measured on the way (D = 128 of the above unless said): 64 rows a
// wave, one wave a SIMD: slower (759 against 505 us for 2048 tokens after 6144
// at D = 256); page numbers from LDS and no load waited for in the loop, so
// that copies stay in flight over the barrier: 285 -> 265 us; priority for the
// wave that computes scores: 265 -> 260 us (D = 256: 460 -> 444); waves of one
// SIMD set half a tile apart: 274 us; a barrier every second tile: 267 us;
// tiles of pages of 64 keys or more copied as one run: no gain; 32-bit offsets
// for the copies and sums of probabilities in pairs: 264 -> 260 us (ragged
// prompts 386 -> 377).
#include "attn_tiles.h"

namespace pq1 {

namespace {

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

// Copies 16 bytes a lane from memory to LDS, lane after lane from `to` on (the
// same for the whole wave).  Written as an instruction because the compiler
// would wait for all copies in flight before each read of LDS that it cannot
// tell apart from them; here the wait is wait_copies and a barrier.
__device__ __forceinline__ uint32_t lds_at(const char* p) {
  return __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const char*)p)));
}
__device__ __forceinline__ void copy16(const char* from, char* to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "s"(lds_at(to)), "v"(from)
               : "m0");
}
// The same from a place that the whole wave shares, plus a lane's offset.
__device__ __forceinline__ void copy16(const char* from, uint32_t offset, char* to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %1"
               :
               : "s"(lds_at(to)), "s"(from), "v"(offset)
               : "m0");
}
// Waits until at most N copies of this wave are in flight.
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

constexpr int kPages = 4096;  // page numbers kept in LDS

struct TileGrid {
  int row_tiles, nsplit, chunk;
};

constexpr int kTileWaves = kTileRows / 32;

template <typename T, typename TO, int D, bool WIDE>
__global__ __launch_bounds__(64 * kTileWaves) void many_rows_kernel(AttnArgs a, TileGrid tg,
                                                                    float* part_o,
                                                                    float2* part_ml) {
  constexpr int NP = kParts<T, TO>;
  constexpr int KT = D == 256 ? 32 : 64;        // keys of a tile
  constexpr int ROWB = 2 * D;                   // bytes of a cache row
  constexpr int TILE = KT * ROWB;
  constexpr int PIECES = D / 8;                 // 16-byte pieces of a row
  constexpr int CROWS = 64 / PIECES;            // rows one copy of a wave fills
  constexpr int COPIES = KT / (CROWS * kTileWaves);
  constexpr int NB = D / 32;                    // blocks of 32 dimensions
  constexpr int EB = KT / 32;                   // blocks of 32 keys
  constexpr int AHEAD = D == 256 ? 3 : 4;       // fragments in flight from LDS
  __shared__ __attribute__((aligned(TILE))) char k_lds[3 * TILE], v_lds[3 * TILE];
  __shared__ int32_t page_lds[kPages + 1];

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
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int rows = s.n * a.G;
  const int Hq = a.Hk * a.G;
  const int page_mask = (1 << a.page_shift) - 1;

  for (int64_t r0 = static_cast<int64_t>(rt) * kTileRows; r0 < rows;
       r0 += static_cast<int64_t>(tg.row_tiles) * kTileRows) {
    const Parts pt = split_keys(a, s, static_cast<int>(r0), kTileRows, tg.chunk, tg.nsplit);
    if (split > 0 && split >= pt.count()) continue;
    const int k0 = pt.start + split * pt.chunk;
    const int k1 = pt.hi - k0 < pt.chunk ? pt.hi : k0 + pt.chunk;

    const int wr0 = static_cast<int>(r0) + 32 * wave;  // this wave's rows
    U4 q[D / 16];
    {
      const int r = wr0 + col;
      const int i = a.by_G.div(r);
      const T* src = static_cast<const T*>(a.q) + (s.q0 + i) * a.q_ts +
                     (h * a.G + r - i * a.G) * a.q_hs + 8 * g;
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
        q[d] = r < rows ? *reinterpret_cast<const U4*>(src + 16 * d) : U4{0, 0, 0, 0};
    }
    F16 o[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n) o[n] = F16{};
    float m = kNegInf, l = 0.0f;
    bool odd_values = false;  // infinities or NaN were taken out of V

    // Pages of keys first .. end - 1 are in LDS: the number, -1 for no page of
    // the cache; or, where K and V take less than 4 GB each, the byte at which
    // the page's rows of this head begin, one more than page 0's for none.
    // Keys past the last take its page, so that every address lies in the
    // cache.  A lane looks up the rows that it copies, a tile ahead.
    int first = 0, end = 0;
    auto page_at = [&](int j) { return page_lds[(j >> a.page_shift) - (first >> a.page_shift)]; };
    auto is_gone = [](int entry) { return WIDE ? entry < 0 : (entry & 1) != 0; };
    auto up_to_end = [&](int j) { return j < end ? j : end - 1; };
    auto gone_of = [&](int j0) {  // keys of a tile on no page of the cache
      const uint64_t bits = __ballot(is_gone(page_at(up_to_end(j0 + lane))));
      return KT == 64 ? bits : bits & 0xffffffffu;
    };
    const int crow = wave * (COPIES * CROWS) + lane / PIECES;  // the row of copy 0
    auto find_pages = [&](int j0, int (&page)[COPIES]) {
#pragma unroll
      for (int c = 0; c < COPIES; ++c) page[c] = page_at(up_to_end(j0 + crow + c * CROWS));
    };
    auto copy = [&](const int (&page)[COPIES], int j0, char* kb, char* vb) {
      const int r = here(crow), piece = here(lane) % PIECES;
      const int kp = 16 * (piece ^ k_bits<D>(r)), vp = 16 * (piece ^ v_bits<D>(r));
      const char* k = static_cast<const char*>(a.k_cache);
      const char* v = static_cast<const char*>(a.v_cache);
#pragma unroll
      for (int c = 0; c < COPIES; ++c) {
        const int in_page = up_to_end(j0 + r + c * CROWS) & page_mask;
        const int kc = kp ^ 16 * k_bits<D>(c * CROWS), vc = vp ^ 16 * v_bits<D>(c * CROWS);
        const int to = (wave * COPIES + c) * 1024;
        if constexpr (WIDE) {
          const int64_t at =
              (((static_cast<int64_t>(page[c] < 0 ? 0 : page[c]) * a.Hk + h) << a.page_shift) +
               in_page) * ROWB;
          copy16(k + at + kc, kb + to);
          copy16(v + at + vc, vb + to);
        } else {
          const uint32_t at = (static_cast<uint32_t>(page[c]) & ~1u) + in_page * ROWB;
          copy16(k, at + kc, kb + to);
          copy16(v, at + vc, vb + to);
        }
      }
    };
    // Values no row sees become zero, and where there are infinities or NaN
    // among the others these too: times a probability of zero they would be
    // NaN in the rows that do not see them.
    auto clean = [&](char* vb, int j0, uint64_t gone) {
      uint32_t odd = 0;
#pragma unroll
      for (int e = 0; e < TILE / 16 / (64 * kTileWaves); ++e) {
        const int at = 64 * kTileWaves * e + here(threadIdx.x);
        const int r = at / PIECES;
        U4* v = reinterpret_cast<U4*>(vb + 16 * at);
        U4 x = *v;
        const bool seen = j0 + r >= pt.lo && j0 + r < pt.hi && !(gone >> r & 1);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          x[w] = seen ? x[w] : 0u;
          odd |= odd_bits<T>(x[w]);
          x[w] = finite_or_zero<T>(x[w]);
        }
        *v = x;
      }
      odd_values |= __syncthreads_or((odd & kOdd) != 0) != 0;
    };

    const int kat = col * ROWB + 16 * (g ^ k_bits<D>(col));
    const int vrow = 4 * g + ((lane & 15) >> 2);           // V row of a transposing read
    const int vpiece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
    const int vat = vrow * ROWB + 16 * (vpiece ^ v_bits<D>(vrow)) + 8 * (lane & 1);

    // S^T = K Q^T.  Fragments are read AHEAD steps before their products; steps
    // that share an address but for a constant follow one another.
    auto scores = [&](const char* kb, F16 (&sc)[EB]) {
      const auto step = [](int n) {
        return D == 256 ? n / 2 + 8 * (n % 2) : n / EB;
      };
      const int kx = here(kat);
      // first in line for the matrix pipe: the other wave of the SIMD does its softmax
      __builtin_amdgcn_s_setprio(1);
      U4 kf[AHEAD];
      auto read = [&](int n) {
        const int e = EB == 2 ? n % 2 : 0, d = step(n);
        return *reinterpret_cast<const U4*>(kb + 32 * e * ROWB + (kx ^ 32 * (d & 7)) +
                                            256 * (d >> 3));
      };
      constexpr int N = EB * D / 16;
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) kf[n] = read(n);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int e = EB == 2 ? n % 2 : 0;
        sc[e] = mfma32(kf[n % AHEAD], q[step(n)], n < EB ? F16{} : sc[e], T{});
        if (n + AHEAD < N) kf[n % AHEAD] = read(n + AHEAD);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (n + AHEAD < N) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    };

    // Softmax of the scores, O^T += V^T P^T.
    auto products = [&](const char* vb, int j0, uint64_t gone, F16 (&sc)[EB]) {
      if (is_edge(pt, j0, KT, gone != 0)) {
        // key numbers relative to the lane's first: compile-time constants
        const int at = j0 + 4 * g;
        const uint64_t lost = gone >> (4 * g);
        int lo = 0, hi = 0;
        const int r = wr0 + here(lane) % 32;
        if (r < rows) visible(a, s, a.by_G.div(r), &lo, &hi);
        lo -= at;
        hi -= at;
#pragma unroll
        for (int e = 0; e < EB; ++e)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = 32 * e + 8 * (i >> 2) + (i & 3);
            sc[e][i] = key < lo || key >= hi    ? kNegInf
                       : (lost >> key & 1) != 0 ? __builtin_nanf("")
                                                : sc[e][i];
          }
      }
      __builtin_amdgcn_s_setprio(0);
      float top = sc[0][0];
#pragma unroll
      for (int e = 0; e < EB; ++e)
#pragma unroll
        for (int i = 0; i < 16; ++i) top = fmaxf(top, sc[e][i]);
      const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top),
                                                       false, false);
      top = fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1]));
      if (__any(top * a.scale_log2 > m + kLag)) {
        const float up = fmaxf(m, scaled_max(top, a.scale_log2));
        const float keep = m == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m - up);
        m = up;
        l *= keep;
#pragma unroll
        for (int n = 0; n < NB; ++n) o[n] *= keep;
      }
      float shift = m == kNegInf ? 0.0f : kUp<T> - m;
      if (__any(is_far(m))) {
        const bool far = is_far(m);
        shift = far ? kUp<T> : shift;
#pragma unroll
        for (int e = 0; e < EB; ++e)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sc[e][i] = far ? near_score(sc[e][i], a.scale_log2, m) : sc[e][i];
      }
      U4 pr[2 * EB][NP];
#pragma unroll
      for (int st = 0; st < 2 * EB; ++st) {
        float p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          p[i] = __builtin_amdgcn_exp2f(fmaf(sc[st / 2][8 * (st % 2) + i], a.scale_log2, shift));
          if constexpr (!kSumParts<T, NP>) l += p[i];
        }
        split_probs<T, NP>(p, pr[st]);
        if constexpr (kSumParts<T, NP>) {
#pragma unroll
          for (int n = 0; n < NP; ++n)
#pragma unroll
            for (int w = 0; w < 4; ++w) l = add_pair<T>(pr[st][n][w], l);
        }
      }
      const int vx = here(vat);
      U4 vf[AHEAD];
      auto read = [&](int n) {
        const int d = n % NB;
        const char* src = vb + 16 * (n / NB) * ROWB + (vx ^ 64 * (d & 3)) + 256 * (d >> 2);
        const U2 x = __builtin_bit_cast(
            U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4*)src));
        const U2 y = __builtin_bit_cast(
            U2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsS4*)(src + 8 * ROWB)));
        return U4{x[0], x[1], y[0], y[1]};
      };
      constexpr int N = 2 * EB * NB;
#pragma unroll
      for (int n = 0; n < AHEAD; ++n) vf[n] = read(n);
#pragma unroll
      for (int n = 0; n < N; ++n) {
#pragma unroll
        for (int z = NP - 1; z >= 0; --z)
          o[n % NB] = mfma32(vf[n % AHEAD], pr[n / NB][z], o[n % NB], T{});
        if (n + AHEAD < N) vf[n % AHEAD] = read(n + AHEAD);
      }
      __builtin_amdgcn_sched_group_barrier(0x100, 2 * AHEAD, 1);
#pragma unroll
      for (int n = 0; n < N; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x008, NP, 1);
        if (n + AHEAD < N) __builtin_amdgcn_sched_group_barrier(0x100, 2, 1);
      }
    };

    // Tile t is computed while t + 2 is copied (past the last tile, its last
    // key again); before the barrier that ends a tile a wave waits until only
    // that copy is in flight, so its part of the next tile is complete.  The
    // page numbers come from LDS, as many as fit at a time: with no other load
    // in the loop, the count of copies in flight is known.
    for (first = k0; first < k1; first = end) {
      const int64_t most = static_cast<int64_t>(first) + (int64_t{kPages - 1} << a.page_shift);
      end = k1 < most ? k1 : static_cast<int>(most - (most - first) % KT);
      const int p0 = first >> a.page_shift, p1 = (end - 1) >> a.page_shift;
      bool lost = false;
      __syncthreads();  // the last tile of the keys before is done
      for (int p = p0 + static_cast<int>(threadIdx.x); p <= p1; p += 64 * kTileWaves) {
        const int page = p < a.max_pages ? table[p] : -1;
        const bool bad = page < 0 || page >= a.pages;
        if constexpr (WIDE)
          page_lds[p - p0] = bad ? -1 : page;
        else
          page_lds[p - p0] = (((static_cast<uint32_t>(bad ? 0 : page) * a.Hk + h) << a.page_shift) *
                              ROWB) | bad;
        lost |= bad;
      }
      const bool any_gone = __syncthreads_or(lost);
      int page[COPIES];
      find_pages(first, page);
      copy(page, first, k_lds, v_lds);
      find_pages(first + KT, page);
      copy(page, first + KT, k_lds + TILE, v_lds + TILE);
      find_pages(first + 2 * KT, page);
      wait_copies<2 * COPIES>();
      __syncthreads();
      // The rows' loads end here: a wait for them inside the loop would be one
      // for the copies as well.
#pragma unroll
      for (int d = 0; d < D / 16; ++d) asm volatile("" : "+v"(q[d]));
      int now = 0, then = 2 * TILE;
#pragma unroll 1
      for (int j0 = first; j0 < end; j0 += KT) {
        const uint64_t gone = any_gone ? gone_of(j0) : 0;
        if (is_edge(pt, j0, KT, gone != 0)) clean(v_lds + now, j0, gone);
        copy(page, j0 + 2 * KT, k_lds + then, v_lds + then);
        find_pages(j0 + 3 * KT, page);
        F16 sc[EB];
        scores(k_lds + now, sc);
        products(v_lds + now, j0, gone, sc);
        wait_copies<2 * COPIES>();
        __syncthreads();
        now = now == 2 * TILE ? 0 : now + TILE;
        then = then == 2 * TILE ? 0 : then + TILE;
      }
      wait_copies<0>();
    }

    {
      const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l),
                                                       false, false);
      const float sum = __uint_as_float(sw[0]) + __uint_as_float(sw[1]);
      const int r = wr0 + col;
      if (r < rows) {
        const int i = a.by_G.div(r);
        const int hq = h * a.G + r - i * a.G;
        const int64_t at_row = static_cast<int64_t>(split) * a.T * Hq + (s.q0 + i) * Hq + hq;
        if (tg.nsplit > 1 && g == 0) part_ml[at_row] = make_float2(m, sum);
        const float inv = 1.0f / sum;
        int lo, hi;
        visible(a, s, i, &lo, &hi);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const int d = 32 * n + 8 * i4 + 4 * g;
            float y[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) y[c] = o[n][4 * i4 + c];
            if (tg.nsplit > 1) {
              store_wide(part_o + at_row * D + d, y);
            } else {
#pragma unroll
              for (int c = 0; c < 4; ++c) y[c] = hi > lo ? y[c] * inv : 0.0f;
              store_wide(static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs + d, y);
            }
          }
      }
    }

    if (odd_values) {
      __syncthreads();
      put_back<T, TO>(a, s, table, h, pt, k0, k1, KT, r0, kTileRows, 64 * kTileWaves, split,
                      tg.nsplit > 1, part_o);
    }
    __syncthreads();  // the next tile of rows takes the buffers
  }
}

template <typename T, typename TO, int D>
hipError_t launch_tiles(const AttnPlan& plan, const AttnArgs& a, void* workspace, hipStream_t s) {
  const TileGrid tg{static_cast<int>(plan.row_tiles), plan.nsplit, plan.chunk};
  float* part_o = static_cast<float*>(workspace);
  float2* part_ml =
      reinterpret_cast<float2*>(part_o + static_cast<int64_t>(plan.nsplit) * a.T * a.Hk * a.G * D);
  const dim3 grid(static_cast<uint32_t>(a.B * a.Hk * plan.row_tiles * plan.nsplit));
  // 32-bit offsets into K and V where they reach (D = 64 of the above: 193 us
  // with 64-bit ones, 186 with these)
  const bool wide = ((static_cast<uint64_t>(a.pages) * a.Hk << a.page_shift) * 2 * D) >> 32 != 0;
  if (wide)
    many_rows_kernel<T, TO, D, true><<<grid, 64 * kTileWaves, 0, s>>>(a, tg, part_o, part_ml);
  else
    many_rows_kernel<T, TO, D, false><<<grid, 64 * kTileWaves, 0, s>>>(a, tg, part_o, part_ml);
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
