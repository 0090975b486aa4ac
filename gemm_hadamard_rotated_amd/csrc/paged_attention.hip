// Attention of new tokens over a paged key/value cache (pq1_paged_attention).
//
// Row (b, i, h) sees keys [lo, hi) of its sequence and computes
//   o = sum_j 2^(c q.k_j - m) v_j / sum_j 2^(c q.k_j - m),   c = scale log2(e),
// with a running maximum m over tiles of keys, so that one pass over the
// cache does: a tile with a larger maximum scales what was summed so far.
#include "attn_device.h"
#include "attn_internal.h"

namespace pq1 {

namespace {

constexpr float kNegInf = -__builtin_inff();

// What a workgroup needs to know of its sequence.
struct Seq {
  int64_t q0;  // first row of q
  int n;       // new tokens
  int kv;      // keys
};

__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int64_t b) {
  int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
  q0 = q0 < 0 ? 0 : q0 > a.T ? a.T : q0;
  q1 = q1 < q0 ? q0 : q1 > a.T ? a.T : q1;
  const int kv = a.kv_len[b];
  return {q0, static_cast<int>(q1 - q0), kv < 0 ? 0 : kv};
}

// Keys [lo, hi) that row i sees.
__device__ __forceinline__ void visible(const AttnArgs& a, const Seq& s, int i, int* lo, int* hi) {
  *lo = 0;
  *hi = s.kv;
  if (a.causal) {
    const int64_t end = static_cast<int64_t>(s.kv) - s.n + i + 1;
    *hi = end < 0 ? 0 : static_cast<int>(end);
    if (a.window > 0 && *hi > a.window) *lo = *hi - a.window;
  }
}

// First cache row of key j for cache head h, or -1 for a page that is not in
// the cache.
__device__ __forceinline__ int64_t key_row(const AttnArgs& a, int64_t b, int h, int j) {
  const int64_t p = j >> a.page_shift;
  if (p >= a.max_pages) return -1;
  const int64_t page = a.table[b * a.max_pages + p];
  if (page < 0 || page >= a.pages) return -1;
  return ((page * a.Hk + h) << a.page_shift) + (j & ((1 << a.page_shift) - 1));
}

// One wave per row: 64 keys at a time, one a lane, for the scores; then every
// lane sums D / 64 dimensions over those keys.
template <typename T, typename TO, int D>
__global__ __launch_bounds__(64) void row_kernel(AttnArgs a, int row_tiles) {
  __shared__ float qs[D];
  __shared__ float ps[64];
  __shared__ int64_t rows[64];
  const int lane = threadIdx.x;
  const int Hq = a.Hk * a.G;
  const int64_t b = blockIdx.x / (static_cast<int64_t>(row_tiles) * Hq);
  const int rem = static_cast<int>(blockIdx.x - b * row_tiles * Hq);
  const int tile = rem / Hq, hq = rem - tile * Hq, h = hq / a.G;
  const Seq s = load_seq(a, b);
  const T* K = static_cast<const T*>(a.k_cache);
  const T* V = static_cast<const T*>(a.v_cache);
  constexpr int N = D / 64;
  for (int i = tile; i < s.n; i += row_tiles) {
    const T* q = static_cast<const T*>(a.q) + (s.q0 + i) * a.q_ts + hq * a.q_hs;
    __syncthreads();
#pragma unroll
    for (int d = 0; d < N; ++d) qs[lane + 64 * d] = static_cast<float>(q[lane + 64 * d]);
    __syncthreads();
    int lo, hi;
    visible(a, s, i, &lo, &hi);
    float m = kNegInf, l = 0.0f, acc[N] = {};
    for (int j0 = lo; j0 < hi; j0 += 64) {
      const int j = j0 + lane;
      float x = kNegInf;
      int64_t row = -1;
      if (j < hi) {
        row = key_row(a, b, h, j);
        x = __builtin_nanf("");
        if (row >= 0) {
          x = 0.0f;
          for (int d = 0; d < D; d += 8) {
            float k[8];
            load_wide(K + row * D + d, k);
#pragma unroll
            for (int e = 0; e < 8; ++e) x = fmaf(qs[d + e], k[e], x);
          }
          x *= a.scale_log2;
        }
      }
      float top = x;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
      top = fmaxf(m, top);
      const float base = top == kNegInf ? 0.0f : top;  // all scores so far -inf
      const float p = j < hi ? exp2f(x - base) : 0.0f;
      float sum = p;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
      const float keep = m == kNegInf ? 0.0f : exp2f(m - base);
      m = top;
      l = l * keep + sum;
      __syncthreads();
      ps[lane] = p;
      rows[lane] = row;
      __syncthreads();
#pragma unroll
      for (int d = 0; d < N; ++d) acc[d] *= keep;
      const int cnt = hi - j0 < 64 ? hi - j0 : 64;
      for (int e = 0; e < cnt; ++e) {
        if (rows[e] < 0) continue;  // its probability is NaN already
#pragma unroll
        for (int d = 0; d < N; ++d)
          acc[d] = fmaf(ps[e], static_cast<float>(V[rows[e] * D + lane + 64 * d]), acc[d]);
      }
    }
    TO* o = static_cast<TO*>(a.out) + (s.q0 + i) * a.o_ts + hq * a.o_hs;
#pragma unroll
    for (int d = 0; d < N; ++d)
      o[lane + 64 * d] = static_cast<TO>(hi > lo ? acc[d] / l : 0.0f);
  }
}

template <typename T, typename TO>
hipError_t launch_dim(const AttnPlan& plan, const AttnArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(a.B * a.Hk * a.G * plan.row_tiles));
  const int rt = static_cast<int>(plan.row_tiles);
  switch (a.D) {
    case 64: row_kernel<T, TO, 64><<<grid, 64, 0, s>>>(a, rt); break;
    case 128: row_kernel<T, TO, 128><<<grid, 64, 0, s>>>(a, rt); break;
    default: row_kernel<T, TO, 256><<<grid, 64, 0, s>>>(a, rt); break;
  }
  return hipGetLastError();
}

}  // namespace

AttnPlan plan_attention(int64_t B, int64_t T, int Hq, int Hk, int D, int64_t max_q,
                        int64_t max_kv) {
  AttnPlan p;
  p.row_tiles = max_q < 1 ? 1 : max_q < T ? max_q : T;
  p.fits = B <= 0x7fffffff / Hq && B * Hq <= 0x7fffffff / p.row_tiles;
  return p;
}

hipError_t launch_attention(const AttnPlan& plan, const AttnArgs& a, int dtype, int out_dtype,
                            void* workspace, hipStream_t s) {
  if (dtype == PQ1_BF16)
    return out_dtype == PQ1_F32 ? launch_dim<bf16, float>(plan, a, s)
                                : launch_dim<bf16, bf16>(plan, a, s);
  return out_dtype == PQ1_F32 ? launch_dim<f16, float>(plan, a, s)
                              : launch_dim<f16, f16>(plan, a, s);
}

}  // namespace pq1
