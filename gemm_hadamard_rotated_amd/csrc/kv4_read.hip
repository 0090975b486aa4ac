// Rows of a 4-bit cache read back as numbers (pq1_kv4_read).
//
// A lane takes 8 codes (4 bytes) at a time and writes 8 numbers, so a wave writes
// whole lines of memory; four such eights of a thread are in flight at once where
// there are many (50000 rows of 4 heads of 256: 79 us with one, 68 with four), all
// their slots first, then all their codes.  Bound: the writes; those rows take 40 us
// now, 6.5 TB/s, a prefix of 333 tokens 2.9 us, as an empty kernel.
#include "attn_device.h"
#include "attn_internal.h"
#include "kv4_format.h"

namespace pq1 {

namespace {

constexpr int kThreads = 256;

struct ReadDims {
  FastDiv per_token;  // eights of a token: of its keys, then of its values
  FastDiv per_head;
  int keys;           // eights of its keys
  int64_t first;      // token of the launch's first workgroup
  uint32_t tokens;    // tokens of the launch
};

__device__ __forceinline__ void widen(uint32_t codes, uint32_t byte, float (&v)[8]) {
  using F2 = __attribute__((ext_vector_type(2))) float;
  const float s = scale_of(byte);
  F2 p[4];
  p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0);
  p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1);
  p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 2);
  p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 3);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = p[i / 2][i % 2];
}

// PAST: past the caches.
template <bool PAST, typename TO>
__device__ __forceinline__ void store_eight(TO* dst, const float (&v)[8]) {
  if constexpr (PAST) {
    using U4 = __attribute__((ext_vector_type(4))) uint32_t;
    constexpr int N = sizeof(TO) * 8 / 16;
    struct Words {
      U4 w[N];
    };
    Pack<TO, 8> r;
#pragma unroll
    for (int i = 0; i < 8; ++i) r.e[i] = static_cast<TO>(v[i]);
    const Words x = __builtin_bit_cast(Words, r);
#pragma unroll
    for (int n = 0; n < N; ++n) __builtin_nontemporal_store(x.w[n], reinterpret_cast<U4*>(dst) + n);
  } else {
    store_wide(dst, v);
  }
}

template <typename TO, int U, bool PAST>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Read4Args a, ReadDims dm) {
  // All slots are read, then all codes: two waits for memory in all.
  uint32_t w[U], h[U], codes[U], byte[U];
  int64_t t[U], slot[U];
  bool mine[U], of_v[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t u = (blockIdx.x * U + k) * kThreads + threadIdx.x;
    uint32_t tl = dm.per_token.div(u);
    w[k] = u - tl * dm.per_token.d;
    mine[k] = tl < dm.tokens;
    tl = mine[k] ? tl : 0;
    t[k] = dm.first + tl;
    slot[k] = a.slots[t[k]];
    const bool value = w[k] >= static_cast<uint32_t>(dm.keys);
    if (value) w[k] -= dm.keys;
    h[k] = dm.per_head.div(w[k]);
    w[k] -= h[k] * dm.per_head.d;
    // keys first, unless only values are wanted
    of_v[k] = value || a.k_out == nullptr;
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const bool stored = slot[k] >= 0 && slot[k] < a.slot_count;
    const int64_t at = stored ? slot[k] : 0;
    const int64_t page = at >> a.page_shift;
    const int64_t row = ((page * a.H + h[k]) << a.page_shift) + (at - (page << a.page_shift));
    const uint32_t c =
        reinterpret_cast<const uint32_t*>((of_v[k] ? a.v : a.k) + row * (a.D / 2))[w[k]];
    const uint32_t s = ((of_v[k] ? a.v_scale : a.k_scale) + row * (a.D / kGroup4))[w[k] / 4];
    codes[k] = stored ? c : 0;
    byte[k] = stored ? s : 0;
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (!mine[k]) continue;
    TO* const dst = (of_v[k] ? static_cast<TO*>(a.v_out) + t[k] * a.v_ts + h[k] * a.v_hs
                             : static_cast<TO*>(a.k_out) + t[k] * a.k_ts + h[k] * a.k_hs) + 8 * w[k];
    float v[8];
    widen(codes[k], byte[k], v);
    store_eight<PAST>(dst, v);
  }
}

template <typename TO, int U, bool PAST>
hipError_t launch_units(const Read4Args& a, ReadDims dm, hipStream_t s) {
  // a launch holds less than 2^32 threads
  const int64_t per_token = dm.per_token.d;
  const int64_t most = ((int64_t{1} << 32) - 2 * U * kThreads) / per_token;
  for (dm.first = 0; dm.first < a.T; dm.first += most) {
    dm.tokens = static_cast<uint32_t>(a.T - dm.first < most ? a.T - dm.first : most);
    const int64_t blocks = (dm.tokens * per_token + U * kThreads - 1) / (U * kThreads);
    kv4_read_kernel<TO, U, PAST><<<dim3(static_cast<uint32_t>(blocks)), kThreads, 0, s>>>(a, dm);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TO>
hipError_t launch(const Read4Args& a, hipStream_t s) {
  ReadDims dm;
  const int64_t keys = static_cast<int64_t>(a.H) * (a.D / 8);
  const bool both = a.k_out != nullptr && a.v_out != nullptr;
  const int64_t per_token = both ? 2 * keys : keys;
  dm.per_token = FastDiv(static_cast<uint32_t>(per_token));
  dm.per_head = FastDiv(a.D / 8);
  dm.keys = static_cast<int>(keys);
  // Up to eight workgroups for each CU: an eight a thread, so that more CUs take part.
  if (a.T * per_token < 256 * 8 * kThreads) return launch_units<TO, 1, false>(a, dm, s);
  // Numbers that fill more than half of the last-level cache (256 MB) are stored
  // past it: most would be gone before they are read, and what the cache held with
  // them (50000 rows of 4 heads of 256, three caches in turn: 68 us through it, 40
  // past it; a plain expansion of bytes of that size 46 and 37).
  const bool past = a.T * per_token * 8 * static_cast<int64_t>(sizeof(TO)) > int64_t{128} << 20;
  return past ? launch_units<TO, 4, true>(a, dm, s) : launch_units<TO, 4, false>(a, dm, s);
}

}  // namespace

hipError_t launch_kv4_read(const Read4Args& a, int out_dtype, hipStream_t s) {
  switch (out_dtype) {
    case PQ1_BF16: return launch<bf16>(a, s);
    case PQ1_F16: return launch<f16>(a, s);
    default: return launch<float>(a, s);
  }
}

}  // namespace pq1
