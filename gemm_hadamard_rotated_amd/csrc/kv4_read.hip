// Rows of a 4-bit cache read back as numbers (pq1_kv4_read).
//
// A lane takes 8 codes (4 bytes) at a time and writes 8 numbers, so a wave writes
// whole lines of memory; four such eights of a thread are in flight at once where
// there are many.  Bound: the writes.
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

template <typename TO>
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

template <typename TO, int U>
__global__ __launch_bounds__(kThreads) void kv4_read_kernel(Read4Args a, ReadDims dm) {
  TO* dst[U];
  uint32_t codes[U], byte[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t u = (blockIdx.x * U + k) * kThreads + threadIdx.x;
    const uint32_t tl = dm.per_token.div(u);
    dst[k] = nullptr;
    codes[k] = byte[k] = 0;
    if (tl >= dm.tokens) continue;
    const int64_t t = dm.first + tl;
    uint32_t w = u - tl * dm.per_token.d;
    const bool value = w >= static_cast<uint32_t>(dm.keys);
    if (value) w -= dm.keys;
    const uint32_t h = dm.per_head.div(w);
    w -= h * dm.per_head.d;
    // keys first, unless only values are wanted
    const bool of_v = value || a.k_out == nullptr;
    dst[k] = (of_v ? static_cast<TO*>(a.v_out) + t * a.v_ts + h * a.v_hs
                   : static_cast<TO*>(a.k_out) + t * a.k_ts + h * a.k_hs) + 8 * w;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.slot_count) continue;
    const int64_t page = slot >> a.page_shift;
    const int64_t row = ((page * a.H + h) << a.page_shift) + (slot - (page << a.page_shift));
    codes[k] = reinterpret_cast<const uint32_t*>((of_v ? a.v : a.k) + row * (a.D / 2))[w];
    byte[k] = ((of_v ? a.v_scale : a.k_scale) + row * (a.D / kGroup4))[w / 4];
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (dst[k] == nullptr) continue;
    float v[8];
    widen<TO>(codes[k], byte[k], v);
    store_wide(dst[k], v);
  }
}

template <typename TO, int U>
hipError_t launch_units(const Read4Args& a, ReadDims dm, hipStream_t s) {
  // a launch holds less than 2^32 threads
  const int64_t per_token = dm.per_token.d;
  const int64_t most = ((int64_t{1} << 32) - 2 * U * kThreads) / per_token;
  for (dm.first = 0; dm.first < a.T; dm.first += most) {
    dm.tokens = static_cast<uint32_t>(a.T - dm.first < most ? a.T - dm.first : most);
    const int64_t blocks = (dm.tokens * per_token + U * kThreads - 1) / (U * kThreads);
    kv4_read_kernel<TO, U><<<dim3(static_cast<uint32_t>(blocks)), kThreads, 0, s>>>(a, dm);
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
  return a.T * per_token < 256 * 8 * kThreads ? launch_units<TO, 1>(a, dm, s)
                                              : launch_units<TO, 4>(a, dm, s);
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
