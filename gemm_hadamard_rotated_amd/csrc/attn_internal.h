// Internal declarations of the attention-layer kernels (rope.hip,
// paged_attention.hip).  Arguments are validated in api_attention.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attn_plan.h"
#include "pq1.h"

namespace pq1 {

// Unsigned division by a run-time constant: n / d for every 32-bit n.
struct FastDiv {
  uint32_t d = 1, mul = 1, shift = 0;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div) {
    uint32_t l = 0;
    while ((uint64_t{1} << l) < div) ++l;
    mul = static_cast<uint32_t>(((uint64_t{1} << 32) * ((uint64_t{1} << l) - div)) / div + 1);
    shift = l;
  }
  // n / d = (mulhi(mul, n) + n) >> shift, the sum taken in 33 bits
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint64_t t = static_cast<uint64_t>(__umulhi(mul, n)) + n;
    return static_cast<uint32_t>(t >> shift);
  }
};

// One launch of the rotation kernel: `x` streams through it into `y`, and in
// an append also keys and values into the cache.
struct RopeArgs {
  const void* x = nullptr;  // rotated stream (queries of an append; may be absent: Hx = 0)
  int64_t x_ts = 0, x_hs = 0;
  void* y = nullptr;
  int64_t y_ts = 0, y_hs = 0;
  const void* k = nullptr;
  int64_t k_ts = 0, k_hs = 0;
  const void* v = nullptr;
  int64_t v_ts = 0, v_hs = 0;
  const int64_t* slots = nullptr;
  void* k_cache = nullptr;
  void* v_cache = nullptr;
  int64_t slot_count = 0;  // pages * page_size
  int page_shift = 0;
  int Hk = 0;
  const int32_t* positions = nullptr;
  const double* freqs = nullptr;
  int64_t T = 0;
  int Hx = 0, D = 0;
  int rot = 0;  // 0: no rotation
  int axes = 1;
  int section[4] = {0, 0, 0, 0};
  bool interleaved = false, adjacent = false, inverse = false;
};
hipError_t launch_rope(const RopeArgs& a, int in_dtype, int out_dtype, hipStream_t s);

struct AttnArgs {
  const void* q = nullptr;
  int64_t q_ts = 0, q_hs = 0;
  void* out = nullptr;
  int64_t o_ts = 0, o_hs = 0;
  const void* k_cache = nullptr;
  const void* v_cache = nullptr;
  int pages = 0;
  int page_shift = 0;
  int Hk = 0, G = 1, D = 0;  // G: query heads of a cache head
  FastDiv by_G;
  const int32_t* table = nullptr;
  int max_pages = 0;  // of a sequence, in its row of the table
  const int32_t* cu_q = nullptr;
  const int32_t* kv_len = nullptr;
  int64_t B = 0, T = 0;
  float scale_log2 = 0;  // scale * log2(e): the softmax runs in powers of two
  bool causal = false;
  int window = 0;
};

hipError_t launch_many_rows(const AttnPlan& plan, const AttnArgs& a, int dtype, int out_dtype,
                            void* workspace, hipStream_t s);
hipError_t launch_attention(const AttnPlan& plan, const AttnArgs& a, int dtype, int out_dtype,
                            void* workspace, hipStream_t s);

}  // namespace pq1
