// Element types of the attention-layer kernels: widening loads and rounding
// stores of 1, 4 or 8 consecutive elements.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace pq1 {

using f16 = _Float16;
using bf16 = __bf16;

template <typename T, int N>
struct alignas(sizeof(T) * N <= 16 ? sizeof(T) * N : 16) Pack {
  T e[N];
};

template <typename T, int N>
__device__ __forceinline__ void load_wide(const T* p, float (&o)[N]) {
  const Pack<T, N> v = *reinterpret_cast<const Pack<T, N>*>(p);
#pragma unroll
  for (int i = 0; i < N; ++i) o[i] = static_cast<float>(v.e[i]);
}

// The conversions round to nearest, ties to even (hardware on gfx950).
template <typename T, int N>
__device__ __forceinline__ void store_wide(T* p, const float (&v)[N]) {
  Pack<T, N> r;
#pragma unroll
  for (int i = 0; i < N; ++i) r.e[i] = static_cast<T>(v[i]);
  *reinterpret_cast<Pack<T, N>*>(p) = r;
}

}  // namespace pq1
