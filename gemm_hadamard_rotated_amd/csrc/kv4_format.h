// The numbers of a 4-bit cache on the device.  A code is e2m1: a sign and one of
// 0, 0.5, 1, 1.5, 2, 3, 4, 6; 32 neighbours of a head share a scale byte b, which
// stands for 2^(b - 127) (255: NaN, whatever the codes).  gfx950 converts pairs of
// codes both ways in one instruction, at the rate of any other vector
// instruction (32 T lanes/s), so nothing else was tried.
#pragma once

#include "attn_device.h"

namespace pq1 {

constexpr int kGroup4 = 32;        // elements that share a scale
constexpr uint32_t kNanScale = 255;

// Exponents that the append gives a scale: values down to half of it are
// normal numbers of fp32 and bf16, or numbers of f16, and six times it is finite.
template <typename T>
constexpr int kLeastExp = __is_same(T, bf16) ? -100 : -23;
template <typename T>
constexpr int kMostExp = __is_same(T, bf16) ? 125 : 13;

__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Two codes (byte SEL of `codes`) as a pair of T.
template <typename T, int SEL>
__device__ __forceinline__ uint32_t pair_of(uint32_t codes, float scale) {
  if constexpr (__is_same(T, bf16))
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
  else
    return __builtin_bit_cast(uint32_t,
                              __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, scale, SEL));
}
// The same with a byte number that unrolling makes a constant.
template <typename T>
__device__ __forceinline__ uint32_t pair_at(uint32_t codes, float scale, int sel) {
  switch (sel) {
    case 0: return pair_of<T, 0>(codes, scale);
    case 1: return pair_of<T, 1>(codes, scale);
    case 2: return pair_of<T, 2>(codes, scale);
    default: return pair_of<T, 3>(codes, scale);
  }
}
// Eight codes as four pairs.
template <typename T>
__device__ __forceinline__ void pairs_of(uint32_t codes, float scale, uint32_t (&out)[4]) {
  out[0] = pair_of<T, 0>(codes, scale);
  out[1] = pair_of<T, 1>(codes, scale);
  out[2] = pair_of<T, 2>(codes, scale);
  out[3] = pair_of<T, 3>(codes, scale);
}

// The codes of a word, all four bits of each, whose values under this scale are
// infinities of T (from `least` on: 4 at twice the largest scale of the append, then
// 2, 1 and 0.5) or NaN (all of them).  The scale is past the append's range.
template <typename T>
__device__ __forceinline__ uint32_t odd_codes(uint32_t codes, uint32_t byte) {
  const int past = static_cast<int>(byte) - (kMostExp<T> + 127);
  const int least = byte == kNanScale ? 0 : past > 3 ? 1 : 8 - 2 * past;
  const uint32_t top =
      ((codes & 0x77777777u) + static_cast<uint32_t>(8 - least) * 0x11111111u) & 0x88888888u;
  return top | (top - (top >> 3));
}

// Scale byte of a group whose largest magnitude has these bits: the least
// exponent e with top <= 7 * 2^e, so that the largest code, 6, is off by no more
// than half the step below it.
template <typename T>
__device__ __forceinline__ uint32_t scale_for(uint32_t top) {
  int e = static_cast<int>(top >> 23) - 127 - 2 + ((top & 0x7fffffu) > 0x600000u);
  e = e < kLeastExp<T> ? kLeastExp<T> : e > kMostExp<T> ? kMostExp<T> : e;
  return top >= 0x7f800000u ? kNanScale : static_cast<uint32_t>(e + 127);
}

// Eight values as codes, to nearest, ties to even codes, past six to six.
__device__ __forceinline__ uint32_t codes_of(const float (&v)[8], uint32_t byte) {
  const float s = scale_of(byte);
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0], v[1], s, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2], v[3], s, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4], v[5], s, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6], v[7], s, 3);
  return byte == kNanScale ? 0u : c;
}

}  // namespace pq1
