// Codes of the 8-bit formats, shared by the state cache and the norm's 8-bit output.
#pragma once

#include "common.hpp"

namespace dr {

// The integer nearest to the exact quotient x / s (ties to even), |x / s| < 128: a candidate from the
// hardware reciprocal, at most one off next to a tie, set right by its remainder, which an fma gives exactly
// (x and q s are multiples of the smaller one's last place and differ by less than 2 s). Twice the remainder is
// compared with s: half of s is no float32 number when s lies below 2^-125.
__device__ __forceinline__ int code_int8(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x), r2 = r + r;
  const bool odd = ((int)q & 1) != 0;
  if (r2 > s || (r2 == s && odd)) q += 1.f;
  if (r2 < -s || (r2 == -s && odd)) q -= 1.f;
  return (int)q;
}
// A row's scale from its largest magnitude `amax` (bits `top`), and what its values are multiplied by.
// int8: amax times the fp32 number next to 1/127 (within 1.5 roundings of amax / 127): the value that torch's division
// of a tensor by 127 gives on the GPU, so that caches written by such a program hold the same codes.
// e4m3: amax = m 2^(E - 126), m in [1/2, 1): amax <= 448 2^j (448 = 7/8 2^9) for j = E - 135, or one more if
// m > 7/8; a subnormal amax (E = 0) takes the least scale; the inverse is exact.
template <bool E4M3>
__device__ __forceinline__ float row_scale(uint32_t top, float* inv) {
  if constexpr (E4M3) {
    const int E = (int)(top >> 23);
    int j = E - 135 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
    j = max(j, -126);
    *inv = __builtin_bit_cast(float, (uint32_t)(127 - j) << 23);
    return __builtin_bit_cast(float, (uint32_t)(j + 127) << 23);
  } else {
    const float scale = fmaxf(__builtin_bit_cast(float, top) * (1.f / 127.f), 0x1p-126f);
    *inv = __builtin_amdgcn_rcpf(scale);
    return scale;
  }
}
// Four values' codes, one byte each.
template <bool E4M3>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float scale, float inv) {
  if constexpr (E4M3) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  } else {
    return (uint32_t)(code_int8(a, scale, inv) & 0xff) | (uint32_t)(code_int8(b, scale, inv) & 0xff) << 8 |
           (uint32_t)(code_int8(c, scale, inv) & 0xff) << 16 | (uint32_t)(code_int8(d, scale, inv) & 0xff) << 24;
  }
}

}  // namespace dr
