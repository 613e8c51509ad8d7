// codes.cuh -- codes of the page-scaled formats: E4M3, or INT8 stored as code + 128.
#pragma once

#include "kvq_common.cuh"

namespace kvq {
namespace runs {

// Four codes of x f, f = 2^-e.  INT8: the sum with 1.5 2^23 + 128 is rounded once, to an integer, and its low byte is
// code + 128; the values are in range (the caller has clamped them where they need not be).
template <bool INT8>
__device__ __forceinline__ uint32_t encode4(float x0, float x1, float x2, float x3, float f) {
  if (INT8) {
    constexpr float kMagic = 12582912.f + 128.f;
    const uint32_t a = __float_as_uint(__fmaf_rn(x0, f, kMagic)), b = __float_as_uint(__fmaf_rn(x1, f, kMagic));
    const uint32_t c = __float_as_uint(__fmaf_rn(x2, f, kMagic)), d = __float_as_uint(__fmaf_rn(x3, f, kMagic));
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
  }
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0 * f, x1 * f), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2 * f, x3 * f), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
template <bool INT8>
__device__ __forceinline__ float decode(uint8_t b) {
  return INT8 ? static_cast<float>(static_cast<int>(b) - 128) : e4m3_bits_to_f32(b);
}

template <bool INT8>
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {  // four codes times f = 2^-d
  return encode4<INT8>(decode<INT8>(w), decode<INT8>(w >> 8), decode<INT8>(w >> 16), decode<INT8>(w >> 24), f);
}
template <bool INT8>
__device__ __forceinline__ uint4 rescale(uint4 w, float f) {
  return make_uint4(rescale4<INT8>(w.x, f), rescale4<INT8>(w.y, f), rescale4<INT8>(w.z, f), rescale4<INT8>(w.w, f));
}

}  // namespace runs
}  // namespace kvq
