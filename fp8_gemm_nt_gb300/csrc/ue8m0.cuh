// Scalar helpers of the scale and element formats, shared by the kernels around the GEMMs.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dg {

// Bits of the device status word (the GEMM kernels set the same ones).
enum : uint32_t { kBadIndexBit = 1u << 6 };

// 2^(e - 127); code 0 is the subnormal 2^-127, code 255 NaN.
__device__ __forceinline__ float ue8m0_value(uint32_t e) {
  return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}

// Least code e in [1, 254] with amax <= 448 * 2^(e - 127); 127 (scale 1) for a group of zeros.
// 448 = 1.75 * 2^8: the mantissa of amax decides whether its own exponent less 8 is enough.
__device__ __forceinline__ int ue8m0_for_amax(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0) return 127;
  const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1 : e > 254 ? 254 : e;
}

// 2^(127 - e) for a code e in [1, 254]: what brings a group to E4M3's range.
__device__ __forceinline__ float ue8m0_inverse(int e) {
  return __uint_as_float(e == 254 ? 0x00400000u : static_cast<uint32_t>(254 - e) << 23);
}

// Four floats -> four E4M3 bytes, round to nearest even; |v| <= 448 or NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ void unpack_bf16(uint32_t w, float& a, float& b) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xFFFF0000u);
}

}  // namespace dg
