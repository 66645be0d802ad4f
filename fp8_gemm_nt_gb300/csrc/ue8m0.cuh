// Scalar helpers of the scale and element formats and of exponentials, shared by the kernels around the GEMMs.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace dg {

// Bits of the device status word (the GEMM kernels set the same ones).
enum : uint32_t { kTimeoutBit = 1u << 5, kBadIndexBit = 1u << 6 };

// Least code e in [1, 254] with amax <= 448 * 2^(e - 127); for 0 the least of all, 1.
// 448 = 1.75 * 2^8: the exponent of amax less 8, one more if the mantissa is above 0.75 = 0x600000 / 2^23,
// which is when adding 0x1FFFFF carries into the exponent.
__device__ __forceinline__ int ue8m0_for_amax(float amax) {
  const int e = static_cast<int>((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 8;
  return min(max(e, 1), 254);
}

// 2^(127 - e) for a code e in [1, 254]: what brings a group to E4M3's range (2^-127 is subnormal).
__device__ __forceinline__ float ue8m0_inverse(int e) {
  return __uint_as_float(max(static_cast<uint32_t>(254 - e) << 23, 0x00400000u));
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

// 2^v and 1 / v within two units of the last place (results below 2^-126 are 0).
__device__ __forceinline__ float exp2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

}  // namespace dg
