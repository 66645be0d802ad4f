// A warp's rows of router logits: how its lanes hold a row, and sums and maxima over it.
#pragma once

#include <cmath>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>

#include "dg.h"
#include "ue8m0.cuh"

namespace dg {
namespace rows {

constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(p))) << 16);
}
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// A lane's logits of a row: kVec consecutive ones (1, or 16 bytes where rows are aligned to that) of every
// 32 * kVec; -infinity, as a masked expert's, past the row's end.
template <class L, int J, int kVec>
struct Lane {
  static constexpr int kCount = J * kVec;
  static __device__ __forceinline__ int index(int lane, int i) { return (i / kVec * 32 + lane) * kVec + i % kVec; }
  static __device__ __forceinline__ void load(const L* row, int lane, int E, float (&v)[kCount]) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int at = index(lane, j * kVec);
#pragma unroll
      for (int c = 0; c < kVec; ++c) v[j * kVec + c] = -INFINITY;
      if (at >= E) continue;
      if constexpr (kVec == 1) {
        v[j] = load_logit(row + at);
      } else {
        const uint4 u = __ldcg(reinterpret_cast<const uint4*>(row + at));
        if constexpr (kVec == 4) {
          v[j * 4] = __uint_as_float(u.x), v[j * 4 + 1] = __uint_as_float(u.y), v[j * 4 + 2] = __uint_as_float(u.z), v[j * 4 + 3] = __uint_as_float(u.w);
        } else {
          unpack_bf16(u.x, v[j * 8], v[j * 8 + 1]);
          unpack_bf16(u.y, v[j * 8 + 2], v[j * 8 + 3]);
          unpack_bf16(u.z, v[j * 8 + 4], v[j * 8 + 5]);
          unpack_bf16(u.w, v[j * 8 + 6], v[j * 8 + 7]);
        }
      }
    }
  }
  static __device__ __forceinline__ void store(L* row, int lane, int E, const float (&v)[kCount]) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int at = index(lane, j * kVec);
      if (at >= E) continue;
      if constexpr (kVec == 1)
        store_grad(row + at, v[j]);
      else if constexpr (kVec == 4)
        *reinterpret_cast<float4*>(row + at) = make_float4(v[j * 4], v[j * 4 + 1], v[j * 4 + 2], v[j * 4 + 3]);
      else
        *reinterpret_cast<uint4*>(row + at) = make_uint4(pack_bf16(v[j * 8], v[j * 8 + 1]), pack_bf16(v[j * 8 + 2], v[j * 8 + 3]),
                                                         pack_bf16(v[j * 8 + 4], v[j * 8 + 5]), pack_bf16(v[j * 8 + 6], v[j * 8 + 7]));
    }
  }
};

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}
template <int N>
__device__ __forceinline__ float max_of(const float (&v)[N]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  return m;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// Calls f with a lane's vectors and their length. `aligned`: every row is a whole number of 16-byte pieces.
template <class L, class F>
dg_status with_shape(int E, bool aligned, F f) {
  constexpr int kWide = 16 / sizeof(L);
  using std::integral_constant;
  if (aligned) {
    const integral_constant<int, kWide> vec;
    if (E <= 32 * kWide) return f(integral_constant<int, 1>(), vec);
    if (E <= 64 * kWide) return f(integral_constant<int, 2>(), vec);
    if (E <= 128 * kWide) return f(integral_constant<int, 4>(), vec);
    if constexpr (kWide == 4) return f(integral_constant<int, 8>(), vec);
  }
  const integral_constant<int, 1> one;
  if (E <= 32) return f(integral_constant<int, 1>(), one);
  if (E <= 64) return f(integral_constant<int, 2>(), one);
  if (E <= 128) return f(integral_constant<int, 4>(), one);
  if (E <= 256) return f(integral_constant<int, 8>(), one);
  if (E <= 512) return f(integral_constant<int, 16>(), one);
  return f(integral_constant<int, 32>(), one);
}
template <class L>
bool whole_pieces(const void* p, size_t ld, int E) {
  constexpr size_t kWide = 16 / sizeof(L);
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % kWide == 0 && E % kWide == 0;
}

}  // namespace rows
}  // namespace dg
