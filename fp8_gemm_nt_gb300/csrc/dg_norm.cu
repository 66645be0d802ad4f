// Residual addition + RMS norm with BF16 and E4M3 outputs, and its gradient.
//
//   s = x + r        rstd = (mean(s^2) + eps)^(-1/2)        y = s * rstd * w
//   q = e4m3(y * 2^-n_g), n_g the least integer with max|y_g| * 2^-n_g <= 448, per group g of 128 columns
//
//   g = dy * w       dx = rstd * (g - s rstd * mean(g * s rstd)) + ds        dw = sum_t dy * s rstd
//
// Every sum and statistic is FP32; s, y and dx are rounded once, where they are stored, and q is
// rounded from the FP32 y.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dg.h"
#include "ptx.cuh"
#include "runtime.h"
#include "ue8m0.cuh"

namespace {

using dg::LaunchContext;

constexpr int kVec = 8;                 // elements a thread takes at once
constexpr int kMaxH = 16384;
constexpr int kThreads = 256;           // threads of a forward block, at most (8 vectors each at kMaxH)
constexpr int kGradThreads = 512;       // and of a gradient block, whose threads hold four arrays (4 vectors each)

// Eight consecutive elements, BF16 or FP32, to and from FP32 (loads at L2: the row may have been
// written by the kernel before this one in the stream, whose end this one overlaps).
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = dg::ld_cg_v4(p);
  dg::unpack_bf16(u.x, v[0], v[1]);
  dg::unpack_bf16(u.y, v[2], v[3]);
  dg::unpack_bf16(u.z, v[4], v[5]);
  dg::unpack_bf16(u.w, v[6], v[7]);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const uint4 a = dg::ld_cg_v4(p), b = dg::ld_cg_v4(p + 4);
  v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
  v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(dg::pack_bf16(v[0], v[1]), dg::pack_bf16(v[2], v[3]),
                                            dg::pack_bf16(v[4], v[5]), dg::pack_bf16(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sum over the block's threads, the same value in each. `part`: one float per warp.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  const int warps = blockDim.x / 32;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  float s = 0;
  for (int i = 0; i < warps; ++i) s += part[i];
  return s;
}

template <class R, class W>
struct NormArgs {
  const __nv_bfloat16* x;
  const R* residual;       // or null
  const W* weight;
  __nv_bfloat16* y;        // or null
  uint8_t* q;              // or null, then sf too
  int32_t* sf;
  R* residual_out;         // or null
  float* rstd;             // or null
  int T, H;
  size_t ldx, ldr, ldo;
  float eps, inv_h;
};

// One row per block; a thread holds V vectors of 8 columns, V * 8 FP32 values in registers.
template <class R, class W, int V>
__global__ void __launch_bounds__(kThreads) norm_kernel(const NormArgs<R, W> a) {
  __shared__ float part[kThreads / 32];
  __shared__ uint8_t codes[kMaxH / 128];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int t = blockIdx.x;
  const int nvec = a.H / kVec;
  float v[V][8];
  float sum = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = j * blockDim.x + threadIdx.x;
    if (c < nvec) {
      load8(a.x + t * a.ldx + c * kVec, v[j]);
      if (a.residual) {
        float r[8];
        load8(a.residual + t * a.ldr + c * kVec, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += r[i];
      }
      if (a.residual_out) store8(a.residual_out + t * a.ldo + c * kVec, v[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fmaf(v[j][i], v[j][i], sum);
    }
  }
  // each thread's share of the mean: a sum over the whole row could leave FP32's range before its mean does
  const float rstd = 1.0f / sqrtf(block_sum(sum * a.inv_h, part) + a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = j * blockDim.x + threadIdx.x;
    if (c < nvec) {
      float w[8];
      load8(a.weight + c * kVec, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = v[j][i] * rstd * w[i];
      if (a.y) store8(a.y + static_cast<long long>(t) * a.H + c * kVec, v[j]);
    }
    if (a.q) {
      // a group is 16 neighbouring threads (H % 128 == 0: all 16 have a vector, or none has); an
      // element that is not finite becomes the NaN code and does not count for the scale
      float m = 0;
      if (c < nvec) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = fabsf(v[j][i]);
          if (!(f < INFINITY)) v[j][i] = NAN;
          m = fmaxf(m, f < INFINITY ? f : 0.0f);
        }
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (c < nvec) {
        const int e = dg::ue8m0_for_amax(m);
        const float k = dg::ue8m0_inverse(e);
        const uint32_t lo = dg::pack_e4m3(v[j][0] * k, v[j][1] * k, v[j][2] * k, v[j][3] * k);
        const uint32_t hi = dg::pack_e4m3(v[j][4] * k, v[j][5] * k, v[j][6] * k, v[j][7] * k);
        *reinterpret_cast<uint2*>(a.q + static_cast<long long>(t) * a.H + c * kVec) = make_uint2(lo, hi);
        if ((c & 15) == 0) codes[c / 16] = static_cast<uint8_t>(e);
      }
    }
  }
  if (!a.q) return;
  __syncthreads();
  const int groups = a.H / 128, words = (groups + 3) / 4;
  const long long t4 = (static_cast<long long>(a.T) + 3) / 4 * 4;
  for (int i = threadIdx.x; i < words; i += blockDim.x) {
    uint32_t word = 0;
    for (int b = 0; b < 4 && 4 * i + b < groups; ++b) word |= static_cast<uint32_t>(codes[4 * i + b]) << (8 * b);
    a.sf[i * t4 + t] = static_cast<int32_t>(word);
    if (t == a.T - 1)
      for (long long p = a.T; p < t4; ++p) a.sf[i * t4 + p] = 0;
  }
}

template <class R, class W>
struct NormGradArgs {
  const __nv_bfloat16* dy;
  const R* s;
  const W* weight;
  const float* rstd;
  const R* ds;             // or null
  __nv_bfloat16* dx;       // or null
  R* dresidual;            // or null
  float* partial;          // [gridDim.x, H]
  int T, H;
};

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...: a thread keeps its columns' share of dw in registers
// over all of them, so dw costs one row of partial sums per block.
template <class R, class W, int V>
__global__ void __launch_bounds__(kGradThreads) norm_grad_kernel(const NormGradArgs<R, W> a) {
  __shared__ float part[2][kGradThreads / 32];
  dg::grid_dependency_wait();
  const int nvec = a.H / kVec;
  constexpr bool kKeep = V <= 2;   // four vectors do not fit the registers: weight and s are then read again, from L2
  float w[kKeep ? V : 1][8], dw[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = j * blockDim.x + threadIdx.x;
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0;
    if (kKeep && c < nvec) load8(a.weight + c * kVec, w[kKeep ? j : 0]);
  }
  int flip = 0;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x, flip ^= 1) {
    const long long row = static_cast<long long>(t) * a.H;
    const float rstd = __ldcg(a.rstd + t);
    float dy[V][8], xhat[kKeep ? V : 1][8];
    float sum = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = j * blockDim.x + threadIdx.x;
      if (c < nvec) {
        load8(a.dy + row + c * kVec, dy[j]);
        float (&xh)[8] = xhat[kKeep ? j : 0];
        load8(a.s + row + c * kVec, xh);
        if (!kKeep) load8(a.weight + c * kVec, w[0]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xh[i] *= rstd;
          dw[j][i] = fmaf(dy[j][i], xh[i], dw[j][i]);
          dy[j][i] *= w[kKeep ? j : 0][i];
          sum = fmaf(dy[j][i], xh[i], sum);
        }
      }
    }
    const float mean = block_sum(sum, part[flip]) / static_cast<float>(a.H);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = j * blockDim.x + threadIdx.x;
      if (c < nvec) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0;
        if (a.ds) load8(a.ds + row + c * kVec, d);
        float (&xh)[8] = xhat[kKeep ? j : 0];
        if (!kKeep) load8(a.s + row + c * kVec, xh);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = fmaf(rstd, fmaf(-(kKeep ? xh[i] : xh[i] * rstd), mean, dy[j][i]), d[i]);
        if (a.dx) store8(a.dx + row + c * kVec, d);
        if (a.dresidual) store8(a.dresidual + row + c * kVec, d);
      }
    }
  }
  dg::grid_launch_dependents();
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = j * blockDim.x + threadIdx.x;
    if (c < nvec) store8(a.partial + static_cast<long long>(blockIdx.x) * a.H + c * kVec, dw[j]);
  }
}

// dw[c] = sum over the blocks' partial sums, in their order: 32 columns per block of 8 warps, each
// warp every eighth row of them.
__global__ void __launch_bounds__(256) norm_dw_kernel(const float* partial, float* dw, int rows, int H) {
  __shared__ float part[8][33];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0;
  if (c < H)
    for (int r = warp; r < rows; r += 8) sum += __ldcg(partial + static_cast<long long>(r) * H + c);
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < H) {
    float v = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][lane];
    dw[c] = v;
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Threads of a row and vectors per thread: the fewest vectors that fit a block, then the warps that they take.
struct Shape {
  int v, threads;
};
Shape row_shape(int H, int max_threads) {
  const int nvec = H / kVec;
  int v = 1;
  while (v * max_threads < nvec) v *= 2;
  return {v, ((nvec + v - 1) / v + 31) / 32 * 32};
}

template <int kMaxV, class F>
dg_status with_v(int v, F f) {
  switch (v) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, kMaxV>());
  }
}

// Calls f with null pointers of the residual stream's type and the weight's.
template <class F>
dg_status with_types(int residual_type, int weight_type, F f) {
  const __nv_bfloat16* b = nullptr;
  const float* s = nullptr;
  if (residual_type == DG_BF16) return weight_type == DG_BF16 ? f(b, b) : f(b, s);
  return weight_type == DG_BF16 ? f(s, b) : f(s, s);
}

bool known_type(int t) { return t == DG_BF16 || t == DG_F32; }
size_t row_bytes(size_t ld, int type) { return ld * (type == DG_BF16 ? 2 : 4); }

}  // namespace

extern "C" {

dg_status dg_add_rms_norm(const void* x, const void* residual, const void* weight, void* residual_out, void* y, void* q,
                          int32_t* sf, float* rstd, const dg_norm_desc* desc, cudaStream_t stream) {
  if (!desc) return DG_ERR_INVALID_ARG;
  const int T = desc->T, H = desc->H, residual_type = desc->residual_type, weight_type = desc->weight_type;
  const size_t ldx = desc->ldx, ldr = desc->ldr, ldo = desc->ldo;
  const float eps = desc->eps;
  if (T < 0 || H <= 0 || H % kVec != 0 || !known_type(residual_type) || !known_type(weight_type)) return DG_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps < INFINITY)) return DG_ERR_INVALID_ARG;
  if ((q != nullptr) != (sf != nullptr) || (T > 0 && !q && !y && !residual_out) || (q && H % 128 != 0)) return DG_ERR_INVALID_ARG;
  if (H > kMaxH) return DG_ERR_UNSUPPORTED;
  if (T == 0) return DG_OK;
  const size_t cols = static_cast<size_t>(H);
  if (!x || !weight || ldx < cols || (residual && ldr < cols) || (residual_out && ldo < cols)) return DG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned16(q) || !aligned16(sf) || (reinterpret_cast<uintptr_t>(rstd) & 3u) || row_bytes(ldx, DG_BF16) % 16 ||
      (residual && row_bytes(ldr, residual_type) % 16) || (residual_out && row_bytes(ldo, residual_type) % 16))
    return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const Shape shape = row_shape(H, kThreads);
  return with_types(residual_type, weight_type, [&](auto* r, auto* w) {
    using R = std::remove_const_t<std::remove_pointer_t<decltype(r)>>;
    using W = std::remove_const_t<std::remove_pointer_t<decltype(w)>>;
    const NormArgs<R, W> a{static_cast<const __nv_bfloat16*>(x), static_cast<const R*>(residual),
                           static_cast<const W*>(weight), static_cast<__nv_bfloat16*>(y), static_cast<uint8_t*>(q), sf,
                           static_cast<R*>(residual_out), rstd, T, H, ldx, ldr, ldo, eps, 1.0f / static_cast<float>(H)};
    return with_v<8>(shape.v, [&](auto v) {
      return dg::launch(norm_kernel<R, W, decltype(v)::value>, static_cast<unsigned>(T), static_cast<unsigned>(shape.threads), 0, stream, ctx.pdl, a);
    });
  });
}

dg_status dg_add_rms_norm_backward(const void* dy, const void* s, const void* weight, const float* rstd, const void* ds,
                                   void* dx, void* dresidual, float* dw, int T, int H, int residual_type,
                                   int weight_type, cudaStream_t stream) {
  if (T < 0 || H <= 0 || H % kVec != 0 || !known_type(residual_type) || !known_type(weight_type) || !dw) return DG_ERR_INVALID_ARG;
  if (H > kMaxH) return DG_ERR_UNSUPPORTED;
  if (T > 0 && (!dy || !s || !weight || !rstd || (!dx && !dresidual))) return DG_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(s) || !aligned16(weight) || !aligned16(ds) || !aligned16(dx) || !aligned16(dresidual) ||
      !aligned16(dw) || (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status e = dg::launch_context(&ctx); e != DG_OK) return e;
  const unsigned dw_blocks = static_cast<unsigned>((H + 31) / 32);
  if (T == 0)   // the sum over no rows
    return dg::launch(norm_dw_kernel, dw_blocks, 256, 0, stream, ctx.pdl, static_cast<const float*>(nullptr), dw, 0, H);
  const int blocks = std::min(T, 2 * ctx.sms);
  dg::StreamWorkspace ws;
  void* partial = nullptr;
  if (dg_status e = ws.acquire(stream, static_cast<size_t>(blocks) * H * sizeof(float), &partial); e != DG_OK) return e;
  const Shape shape = row_shape(H, kGradThreads);
  const dg_status e = with_types(residual_type, weight_type, [&](auto* r, auto* w) {
    using R = std::remove_const_t<std::remove_pointer_t<decltype(r)>>;
    using W = std::remove_const_t<std::remove_pointer_t<decltype(w)>>;
    const NormGradArgs<R, W> a{static_cast<const __nv_bfloat16*>(dy), static_cast<const R*>(s), static_cast<const W*>(weight),
                               rstd, static_cast<const R*>(ds), static_cast<__nv_bfloat16*>(dx), static_cast<R*>(dresidual),
                               static_cast<float*>(partial), T, H};
    return with_v<4>(shape.v, [&](auto v) {
      return dg::launch(norm_grad_kernel<R, W, decltype(v)::value>, static_cast<unsigned>(blocks), static_cast<unsigned>(shape.threads), 0, stream, ctx.pdl, a);
    });
  });
  if (e != DG_OK) return e;
  return dg::launch(norm_dw_kernel, dw_blocks, 256, 0, stream, ctx.pdl, static_cast<const float*>(partial), dw, blocks, H);
}

}  // extern "C"
