// Top-k router of a mixture of experts, and its gradient.
//
//   ids     = the k experts of the largest logits, largest first, equal logits by lowest index
//   p       = softmax of the row's logits, or their sigmoid
//   weights = scale * p[ids] (divided by its sum over the chosen if `renormalize`)
//
// An expert whose logit is -inf or NaN is masked: never chosen, and no part of the softmax. Slots for
// which no expert is left get id -1 and weight 0.
//
// One warp per row. The experts' values stay in registers, expert 32 j + lane in register j of a
// lane; a choice is two warp-wide reductions, the largest key and the lowest index that has it.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "dg.h"
#include "ptx.cuh"
#include "runtime.h"
#include "ue8m0.cuh"

namespace {

using dg::LaunchContext;

constexpr int kWarps = 8;               // rows per block
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;            // a lane of the warp holds a slot
constexpr uint32_t kAll = 0xFFFFFFFFu;

__device__ __forceinline__ float load_logit(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(p))) << 16);
}
__device__ __forceinline__ void store_grad(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_grad(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Unsigned keys in the order of the values (-0 as +0); 0 for a masked expert (-inf, NaN).
__device__ __forceinline__ uint32_t order_key(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

template <class L>
struct RouteArgs {
  const L* logits;
  int32_t* ids;
  float* weights;
  int T, E, k;
  size_t ld;
  int sigmoid, renorm;
  float scale;
};

template <class L, int P>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs<L> a) {
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (t >= a.T) return;
  const L* row = a.logits + t * a.ld;
  uint32_t key[P];
#pragma unroll
  for (int j = 0; j < P; ++j) {
    const int e = 32 * j + lane;
    key[j] = e < a.E ? order_key(load_logit(row + e)) : 0;
  }
  float total = 0;   // of the softmax over every expert, relative to the largest
  uint32_t top = 0;
  if (!a.sigmoid && !a.renorm) {
#pragma unroll
    for (int j = 0; j < P; ++j) top = max(top, key[j]);
    top = __reduce_max_sync(kAll, top);
    const float largest = key_value(top);
#pragma unroll
    for (int j = 0; j < P; ++j)
      if (key[j]) total += expf(key_value(key[j]) - largest);
    total = warp_sum(total);
  }
  int my_id = -1;
  uint32_t my_key = 0;
  for (int i = 0; i < a.k; ++i) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int j = P - 1; j >= 0; --j)
      if (key[j] >= best) best = key[j], at = j;      // the lowest of equal ones
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m == 0) break;
    const int e = static_cast<int>(__reduce_min_sync(kAll, best == m ? static_cast<uint32_t>(32 * at + lane) : kAll));
    if (lane == i) my_id = e, my_key = m;
#pragma unroll
    for (int j = 0; j < P; ++j)
      if (32 * j + lane == e) key[j] = 0;
    if (i == 0) top = m;
  }
  float w = 0;
  if (my_id >= 0) w = a.sigmoid ? sigmoid(key_value(my_key)) : expf(key_value(my_key) - key_value(top));
  if (a.renorm) total = warp_sum(w);
  if (a.renorm || !a.sigmoid) w = total > 0 ? w / total : total == 0 ? 0.0f : NAN;
  if (lane < a.k) {
    a.ids[t * a.k + lane] = my_id;
    a.weights[t * a.k + lane] = my_id >= 0 ? a.scale * w : 0.0f;
  }
}

template <class L>
struct RouteGradArgs {
  const L* logits;
  const int32_t* ids;
  const float* dweights;
  L* dlogits;
  uint32_t* status;
  int T, E, k;
  size_t ld;
  int sigmoid, renorm;
  float scale;
};

// With q the weights before `scale` and d the gradients of the weights times `scale`, over the chosen j:
//   softmax, renormalised : dl_j = q_j (d_j - sum q d)             (q is the softmax over the chosen)
//   softmax               : dl_i = p_i ([i chosen] d_i - sum p d)  for every expert i
//   sigmoid, renormalised : dl_j = q_j (d_j - sum q d) (1 - p_j)
//   sigmoid               : dl_j = d_j p_j (1 - p_j)
template <class L, int P>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const RouteGradArgs<L> a) {
  __shared__ float row_out[kWarps][32 * P];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (t >= a.T) return;
  const L* row = a.logits + t * a.ld;
  float* out = row_out[threadIdx.x / 32];
  int id = lane < a.k ? __ldcg(a.ids + t * a.k + lane) : -1;
  if (id < -1 || id >= a.E) {
    atomicOr(a.status, dg::kBadIndexBit);
    id = -1;
  }
  const float x = id >= 0 ? load_logit(row + id) : -INFINITY;
  const bool chosen = id >= 0 && x > -INFINITY;
  const float d = chosen ? a.scale * __ldcg(a.dweights + t * a.k + lane) : 0.0f;
  float dl;
  float all[P];
#pragma unroll
  for (int j = 0; j < P; ++j) all[j] = 0;
  if (a.sigmoid) {
    const float p = chosen ? sigmoid(x) : 0.0f;
    float q = p, lean = d;
    if (a.renorm) {
      const float total = warp_sum(p);
      q = total > 0 ? p / total : 0.0f;
      lean = d - warp_sum(q * d);
    }
    dl = q * lean * (1.0f / (1.0f + expf(x)));      // 1 - p, without the cancellation
  } else if (a.renorm) {
    const uint32_t top = __reduce_max_sync(kAll, chosen ? order_key(x) : 0);
    const float p = chosen ? expf(x - key_value(top)) : 0.0f;
    const float total = warp_sum(p);
    const float q = total > 0 ? p / total : 0.0f;
    dl = q * (d - warp_sum(q * d));
  } else {
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      const int e = 32 * j + lane;
      all[j] = e < a.E ? load_logit(row + e) : -INFINITY;
      top = max(top, order_key(all[j]));
    }
    top = __reduce_max_sync(kAll, top);
    const float largest = key_value(top);
    float total = 0;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      all[j] = order_key(all[j]) ? expf(all[j] - largest) : 0.0f;
      total += all[j];
    }
    total = warp_sum(total);
    const float inv = total > 0 ? 1.0f / total : 0.0f;
    const float p = chosen ? expf(x - largest) * inv : 0.0f;
    const float inner = warp_sum(p * d);
    dl = p * (d - inner);
#pragma unroll
    for (int j = 0; j < P; ++j) all[j] *= -inv * inner;
  }
#pragma unroll
  for (int j = 0; j < P; ++j) out[32 * j + lane] = all[j];
  __syncwarp();
  if (chosen) out[id] = dl;
  __syncwarp();
  L* to = a.dlogits + t * a.E;
#pragma unroll
  for (int j = 0; j < P; ++j)
    if (32 * j + lane < a.E) store_grad(to + 32 * j + lane, out[32 * j + lane]);
}

template <class F>
dg_status with_p(int E, F f) {
  if (E <= 32) return f(std::integral_constant<int, 1>());
  if (E <= 64) return f(std::integral_constant<int, 2>());
  if (E <= 128) return f(std::integral_constant<int, 4>());
  if (E <= 256) return f(std::integral_constant<int, 8>());
  if (E <= 512) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

dg_status check(const void* logits, const void* ids, const void* weights, const dg_route_desc* desc) {
  if (!desc) return DG_ERR_INVALID_ARG;
  const auto [T, E, topk, ld, logits_type, scoring, renormalize, scale] = *desc;
  if (T < 0 || E <= 0 || topk <= 0 || topk > E || ld < static_cast<size_t>(E) || (logits_type != DG_BF16 && logits_type != DG_F32))
    return DG_ERR_INVALID_ARG;
  if ((scoring != DG_ROUTE_SOFTMAX && scoring != DG_ROUTE_SIGMOID) || (renormalize != 0 && renormalize != 1) || !std::isfinite(scale))
    return DG_ERR_INVALID_ARG;
  if (E > kMaxExperts || topk > kMaxTopk) return DG_ERR_UNSUPPORTED;
  if (T == 0) return DG_OK;
  if (!logits || !ids || !weights) return DG_ERR_INVALID_ARG;
  const uintptr_t lm = logits_type == DG_BF16 ? 1 : 3;
  if ((reinterpret_cast<uintptr_t>(logits) & lm) || ((reinterpret_cast<uintptr_t>(ids) | reinterpret_cast<uintptr_t>(weights)) & 3u))
    return DG_ERR_MISALIGNED;
  return DG_OK;
}

unsigned row_blocks(int T) { return static_cast<unsigned>((static_cast<long long>(T) + kWarps - 1) / kWarps); }

}  // namespace

extern "C" {

dg_status dg_moe_route(const void* logits, int32_t* topk_ids, float* topk_weights, const dg_route_desc* desc,
                       cudaStream_t stream) {
  if (dg_status s = check(logits, topk_ids, topk_weights, desc); s != DG_OK) return s;
  if (desc->T == 0) return DG_OK;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  auto run = [&](auto* type) {
    using L = std::remove_pointer_t<decltype(type)>;
    const RouteArgs<L> a{static_cast<const L*>(logits), topk_ids, topk_weights, desc->T, desc->E, desc->topk, desc->ld,
                         desc->scoring == DG_ROUTE_SIGMOID, desc->renormalize, desc->scale};
    return with_p(desc->E, [&](auto p) {
      return dg::launch(route_kernel<L, decltype(p)::value>, row_blocks(desc->T), kWarps * 32, 0, stream, ctx.pdl, a);
    });
  };
  return desc->logits_type == DG_BF16 ? run(static_cast<__nv_bfloat16*>(nullptr)) : run(static_cast<float*>(nullptr));
}

dg_status dg_moe_route_backward(const void* logits, const int32_t* topk_ids, const float* dweights, void* dlogits,
                                const dg_route_desc* desc, cudaStream_t stream) {
  if (dg_status s = check(logits, topk_ids, dweights, desc); s != DG_OK) return s;
  if (desc->T == 0) return DG_OK;
  if (!dlogits) return DG_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(dlogits) & (desc->logits_type == DG_BF16 ? 1u : 3u)) return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  auto run = [&](auto* type) {
    using L = std::remove_pointer_t<decltype(type)>;
    const RouteGradArgs<L> a{static_cast<const L*>(logits), topk_ids, dweights, static_cast<L*>(dlogits), ctx.status,
                             desc->T, desc->E, desc->topk, desc->ld, desc->scoring == DG_ROUTE_SIGMOID, desc->renormalize, desc->scale};
    return with_p(desc->E, [&](auto p) {
      return dg::launch(route_grad_kernel<L, decltype(p)::value>, row_blocks(desc->T), kWarps * 32, 0, stream, ctx.pdl, a);
    });
  };
  return desc->logits_type == DG_BF16 ? run(static_cast<__nv_bfloat16*>(nullptr)) : run(static_cast<float*>(nullptr));
}

}  // extern "C"
