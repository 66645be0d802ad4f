// Top-k router of a mixture of experts, and its gradient.
//
//   ids     = the k experts of the largest logits, largest first, equal logits by lowest index
//   p       = softmax of the row's logits, or their sigmoid
//   weights = scale * p[ids] (divided by its sum over the chosen if `renormalize`)
//
// An expert whose logit is -inf or NaN is masked: never chosen, and no part of the softmax. Slots for
// which no expert is left get id -1 and weight 0.
//
// A warp takes a row, its logits in registers. A choice of k among all E by
// k rounds over every register costs about 50 instructions a round, more than reading the row allows; so
// most of the row is sorted out first. The k-th largest of the 32 lanes' own maxima is a lower bound of
// the k-th largest logit; what reaches it (k and a few) is gathered, one per lane, and each candidate
// counts those before it. Rows with more than 32 candidates (large k, many equal logits) take the rounds
// over all. Where there are many rows and k is at most 8, a warp takes two.
//
// 65536 rows of 256 FP32 logits, k = 8: 24 us, 2.9 TB/s, bound by issued instructions (29.4 us with a row a warp, 500
// instructions a row; 70 us by rounds alone). Blocks that loop over rows with the next row's loads in flight
// were slower (34 us: the registers cost more warps than the loads cost time).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <type_traits>

#include "dg.h"
#include "logit_rows.cuh"
#include "ptx.cuh"
#include "runtime.h"
#include "ue8m0.cuh"

namespace {

using namespace dg::rows;
using dg::LaunchContext;

constexpr int kWarps = 8;               // rows per block
constexpr int kMaxExperts = 1024;
constexpr int kMaxTopk = 32;            // a lane of the warp holds a slot
// Two rows a warp: for k that seldom leaves more than 16 candidates, few enough logits per lane to hold both rows, and
// rows enough for half the warps to fill the SMs. Two rows against one, 256 FP32 logits, k = 8: 65536 rows 24.0 and
// 29.1 us, 16384 rows 7.6 and 8.9, 4096 rows 3.7 and 3.8, 1024 rows 3.3 and 2.7; 65536 rows of k = 12: 32.0 and 34.9,
// k = 16: 42.7 and 41.2; of 512 logits 36.8 and 38.5. The limits keep to where it gains a tenth or more, short of
// where it begins to gain: at 4096 rows, k = 12 and 512 logits it would by 3 to 8 %, at 1024 rows and k = 16 it loses.
constexpr int kPairTopk = 8, kPairLogits = 8, kPairRows = 8192;

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

// What is known of a row once its candidates, n of them, have been gathered as (logit, expert).
struct Candidates {
  float top, total;      // the largest logit, and the softmax's sum over every expert relative to it
  int n;
};

template <class At, int P, class L>
__device__ __forceinline__ Candidates gather(const RouteArgs<L>& a, float (&v)[P], int lane, float2* candidates) {
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = fmaxf(v[i], -INFINITY);        // NaN is masked as -inf is
  const float mine = max_of(v), top = warp_max(mine);
  float total = 0;
  if (!a.sigmoid && !a.renorm && top > -INFINITY) {
#pragma unroll
    for (int i = 0; i < P; ++i) total += expf(v[i] - top);
    total = warp_sum(total);
  }
  if (P == 1) {
    candidates[lane] = make_float2(v[0], __int_as_float(lane));
    __syncwarp();
    return {top, total, 32};
  }
  float left = mine, bound = top;
  for (int i = 1; i < a.k; ++i) {
    left = left == bound ? -INFINITY : left;
    bound = warp_max(left);
  }
  bound = fmaxf(bound, -3.402823466e38f);                       // any logit that is not masked
  int count = 0;
#pragma unroll
  for (int i = 0; i < P; ++i) count += v[i] >= bound;
  int at = count;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kAll, at, o);
    if (lane >= o) at += x;
  }
  const int n = __shfl_sync(kAll, at, 31);
  if (n <= 32) {
    at -= count;
    if (count > 0) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (v[i] >= bound) candidates[at++] = make_float2(v[i], __int_as_float(At::index(lane, i)));
    }
    __syncwarp();
  }
  return {top, total, n};
}

// How many of n candidates come before one: larger ones, and equal ones of a lower index.
__device__ __forceinline__ int rank_of(float2 cand, const float2* candidates, int n) {
  const int id = __float_as_int(cand.y);
  int before = 0;
  for (int i = 0; i < n; ++i) {
    const float2 c = candidates[i];
    before += c.x > cand.x || (c.x == cand.x && __float_as_int(c.y) < id);
  }
  return before;
}

// The weight of a chosen expert before `scale`; `total`: of the softmax or, renormalised, of the chosen.
template <class L>
__device__ __forceinline__ float weight_of(const RouteArgs<L>& a, float w, float total) {
  if (!a.renorm && a.sigmoid) return w;
  return total > 0 ? w / total : total == 0 ? 0.0f : NAN;
}

// A row's choice and its outputs, by the whole warp.
template <class At, int P, class L>
__device__ __forceinline__ void choose(const RouteArgs<L>& a, long long t, float (&v)[P], const Candidates& row, int lane, const float2* candidates, float2* slots) {
  int found = 0;
  if (row.n <= 32) {
    const float2 cand = lane < row.n ? candidates[lane] : make_float2(-INFINITY, 0);
    const bool live = cand.x > -INFINITY;
    const int before = rank_of(cand, candidates, row.n);
    found = min(a.k, __popc(__ballot_sync(kAll, live)));
    if (live && before < a.k) slots[before] = cand;
  } else {
    for (; found < a.k; ++found) {
      const float m = warp_max(max_of(v));
      if (!(m > -INFINITY)) break;
      uint32_t id = kAll;
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (v[i] == m) id = min(id, static_cast<uint32_t>(At::index(lane, i)));
      id = __reduce_min_sync(kAll, id);
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (At::index(lane, i) == static_cast<int>(id)) v[i] = -INFINITY;
      if (lane == 0) slots[found] = make_float2(m, __int_as_float(static_cast<int>(id)));
    }
  }
  __syncwarp();
  const bool have = lane < found;
  const float2 slot = slots[lane];
  float w = 0;
  if (have) w = a.sigmoid ? sigmoid(slot.x) : expf(slot.x - row.top);
  w = weight_of(a, w, a.renorm ? warp_sum(w) : row.total);
  if (lane < a.k) {
    a.ids[t * a.k + lane] = have ? __float_as_int(slot.y) : -1;
    a.weights[t * a.k + lane] = have ? a.scale * w : 0.0f;
  }
}

template <class L, int J, int kVec>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs<L> a) {
  using At = Lane<L, J, kVec>;
  __shared__ float2 gathered[kWarps][32], chosen[kWarps][32];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= a.T) return;
  float v[At::kCount];
  At::load(a.logits + t * a.ld, lane, a.E, v);
  const Candidates row = gather<At>(a, v, lane, gathered[warp]);
  choose<At>(a, t, v, row, lane, gathered[warp], chosen[warp]);
}

// Two rows a warp. Each is gathered by all lanes; the order of its candidates, the weights and the outputs, which
// need few, by 16 lanes for either row at once, if neither has more candidates.
template <class L, int J, int kVec>
__global__ void __launch_bounds__(kWarps * 32) route_pair_kernel(const RouteArgs<L> a) {
  using At = Lane<L, J, kVec>;
  __shared__ float2 gathered[kWarps][2][32], chosen[kWarps][32];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const long long t = 2 * (static_cast<long long>(blockIdx.x) * kWarps + warp);
  if (t >= a.T) return;
  const bool two = t + 1 < a.T;
  float v[2][At::kCount];
  At::load(a.logits + t * a.ld, lane, a.E, v[0]);
  At::load(a.logits + (two ? t + 1 : t) * a.ld, lane, a.E, v[1]);
  float2(&candidates)[2][32] = gathered[warp];
  float2* const slots = chosen[warp];
  const Candidates row0 = gather<At>(a, v[0], lane, candidates[0]), row1 = gather<At>(a, v[1], lane, candidates[1]);
  if (max(row0.n, row1.n) > 16) {
    choose<At>(a, t, v[0], row0, lane, candidates[0], slots);
    __syncwarp();
    if (two) choose<At>(a, t + 1, v[1], row1, lane, candidates[1], slots);
    return;
  }
  const int at = lane & 15;
  const bool second = lane >= 16;
  const int n = second ? row1.n : row0.n;
  const float2* const mine = candidates[second];
  const float2 cand = at < n ? mine[at] : make_float2(-INFINITY, 0);
  const bool live = cand.x > -INFINITY;
  const int before = rank_of(cand, mine, n);
  const int found = min(a.k, __popc(__ballot_sync(kAll, live) & (second ? 0xFFFF0000u : 0xFFFFu)));
  if (live && before < a.k) slots[16 * second + before] = cand;
  __syncwarp();
  const bool have = at < found;
  const float2 slot = slots[lane];
  float w = 0, total = second ? row1.total : row0.total;
  if (have) w = a.sigmoid ? sigmoid(slot.x) : expf(slot.x - (second ? row1.top : row0.top));
  if (a.renorm) {
    total = w;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  }
  w = weight_of(a, w, total);
  if (at < a.k && (two || !second)) {
    const long long to = (t + second) * a.k + at;
    a.ids[to] = have ? __float_as_int(slot.y) : -1;
    a.weights[to] = have ? a.scale * w : 0.0f;
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
//
// Every lane writes its share of the row; the lanes that have a chosen slot then write over it.
template <class L, int J, int kVec>
__global__ void __launch_bounds__(kWarps * 32) route_grad_kernel(const RouteGradArgs<L> a) {
  using At = Lane<L, J, kVec>;
  constexpr int P = At::kCount;
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (t >= a.T) return;
  const L* row = a.logits + t * a.ld;
  float all[P];
  const bool dense = !a.sigmoid && !a.renorm;
  if (dense) At::load(row, lane, a.E, all);           // in flight while the ids are followed
  int id = lane < a.k ? __ldcg(a.ids + t * a.k + lane) : -1;
  if (id < -1 || id >= a.E) {
    atomicOr(a.status, dg::kBadIndexBit);
    id = -1;
  }
  const float g = id >= 0 ? __ldcg(a.dweights + t * a.k + lane) : 0.0f;
  const float x = id >= 0 ? load_logit(row + id) : -INFINITY;
  const bool chosen = x > -INFINITY;
  const float d = chosen ? a.scale * g : 0.0f;
  float dl;
  if (dense) {
#pragma unroll
    for (int i = 0; i < P; ++i) all[i] = fmaxf(all[i], -INFINITY);
    const float top = warp_max(max_of(all)), base = top > -INFINITY ? top : 0.0f;
    float total = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      all[i] = expf(all[i] - base);
      total += all[i];
    }
    total = warp_sum(total);
    const float inv = total > 0 ? 1.0f / total : total == 0 ? 0.0f : NAN;
    const float p = chosen ? expf(x - base) * inv : 0.0f;
    const float inner = warp_sum(p * d);
    dl = p * (d - inner);
#pragma unroll
    for (int i = 0; i < P; ++i) all[i] *= -inv * inner;
  } else {
#pragma unroll
    for (int i = 0; i < P; ++i) all[i] = 0;
    const float top = warp_max(chosen ? x : -INFINITY);
    const float p = !chosen ? 0.0f : a.sigmoid ? sigmoid(x) : expf(x - top);
    float q = p, lean = d;
    if (a.renorm) {
      const float total = warp_sum(p);
      q = total > 0 ? p / total : total == 0 ? 0.0f : NAN;
      lean = d - warp_sum(q * d);
    }
    dl = q * lean;
    if (a.sigmoid) dl *= 1.0f / (1.0f + expf(x));      // 1 - p, without the cancellation
  }
  L* to = a.dlogits + t * a.E;
  At::store(to, lane, a.E, all);
  __syncwarp();
  if (chosen) store_grad(to + id, dl);
}

// Elements between the rows of the logits; a single row has no next one, whatever its stride says.
size_t row_stride(const dg_route_desc& d) { return d.T > 1 ? d.ld : static_cast<size_t>(d.E); }

dg_status check(const void* logits, const void* ids, const void* weights, const dg_route_desc* desc) {
  if (!desc) return DG_ERR_INVALID_ARG;
  const auto [T, E, topk, ld, logits_type, scoring, renormalize, scale] = *desc;
  if (T < 0 || E <= 0 || topk <= 0 || topk > E || row_stride(*desc) < static_cast<size_t>(E) || (logits_type != DG_BF16 && logits_type != DG_F32))
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
  const size_t ld = row_stride(*desc);
  auto run = [&](auto* type) {
    using L = std::remove_pointer_t<decltype(type)>;
    const RouteArgs<L> a{static_cast<const L*>(logits), topk_ids, topk_weights, desc->T, desc->E, desc->topk, ld,
                         desc->scoring == DG_ROUTE_SIGMOID, desc->renormalize, desc->scale};
    // 16-byte loads only where every lane has one: the bound is among the lanes' maxima (65536 rows of 64 BF16 logits,
    // k = 8: 25 us, against 39 us with 8 lanes at work)
    const bool wide = desc->E >= 32 * static_cast<int>(16 / sizeof(L)) && whole_pieces<L>(logits, ld, desc->E);
    return with_shape<L>(desc->E, wide, [&](auto j, auto vec) {
      constexpr int kLogits = decltype(j)::value * decltype(vec)::value;
      if constexpr (kLogits > 1 && kLogits <= kPairLogits)
        if (desc->topk <= kPairTopk && desc->T >= kPairRows)
          return dg::launch(route_pair_kernel<L, decltype(j)::value, decltype(vec)::value>, row_blocks(desc->T / 2 + desc->T % 2), kWarps * 32, 0, stream, ctx.pdl, a);
      return dg::launch(route_kernel<L, decltype(j)::value, decltype(vec)::value>, row_blocks(desc->T), kWarps * 32, 0, stream, ctx.pdl, a);
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
  const size_t ld = row_stride(*desc);
  auto run = [&](auto* type) {
    using L = std::remove_pointer_t<decltype(type)>;
    const RouteGradArgs<L> a{static_cast<const L*>(logits), topk_ids, dweights, static_cast<L*>(dlogits), ctx.status,
                             desc->T, desc->E, desc->topk, ld, desc->scoring == DG_ROUTE_SIGMOID, desc->renormalize, desc->scale};
    const bool aligned = whole_pieces<L>(logits, ld, desc->E) && whole_pieces<L>(dlogits, desc->E, desc->E);
    return with_shape<L>(desc->E, aligned, [&](auto j, auto vec) {
      return dg::launch(route_grad_kernel<L, decltype(j)::value, decltype(vec)::value>, row_blocks(desc->T), kWarps * 32, 0, stream, ctx.pdl, a);
    });
  };
  return desc->logits_type == DG_BF16 ? run(static_cast<__nv_bfloat16*>(nullptr)) : run(static_cast<float*>(nullptr));
}

}  // extern "C"
