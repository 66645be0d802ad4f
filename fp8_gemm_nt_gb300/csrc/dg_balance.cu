// Balance loss of a mixture of experts' router with its counts per expert, and its gradient.
//
//   p = softmax over a row's experts that are not masked, of x or of log sigmoid(x)
//   f = counts / sum of counts,   P = mean of p over the live rows,   loss = coef E sum f P
//   dloss/dx_e = coef E / live p_e (f_e - sum_j p_j f_j), with sigmoid scores times 1 - sigmoid(x_e)
//
// A warp takes rows in turn and keeps its sums over rows (or f, the same for every row) in registers. Forward, it works on
// two rows or four side by side while the next ones load; its sums are joined per block, then over the blocks by the last
// one to finish, in a fixed order; the counts are integers, whose atomics have no order to keep. A block that is alone (one
// round of its warps covers the rows) keeps all of it to itself: 64 rows take 3 us instead of 6. 65536 rows of 256 FP32
// logits: 17.3 us, of which some 4 are the chain of sums at the end; the rest is two thirds of the issue slots.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "dg.h"
#include "logit_rows.cuh"
#include "ptx.cuh"
#include "runtime.h"
#include "ue8m0.cuh"

namespace {

using namespace dg::rows;
using dg::exp2_fast;
using dg::kLog2e;
using dg::LaunchContext;
using dg::reciprocal;

// Warps of a block, one block an SM: as many as the registers of a lane's P logits leave room for.
template <int P>
constexpr int kWarpsOf = P > 16 ? 8 : P > 8 ? 16 : 32;
// Rows that a warp of it works on at once, side by side.
template <int P>
constexpr int kRowsOf = P > 8 ? 1 : P == 8 ? 2 : 4;
// The gradient's blocks, of 8 warps, that an SM holds at once.
constexpr int kGradWarps = 8;
template <int P>
constexpr int kGradBlocks = P > 16 ? 1 : P > 8 ? 2 : P == 8 ? 4 : 5;
constexpr int kMaxExperts = 1024, kMaxTopk = 32;

// Sums over the warp of R values, R chains of shuffles side by side.
template <int R>
__device__ __forceinline__ void warp_sums(float (&v)[R]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
    for (int r = 0; r < R; ++r) v[r] += __shfl_xor_sync(kAll, v[r], o);
  }
}

// The scores p of R rows of logits up to a common factor of each, and the factor that makes them add up to one (0 for a
// row without any). Sigmoids are taken relative to the largest where all are small, which keeps them from underflowing
// together: sigmoid(x) / sigmoid(top) is exp(x - top) / (1 + exp(x)) but for a factor that the row has in common. kRest:
// also rest = 1 - sigmoid(x), without the cancellation, where p is not 0.
// The rounded difference and its product with log2 e put a score |x - top| 2^-23 of itself off, the approximations 2^-22: its
// last bits where it counts in a sum, 2^-20 where it is e^-10 of the largest, 2^-16 at e^-80. expf would spare half of the
// first term; with it and with divisions 65536 rows of 256 FP32 logits took 27.9 us where these took 20.
template <bool kSigmoid, bool kRest, int R, int P>
__device__ __forceinline__ void scores(const float (&x)[R][P], float (&p)[R][P], float (&rest)[R][P], float (&by)[R], bool (&live)[R]) {
  float total[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
#pragma unroll
    for (int i = 0; i < P; ++i) p[r][i] = fmaxf(x[r][i], -INFINITY);        // NaN is masked as -inf is
    by[r] = warp_max(max_of(p[r]));
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float top = by[r];
    live[r] = top > -INFINITY;
    const float base = live[r] ? top : 0.0f;      // (subtracted first: rows of the type's lowest value differ by 0)
    if constexpr (kSigmoid) {
      if (top > 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float e = exp2_fast(-kLog2e * p[r][i]);
          if constexpr (kRest) e = fminf(e, 3.0e38f);
          p[r][i] = reciprocal(1.0f + e);
          if constexpr (kRest) rest[r][i] = e * p[r][i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float one = reciprocal(1.0f + exp2_fast(kLog2e * p[r][i]));
          if constexpr (kRest) rest[r][i] = one;
          p[r][i] = one * exp2_fast((p[r][i] - base) * kLog2e);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) p[r][i] = exp2_fast((p[r][i] - base) * kLog2e);
    }
    total[r] = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) total[r] += p[r][i];
  }
  warp_sums(total);
#pragma unroll
  for (int r = 0; r < R; ++r) by[r] = live[r] ? reciprocal(total[r]) : 0.0f;
}

// Has the lines of a row brought to L2, by a warp. Forward, for rows that are worked on alone, two ahead: 65536 of 512 FP32
// logits 34.2 -> 29.3 us (narrower ones, with more loads of their own under way: the same).
template <class L>
__device__ __forceinline__ void prefetch_row(const L* row, int lane, int E) {
  if (lane * 128 < E * static_cast<int>(sizeof(L)))
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(row) + lane * 128));
}

template <class L>
struct BalanceArgs {
  const L* logits;
  const int32_t* ids;
  int32_t* counts;
  int32_t* live_rows;
  float* prob_mean;
  float* loss;
  float* partial;       // [blocks][E]; this and the next not read by a block that is alone
  int* counters;        // blocks that have finished, live rows, and from kCountsAt on the counts; zero between launches
  uint32_t* status;
  int T, E, slots;
  size_t ld;
  float coef;
};
constexpr int kCountsAt = 64;

template <class L, int J, int kVec, bool kSigmoid>
__global__ void __launch_bounds__(kWarpsOf<J * kVec> * 32, 1) balance_kernel(const BalanceArgs<L> a) {
  using At = Lane<L, J, kVec>;
  constexpr int P = At::kCount, kWarps = kWarpsOf<P>;
  extern __shared__ float sums[];                           // [kWarps][E], then [E] counts
  int* const hist = reinterpret_cast<int*>(sums + kWarps * a.E);
  __shared__ int live_warps[kWarps];
  __shared__ float joined[kWarps];
  __shared__ bool last;
  __shared__ int all_live;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  for (int e = threadIdx.x; e < a.E; e += kWarps * 32) hist[e] = 0;
  __syncthreads();
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();

  // (rows and slots are below 2^31, and a few steps more below 2^32)
  const uint32_t step = gridDim.x * kWarps, T = static_cast<uint32_t>(a.T), slots = static_cast<uint32_t>(a.slots);
  uint32_t t = blockIdx.x * kWarps + warp;
  constexpr int R = kRowsOf<P>;
  float next[R][P], acc[P];
#pragma unroll
  for (int i = 0; i < P; ++i) acc[i] = 0;
  // (in place of rows past the last a warp loads its first one again, and does not count it: the loads stay free of
  // branches)
  const uint32_t own = t;
  auto row = [&](uint32_t at) { return a.logits + (at < T ? at : own) * a.ld; };
  if (t < T) {
#pragma unroll
    for (int r = 0; r < R; ++r) At::load(row(t + r * step), lane, a.E, next[r]);
  }
  // the block's share of the slots, while the first rows arrive
  constexpr int kBatch = 4;
  for (uint32_t s = blockIdx.x * (kWarps * 32) + threadIdx.x; s < slots; s += kBatch * step * 32) {
    int id[kBatch];
#pragma unroll
    for (int n = 0; n < kBatch; ++n) id[n] = s + n * step * 32 < slots ? __ldcg(a.ids + s + n * step * 32) : -1;
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      if (id[n] >= 0 && id[n] < a.E)
        atomicAdd(hist + id[n], 1);
      else if (id[n] != -1)
        atomicOr(a.status, dg::kBadIndexBit);
    }
  }
  int rows = 0;
  for (; t < T; t += R * step) {
    float p[R][P], none[R][P], by[R];
    bool live[R];
    if constexpr (R == 1)
      if (t + 2 * step < T) prefetch_row(a.logits + (t + 2 * step) * a.ld, lane, a.E);
    scores<kSigmoid, false>(next, p, none, by, live);
    if (t + R * step < T) {
#pragma unroll
      for (int r = 0; r < R; ++r) At::load(row(t + (R + r) * step), lane, a.E, next[r]);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (t + r * step >= T) break;
      rows += live[r];
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i] = fmaf(p[r][i], by[r], acc[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = At::index(lane, i);
    if (e < a.E) sums[warp * a.E + e] = acc[i];
  }
  if (lane == 0) live_warps[warp] = rows;
  __syncthreads();
  const bool alone = gridDim.x == 1;
  int live = 0;
  if (threadIdx.x < 32) live = __reduce_add_sync(kAll, lane < kWarps ? live_warps[lane] : 0);
  for (int e = threadIdx.x; e < a.E; e += kWarps * 32) {
    float s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w * a.E + e];
    if (alone) {
      sums[e] = s;
      continue;
    }
    a.partial[static_cast<size_t>(blockIdx.x) * a.E + e] = s;
    if (hist[e] > 0) atomicAdd(a.counters + kCountsAt + e, hist[e]);
  }
  if (threadIdx.x == 0) {
    all_live = live;
    if (!alone && live > 0) atomicAdd(a.counters + 1, live);
  }
  __syncthreads();
  int shares = 1;
  if (!alone) {
    if (threadIdx.x == 0) {
      __threadfence();       // what the block has written is seen before its arrival, and after it what the others have
      last = atomicAdd(a.counters, 1) == static_cast<int>(gridDim.x) - 1;
      __threadfence();
    }
    __syncthreads();
    if (!last) return;
    // the partial sums of an expert, or of four, by several threads, a share of the blocks each, and their sums in the
    // threads' order
    const int four = a.E % 4 == 0 ? 4 : 1, columns = a.E / four;
    shares = min(max(kWarps * 32 / columns, 1), kWarps);
    if (threadIdx.x == 0) all_live = __ldcg(a.counters + 1);
    for (int e = threadIdx.x; e < a.E; e += kWarps * 32) hist[e] = __ldcg(a.counters + kCountsAt + e);
    for (int i = threadIdx.x; i < shares * columns; i += kWarps * 32) {
      const int e = i % columns * four, share = i / columns;
      const unsigned from = gridDim.x * share / shares, to = gridDim.x * (share + 1) / shares;
      if (four == 4) {
        float4 s = make_float4(0, 0, 0, 0);
#pragma unroll 8
        for (unsigned b = from; b < to; ++b) {
          const float4 v = __ldcg(reinterpret_cast<const float4*>(a.partial + static_cast<size_t>(b) * a.E + e));
          s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
        }
        sums[share * a.E + e] = s.x, sums[share * a.E + e + 1] = s.y, sums[share * a.E + e + 2] = s.z, sums[share * a.E + e + 3] = s.w;
      } else {
        float s = 0;
#pragma unroll 8
        for (unsigned b = from; b < to; ++b) s += __ldcg(a.partial + static_cast<size_t>(b) * a.E + e);
        sums[share * a.E + e] = s;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kWarps * 32) a.counters[kCountsAt + e] = 0;
    if (threadIdx.x == 0) a.counters[0] = a.counters[1] = 0;
  }

  const float inv = 1.0f / static_cast<float>(max(all_live, 1));
  float inner = 0;
  int total = 0;
  for (int e = threadIdx.x; e < a.E; e += kWarps * 32) {
    float s = 0;
    for (int i = 0; i < shares; ++i) s += sums[i * a.E + e];
    const int c = hist[e];
    a.counts[e] = c;
    a.prob_mean[e] = s * inv;
    inner += static_cast<float>(c) * (s * inv);
    total += c;
  }
  inner = warp_sum(inner);
  total = __reduce_add_sync(kAll, total);
  if (lane == 0) joined[warp] = inner, live_warps[warp] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = 0;
    int c = 0;
    for (int w = 0; w < kWarps; ++w) s += joined[w], c += live_warps[w];
    *a.live_rows = all_live;
    *a.loss = a.coef * static_cast<float>(a.E) * (s / static_cast<float>(max(c, 1)));
  }
}

template <class L>
struct BalanceGradArgs {
  const L* logits;
  const int32_t* counts;
  const int32_t* live_rows;
  const float* dloss;
  const L* base;
  L* dlogits;
  int T, E;
  size_t ld;
  float coef;
};

// Warps keep f in registers and take rows in turn, as many of them as registers allow, to cover each other's loads. The
// counts are read once by a block: reads of the same few lines of L2 wait for one another (65536 rows of 256 FP32 logits with
// a base: 33.4 us, 6.0 TB/s, 0.90 of HBM's copy rate; 41.6 with the counts read by each warp, 152 with a warp for each row;
// 4096 rows: 4.7 us, 13 by each warp).
template <class L, int J, int kVec, bool kSigmoid, bool kBase>
__global__ void __launch_bounds__(kGradWarps * 32, kGradBlocks<J * kVec>) balance_grad_kernel(const BalanceGradArgs<L> a) {
  using At = Lane<L, J, kVec>;
  constexpr int P = At::kCount;
  __shared__ float shares[kMaxExperts], scale;               // the experts' slots; what every gradient is multiplied by
  __shared__ long long totals[kGradWarps];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long step = static_cast<long long>(gridDim.x) * kGradWarps;
  long long t = static_cast<long long>(blockIdx.x) * kGradWarps + threadIdx.x / 32;
  if (t < a.T) {
    prefetch_row(a.logits + t * a.ld, lane, a.E);
    if constexpr (kBase) prefetch_row(a.base + t * a.E, lane, a.E);
  }
  long long total = 0;
  for (int e = threadIdx.x; e < a.E; e += kGradWarps * 32) {
    const int c = max(__ldcg(a.counts + e), 0);
    shares[e] = static_cast<float>(c);
    total += c;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  if (lane == 0) totals[threadIdx.x / 32] = total;
  if (threadIdx.x == 0) scale = __ldcg(a.dloss) * (a.coef * static_cast<float>(a.E)) / static_cast<float>(max(__ldcg(a.live_rows), 1));
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kGradWarps; ++w) total += totals[w];
  const float inv = 1.0f / static_cast<float>(total > 1 ? total : 1);
  float f[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int e = At::index(lane, i);
    f[i] = e < a.E ? shares[e] * inv : 0.0f;
  }
  for (; t < a.T; t += step) {
    float x[1][P], d[P], p[1][P], rest[1][P], by[1], inner[1] = {0};
    bool live[1];
    At::load(a.logits + t * a.ld, lane, a.E, x[0]);
    if constexpr (kBase) At::load(a.base + t * a.E, lane, a.E, d);
    scores<kSigmoid, true>(x, p, rest, by, live);
#pragma unroll
    for (int i = 0; i < P; ++i) inner[0] = fmaf(p[0][i], f[i], inner[0]);
    warp_sums(inner);
    const float mean = inner[0] * by[0], all = scale * by[0];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float g = all * p[0][i] * (f[i] - mean);
      if constexpr (kSigmoid) g *= rest[0][i];
      x[0][i] = (kBase ? d[i] : 0.0f) + (p[0][i] == 0.0f ? 0.0f : g);
    }
    At::store(a.dlogits + t * a.E, lane, a.E, x[0]);
  }
}

size_t row_stride(const dg_balance_desc& d) { return d.T > 1 ? d.ld : static_cast<size_t>(d.E); }

dg_status check(const void* logits, const dg_balance_desc* desc) {
  if (!desc) return DG_ERR_INVALID_ARG;
  if (desc->T < 0 || desc->E <= 0 || row_stride(*desc) < static_cast<size_t>(desc->E)) return DG_ERR_INVALID_ARG;
  if (desc->logits_type != DG_BF16 && desc->logits_type != DG_F32) return DG_ERR_INVALID_ARG;
  if ((desc->scoring != DG_ROUTE_SOFTMAX && desc->scoring != DG_ROUTE_SIGMOID) || !std::isfinite(desc->coef)) return DG_ERR_INVALID_ARG;
  if (desc->E > kMaxExperts) return DG_ERR_UNSUPPORTED;
  if (desc->T == 0) return DG_OK;
  if (!logits) return DG_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(logits) & (desc->logits_type == DG_BF16 ? 1 : 3) ? DG_ERR_MISALIGNED : DG_OK;
}
bool words(std::initializer_list<const void*> all) {
  uintptr_t any = 0;
  for (const void* p : all) any |= reinterpret_cast<uintptr_t>(p);
  return (any & 3u) == 0;
}

// Whether pieces of 16 bytes leave no more logits to a lane than single ones do: 65536 rows of 64 BF16 logits, sigmoid scores,
// 12.3 us with single ones, 22.3 with pieces, and their gradient 14.0 and 33.7.
template <class L>
bool wide(int E) { return E > 16 * static_cast<int>(16 / sizeof(L)); }

// Blocks that take `rows` rows at a time, `most` at most.
unsigned blocks_for(int T, int rows, int most) {
  return static_cast<unsigned>(std::max(1, std::min(T / rows + (T % rows != 0), most)));
}

}  // namespace

extern "C" {

dg_status dg_moe_balance_loss(const void* logits, const int32_t* topk_ids, int32_t* counts, int32_t* live_rows, float* prob_mean,
                              float* loss, const dg_balance_desc* desc, cudaStream_t stream) {
  if (dg_status s = check(logits, desc); s != DG_OK) return s;
  if (desc->topk <= 0 || !counts || !live_rows || !prob_mean || !loss || (desc->T > 0 && !topk_ids)) return DG_ERR_INVALID_ARG;
  if (desc->topk > kMaxTopk || static_cast<long long>(desc->T) * desc->topk > 0x7FFFFFFFll) return DG_ERR_UNSUPPORTED;
  if (!words({topk_ids, counts, live_rows, prob_mean, loss})) return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const size_t ld = row_stride(*desc);
  auto run = [&](auto* type) {
    using L = std::remove_pointer_t<decltype(type)>;
    BalanceArgs<L> a{static_cast<const L*>(logits), topk_ids, counts, live_rows, prob_mean, loss, nullptr, nullptr, ctx.status,
                     desc->T, desc->E, desc->T * desc->topk, ld, desc->coef};
    return with_shape<L>(desc->E, wide<L>(desc->E) && whole_pieces<L>(logits, ld, desc->E), [&](auto j, auto vec) {
      constexpr int P = decltype(j)::value * decltype(vec)::value, kWarps = kWarpsOf<P>;
      // (a lane's P logits are of 32 P experts at most: 37 KB, less than a kernel has to ask for)
      static_assert((kWarps + 1) * std::min(32 * P, kMaxExperts) * sizeof(float) <= 40 * 1024, "shared memory");
      const size_t smem = static_cast<size_t>(kWarps + 1) * desc->E * sizeof(float);
      auto kernel = desc->scoring == DG_ROUTE_SIGMOID ? balance_kernel<L, decltype(j)::value, decltype(vec)::value, true>
                                                      : balance_kernel<L, decltype(j)::value, decltype(vec)::value, false>;
      const unsigned blocks = blocks_for(desc->T, kWarps * kRowsOf<P>, ctx.sms);
      dg::StreamWorkspace ws;      // (what a block alone has no use for: a stream without one can be captured)
      void* scratch = nullptr;
      if (blocks > 1)
        if (dg_status s = ws.acquire(stream, static_cast<size_t>(ctx.sms) * desc->E * sizeof(float), &scratch); s != DG_OK) return s;
      a.partial = static_cast<float*>(scratch), a.counters = ws.counters();
      return dg::launch(kernel, blocks, kWarps * 32, smem, stream, ctx.pdl, a);
    });
  };
  return desc->logits_type == DG_BF16 ? run(static_cast<__nv_bfloat16*>(nullptr)) : run(static_cast<float*>(nullptr));
}

dg_status dg_moe_balance_loss_backward(const void* logits, const int32_t* counts, const int32_t* live_rows, const float* dloss,
                                       const void* base, void* dlogits, const dg_balance_desc* desc, cudaStream_t stream) {
  if (dg_status s = check(logits, desc); s != DG_OK) return s;
  if (desc->T == 0) return DG_OK;
  if (!counts || !live_rows || !dloss || !dlogits) return DG_ERR_INVALID_ARG;
  const uintptr_t of = desc->logits_type == DG_BF16 ? 1 : 3;
  if (!words({counts, live_rows, dloss}) || ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(dlogits)) & of))
    return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const size_t ld = row_stride(*desc);
  auto run = [&](auto* type) {
    using L = std::remove_pointer_t<decltype(type)>;
    const BalanceGradArgs<L> a{static_cast<const L*>(logits), counts, live_rows, dloss, static_cast<const L*>(base), static_cast<L*>(dlogits),
                               desc->T, desc->E, ld, desc->coef};
    const bool aligned = wide<L>(desc->E) && whole_pieces<L>(logits, ld, desc->E) && whole_pieces<L>(dlogits, desc->E, desc->E) &&
                         whole_pieces<L>(base, desc->E, desc->E);
    return with_shape<L>(desc->E, aligned, [&](auto j, auto vec) {
      constexpr int J = decltype(j)::value, kVec = decltype(vec)::value;
      const bool sig = desc->scoring == DG_ROUTE_SIGMOID;
      auto kernel = base ? (sig ? balance_grad_kernel<L, J, kVec, true, true> : balance_grad_kernel<L, J, kVec, false, true>)
                         : (sig ? balance_grad_kernel<L, J, kVec, true, false> : balance_grad_kernel<L, J, kVec, false, false>);
      return dg::launch(kernel, blocks_for(desc->T, kGradWarps, kGradBlocks<J * kVec> * ctx.sms), kGradWarps * 32, 0, stream, ctx.pdl, a);
    });
  };
  return desc->logits_type == DG_BF16 ? run(static_cast<__nv_bfloat16*>(nullptr)) : run(static_cast<float*>(nullptr));
}

}  // extern "C"
