// A whole mixture-of-experts layer for a few tokens (at most 32), in two kernels:
//
//   y[t] = c[t] + sum over the slots j of token t with an expert e = ids[t, j]:
//              weights[t, j] * W2_e (silu(G_e x_t) * (U_e x_t)),      (G_e; U_e) = W13_e
//
// x is E4M3 with one UE8M0 scale per 128 columns; the experts' weights are E4M3 with one scale per
// 128 x 128 block, or E2M1 with one per row per 32 columns: the grouped GEMMs' operands.
//
// At a few tokens an expert has one to a handful of rows, so the time is that of reading the weights
// of the experts in use, once. Both kernels stream them with TMA into rings in shared memory. A warp
// multiplies 16 weight rows (or 32) by up to 8 tokens (or 16) with m16n8 MMAs: the weights are the M
// operand, an expert's tokens the N columns. The first product's operands are both E4M3 (E2M1 is one
// with two exponent bits, moved into place), the second's FP16, which holds E4M3 and E2M1 exactly.
// Accumulation is FP32, and the scales are applied to FP32 partial sums.
//
// An expert's tokens are compacted into jobs of at most 8 (16) columns; each distinct (expert, token)
// pair is a slot. The first kernel writes h = weight * silu(g) * u of every slot to the workspace, in
// FP16 with one power-of-two scale per 64 or 128 columns (11 bits of every value within 2^-29 of the
// largest; plain FP32 would double what the second kernel reads). The second kernel owns output rows: a
// block sums all experts for its 16 (32) rows of W2 and every token, in an order that depends on the
// sizes alone, and writes each output once. No atomics on values.
//
// Where a layer has fewer pieces of work than the GPU has room for blocks, a cluster of blocks shares a
// piece, each with a part of K, and sums through distributed shared memory in the order of its ranks.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "debug_state.h"
#include "dg.h"
#include "ptx.cuh"
#include "runtime.h"
#include "ue8m0.cuh"

namespace {

using dg::LaunchContext;

constexpr int kMaxTokens = 32;          // a token is a bit of an expert's mask
constexpr int kMaxTopk = 16;
constexpr int kMaxExperts = 1024;
constexpr int kMaxH = 16384;
constexpr int kMaxSlots = kMaxTokens * kMaxTopk;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kHBytes = 272;            // 128 columns of h of a slot: 256 bytes of FP16, FP32 scales of both halves, padding
constexpr int kMaxSmem = 216 * 1024;
constexpr int kHalfSm = 104 * 1024;     // dynamic shared memory of a block of which two are resident

struct MoeArgs {
  const uint8_t* x;        // [T, H] E4M3
  const int32_t* sfx;      // [KP(H), ceil4(T)]
  const uint8_t* w13;      // [E, 2 I, H] (H / 2 bytes a row for E2M1)
  const int32_t* sf13;
  const uint8_t* w2;       // [E, H, I]
  const int32_t* sf2;
  const int32_t* ids;      // [T, k]
  const float* weights;    // [T, k]
  const __nv_bfloat16* c;  // [T, H] or null
  __nv_bfloat16* y;        // [T, H]
  uint8_t* h;              // [slots, I / 128, kHBytes]
  uint32_t* status;
  unsigned long long timeout_ns;   // of a wait for a copy
  int fault;                       // failure injection: no copies
  int T, k, E, H, I;
};

// -------------------------------------------------------------------------------------------
// Who needs which expert
// -------------------------------------------------------------------------------------------

struct Routing {
  uint16_t job_expert[kMaxSlots];
  uint16_t job_slot[kMaxSlots];         // first slot of a job; a job's slots are consecutive
  uint8_t job_count[kMaxSlots];
  uint8_t token[kMaxSlots];
  float coef[kMaxSlots];                // weight of a slot (the sum, where a token names an expert twice)
  int warp_sum[17];
  int jobs;
};

// Needed only while the routing is built: lies where the rings will.
struct RoutingScratch {
  uint32_t mask[kMaxExperts];           // tokens of an expert
  uint16_t first_slot[kMaxExperts];
  int32_t ids[kMaxSlots];
  float weights[kMaxSlots];
};

// Builds the routing of the block from the ids, in the order of experts and tokens: the same in
// every block of both kernels. `kCols`: columns of a job.
template <int kCols, int kThreads>
__device__ __forceinline__ void build_routing(const MoeArgs& a, Routing& r, RoutingScratch& s, bool report) {
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, slots = a.T * a.k;
  for (int i = tid; i < slots; i += kThreads) {
    s.ids[i] = dg::ld_cg_s32(a.ids + i);
    s.weights[i] = __ldcg(a.weights + i);
  }
  for (int e = tid; e < a.E; e += kThreads) s.mask[e] = 0;
  __syncthreads();
  for (int i = tid; i < slots; i += kThreads) {
    const int e = s.ids[i];
    if (e >= 0 && e < a.E) atomicOr(&s.mask[e], 1u << (i / a.k));
    else if (e != -1 && report) atomicOr(a.status, dg::kBadIndexBit);
  }
  __syncthreads();
  // jobs and slots before each expert: kPer experts per thread, jobs in the upper half of a word
  int n[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * tid + i;
    const int tokens = e < a.E ? __popc(s.mask[e]) : 0;
    n[i] = ((tokens + kCols - 1) / kCols) << 16 | tokens;
    sum += n[i];
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kAll, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) r.warp_sum[warp] = before;
  before -= sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += r.warp_sum[w];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = kPer * tid + i;
    if (e < a.E) {
      const int slot = before & 0xFFFF, tokens = n[i] & 0xFFFF;
      s.first_slot[e] = static_cast<uint16_t>(slot);
      int job = before >> 16;
      for (int c = 0; c < tokens; c += kCols, ++job) {
        r.job_expert[job] = static_cast<uint16_t>(e);
        r.job_slot[job] = static_cast<uint16_t>(slot + c);
        r.job_count[job] = static_cast<uint8_t>(min(kCols, tokens - c));
      }
      before += n[i];
    }
  }
  if (tid == kThreads - 1) r.jobs = before >> 16;
  __syncthreads();
  for (int i = tid; i < slots; i += kThreads) {
    const int e = s.ids[i];
    if (e < 0 || e >= a.E) continue;
    const int t = i / a.k;
    bool first = true;
    float w = 0;
    for (int j = t * a.k; j < (t + 1) * a.k; ++j)
      if (s.ids[j] == e) {
        first = first && j >= i;
        w += s.weights[j];
      }
    if (first) {
      const int slot = s.first_slot[e] + __popc(s.mask[e] & ((1u << t) - 1));
      r.token[slot] = static_cast<uint8_t>(t);
      r.coef[slot] = w;
    }
  }
  __syncthreads();
}

// -------------------------------------------------------------------------------------------
// Elements, MMAs, copies
// -------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

// Four E2M1 codes as E4M3 of 2^-6 of their values: the sign to bit 7, the two exponent bits and the
// mantissa bit to the lowest exponent bits and the highest mantissa bit (E2M1's subnormal 0.5 becomes
// the subnormal 2^-7). Even elements of eight are the low nibbles, odd ones the high nibbles.
__device__ __forceinline__ uint32_t e4m3_of_even(uint32_t w) { return (w << 4 & 0x80808080u) | (w << 2 & 0x1C1C1C1Cu); }
__device__ __forceinline__ uint32_t e4m3_of_odd(uint32_t w) { return (w & 0x80808080u) | (w >> 2 & 0x1C1C1C1Cu); }

// The same as the upper bytes of FP16 of 2^-14 of their values (the lower bytes are 0), and two of them as a
// pair: bytes 0 and 1, or 2 and 3, of b.
__device__ __forceinline__ uint32_t f16_of_even(uint32_t w) { return (w << 4 & 0x80808080u) | (w << 1 & 0x0E0E0E0Eu); }
__device__ __forceinline__ uint32_t f16_of_odd(uint32_t w) { return (w & 0x80808080u) | (w >> 3 & 0x0E0E0E0Eu); }
__device__ __forceinline__ uint32_t lower_pair(uint32_t b) { return __byte_perm(b, 0, 0x1404); }
__device__ __forceinline__ uint32_t upper_pair(uint32_t b) { return __byte_perm(b, 0, 0x3424); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same on a sum that starts at zero.
__device__ __forceinline__ void mma_e4m3_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
               : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Plain loads of shared memory: the waits before them clobber memory, so they stay after those, and the
// compiler may otherwise move them ahead of other work.
template <class T>
__device__ __forceinline__ T lds(const uint8_t* p) { return *reinterpret_cast<const T*>(p); }
__device__ __forceinline__ uint2 ld_cg_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ float float_of(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Untiled bulk copy (16-byte aligned addresses and size) that completes on `bar`.
__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dg::smem_addr(to)),
               "l"(from), "r"(bytes), "r"(dg::smem_addr(bar))
               : "memory");
}

// The K order of a product is free. Within 128 columns, lane 4 g + q (g the row or column of the MMA
// fragment) takes, in the E4M3 form, columns 64 p + 16 q .. + 15 of half p: one 128-bit load of a row holds
// its fragments of two (four) MMAs. In the E2M1 form it takes columns 32 b + 8 q .. + 7 of block b: the
// columns of an MMA then share a scale.
//
// TMA permutes the 16-byte chunks of a row (the 128-byte swizzle for E4M3, the 64-byte one for E2M1).
// The eight lanes of a 128-bit load's phase are two rows of four chunks; they cover every bank once if the
// rows differ by four, so row g of a fragment is row g / 2 + 4 (g % 2) of eight in memory. E2M1's 32-bit
// loads (eight rows of one chunk) meet no bank twice in any order of the rows.
template <bool kFp4>
struct Rows {
  static constexpr int kBytes = kFp4 ? 64 : 128;            // of 128 columns
  static __device__ __forceinline__ int of(int g) { return kFp4 ? g : g / 2 + 4 * (g & 1); }
  static __device__ __forceinline__ int chunk(int row, int c) {
    return kFp4 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4) : row * 128 + ((c ^ (row & 7)) << 4);
  }
};

// FP32 values of the four UE8M0 codes of a word: the code in the exponent's place, unless a code is 0 (2^-127,
// a subnormal) or 255 (NaN). A byte of v is 0 where (v - 0x01010101) & ~v has its top bit (or a byte below
// is 0, which is as good a reason to look closer).
__device__ __forceinline__ float4 four_scales(uint32_t w) {
  if (((w - 0x01010101u) & ~w & 0x80808080u) || ((~w - 0x01010101u) & w & 0x80808080u))
    return make_float4(dg::ue8m0_value(w & 255), dg::ue8m0_value(w >> 8 & 255), dg::ue8m0_value(w >> 16 & 255), dg::ue8m0_value(w >> 24));
  return make_float4(__uint_as_float(w << 23 & 0x7F800000u), __uint_as_float(w << 15 & 0x7F800000u), __uint_as_float(w << 7 & 0x7F800000u),
                     __uint_as_float(w >> 1 & 0x7F800000u));
}

// A wait that has run out once is not repeated: the kernel then runs through on what is in its rings, with
// every barrier met, and the status word says that its results are void.
__device__ __forceinline__ bool wait_full(uint64_t* bar, uint32_t parity, const MoeArgs& a, bool ok) {
  if (ok && dg::mbar_wait(bar, parity, a.timeout_ns)) return true;
  if (ok) atomicOr(a.status, dg::kTimeoutBit);
  return false;
}

__host__ __device__ constexpr int round_up(int v, int to) { return (v + to - 1) / to * to; }

// Shapes. kBig (more than 8 tokens): experts then have several tokens; 16 columns, and for E2M1, whose
// tokens' side and conversions cost as much as its bytes, 32 rows a warp.
template <bool kFp4, bool kBig>
struct Up {
  static constexpr int kM = kFp4 && kBig ? 2 : 1, kCols = kBig ? 16 : 8;
  static constexpr int kWarps = kBig && !kFp4 ? 16 : 8, kThreads = 32 * kWarps;
  static constexpr int kBlock = 8 * kM * kWarps;                    // columns of h of a block, 64 or 128
  static constexpr int kBlocksPerSm = kBig && !kFp4 ? 1 : 2;
  static constexpr int kStages = kFp4 ? (kBig ? 4 : 8) : 5;
  static constexpr int kAhead = kStages - 2;                        // copies run this far ahead of the products
  // a stage: kBlock gate rows and as many up rows of 128 columns, the tokens' 128 bytes, E2M1's scales. A
  // token's row is spaced so that the lanes of a load of it (two rows of 64 bytes, four of 32) cover the banks.
  static constexpr int kBox = kBlock * Rows<kFp4>::kBytes;
  static constexpr int kTokenStride = kFp4 ? 160 : 192;
  static constexpr int kTokens = 2 * kBox, kScales = kTokens + kCols * kTokenStride;
  static constexpr int kStage = round_up(kScales + (kFp4 ? 8 * kBlock : 0), 1024);
  static constexpr int kRing = kStages * kStage;
  static constexpr int kExpanded = kFp4 ? kWarps * 256 * kM : 0;    // E2M1: a warp's scales as FP32
  // then the tokens' scales [groups, T], for E4M3 each warp's two scales of every group, and a cluster's
  // partial sums of two units
  static constexpr int kSums = kM * kCols / 2;                      // a thread's
  static __host__ __device__ int partials(int groups, int T) {
    return kRing + kExpanded + round_up((groups * T + 1) / 2 * 8 + (kFp4 ? 0 : kWarps * groups * 8), 16);
  }
  static int smem(int groups, int T, int cluster) { return 1024 + partials(groups, T) + (cluster > 1 ? 2 * kThreads * kSums * 4 : 0); }
};
template <bool kFp4, bool kBig>
struct Down {
  static constexpr int kM = kFp4 && kBig ? 2 : 1;
  // with 32 rows, 16 columns' fragments and sums would not fit the registers: an expert of more than 8 tokens
  // is then two jobs, the second of which finds the weights in L2
  static constexpr int kCols = kBig && kM == 1 ? 16 : 8;
  static constexpr int kRows = 16 * kM, kWarps = 16, kThreads = 32 * kWarps;
  static constexpr int kStages = kFp4 ? (kBig ? 4 : 6) : 4;
  static constexpr int kBox = kRows * Rows<kFp4>::kBytes;           // a stage of a warp
  static constexpr int kRing = kWarps * kStages * kBox;
  // E4M3: the packed word of the rows' 128-row block (with its neighbours); E2M1: a word per row
  static constexpr int kScaleBytes = kFp4 ? 4 * kRows : 16;
  static constexpr int kScales = kWarps * kStages * kScaleBytes;
  static constexpr int kExpanded = kFp4 ? kWarps * 256 * kM : 0;
  // then every warp's sums of a tile, [warps][T][kRows], and the block's
  static int smem(int T) { return 1024 + kRing + kScales + kExpanded + (kWarps + 1) * T * kRows * 4; }
};

__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}

__device__ __forceinline__ int cluster_blocks() {
  int n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}

__device__ __forceinline__ uint8_t* aligned_1k(uint8_t* p) {
  return p + ((1024u - (dg::smem_addr(p) & 1023u)) & 1023u);
}

// -------------------------------------------------------------------------------------------
// First kernel: h = weight * silu(G x) * (U x)
// -------------------------------------------------------------------------------------------
//
// A unit is kBlock columns of h of a job: kBlock gate rows and kBlock up rows of W13, a warp 8 kM of each. A
// stage is 128 columns of all of them and of the job's tokens. The warps take turns at issuing its copies,
// two stages less than the ring is long ahead: a warp may then lag another by two stages before its turn
// has to wait for it. (A warp for the copies alone would leave the others 96 registers instead of 128.)

template <bool kFp4, bool kBig>
__global__ void __launch_bounds__(Up<kFp4, kBig>::kThreads, Up<kFp4, kBig>::kBlocksPerSm)
    moe_up_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
  using C = Up<kFp4, kBig>;
  using R = Rows<kFp4>;
  constexpr int kM = C::kM, NT = C::kCols / 8, kStages = C::kStages, kWarps = C::kWarps;
  extern __shared__ uint8_t raw[];
  __shared__ Routing r;
  __shared__ float block_max[2][kWarps][C::kCols];
  __shared__ uint64_t full[kStages], empty[kStages];
  uint8_t* const ring = aligned_1k(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      dg::mbar_init(&full[i], 1);
      dg::mbar_init(&empty[i], kWarps);
    }
    dg::fence_mbarrier_init();
    dg::tma_prefetch_desc(&map);
  }
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int t4 = (a.T + 3) / 4 * 4;
  const int groups = a.H / 128, blocks = a.I / C::kBlock;
  build_routing<C::kCols, C::kThreads>(a, r, *reinterpret_cast<RoutingScratch*>(ring), blockIdx.x == 0);
  float* expanded = reinterpret_cast<float*>(ring + C::kRing) + warp * 64 * kM;
  float* sx = reinterpret_cast<float*>(ring + C::kRing + C::kExpanded);
  for (int i = threadIdx.x; i < (groups + 3) / 4 * a.T; i += C::kThreads) {
    const int w = i / a.T, t = i % a.T;
    const uint32_t v = dg::ld_cg_s32(a.sfx + w * t4 + t);
    for (int b = 0; b < 4 && 4 * w + b < groups; ++b) sx[(4 * w + b) * a.T + t] = dg::ue8m0_value(v >> (8 * b) & 255);
  }
  dg::fence_proxy_async_smem();        // the scratch in the ring was written by threads; copies write there next
  __syncthreads();
  const int units = r.jobs * blocks;
  // the cluster's share of the units, and this block's of their column groups
  const int ranks = cluster_blocks(), rank = ranks > 1 ? dg::cluster_cta_rank() : 0;
  const int first_unit = blockIdx.x / ranks, unit_step = gridDim.x / ranks;
  const int group_begin = rank * groups / ranks, group_end = (rank + 1) * groups / ranks;
  bool ok = true;

  // the stage to copy: column group fg of unit fu, the issued'th of the block
  int fu = first_unit, fg = group_begin, fstage = 0, issued = 0;
  uint32_t fphase = 1;
  auto fetch = [&] {
    if (fu >= units) return;
    if (issued % kWarps == warp && a.fault == 0) {
      const int job = fu / blocks, e = r.job_expert[job], i0 = fu % blocks * C::kBlock, slot = r.job_slot[job], count = r.job_count[job];
      ok = wait_full(&empty[fstage], fphase, a, ok);
      if (__all_sync(kAll, ok)) {
        uint8_t* to = ring + fstage * C::kStage;
        if (lane == 0) {
          const int row = e * 2 * a.I + i0;
          dg::mbar_arrive_expect_tx(&full[fstage], 2 * C::kBox + count * 128 + (kFp4 ? 8 * C::kBlock : 0));
          dg::tma_load_2d(to, &map, &full[fstage], fg * R::kBytes, row);
          dg::tma_load_2d(to + C::kBox, &map, &full[fstage], fg * R::kBytes, row + a.I);
          if (kFp4) {
            const int32_t* from = a.sf13 + (static_cast<long long>(e) * groups + fg) * 2 * a.I + i0;
            bulk_load(to + C::kScales, from, 4 * C::kBlock, &full[fstage]);
            bulk_load(to + C::kScales + 4 * C::kBlock, from + a.I, 4 * C::kBlock, &full[fstage]);
          }
        }
        __syncwarp();
        if (lane < count)
          bulk_load(to + C::kTokens + lane * C::kTokenStride, a.x + static_cast<long long>(r.token[slot + lane]) * a.H + fg * 128, 128, &full[fstage]);
      }
    }
    ++issued;
    if (++fstage == kStages) fstage = 0, fphase ^= 1;
    if (++fg == group_end) fg = group_begin, fu += unit_step;
  };

  const int g8 = lane / 4, q4 = lane & 3, row8 = R::of(g8);
  float2* sw = reinterpret_cast<float2*>(sx + (groups * a.T + 1) / 2 * 2) + warp * groups;
  // E4M3: packed scale word `lane` of a unit's gate and up rows, read a unit ahead
  uint32_t next_gate = 0, next_up = 0;
  auto load_scales = [&](int u) {
    const int e = r.job_expert[u / blocks], i0 = u % blocks * C::kBlock, n4 = (a.I / 64 + 3) / 4 * 4;
    if (lane < (groups + 3) / 4) {
      const int32_t* sf = a.sf13 + (static_cast<long long>(e) * ((groups + 3) / 4) + lane) * n4;
      next_gate = dg::ld_cg_s32(sf + i0 / 128);
      next_up = dg::ld_cg_s32(sf + (a.I + i0) / 128);
    }
  };
  for (int i = 0; i < C::kAhead; ++i) fetch();
  if (!kFp4 && first_unit < units) load_scales(first_unit);
  int stage = 0, flip = 0;
  uint32_t phase = 0;
  for (int u = first_unit; u < units; u += unit_step, flip ^= 1) {
    const int job = u / blocks, blk = u % blocks, slot = r.job_slot[job], count = r.job_count[job];
    float sum[kM][NT][4];
    const float* sxt[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int m = 0; m < kM; ++m) sum[m][n][0] = sum[m][n][1] = sum[m][n][2] = sum[m][n][3] = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        sxt[n][i] = sx + (col < count ? r.token[slot + col] : 0);
      }
    }
    if constexpr (!kFp4) {
      __syncwarp();
      if (lane < (groups + 3) / 4) {
        const float4 gate = four_scales(next_gate), up = four_scales(next_up);
        sw[4 * lane] = make_float2(gate.x, up.x);
        if (4 * lane + 1 < groups) sw[4 * lane + 1] = make_float2(gate.y, up.y);
        if (4 * lane + 2 < groups) sw[4 * lane + 2] = make_float2(gate.z, up.z);
        if (4 * lane + 3 < groups) sw[4 * lane + 3] = make_float2(gate.w, up.w);
      }
      __syncwarp();
      if (u + unit_step < units) load_scales(u + unit_step);
    }
    for (int g = group_begin; g < group_end; ++g) {
      fetch();
      ok = wait_full(&full[stage], phase, a, ok);
      const uint8_t* at = ring + stage * C::kStage;
      const uint8_t* gate = at + warp * 8 * kM * R::kBytes;
      const uint8_t* up = gate + C::kBox;
      const uint8_t* tokens = at + C::kTokens + g8 * C::kTokenStride;
      // one item, for N eights of columns (a branch for the second eight inside would cost those that have one)
      auto item = [&](auto eights) {
        constexpr int N = decltype(eights)::value;
        float acc[kM][N][4];
        if constexpr (!kFp4) {
          uint4 w0[2], w1[2], x[N][2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            w0[p] = lds<uint4>(gate + R::chunk(row8, 4 * p + q4)), w1[p] = lds<uint4>(up + R::chunk(row8, 4 * p + q4));
#pragma unroll
            for (int n = 0; n < N; ++n)
              x[n][p] = lds<uint4>(tokens + n * 8 * C::kTokenStride + 64 * p + 16 * q4);
          }
#pragma unroll
          for (int n = 0; n < N; ++n)
            {
              mma_e4m3_zero(acc[0][n], w0[0].x, w1[0].x, w0[0].y, w1[0].y, x[n][0].x, x[n][0].y);
              mma_e4m3(acc[0][n], w0[0].z, w1[0].z, w0[0].w, w1[0].w, x[n][0].z, x[n][0].w);
              mma_e4m3(acc[0][n], w0[1].x, w1[1].x, w0[1].y, w1[1].y, x[n][1].x, x[n][1].y);
              mma_e4m3(acc[0][n], w0[1].z, w1[1].z, w0[1].w, w1[1].w, x[n][1].z, x[n][1].w);
            }
        } else {
          // the warp's scales, 8 kM gate rows and then as many up rows, as FP32: each converted by one lane
          const uint8_t* packed = at + C::kScales + warp * 32 * kM + (lane / 16) * 4 * C::kBlock;
          if constexpr (kM == 1) {
            const uint32_t w = lds<uint32_t>(packed + lane % 16 / 2 * 4) >> (lane & 1) * 16;
            reinterpret_cast<float2*>(expanded)[lane] = make_float2(dg::ue8m0_value(w & 255), dg::ue8m0_value(w >> 8 & 255));
          } else {
            reinterpret_cast<float4*>(expanded)[lane] = four_scales(lds<uint32_t>(packed + lane % 16 * 4));
          }
          __syncwarp();
          float4 scale[kM][2];
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            scale[m][0] = reinterpret_cast<const float4*>(expanded)[8 * m + g8];
            scale[m][1] = reinterpret_cast<const float4*>(expanded)[8 * kM + 8 * m + g8];
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            uint32_t even[N], odd[N];
#pragma unroll
            for (int n = 0; n < N; ++n)
              {
                const uint2 x = lds<uint2>(tokens + n * 8 * C::kTokenStride + 32 * b + 8 * q4);
                even[n] = __byte_perm(x.x, x.y, 0x6420), odd[n] = __byte_perm(x.x, x.y, 0x7531);
              }
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              const uint32_t u0 = lds<uint32_t>(gate + m * 8 * R::kBytes + R::chunk(row8, b) + 4 * q4);
              const uint32_t u1 = lds<uint32_t>(up + m * 8 * R::kBytes + R::chunk(row8, b) + 4 * q4);
              const uint32_t a0 = e4m3_of_even(u0), a1 = e4m3_of_even(u1), a2 = e4m3_of_odd(u0), a3 = e4m3_of_odd(u1);
              const float e0 = float_of(scale[m][0], b), e1 = float_of(scale[m][1], b);
#pragma unroll
              for (int n = 0; n < N; ++n)
                {
                  float part[4];
                  mma_e4m3_zero(part, a0, a1, a2, a3, even[n], odd[n]);
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const float e = i < 2 ? e0 : e1;
                    acc[m][n][i] = b == 0 ? e * part[i] : fmaf(e, part[i], acc[m][n][i]);
                  }
                }
            }
          }
        }
        __syncwarp();
        if (lane == 0) dg::mbar_arrive(&empty[stage]);
        const float2 s = kFp4 ? make_float2(1.0f, 1.0f) : sw[g];
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float t = sxt[n][i][g * a.T], tx = kFp4 ? t : t * s.x, ty = kFp4 ? t : t * s.y;
#pragma unroll
              for (int m = 0; m < kM; ++m) {
                sum[m][n][i] = fmaf(tx, acc[m][n][i], sum[m][n][i]);
                sum[m][n][2 + i] = fmaf(ty, acc[m][n][2 + i], sum[m][n][2 + i]);
              }
            }
      };
      if (NT == 1 || count <= 8) item(std::integral_constant<int, 1>());
      else item(std::integral_constant<int, NT>());
      if (++stage == kStages) stage = 0, phase ^= 1;
    }
    if (ranks > 1) {
      // the first block of the cluster adds the others' sums to its own
      float4* mine = reinterpret_cast<float4*>(ring + C::partials(groups, a.T)) + flip * C::kThreads * (C::kSums / 4);
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          mine[(m * NT + n) * C::kThreads + threadIdx.x] = make_float4(sum[m][n][0], sum[m][n][1], sum[m][n][2], sum[m][n][3]);
      dg::cluster_sync();
      if (rank != 0) continue;
      for (int other = 1; other < ranks; ++other) {
        const uint32_t theirs = dg::map_to_rank(mine, other);
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 v = dg::ld_shared_cluster_v4(theirs + ((m * NT + n) * C::kThreads + threadIdx.x) * 16);
            sum[m][n][0] += __uint_as_float(v.x), sum[m][n][1] += __uint_as_float(v.y);
            sum[m][n][2] += __uint_as_float(v.z), sum[m][n][3] += __uint_as_float(v.w);
          }
      }
    }
    // column blk * kBlock + (warp * kM + m) * 8 + row8 of h for tokens 2 q4, 2 q4 + 1 of each eight: gate in
    // sum[0..1], up in sum[2..3] (E2M1 went into the MMAs as 2^-6 of itself)
    constexpr float kUnit = kFp4 ? 64.0f : 1.0f;
    float hv[kM][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        const float w = col < count ? r.coef[slot + col] : 0.0f;
        float top = 0;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const float gate = sum[m][n][i] * kUnit;
          hv[m][n][i] = col < count ? w * (gate / (1.0f + expf(-gate)) * (sum[m][n][2 + i] * kUnit)) : 0.0f;
          const float v = fabsf(hv[m][n][i]);
          top = fmaxf(top, v < INFINITY ? v : 0.0f);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        if (g8 == 0) block_max[flip][warp][col] = top;
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        if (col >= count) continue;
        float top = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, block_max[flip][w][col]);
        // the largest to [2^14, 2^15); both powers stay normal
        const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 254) - 127 - 14;
        const float to_half = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        const float back = __uint_as_float(static_cast<uint32_t>(127 + ex + (kFp4 ? 14 : 0)) << 23);   // E2M1 enters the MMAs as 2^-14 of itself
        uint8_t* row = a.h + (static_cast<long long>(slot + col) * (a.I / 128) + blk * C::kBlock / 128) * kHBytes;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          // where the second kernel's lanes find this column of the 128: E4M3 as 16-byte pieces of two loads,
          // each of 64 bytes over four lanes; E2M1 the even ones of every eight, then the odd ones
          const int cc = blk * C::kBlock % 128 + (warp * kM + m) * 8 + row8;
          const int place = kFp4 ? (cc / 8 * 8 + cc % 2 * 4 + cc % 8 / 2) * 2 : cc / 64 * 128 + cc % 16 / 8 * 64 + cc % 64 / 16 * 16 + cc % 8 * 2;
          *reinterpret_cast<__half*>(row + place) = __float2half_rn(hv[m][n][i] * to_half);
        }
        if (warp == 0 && g8 == 0) {
          float* to = reinterpret_cast<float*>(row + 256);
          if (C::kBlock == 128) to[0] = to[1] = back;
          else to[blk & 1] = back;
        }
      }
  }
  // no copy may be under way when the block ends, and no block of a cluster be gone whose sums are read
  if (!ok && a.fault == 0)
    for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
      if (!dg::mbar_wait(&full[i % kStages], i / kStages & 1, a.timeout_ns)) break;
  if (ranks > 1) dg::cluster_sync();
}

// -------------------------------------------------------------------------------------------
// Second kernel: y = c + W2 h
// -------------------------------------------------------------------------------------------
//
// A tile is kRows output rows and all tokens. Its items are 128 columns of W2 of a job each; a warp takes a
// run of them, with a ring of its own that its first lane fills. The tokens' side is small, shared by all
// tiles and stays in L2: a warp reads its fragments of it straight into registers, an item ahead.

template <bool kFp4, bool kBig>
__global__ void __launch_bounds__(Down<kFp4, kBig>::kThreads, 1) moe_down_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
  using C = Down<kFp4, kBig>;
  using R = Rows<kFp4>;
  constexpr int kM = C::kM, NT = C::kCols / 8, kStages = C::kStages, kWarps = C::kWarps;
  extern __shared__ uint8_t raw[];
  __shared__ Routing r;
  __shared__ uint64_t full_bars[kWarps][kStages];
  uint8_t* const rings = aligned_1k(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3, row8 = R::of(g8);
  uint64_t* full = full_bars[warp];
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) dg::mbar_init(&full[i], 1);
    dg::fence_mbarrier_init();
    if (warp == 0) dg::tma_prefetch_desc(&map);
  }
  // The first kernel let this one start only after its own wait: ids and weights are there, h is not yet.
  build_routing<C::kCols, C::kThreads>(a, r, *reinterpret_cast<RoutingScratch*>(rings), false);

  const int groups = a.I / 128, items = r.jobs * groups, tiles = a.H / C::kRows;
  const int n4 = kFp4 ? a.H : (a.H / 128 + 3) / 4 * 4;
  uint8_t* const ring = rings + warp * kStages * C::kBox;
  uint8_t* const scales = rings + C::kRing + warp * kStages * C::kScaleBytes;
  float* expanded = reinterpret_cast<float*>(rings + C::kRing + C::kScales) + warp * 64 * kM;
  float* sums = reinterpret_cast<float*>(rings + C::kRing + C::kScales + C::kExpanded);
  for (int i = threadIdx.x; i < kWarps * a.T * C::kRows; i += C::kThreads) sums[i] = 0;
  dg::fence_proxy_async_smem();        // the scratch in the rings was written by threads; copies write there next
  __syncthreads();

  // the cluster's tiles, and this warp's run of their items among all of the cluster's warps
  const int ranks = cluster_blocks(), rank = ranks > 1 ? dg::cluster_cta_rank() : 0;
  const int first_tile = blockIdx.x / ranks, tile_step = gridDim.x / ranks;
  const int place = rank * kWarps + warp, places = ranks * kWarps;
  const int begin = place * items / places, end = (place + 1) * items / places, begin_job = begin / groups, begin_g = begin % groups;
  int ft = begin < end && a.fault == 0 ? first_tile : tiles, fi = begin, fjob = begin_job, fg = begin_g, fstage = 0, issued = 0;
  auto fetch = [&] {
    if (ft >= tiles) return;
    if (lane == 0) {
      const int e = r.job_expert[fjob], row = ft * C::kRows;
      dg::mbar_arrive_expect_tx(&full[fstage], C::kBox + C::kScaleBytes);
      dg::tma_load_2d(ring + fstage * C::kBox, &map, &full[fstage], fg * R::kBytes, e * a.H + row);
      const int32_t* sf = kFp4 ? a.sf2 + (static_cast<long long>(e) * groups + fg) * n4 + row
                               : a.sf2 + (static_cast<long long>(e) * ((groups + 3) / 4) + fg / 4) * n4 + (row / 128 & ~3);
      bulk_load(scales + fstage * C::kScaleBytes, sf, C::kScaleBytes, &full[fstage]);
    }
    ++issued;
    if (++fstage == kStages) fstage = 0;
    if (++fi == end) fi = begin, fjob = begin_job, fg = begin_g, ft += tile_step;
    else if (++fg == groups) fg = 0, ++fjob;
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();

  // this lane's fragments of an item's tokens (as FP16 pairs) and the scales of its two columns
  constexpr bool kAhead = NT == 1;     // sixteen columns' fragments leave no registers for a second set
  uint4 hr[NT][4];
  uint2 hs[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    hs[n][0] = hs[n][1] = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) hr[n][i] = make_uint4(0, 0, 0, 0);
  }
  const uint32_t slot_bytes = groups * kHBytes;                     // at most 512 slots of 128 groups: 32 bits are enough
  auto load_h = [&](int job, int g) {
    const int slot = r.job_slot[job], count = r.job_count[job];
    const uint8_t* base = a.h + (slot * slot_bytes + g * kHBytes);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (n * 8 + g8 < count) {
        const uint8_t* from = base + (n * 8 + g8) * slot_bytes + q4 * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) hr[n][i] = dg::ld_cg_v4(from + i * 64);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (n * 8 + 2 * q4 + i < count) hs[n][i] = ld_cg_v2(base + (n * 8 + 2 * q4 + i) * slot_bytes + 256);
    }
  };
  if (begin < end && first_tile < tiles) load_h(begin_job, begin_g);

  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  for (int tile = first_tile; tile < tiles; tile += tile_step) {
    float* mine = sums + warp * a.T * C::kRows;
    float sum[kM][NT][4];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) sum[m][n][0] = sum[m][n][1] = sum[m][n][2] = sum[m][n][3] = 0;
    int job = begin_job, g = begin_g;
    for (int it = begin; it < end; ++it) {
      const int slot = r.job_slot[job], count = r.job_count[job];
      const bool last = it + 1 == end, turn = g + 1 == groups;
      auto load_next = [&] {
        if (!last) load_h(turn ? job + 1 : job, turn ? 0 : g + 1);
        else if (tile + tile_step < tiles) load_h(begin_job, begin_g);
      };
      uint4 hc[NT][4];
      uint2 sc[NT][2];
      if constexpr (kAhead) {
#pragma unroll
        for (int i = 0; i < 4; ++i) hc[0][i] = hr[0][i];
        sc[0][0] = hs[0][0], sc[0][1] = hs[0][1];
        load_next();
      }
      auto frag = [&](int n, int i, int w) { return word_of(kAhead ? hc[n][i] : hr[n][i], w); };
      auto col_scale = [&](int n, int i, int p) {
        const uint2 v = kAhead ? sc[n][i] : hs[n][i];
        return __uint_as_float(p ? v.y : v.x);
      };
      ok = wait_full(&full[stage], phase, a, ok);
      const uint8_t* at = ring + stage * C::kBox;
      const uint8_t* packed = scales + stage * C::kScaleBytes;
      // one item, for N eights of columns
      auto item = [&](auto eights) {
        constexpr int N = decltype(eights)::value;
        if constexpr (!kFp4) {
          const float s = dg::ue8m0_value(lds<uint32_t>(packed + (tile * C::kRows / 128 & 3) * 4) >> (8 * (g & 3)) & 255);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint4 w0 = lds<uint4>(at + R::chunk(row8, 4 * p + q4)), w1 = lds<uint4>(at + R::chunk(8 + row8, 4 * p + q4));
            float acc[N][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u0 = word_of(w0, i), u1 = word_of(w1, i);
              const uint32_t a0 = half2_of_e4m3(u0), a2 = half2_of_e4m3(u0 >> 16), a1 = half2_of_e4m3(u1), a3 = half2_of_e4m3(u1 >> 16);
#pragma unroll
              for (int n = 0; n < N; ++n) {
                const uint32_t b0 = frag(n, 2 * p + i / 2, i % 2 * 2), b1 = frag(n, 2 * p + i / 2, i % 2 * 2 + 1);
                if (i == 0) mma_f16_zero(acc[n], a0, a1, a2, a3, b0, b1);
                else mma_f16(acc[n], a0, a1, a2, a3, b0, b1);
              }
            }
#pragma unroll
            for (int n = 0; n < N; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float t = s * col_scale(n, i, p);
                sum[0][n][i] = fmaf(t, acc[n][i], sum[0][n][i]);
                sum[0][n][2 + i] = fmaf(t, acc[n][2 + i], sum[0][n][2 + i]);
              }
          }
        } else {
          // the rows' scales as FP32, each converted by one lane
          if constexpr (kM == 1) {
            const uint32_t w = lds<uint32_t>(packed + lane / 2 * 4) >> (lane & 1) * 16;
            reinterpret_cast<float2*>(expanded)[lane] = make_float2(dg::ue8m0_value(w & 255), dg::ue8m0_value(w >> 8 & 255));
          } else {
            reinterpret_cast<float4*>(expanded)[lane] = four_scales(lds<uint32_t>(packed + lane * 4));
          }
          __syncwarp();
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const float4 s0 = reinterpret_cast<const float4*>(expanded)[16 * m + g8], s1 = reinterpret_cast<const float4*>(expanded)[16 * m + 8 + g8];
            float half[N][4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint32_t u0 = lds<uint32_t>(at + R::chunk(16 * m + row8, b) + 4 * q4), u1 = lds<uint32_t>(at + R::chunk(16 * m + 8 + row8, b) + 4 * q4);
              const uint32_t even0 = f16_of_even(u0), even1 = f16_of_even(u1), odd0 = f16_of_odd(u0), odd1 = f16_of_odd(u1);
              const float e0 = float_of(s0, b), e1 = float_of(s1, b);
#pragma unroll
              for (int n = 0; n < N; ++n) {
                float part[4];
                mma_f16_zero(part, lower_pair(even0), lower_pair(even1), upper_pair(even0), upper_pair(even1), frag(n, b, 0), frag(n, b, 1));
                mma_f16(part, lower_pair(odd0), lower_pair(odd1), upper_pair(odd0), upper_pair(odd1), frag(n, b, 2), frag(n, b, 3));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float e = i < 2 ? e0 : e1;
                  half[n][i] = b % 2 == 0 ? e * part[i] : fmaf(e, part[i], half[n][i]);
                  if (b % 2 == 1) sum[m][n][i] = fmaf(col_scale(n, i % 2, b / 2), half[n][i], sum[m][n][i]);
                }
              }
            }
          }
        }
      };
      if (NT == 1 || count <= 8) item(std::integral_constant<int, 1>());
      else item(std::integral_constant<int, NT>());
      __syncwarp();        // every lane has read the stage
      if constexpr (!kAhead) load_next();
      if (++stage == kStages) stage = 0, phase ^= 1;
      fetch();
      if (last || turn) {
        // rows row8 and row8 + 8 of each 16 for the job's tokens, into the warp's sums
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = n * 8 + 2 * q4 + i;
            if (col < count) {
              float* to = mine + r.token[slot + col] * C::kRows + row8;
#pragma unroll
              for (int m = 0; m < kM; ++m) {
                to[16 * m] += sum[m][n][i];
                to[16 * m + 8] += sum[m][n][2 + i];
              }
            }
#pragma unroll
            for (int m = 0; m < kM; ++m) sum[m][n][i] = sum[m][n][2 + i] = 0;
          }
        __syncwarp();
      }
      g = turn ? 0 : g + 1;
      job += turn;
    }
    __syncthreads();
    // the warps' sums, then the cluster's; each block of a cluster writes its share of the tile
    const int values = a.T * C::kRows;
    float* total = sums + kWarps * values;
    for (int i = threadIdx.x; i < values; i += C::kThreads) {
      float v = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v += sums[w * values + i];
        sums[w * values + i] = 0;
      }
      total[i] = v;
    }
    if (ranks > 1) dg::cluster_sync();
    else __syncthreads();
    for (int i = rank * values / ranks + threadIdx.x; i < (rank + 1) * values / ranks; i += C::kThreads) {
      const long long to = static_cast<long long>(i / C::kRows) * a.H + tile * C::kRows + i % C::kRows;
      float v = a.c ? __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(a.c) + to))) : 0.0f;
      if (ranks == 1) v += total[i];
      else
        for (int other = 0; other < ranks; ++other) v += ld_shared_cluster_f32(dg::map_to_rank(total + i, other));
      a.y[to] = __float2bfloat16_rn(v);
    }
    if (ranks > 1) dg::cluster_sync();
    else __syncthreads();
  }
  // no copy may be under way when the block ends
  if (!ok && a.fault == 0)
    for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
      if (!dg::mbar_wait(&full[i % kStages], i / kStages & 1, a.timeout_ns)) break;
}

// -------------------------------------------------------------------------------------------

template <bool kFp4, bool kBig>
dg_status run_layer(const MoeArgs& a, const LaunchContext& ctx, cudaStream_t stream) {
  using U = Up<kFp4, kBig>;
  using D = Down<kFp4, kBig>;
  static_assert(sizeof(RoutingScratch) <= U::kRing && sizeof(RoutingScratch) <= D::kRing, "scratch in the rings");
  static_assert(U::kBlock == 64 || U::kBlock == 128, "h has two scales per 128 columns");
  // Blocks of a cluster: as many, a power of two up to 8, as fit the SMs for the units (tiles) that there are at
  // most, if each still has K groups (items for its warps) to work on.
  const int groups = a.H / 128, units = std::min(a.T * a.k, a.E) * (a.I / U::kBlock), tiles = a.H / D::kRows;
  const int items = std::min(a.T * a.k, a.E) * (a.I / 128);
  const int up_room = ctx.sms * (U::kBlocksPerSm == 2 && U::smem(groups, a.T, 2) <= kHalfSm ? 2 : 1);
  int up_cluster = 1, down_cluster = 1;
  while (up_cluster < 8 && 2 * up_cluster * units <= up_room && 2 * up_cluster <= groups) up_cluster *= 2;
  while (down_cluster < 8 && 2 * down_cluster * tiles <= ctx.sms && 2 * down_cluster * D::kWarps <= items) down_cluster *= 2;
  const int up_smem = U::smem(groups, a.T, up_cluster), down_smem = D::smem(a.T);
  if (up_smem > kMaxSmem || down_smem > kMaxSmem) return DG_ERR_UNSUPPORTED;
  // once per thread and device: the limit, above what any shape needs
  static thread_local int ready = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && ready != dev) {
    e = cudaFuncSetAttribute(moe_up_kernel<kFp4, kBig>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<kFp4, kBig>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return dg::record_cuda_error(e);
  const int per = kFp4 ? 2 : 1;
  CUtensorMap up_map, down_map;
  if (!dg::byte_rows_map(&up_map, a.w13, static_cast<uint64_t>(a.E) * 2 * a.I, a.H / per, U::kBlock, Rows<kFp4>::kBytes) ||
      !dg::byte_rows_map(&down_map, a.w2, static_cast<uint64_t>(a.E) * a.H, a.I / per, D::kRows, Rows<kFp4>::kBytes))
    return DG_ERR_CUDA;
  const int up_clusters = up_cluster > 1 ? units : std::min(units, U::kBlocksPerSm * ctx.sms);
  const int down_clusters = std::min(tiles, std::max(1, ctx.sms / down_cluster));
  if (dg_status s = dg::launch_clusters(moe_up_kernel<kFp4, kBig>, static_cast<unsigned>(up_clusters * up_cluster), static_cast<unsigned>(up_cluster),
                                        U::kThreads, static_cast<size_t>(up_smem), stream, ctx.pdl, up_map, a); s != DG_OK) return s;
  return dg::launch_clusters(moe_down_kernel<kFp4, kBig>, static_cast<unsigned>(down_clusters * down_cluster), static_cast<unsigned>(down_cluster),
                             D::kThreads, static_cast<size_t>(down_smem), stream, ctx.pdl, down_map, a);
}

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <bool kFp4>
dg_status few_tokens(const void* x, const int32_t* sfx, const void* w13, const int32_t* sf13, const void* w2,
                     const int32_t* sf2, const int32_t* ids, const float* weights, const void* c, void* y, int T, int topk,
                     int E, int H, int I, cudaStream_t stream) {
  if (T < 0 || topk <= 0 || E <= 0 || H <= 0 || I <= 0 || H % 128 != 0 || I % 128 != 0) return DG_ERR_INVALID_ARG;
  if (T > kMaxTokens || topk > kMaxTopk || E > kMaxExperts || H > kMaxH || I > kMaxH) return DG_ERR_UNSUPPORTED;
  if (T == 0) return DG_OK;
  if (!x || !sfx || !w13 || !sf13 || !w2 || !sf2 || !ids || !weights || !y) return DG_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(sfx, 16) || !aligned(w13, 16) || !aligned(sf13, 16) || !aligned(w2, 16) || !aligned(sf2, 16) ||
      !aligned(ids, 4) || !aligned(weights, 4) || !aligned(c, 16) || !aligned(y, 16))
    return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  dg::StreamWorkspace ws;
  void* h = nullptr;
  if (dg_status s = ws.acquire(stream, static_cast<size_t>(T) * topk * (I / 128) * kHBytes, &h); s != DG_OK) return s;
  const MoeArgs a{static_cast<const uint8_t*>(x), sfx, static_cast<const uint8_t*>(w13), sf13, static_cast<const uint8_t*>(w2), sf2,
                  ids, weights, static_cast<const __nv_bfloat16*>(c), static_cast<__nv_bfloat16*>(y), static_cast<uint8_t*>(h),
                  ctx.status, dg::pipeline_wait_timeout_ns(), dg::debug_fault_mode(), T, topk, E, H, I};
  return T <= 8 ? run_layer<kFp4, false>(a, ctx, stream) : run_layer<kFp4, true>(a, ctx, stream);
}

}  // namespace

extern "C" {

dg_status dg_moe_fp8_few_tokens(const void* x, const int32_t* sfx, const void* w13, const int32_t* sf13, const void* w2,
                                const int32_t* sf2, const int32_t* topk_ids, const float* topk_weights, const void* c,
                                void* y, int T, int topk, int E, int H, int I, cudaStream_t stream) {
  return few_tokens<false>(x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, T, topk, E, H, I, stream);
}

dg_status dg_moe_fp8_fp4_few_tokens(const void* x, const int32_t* sfx, const void* w13, const int32_t* sf13, const void* w2,
                                    const int32_t* sf2, const int32_t* topk_ids, const float* topk_weights, const void* c,
                                    void* y, int T, int topk, int E, int H, int I, cudaStream_t stream) {
  return few_tokens<true>(x, sfx, w13, sf13, w2, sf2, topk_ids, topk_weights, c, y, T, topk, E, H, I, stream);
}

}  // extern "C"
