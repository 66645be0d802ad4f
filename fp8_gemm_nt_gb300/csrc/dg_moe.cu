// A whole mixture-of-experts layer for a few tokens (at most 32), in two kernels:
//
//   y[t] = c[t] + sum over the slots j of token t with an expert e = ids[t, j]:
//              weights[t, j] * W2_e (silu(G_e x_t) * (U_e x_t)),      (G_e; U_e) = W13_e
//
// x is E4M3 with one UE8M0 scale per 128 columns; the experts' weights are E4M3 with one scale per
// 128 x 128 block, or E2M1 with one per row per 32 columns: the grouped GEMMs' operands.
//
// At a few tokens an expert has one to a handful of rows, so the time is that of reading the weights
// of the experts in use, once. The grouped GEMMs make the tokens the 128 rows of an MMA and would fill
// one to four of them; here the weights are the M operand (128 rows) and an expert's tokens the N columns
// of block-scaled tcgen05 MMAs, which take E4M3 and E2M1 as they are, with their scales: TMA brings the
// weights to shared memory and no instruction touches them on the way.
//
// An expert's tokens are compacted into jobs (of at most 16 in the first product, 8 in the second); each distinct
// (expert, token) pair is a slot. The first kernel computes h = weight * silu(g) * u of every slot. The second
// product also has to be E4M3 by the weights' type, and four bits would be too few: h is written as the sum of four
// E4M3 terms, each the remainder of those before it times 16, under one power of two for each 64 columns that brings
// their largest to (224, 448]. A term rounds to within 2^-4 of itself or 2^-10 of its scale, so h is within 2^-16 of
// itself or 2^-22 of the scale, which is 2^-29.8 of the largest: with that y is as near to the exact sum as its
// rounding to BF16 lets it be (a sum whose leading bits c cancels is 2^-18.5 off, 2^-16 with three terms, which are
// up to 4 % faster, with many tokens of few experts). The four terms are four columns, whose scales are 16 times
// smaller each, and whose sums the second kernel adds up. It owns output rows, sums all experts for 128 rows of W2
// and every token in an order that depends on the sizes and the ids alone, and writes each output once. No atomics on
// values.
//
// A pipeline is a warp each for the weights' copies, the tokens' side, the weights' scales and the MMAs, and
// four that read the sums from TMEM, with a ring of stages of 128 columns. A block (one to an SM) is two
// pipelines, halves that share nothing but the routing: a stage takes one about 345 clocks, in
// which HBM brings an SM 8.1 KB, an E2M1 stage is 8.5 KB, and waits come on top.
//
// The pieces (64 columns of h of a job; 128 output rows) are few and large, so their stages are dealt out
// evenly, each pipeline a run of them, unless whole pieces do nearly as well (Deal). A piece that is cut is summed
// by the last of its pipelines to finish: each writes its FP32 part to the workspace, and the last adds all parts
// in the order of the pipelines, so that the result does not depend on which one it was. Nobody waits.
//
// Bound by HBM, but for about 15 us at the ends (ids to the first weights, last sums of h to the second product,
// joins). Experts of 7168 x 2048: E4M3, 32 tokens of 8 experts each among 64 (2.76 GB): 428 us, 6.4 TB/s; one token
// (352 MB): 65 us; E2M1, 16 tokens among 32 (736 MB): 137 us. With mma.sync, whose E4M3 products are emulated by
// FP16 ones, it was 464, 67 and 256 us.
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
constexpr int kCols = 16;               // tokens of a job of the first kernel
constexpr int kTerms = 4;               // E4M3 terms of a value of h
constexpr int kDownCols = 8;            // tokens of a job of the second kernel: 32 columns of their terms
constexpr int kBlock = 64;              // columns of h of a unit of the first kernel, which share a scale
constexpr int kHalf = 256;              // threads of a pipeline
constexpr int kThreads = 2 * kHalf;
constexpr int kMaxStages = 8;
constexpr int kJoin = 16;               // stages that take as long as joining the parts of a piece
constexpr int kMinShare = 8;            // stages of a pipeline, at least
constexpr int kMaxSmem = 221 * 1024;    // dynamic

struct MoeArgs {
  const uint8_t* x;        // [T, H] E4M3
  const int32_t* sfx;      // [KP(H), ceil4(T)]
  const int32_t* sf13;     // scales of w13 [E, 2 I, H]
  const int32_t* sf2;      // scales of w2 [E, H, I]
  const int32_t* ids;      // [T, k]
  const float* weights;    // [T, k]
  const __nv_bfloat16* c;  // [T, H] or null
  __nv_bfloat16* y;        // [T, H]
  uint8_t* h;              // [slots, kTerms, I] E4M3
  uint32_t* hs;            // [I / 128, slots, kTerms]: the codes of a term's four 32-column blocks of 128
  uint32_t* status;
  unsigned long long timeout_ns;   // of a wait
  int fault;                       // failure injection: no copies of weights
  int T, k, E, H, I;
  int cols;                              // tokens of a job, at most
  int stages, stage_bytes, scale_bytes;  // of a pipeline's ring
  int rest_bytes;                        // of a pipeline's shared memory beside the rings
  float* parts;                          // [pipelines][2] parts of cut pieces: [kCols][128], [T][128]
  int* arrivals;                         // per first pipeline of a cut piece; zero between launches
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
// every block of both kernels. Ends without a barrier.
template <int kThreads>
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
    n[i] = ((tokens + a.cols - 1) / a.cols) << 16 | tokens;
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
      for (int c = 0; c < tokens; c += a.cols, ++job) {
        r.job_expert[job] = static_cast<uint16_t>(e);
        r.job_slot[job] = static_cast<uint16_t>(slot + c);
        r.job_count[job] = static_cast<uint8_t>(min(a.cols, tokens - c));
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
}

// -------------------------------------------------------------------------------------------
// The products of both kernels
// -------------------------------------------------------------------------------------------

// Untiled bulk copy (16-byte aligned addresses and size) that completes on `bar`.
__device__ __forceinline__ void bulk_load(void* to, const void* from, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dg::smem_addr(to)),
               "l"(from), "r"(bytes), "r"(dg::smem_addr(bar))
               : "memory");
}
// Asynchronous copy of a word, and the thread's arrival at a barrier when its copies so far are done.
__device__ __forceinline__ void cp_async_4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(dg::smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void named_barrier(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// A stage: 128 weight rows of 128 columns (128-byte rows in the 128-byte swizzle; E2M1 spread by TMA, 16 elements to 8 bytes
// and 8 of padding), the tokens' rows in the same form, and scale words as tcgen05.cp takes them, 32 rows of 16 bytes (row
// r: the words of rows r, r + 32, ...): the weights', the tokens', and for E2M1 the weights' as loaded, one per row.
constexpr int kWeights = 128 * 128, kTile = 512;
constexpr int kTileA = 0, kTileB = kTile, kRaw = 2 * kTile;

struct Pipe {
  uint64_t full[kMaxStages], ready[kMaxStages], empty[kMaxStages], sum_full[2], sum_empty[2], drain;
};
struct Shared {
  Routing r;
  Pipe pipe[2];
  uint32_t tmem;
  int arrived[2];
  volatile uint32_t abort;
};

// A run of K groups of one job against 128 weight rows (two boxes of 64): one sum in TMEM.
struct Run {
  int job, expert, slot, count;
  int row0, row1;          // of the boxes, in the [E * N, K] weight matrix
  int begin, end;          // K groups
  int unit;                // first kernel: (job, 64 columns of h); `piece` the columns' index
  int piece;               // second kernel: the tile
  bool done;               // the pipeline's last run of the piece
};

// The stages of all pieces, dealt out to at most `most` pipelines in runs of equal length (to one). Where the longest
// run of whole pieces is at most kJoin stages longer than an equal share, pieces stay whole: joining the parts of a
// cut one takes about 3 us, a stage that does not wait for memory 0.2 us (one token, 8 experts of 7168 x 2048 in
// E4M3: 66.8 us with all stages dealt evenly, 65.0 us this way; twelve layers of 3 to 27 tokens and 0.6 to 100 MB: 372
// and 350 us; with kJoin 40, 366 us). At least kMinShare stages each, since the parts are joined by one pipeline: the
// twelve take 350 us with 4, 334 us with 8, 365 us with 24. At most 2^24 stages.
struct Deal {
  int unit, pipes, share, longer;  // `longer` pipelines have `share` + 1 units of `unit` stages, the others `share`
  __device__ __forceinline__ Deal(int pieces, int per, int most) {
    const int stages = pieces * per;
    const bool whole = (pieces + most - 1) / most * per <= stages / most + kJoin;
    unit = whole ? per : 1;
    const int units = whole ? pieces : stages;
    pipes = max(1, min(most, whole ? pieces : (stages + kMinShare - 1) / kMinShare));
    share = units / pipes;
    longer = units - share * pipes;
  }
  __device__ __forceinline__ int begin(int p) const { return unit * (min(p, pipes) * share + min(p, longer)); }
  // of a stage of a piece that was cut
  __device__ __forceinline__ int owner(int stage) const {
    const int before = longer * (share + 1);
    return stage < before ? stage / (share + 1) : longer + (stage - before) / share;
  }
};

// A pipeline's runs in order. First kernel: the pieces are units (job, 64 columns of h), each 64 gate rows and
// their up rows, a stage a K group. Second kernel: tiles of 128 output rows, a stage a (job, K group); a run ends
// with its job.
template <bool kDown>
struct Walk {
  const MoeArgs& a;
  const Routing& r;
  int at, end;
  int groups, per;         // K groups, and stages of a piece
  __device__ __forceinline__ Walk(const MoeArgs& args, const Routing& routing, const Deal& deal, int pipe) : a(args), r(routing) {
    groups = (kDown ? a.I : a.H) / 128;
    per = kDown ? r.jobs * groups : groups;
    at = deal.begin(pipe);
    end = deal.begin(pipe + 1);
  }
  __device__ __forceinline__ bool next(Run& s) {
    if (at >= end) return false;
    const int piece = at / per, in = at - piece * per;
    if (kDown) {
      s.job = in / groups;
      s.piece = piece;
      s.begin = in - s.job * groups;
    } else {
      const int blocks = a.I / kBlock;
      s.unit = piece;
      s.job = piece / blocks;
      s.piece = piece - s.job * blocks;
      s.begin = in;
    }
    s.end = min(groups, s.begin + end - at);
    at += s.end - s.begin;
    s.done = at >= end || in + s.end - s.begin == per;
    s.expert = r.job_expert[s.job];
    s.slot = r.job_slot[s.job];
    s.count = r.job_count[s.job];
    s.row0 = kDown ? s.expert * a.H + s.piece * 128 : s.expert * 2 * a.I + s.piece * kBlock;
    s.row1 = kDown ? s.row0 + 64 : s.row0 + a.I;
    return true;
  }
};

__device__ __forceinline__ void add(float4& a, const float4& b) { a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w; }

// FP32 value of an E4M3 code.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(d)));
}

// 64 columns of h of a slot, by a warp, two columns a lane: their terms and their scale, from the sums of
// the gate's rows and of the up's.
__device__ __forceinline__ void store_inner(const MoeArgs& a, float coef, int slot, int block, float2 gate, float2 up, int lane) {
  float h[2] = {coef * (gate.x / (1.0f + expf(-gate.x)) * up.x), coef * (gate.y / (1.0f + expf(-gate.y)) * up.y)};
  float top = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float m = fabsf(h[i]);
    top = m < INFINITY ? fmaxf(top, m) : top;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
  // the last term's scale is 2^-12 of the first's: its code stays at least 1
  const int e = max(dg::ue8m0_for_amax(top), 4 * kTerms - 3);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float full = h[i] * dg::ue8m0_inverse(e);
    h[i] = full - full == 0.0f ? full : NAN;        // an infinity (NaN - infinity) becomes NaN
  }
  uint8_t* to = a.h + static_cast<long long>(slot) * kTerms * a.I + block * kBlock + 2 * lane;
  uint16_t* code_to = reinterpret_cast<uint16_t*>(a.hs + (static_cast<long long>(block / 2) * a.T * a.k + slot) * kTerms) + block % 2;
#pragma unroll
  for (int j = 0; j < kTerms; ++j) {
    const uint32_t code = dg::pack_e4m3(h[0], h[1], 0, 0);
    *reinterpret_cast<uint16_t*>(to + static_cast<long long>(j) * a.I) = static_cast<uint16_t>(code);
    h[0] = (h[0] - e4m3_value(code & 255)) * 16.0f;
    h[1] = (h[1] - e4m3_value(code >> 8 & 255)) * 16.0f;
    if (lane == 0) code_to[2 * j] = static_cast<uint16_t>((e - 4 * j) * 0x0101);
  }
}

template <bool kFp4, bool kDown>
__global__ void __launch_bounds__(kThreads, 1) moe_kernel(const __grid_constant__ CUtensorMap map, const MoeArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ Shared s;
  uint8_t* const base = raw + ((1024u - (dg::smem_addr(raw) & 1023u)) & 1023u);
  const int lane = threadIdx.x & 31, half = threadIdx.x / kHalf, warp = threadIdx.x % kHalf / 32;
  Pipe& pipe = s.pipe[half];
  constexpr int kSumCols = kDown ? 32 : 16, kTmemCols = kDown ? 128 : 64;     // two sums, then two buffers of each side's scales
  if (threadIdx.x % kHalf == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      dg::mbar_init(&pipe.full[i], 1);
      dg::mbar_init(&pipe.ready[i], 33);
      dg::mbar_init(&pipe.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      dg::mbar_init(&pipe.sum_full[i], 1);
      dg::mbar_init(&pipe.sum_empty[i], 4);
    }
    dg::mbar_init(&pipe.drain, 1);
    dg::fence_mbarrier_init();
  }
  if (threadIdx.x == 0) {
    s.abort = 0;
    dg::tma_prefetch_desc(&map);
  }
  if (threadIdx.x / 32 == 1) {
    dg::tmem_alloc(&s.tmem, 2 * kTmemCols);
    dg::tmem_relinquish();
  }
  if (!kDown) {
    dg::grid_dependency_wait();
    dg::grid_launch_dependents();
  }
  // the halves' rings and their scales, then for each half the first kernel's sums of a unit, the second's output
  // [T][128]
  uint8_t* const ring = base + half * a.stages * a.stage_bytes;
  uint8_t* const scales = base + 2 * a.stages * a.stage_bytes + half * a.stages * a.scale_bytes;
  float* const rest = reinterpret_cast<float*>(base + 2 * a.stages * (a.stage_bytes + a.scale_bytes) + half * a.rest_bytes);
  if (kDown)
    for (int i = threadIdx.x % kHalf; i < a.T * 128; i += kHalf) rest[i] = 0;
  // (The first kernel let the second start only after its own wait: ids and weights are there, h is not yet.)
  build_routing<kThreads>(a, s.r, *reinterpret_cast<RoutingScratch*>(base), !kDown && blockIdx.x == 0);
  dg::fence_proxy_async_smem();        // written by threads, read and overwritten by copies and MMAs
  dg::tc_fence_before();
  __syncthreads();
  dg::tc_fence_after();

  const int groups = (kDown ? a.I : a.H) / 128;
  const uint32_t tmem = s.tmem + half * kTmemCols;
  const int me = blockIdx.x + half * gridDim.x;
  const int pieces = kDown ? a.H / 128 : s.r.jobs * (a.I / kBlock);
  const Deal deal(pieces, kDown ? s.r.jobs * groups : groups, 2 * static_cast<int>(gridDim.x));
  Walk<kDown> walk(a, s.r, deal, me);
  Run run;
  // A wait that runs out is recorded, and every role then leaves its loop (the epilogue runs through it without
  // waiting, since its warps meet at barriers).
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (dg::mbar_try_wait(dg::smem_addr(bar), parity)) return true;
    if (s.abort) return false;
    if (dg::mbar_wait(bar, parity, a.timeout_ns)) return true;
    atomicOr(a.status, dg::kTimeoutBit);
    s.abort = 1;
    return false;
  };

  if (warp == 0) {
    // ---------------------------------------------- the weights' copies
    if (lane == 0 && a.fault == 0) {
      int stage = 0, issued = 0;
      uint32_t phase = 1;
      bool ok = true;
      while (ok && walk.next(run)) {
        for (int g = run.begin; g < run.end; ++g) {
          if (!(ok = wait(&pipe.empty[stage], phase))) break;
          uint8_t* to = ring + stage * a.stage_bytes;
          uint64_t* bar = &pipe.full[stage];
          dg::mbar_arrive_expect_tx(bar, kFp4 ? kWeights / 2 + kTile : kWeights);
          dg::tma_load_2d(to, &map, bar, g * 128, run.row0);
          dg::tma_load_2d(to + kWeights / 2, &map, bar, g * 128, run.row1);
          if (kFp4) {
            // scale words [E, groups, N]
            const int n = kDown ? a.H : 2 * a.I;
            const int32_t* words = (kDown ? a.sf2 : a.sf13) + (static_cast<long long>(run.expert) * groups + g) * n - static_cast<long long>(run.expert) * n;
            uint8_t* raw_words = scales + stage * a.scale_bytes + kRaw;
            bulk_load(raw_words, words + run.row0, kTile / 2, bar);
            bulk_load(raw_words + kTile / 2, words + run.row1, kTile / 2, bar);
          }
          ++issued;
          if (++stage == a.stages) stage = 0, phase ^= 1;
        }
      }
      // no copy may be under way when the block ends
      for (int i = max(issued - a.stages, 0); i < issued; ++i)
        if (!dg::mbar_wait(&pipe.full[i % a.stages], i / a.stages & 1, a.timeout_ns)) break;
    }
  } else if (warp == 1) {
    // ---------------------------------------------- the MMAs. The whole warp runs the loop and one elected thread
    // issues: behind a branch on the lane, the seven instructions of a stage took 530 clocks to issue (the compiler
    // did not know the descriptors to be uniform), which bounded E2M1: 16 tokens, 174 us that way, 135 us this way.
    const uint64_t a_desc = dg::make_smem_desc(dg::smem_addr(ring), 16, 1024, dg::kLayoutSwizzle128B);
    const uint64_t b_desc = a_desc + (kWeights >> 4);
    const uint64_t sf_desc = dg::make_smem_desc(dg::smem_addr(scales), 0, 128, dg::kLayoutNone);
    int stage = 0;
    uint32_t phase = 0, n = 0, buffer = 0;
    bool ok = true;
    while (ok && walk.next(run)) {
      const uint32_t sum = n & 1, d = tmem + sum * kSumCols;
      if (!(ok = __all_sync(kAll, wait(&pipe.sum_empty[sum], (n >> 1 & 1) ^ 1)))) break;
      dg::tc_fence_after();
      // rows past the last of the tokens' hold anything: they are columns of the sums that nobody reads
      const uint32_t cols = kDown && kTerms * run.count > 16 ? 32 : 16;
      const uint32_t idesc = dg::make_idesc_mxf8_e4m3(128, 0) | (cols >> 3) << 17 | (kFp4 ? 5u << 7 : 0u);
      for (int g = run.begin; g < run.end; ++g) {
        if (!(ok = __all_sync(kAll, wait(&pipe.full[stage], phase) && wait(&pipe.ready[stage], phase)))) break;
        dg::fence_proxy_async_smem();       // of what the barriers say has arrived by cp.async
        dg::tc_fence_after();
        const uint64_t off = static_cast<uint64_t>(stage * a.stage_bytes) >> 4, sf_off = static_cast<uint64_t>(stage * a.scale_bytes) >> 4;
        const uint32_t sfa = tmem + 2 * kSumCols + 4 * buffer, sfb = sfa + 8;
        buffer ^= 1;
        if (dg::elect_one()) {
          dg::tmem_copy_32x128b_warpx4(sfa, sf_desc + sf_off + (kTileA >> 4));
          dg::tmem_copy_32x128b_warpx4(sfb, sf_desc + sf_off + (kTileB >> 4));
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // bytes of the scale words: the four 32-column blocks of E2M1 rows and of h, or the K group of four
            const uint32_t id = dg::idesc_with_sf_id(idesc, kFp4 ? k : g & 3, kDown ? k : g & 3);
            dg::mma_mxf8_block_scale(d, a_desc + off + 2 * k, b_desc + off + 2 * k, id, sfa, sfb, g != run.begin || k != 0);
          }
          dg::tc_commit(&pipe.empty[stage]);
          if (g + 1 == run.end) dg::tc_commit(&pipe.sum_full[sum]);
        }
        __syncwarp();
        if (++stage == a.stages) stage = 0, phase ^= 1;
      }
      ++n;
    }
    // all that was issued has to be done before TMEM is given back
    if (dg::elect_one()) dg::tc_commit(&pipe.drain);
    dg::mbar_wait(&pipe.drain, 0, a.timeout_ns);
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------- the tokens' side: rows and scale words
    if (kDown) {
      dg::grid_dependency_wait();
      dg::grid_launch_dependents();
    }
    int stage = 0;
    uint32_t phase = 1;
    bool ok = true;
    const int t4 = (a.T + 3) / 4 * 4;
    while (ok && walk.next(run)) {
      const int rows = kDown ? kTerms * run.count : run.count;
      for (int g = run.begin; g < run.end; ++g) {
        ok = __all_sync(kAll, wait(&pipe.empty[stage], phase));
        if (!ok) break;
        const uint32_t to = dg::smem_addr(ring) + stage * a.stage_bytes + kWeights;
        for (int i = lane; i < rows * 8; i += 32) {
          const int row = i / 8, c = i & 7;
          const uint8_t* from = kDown ? a.h + static_cast<long long>(run.slot * kTerms + row) * a.I : a.x + static_cast<long long>(s.r.token[run.slot + row]) * a.H;
          dg::cp_async_16(to + row * 128 + ((c ^ (row & 7)) << 4), from + g * 128 + c * 16);
        }
        if (lane < rows)
          cp_async_4(dg::smem_addr(scales) + stage * a.scale_bytes + kTileB + lane * 16,
                     kDown ? reinterpret_cast<const int32_t*>(a.hs) + (static_cast<long long>(g) * a.T * a.k + run.slot) * kTerms + lane
                           : a.sfx + g / 4 * t4 + s.r.token[run.slot + lane]);
        cp_async_arrive(&pipe.ready[stage]);
        if (++stage == a.stages) stage = 0, phase ^= 1;
      }
    }
    cp_async_wait_all();
  } else if (warp == 3) {
    // ---------------------------------------------- the weights' scales to the form of tcgen05.cp
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    // E4M3: packed word `lane` of the boxes' 128-row blocks, loaded a run ahead
    Walk<kDown> ahead = walk;
    Run next_run;
    uint32_t next0 = 0, next1 = 0;
    auto load_words = [&] {
      if (!ahead.next(next_run)) return;
      const int n = kDown ? a.H : 2 * a.I, n4 = (n / 128 + 3) / 4 * 4, words = (groups + 3) / 4;
      const int32_t* sf = (kDown ? a.sf2 : a.sf13) + (static_cast<long long>(next_run.expert) * words + lane) * n4;
      if (lane < words) {
        next0 = dg::ld_cg_s32(sf + (next_run.row0 - next_run.expert * n) / 128);
        next1 = dg::ld_cg_s32(sf + (next_run.row1 - next_run.expert * n) / 128);
      }
    };
    if (!kFp4) load_words();
    while (ok && walk.next(run)) {
      const uint32_t word0 = next0, word1 = next1;
      if (!kFp4) load_words();
      for (int g = run.begin; g < run.end; ++g) {
        // E2M1's words come with the weights; E4M3's are here, and wait only for the stage to be free
        ok = __all_sync(kAll, kFp4 ? wait(&pipe.full[stage], phase) : wait(&pipe.empty[stage], phase ^ 1));
        if (!ok) break;
        const uint32_t area = dg::smem_addr(scales) + stage * a.scale_bytes;
        uint32_t w[4];
        if (kFp4) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = dg::ld_shared_u32(area + kRaw + 4 * (lane + 32 * j));
        } else {
          w[0] = w[1] = __shfl_sync(kAll, word0, g / 4);
          w[2] = w[3] = __shfl_sync(kAll, word1, g / 4);
        }
        dg::st_shared_v4(area + kTileA + 16 * lane, w[0], w[1], w[2], w[3]);
        dg::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) dg::mbar_arrive(&pipe.ready[stage]);
        if (++stage == a.stages) stage = 0, phase ^= 1;
      }
    }
  } else {
    // ---------------------------------------------- the sums: warps 4 to 7, a row of 128 per thread
    const int quad = warp - 4, row = quad * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    uint32_t n = 0;
    // Parts and counts are the first kernel's until it has ended, and the waits below do not keep to that when they run out.
    if (kDown) dg::grid_dependency_wait();
    while (walk.next(run)) {
      const uint32_t sum = n & 1, from = tmem + lanes + sum * kSumCols;
      wait(&pipe.sum_full[sum], n >> 1 & 1);
      __syncwarp();
      dg::tc_fence_after();
      auto release = [&] {
        dg::tc_fence_before();
        __syncwarp();
        if (lane == 0) dg::mbar_arrive(&pipe.sum_empty[sum]);
        ++n;
      };
      // a piece that other pipelines have parts of: 1 if this one is the last to bring its own
      auto last_of = [&](int piece_begin, int per, int* first, int* last) {
        *first = deal.owner(piece_begin);
        *last = deal.owner(piece_begin + per - 1);
        named_barrier(1 + 2 * half, 128);
        if (warp == 4 && lane == 0) {
          // the fences stand between the barriers and the count, in the thread that counts: the first then covers what
          // all 128 threads wrote, the second what they read next
          __threadfence();
          const int before = atomicAdd(a.arrivals + *first, 1);
          __threadfence();
          s.arrived[half] = before == *last - *first;
          if (before == *last - *first) a.arrivals[*first] = 0;
        }
        named_barrier(1 + 2 * half, 128);
        return s.arrived[half] != 0;
      };
      // where pipeline p put its part of the piece: a piece that it did not begin is its first
      auto part_of = [&](int p, int piece_begin) {
        return a.parts + (2ll * p + (deal.begin(p) > piece_begin ? 0 : 1)) * (128 * (kDown ? a.T : kCols));
      };
      if constexpr (kDown) {
        // this row of the job's tokens, the sum of four terms each: no other thread has it
        float* const out = rest;
        uint32_t v[kTerms * kDownCols];
        dg::tmem_load_32x32b_x32(from, v);
        dg::tmem_load_wait();
#pragma unroll
        for (int i = 0; i < kDownCols; ++i)
          if (i < run.count)
            out[s.r.token[run.slot + i] * 128 + row] +=
                (__uint_as_float(v[4 * i]) + __uint_as_float(v[4 * i + 1])) + (__uint_as_float(v[4 * i + 2]) + __uint_as_float(v[4 * i + 3]));
        release();
        if (!run.done) continue;
        const int per = s.r.jobs * groups;
        const int begin = run.piece * per;
        const bool whole = deal.begin(me) <= begin && deal.begin(me + 1) >= begin + per;
        int first = me, last = me;
        bool write = true;
        if (!whole) {
          float* mine = part_of(me, begin);
#pragma unroll 1
          for (int t = 0; t < a.T; ++t) mine[t * 128 + row] = out[t * 128 + row];
          write = last_of(begin, per, &first, &last);
        }
        if (whole || write) {
          // four columns of a token each: a warp a token, and as many of its parts at once as the registers hold
          if (whole) named_barrier(1 + 2 * half, 128);
          for (int t = quad; t < a.T; t += 4) {
            const long long to = static_cast<long long>(t) * a.H + run.piece * 128 + 4 * lane;
            float4 total = make_float4(0, 0, 0, 0);
            if (a.c) {
              const uint2 c = __ldcg(reinterpret_cast<const uint2*>(a.c + to));
              dg::unpack_bf16(c.x, total.x, total.y);
              dg::unpack_bf16(c.y, total.z, total.w);
            }
            if (whole) add(total, *reinterpret_cast<const float4*>(out + t * 128 + 4 * lane));
            else
              for (int p = first; p <= last; p += 16) {
                float4 part[16];
#pragma unroll
                for (int i = 0; i < 16; ++i)
                  part[i] = p + i <= last ? __ldcg(reinterpret_cast<const float4*>(part_of(p + i, begin) + t * 128) + lane) : make_float4(0, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i) add(total, part[i]);
              }
            *reinterpret_cast<uint2*>(a.y + to) = make_uint2(dg::pack_bf16(total.x, total.y), dg::pack_bf16(total.z, total.w));
          }
          if (whole) named_barrier(1 + 2 * half, 128);
        }
#pragma unroll 4
        for (int t = 0; t < a.T; ++t) out[t * 128 + row] = 0;
      } else {
        // sums as [token][row]; rows 0 to 63 are the gate's, 64 to 127 the up's of the same columns of h. The loop
        // over the tokens is a loop in the code too: it runs once or twice per launch, and unrolled over 16 tokens
        // its instructions took 15 us to arrive from memory
        uint32_t v[kCols];
        dg::tmem_load_32x32b_x16(from, v);
        dg::tmem_load_wait();
        release();
        const bool whole = run.end - run.begin == groups;
        const int begin = run.unit * groups;
        float* mine = whole ? rest : part_of(me, begin);
#pragma unroll
        for (int i = 0; i < kCols; ++i)
          if (i < run.count) mine[i * 128 + row] = __uint_as_float(v[i]);
        int first = me, last = me;
        if (whole) named_barrier(1 + 2 * half, 128);
        else if (!last_of(begin, groups, &first, &last)) continue;
#pragma unroll 1
        for (int i = quad; i < run.count; i += 4) {
          float2 gate = make_float2(0, 0), up = make_float2(0, 0);
          if (whole) {
            gate = *reinterpret_cast<const float2*>(rest + i * 128 + 2 * lane);
            up = *reinterpret_cast<const float2*>(rest + i * 128 + 64 + 2 * lane);
          } else {
#pragma unroll 1
            for (int p = first; p <= last; p += 4) {
              float2 part[4][2];
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                  part[j][n] = p + j <= last ? __ldcg(reinterpret_cast<const float2*>(part_of(p + j, begin) + i * 128 + n * 64) + lane) : make_float2(0, 0);
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                gate.x += part[j][0].x, gate.y += part[j][0].y;
                up.x += part[j][1].x, up.y += part[j][1].y;
              }
            }
          }
          store_inner(a, s.r.coef[run.slot + i], run.slot + i, run.piece, gate, up, lane);
        }
        if (whole) named_barrier(1 + 2 * half, 128);
      }
    }
    if (kDown && s.r.jobs == 0) {
      // no expert at all: the addend alone
      for (int i = me * 128 + row; i < a.T * a.H; i += 2 * gridDim.x * 128)
        a.y[i] = a.c ? a.c[i] : __float2bfloat16_rn(0.0f);
    }
  }

  __syncwarp();
  __syncthreads();
  if (threadIdx.x / 32 == 1) dg::tmem_dealloc(s.tmem, 2 * kTmemCols);
}

// -------------------------------------------------------------------------------------------

template <bool kFp4>
dg_status run_layer(MoeArgs a, const void* w13, const void* w2, const LaunchContext& ctx, cudaStream_t stream) {
  // once per thread and device: the limit, above what any shape needs
  static thread_local int ready = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && ready != dev) {
    e = cudaFuncSetAttribute(moe_kernel<kFp4, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_kernel<kFp4, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return dg::record_cuda_error(e);
  // Tokens of a job: 16 are the least columns of an MMA. In the second product each is four rows, 32 at most.
  MoeArgs up = a, down = a;
  up.cols = kCols;
  down.cols = kDownCols;
  CUtensorMap up_map, down_map;
  if (!dg::weight_rows_map(&up_map, w13, static_cast<uint64_t>(a.E) * 2 * a.I, a.H, 64, kFp4) ||
      !dg::weight_rows_map(&down_map, w2, static_cast<uint64_t>(a.E) * a.H, a.I, 64, kFp4))
    return DG_ERR_CUDA;
  // as many blocks as there are SMs, or shares of the stages of the jobs there are at most
  auto grid = [&](const MoeArgs& m, long long stages_of_a_job) {
    const int jobs = std::min(a.T * a.k, a.E + (a.T * a.k + m.cols - 1) / m.cols);
    return static_cast<unsigned>(std::max(1ll, std::min<long long>(ctx.sms, (jobs * stages_of_a_job + kMinShare - 1) / kMinShare)));
  };
  auto shared_bytes = [&](MoeArgs& m, int rows, int rest) {
    m.stage_bytes = kWeights + (rows + 7) / 8 * 1024;
    m.scale_bytes = kTile * (kFp4 ? 3 : 2);
    m.rest_bytes = rest;
    m.stages = std::min(kMaxStages, (kMaxSmem - 1024 - 2 * rest) / (2 * (m.stage_bytes + m.scale_bytes)));
    return static_cast<size_t>(1024 + 2 * (m.stages * (m.stage_bytes + m.scale_bytes) + rest));
  };
  const int up_rows = std::min(a.T, kCols);
  const size_t up_smem = shared_bytes(up, up_rows, up_rows * 128 * 4);
  const size_t down_smem = shared_bytes(down, kTerms * std::min(a.T, down.cols), a.T * 128 * 4);
  if (dg_status s = dg::launch(moe_kernel<kFp4, false>, grid(up, static_cast<long long>(a.I / kBlock) * (a.H / 128)), kThreads, up_smem, stream, ctx.pdl,
                               up_map, up); s != DG_OK) return s;
  return dg::launch(moe_kernel<kFp4, true>, grid(down, static_cast<long long>(a.H / 128) * (a.I / 128)), kThreads, down_smem, stream, ctx.pdl, down_map, down);
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
  if (kFp4 && (!aligned(w13, 32) || !aligned(w2, 32))) return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const size_t slots = static_cast<size_t>(T) * topk, scale_words = (slots * (I / 128) * kTerms + 3) / 4 * 4;
  const size_t part_floats = 2ull * 2 * ctx.sms * 128 * std::max(T, kCols), h_bytes = (slots * kTerms * I + 15) / 16 * 16;
  dg::StreamWorkspace ws;
  void* scratch = nullptr;
  if (dg_status s = ws.acquire(stream, scale_words * 4 + h_bytes + part_floats * 4, &scratch); s != DG_OK) return s;
  MoeArgs a{};
  a.x = static_cast<const uint8_t*>(x), a.sfx = sfx, a.sf13 = sf13, a.sf2 = sf2, a.ids = ids, a.weights = weights;
  a.c = static_cast<const __nv_bfloat16*>(c), a.y = static_cast<__nv_bfloat16*>(y);
  a.hs = static_cast<uint32_t*>(scratch), a.h = static_cast<uint8_t*>(scratch) + scale_words * 4;
  a.parts = reinterpret_cast<float*>(a.h + h_bytes), a.arrivals = ws.counters();
  a.status = ctx.status, a.timeout_ns = dg::pipeline_wait_timeout_ns(), a.fault = dg::debug_fault_mode();
  a.T = T, a.k = topk, a.E = E, a.H = H, a.I = I;
  return run_layer<kFp4>(a, w13, w2, ctx, stream);
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
