// A whole mixture-of-experts layer for a few tokens (at most 32), in two kernels:
//
//   y[t] = c[t] + sum over the slots j of token t with an expert e = ids[t, j]:
//              weights[t, j] * W2_e (silu(G_e x_t) * (U_e x_t)),      (G_e; U_e) = W13_e
//
// x is E4M3 with one UE8M0 scale per 128 columns; the experts' weights are E4M3 with one scale per
// 128 x 128 block, or E2M1 with one per row per 32 columns: the grouped GEMMs' operands.
//
// At a few tokens an expert has one to a handful of rows, so the time is that of reading the weights
// of the experts in use, once. Both kernels stream them: every warp has a ring of its own in shared
// memory that it fills with asynchronous copies, so that no warp waits for another between copies.
// A warp multiplies 16 weight rows (or 32) by up to 8 tokens (or 16) with m16n8 MMAs: the weights are
// the M operand, an expert's tokens the N columns. The first product's operands are both E4M3 (E2M1 is
// one with two exponent bits, moved into place), the second's FP16, which holds E4M3 and E2M1 exactly.
// Accumulation is FP32, and the scales are applied to FP32 partial sums.
//
// An expert's tokens are compacted into jobs of at most 8 (16) columns; each distinct (expert, token)
// pair is a slot. The first kernel writes h = weight * silu(g) * u of every slot to the workspace, in
// FP16 with one power-of-two scale per 64 or 128 columns (11 bits of every value within 2^-29 of the
// largest; plain FP32 would double what the second kernel reads). The second kernel owns output rows: a
// block sums all experts for its 16 (32) rows of W2 and every token, in an order that depends on the
// sizes alone, and writes each output once. No atomics on values.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
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

constexpr int kMaxTokens = 32;          // a token is a bit of an expert's mask
constexpr int kMaxTopk = 16;
constexpr int kMaxExperts = 1024;
constexpr int kMaxH = 16384;
constexpr int kMaxSlots = kMaxTokens * kMaxTopk;
constexpr int kUpWarps = 8;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr int kHBytes = 272;            // 128 columns of h of a slot: 256 bytes of FP16, FP32 scales of both halves, padding
constexpr int kMaxSmem = 216 * 1024;

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
  int warp_sum[16];
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
  constexpr int kPer = kMaxExperts / kThreads;
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
// A warp's piece of the weights: 16 kM rows x 128 columns
// -------------------------------------------------------------------------------------------

__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

__device__ __forceinline__ uint32_t half2_of_e2m1(uint32_t two) {
  uint32_t d;
  asm("{ .reg .b8 b; cvt.u8.u32 b, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(d) : "r"(two));
  return d;
}

// Four E2M1 codes as E4M3 of 2^-6 of their values: the sign to bit 7, the two exponent bits and the
// mantissa bit to the lowest exponent bits and the highest mantissa bit (E2M1's subnormal 0.5 becomes
// the subnormal 2^-7). Even elements of eight are the low nibbles, odd ones the high nibbles.
__device__ __forceinline__ uint32_t e4m3_of_even(uint32_t w) { return (w << 4 & 0x80808080u) | (w << 2 & 0x1C1C1C1Cu); }
__device__ __forceinline__ uint32_t e4m3_of_odd(uint32_t w) { return (w & 0x80808080u) | (w >> 2 & 0x1C1C1C1Cu); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t p) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(p));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t p) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(p));
  return v;
}
__device__ __forceinline__ uint2 ld_cg_v2(const void* p) {
  uint2 v;
  asm volatile("ld.global.cg.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ float float_of(const uint4& v, int i) { return __uint_as_float(word_of(v, i)); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// The K order of a product is free. Within 128 columns, lane 4 g + q (g the row or column of the MMA
// fragment) takes, in the E4M3 form, columns 64 p + 16 q .. + 15 of half p: one 128-bit load of a row holds
// its fragments of two (four) MMAs. In the E2M1 form it takes columns 32 b + 8 q .. + 7 of block b: the
// columns of an MMA then share a scale.
//
// Rings hold 128-byte rows of E4M3 and 64-byte rows of E2M1, in 16-byte chunks that are permuted so that
// the lanes of one shared load cover every bank once: two rows of four chunks (128-bit loads of E4M3),
// eight rows of one (32-bit loads of E2M1), four rows of two (64-bit loads of the E2M1 form's tokens).
__device__ __forceinline__ int chunk_e4m3(int row, int c) { return row * 128 + ((c ^ ((row & 1) << 2)) << 4); }
__device__ __forceinline__ int chunk_e2m1(int row, int c) { return row * 64 + ((c ^ ((row >> 1) & 3)) << 4); }
__device__ __forceinline__ int chunk_pair(int row, int c) { return row * 128 + ((c ^ ((row & 3) << 1)) << 4); }

template <bool kFp4, int kM>
struct Piece {
  static constexpr int kRowBytes = kFp4 ? 64 : 128;
  static constexpr int kBytes = 16 * kM * kRowBytes;
  static constexpr int kCopyRows = 512 / kRowBytes;         // rows of one copy by a whole warp, 16 bytes a lane
  static constexpr int kCopies = 16 * kM / kCopyRows;
  // E4M3: a packed word of one 128-row block (with its neighbours); E2M1: one per row
  static constexpr int kScaleBytes = kFp4 ? 64 * kM : 16;

  static __device__ __forceinline__ int chunk(int row, int c) { return kFp4 ? chunk_e2m1(row, c) : chunk_e4m3(row, c); }
  // this lane's row (of the first copy), first byte of it and place in a stage; copy i is kCopyRows rows further
  static __device__ __forceinline__ int row(int lane) { return lane / (kRowBytes / 16); }
  static __device__ __forceinline__ int column(int lane) { return lane % (kRowBytes / 16) * 16; }
  static __device__ __forceinline__ int place(int lane) { return chunk(row(lane), lane % (kRowBytes / 16)); }

  // E2M1: the stage's scales (4 of every row) as FP32, times `by`, at `to` [16 kM][4]. Ends with the warp's
  // writes visible.
  static __device__ __forceinline__ void expand_scales(uint32_t scales, float* to, int lane, float by) {
    if constexpr (kM == 1) {
      const uint32_t w = lds32(scales + lane / 2 * 4) >> (lane & 1) * 16;
      reinterpret_cast<float2*>(to)[lane] = make_float2(dg::ue8m0_value(w & 255) * by, dg::ue8m0_value(w >> 8 & 255) * by);
    } else {
      const uint32_t w = lds32(scales + lane * 4);
      reinterpret_cast<float4*>(to)[lane] = make_float4(dg::ue8m0_value(w & 255) * by, dg::ue8m0_value(w >> 8 & 255) * by,
                                                        dg::ue8m0_value(w >> 16 & 255) * by, dg::ue8m0_value(w >> 24) * by);
    }
    __syncwarp();
  }
};
static_assert(Piece<true, 1>::kCopyRows == 8 && Piece<false, 1>::kCopyRows == 4, "the permutations repeat every 2 and 8 rows");

// Shapes. kBig (more than 8 tokens): experts then have several tokens, and reading the tokens' side again
// for every 16 weight rows would cost as much as the weights; a warp's pieces have 32 rows and 16 columns.
template <bool kFp4, bool kBig>
struct Up {
  static constexpr int kM = kBig ? 2 : 1, kCols = kBig ? 16 : 8;
  static constexpr int kBlock = 8 * kM * kUpWarps;          // columns of h of a block
  static constexpr int kStages = kBig ? (kFp4 ? 5 : 4) : (kFp4 ? 5 : 4);
  static constexpr int kBlocksPerSm = kBig ? 1 : 2;
  using P = Piece<kFp4, kM>;
  static constexpr int kStage = P::kBytes + (kFp4 ? P::kScaleBytes : 0) + kCols * 128;
  static constexpr int kRing = kUpWarps * kStages * kStage;
  static constexpr int kExpanded = kFp4 ? kUpWarps * 256 * kM : 0;   // E2M1: the piece's scales as FP32, per warp
  // then the tokens' scales [groups, T], and for E4M3 each warp's two scales of every group
  static int smem(int groups, int T) { return kRing + kExpanded + (groups * T + 1) / 2 * 8 + (kFp4 ? 0 : kUpWarps * groups * 8); }
};
template <bool kFp4, bool kBig>
struct Down {
  static constexpr int kM = kBig ? 2 : 1, kCols = kBig ? 16 : 8;
  static constexpr int kRows = 16 * kM;
  static constexpr int kWarps = kBig ? 8 : 16;
  static constexpr int kStages = kFp4 ? 5 : 4;
  using P = Piece<kFp4, kM>;
  static constexpr int kStage = P::kBytes + P::kScaleBytes;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kExpanded = kFp4 ? kWarps * 256 * kM : 0;
  // then every warp's sums of a tile, twice: [2][warps][T][kRows]
  static int smem(int T) { return kRing + kExpanded + 2 * kWarps * T * kRows * 4; }
};

// -------------------------------------------------------------------------------------------
// First kernel: h = weight * silu(G x) * (U x)
// -------------------------------------------------------------------------------------------

template <bool kFp4, bool kBig>
__global__ void __launch_bounds__(32 * kUpWarps, Up<kFp4, kBig>::kBlocksPerSm) moe_up_kernel(const MoeArgs a) {
  using C = Up<kFp4, kBig>;
  using P = typename C::P;
  constexpr int kM = C::kM, NT = C::kCols / 8, kStages = C::kStages;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Routing r;
  __shared__ float block_max[2][kUpWarps][C::kCols];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3;
  const int t4 = (a.T + 3) / 4 * 4;
  const int groups = a.H / 128, blocks = a.I / C::kBlock;
  build_routing<C::kCols, 32 * kUpWarps>(a, r, *reinterpret_cast<RoutingScratch*>(dyn), blockIdx.x == 0);
  float* expanded = reinterpret_cast<float*>(dyn + C::kRing) + warp * 64 * kM;
  float* sx = reinterpret_cast<float*>(dyn + C::kRing + C::kExpanded);
  float2* sw = reinterpret_cast<float2*>(sx + (groups * a.T + 1) / 2 * 2) + warp * groups;
  for (int i = threadIdx.x; i < (groups + 3) / 4 * a.T; i += 32 * kUpWarps) {
    const int w = i / a.T, t = i % a.T;
    const uint32_t v = dg::ld_cg_s32(a.sfx + w * t4 + t);
    for (int b = 0; b < 4 && 4 * w + b < groups; ++b) sx[(4 * w + b) * a.T + t] = dg::ue8m0_value(v >> (8 * b) & 255);
  }
  __syncthreads();

  const int units = r.jobs * blocks;
  const uint32_t ring = dg::smem_addr(dyn) + warp * kStages * C::kStage;
  constexpr int kTokens = P::kBytes + (kFp4 ? P::kScaleBytes : 0);  // where a stage's tokens begin
  const long long row_bytes = kFp4 ? a.H / 2 : a.H;
  const int n4 = kFp4 ? 2 * a.I : (a.I / 64 + 3) / 4 * 4;           // words of a scale row (2 I is a multiple of 4)
  // the copies run kStages - 1 pieces ahead of the products, over the block's units one after another
  int fu = blockIdx.x, fg = 0, fcount = 0;
  uint32_t fto = ring;
  const uint8_t* gate_from = nullptr;
  const uint8_t* up_from = nullptr;
  const int32_t* scale_from = nullptr;
  const uint8_t* x_from[2 * NT];                                    // columns lane / 8 + 4 i of the job
  uint32_t next_gate = 0, next_up = 0;                              // E4M3: packed scale word `lane` of the unit
  auto load_scales = [&](int u) {
    const int e = r.job_expert[u / blocks], i0 = u % blocks * C::kBlock;
    if (lane < (groups + 3) / 4) {
      const int32_t* sf = a.sf13 + (static_cast<long long>(e) * ((groups + 3) / 4) + lane) * n4;
      next_gate = dg::ld_cg_s32(sf + i0 / 128);
      next_up = dg::ld_cg_s32(sf + (a.I + i0) / 128);
    }
  };
  auto fetch = [&] {
    if (fu < units) {
      if (fg == 0) {
        const int job = fu / blocks, e = r.job_expert[job], i0 = fu % blocks * C::kBlock + warp * 8 * kM;
        gate_from = a.w13 + (static_cast<long long>(e) * 2 * a.I + i0 + P::row(lane)) * row_bytes + P::column(lane);
        up_from = gate_from + a.I * row_bytes;
        fcount = r.job_count[job];
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) {
          const int col = lane / 8 + 4 * i;
          x_from[i] = col < fcount ? a.x + static_cast<long long>(r.token[r.job_slot[job] + col]) * a.H + (lane & 7) * 16 : nullptr;
        }
        if (kFp4) {
          const int part = lane & 3;
          scale_from = a.sf13 + static_cast<long long>(e) * groups * n4 + i0 + lane / 4 * 8 + (part < 2 ? 4 * part : a.I + 4 * part - 8);
        } else if (groups >= kStages - 1) {
          load_scales(fu);
        }
      }
      const uint32_t to = fto + P::place(lane);
      constexpr int kHalf = 8 / P::kCopyRows;                       // copies of a tile's 8 gate rows, then as many of its up rows
#pragma unroll
      for (int i = 0; i < P::kCopies; ++i) {
        const int rows = i / (2 * kHalf) * 8 + i % kHalf * P::kCopyRows;
        dg::cp_async_16(to + i * 512, (i / kHalf % 2 ? up_from : gate_from) + rows * row_bytes);
      }
      gate_from += P::kRowBytes;
      up_from += P::kRowBytes;
      if (kFp4) {
        if (lane < 4 * kM) dg::cp_async_16(fto + P::kBytes + 16 * lane, scale_from);
        scale_from += n4;
      }
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i)
        if (x_from[i]) {
          const int col = lane / 8 + 4 * i, c = lane & 7;
          dg::cp_async_16(fto + kTokens + (kFp4 ? chunk_pair(col, c) : chunk_e4m3(col, c)), x_from[i]);
          x_from[i] += 128;
        }
      if (++fg == groups) fg = 0, fu += gridDim.x;
    }
    fto = fto + C::kStage == ring + kStages * C::kStage ? ring : fto + C::kStage;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  int flip = 0;
  uint32_t at = ring;
  for (int u = blockIdx.x; u < units; u += gridDim.x, flip ^= 1) {
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
      // the unit's scales as FP32, read while the unit before was computed (unless the copies, kStages - 1
      // pieces ahead, are then past the next unit's start)
      if (groups < kStages - 1) load_scales(u);
      __syncwarp();
      if (lane < (groups + 3) / 4)
        for (int b = 0; b < 4 && 4 * lane + b < groups; ++b)
          sw[4 * lane + b] = make_float2(dg::ue8m0_value(next_gate >> (8 * b) & 255), dg::ue8m0_value(next_up >> (8 * b) & 255));
      __syncwarp();
    }
    for (int g = 0; g < groups; ++g) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      fetch();
      const uint32_t tokens = at + kTokens;
      float acc[kM][NT][4];
#pragma unroll
      for (int m = 0; m < kM; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0;
      if constexpr (!kFp4) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint4 x[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n == 0 || n * 8 < count) x[n] = lds128(tokens + chunk_e4m3(8 * n + g8, 4 * p + q4));
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const uint4 w0 = lds128(at + P::chunk(16 * m + g8, 4 * p + q4)), w1 = lds128(at + P::chunk(16 * m + 8 + g8, 4 * p + q4));
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n == 0 || n * 8 < count) {
                mma_e4m3(acc[m][n], w0.x, w1.x, w0.y, w1.y, x[n].x, x[n].y);
                mma_e4m3(acc[m][n], w0.z, w1.z, w0.w, w1.w, x[n].z, x[n].w);
              }
          }
        }
        const float2 s = sw[g];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = sxt[n][i][g * a.T], tx = t * s.x, ty = t * s.y;
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              sum[m][n][i] = fmaf(tx, acc[m][n][i], sum[m][n][i]);
              sum[m][n][2 + i] = fmaf(ty, acc[m][n][2 + i], sum[m][n][2 + i]);
            }
          }
      } else {
        P::expand_scales(at + P::kBytes, expanded, lane, 64.0f);    // E2M1 enters the MMAs as 2^-6 of itself
        uint4 scale[kM][2];
#pragma unroll
        for (int m = 0; m < kM; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) scale[m][i] = reinterpret_cast<const uint4*>(expanded)[16 * m + 8 * i + g8];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          uint32_t even[NT], odd[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (n == 0 || n * 8 < count) {
              const uint2 x = lds64(tokens + chunk_pair(8 * n + g8, 2 * b + q4 / 2) + 8 * (q4 & 1));
              even[n] = __byte_perm(x.x, x.y, 0x6420), odd[n] = __byte_perm(x.x, x.y, 0x7531);
            }
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const uint32_t u0 = lds32(at + P::chunk(16 * m + g8, b) + 4 * q4), u1 = lds32(at + P::chunk(16 * m + 8 + g8, b) + 4 * q4);
            const uint32_t a0 = e4m3_of_even(u0), a1 = e4m3_of_even(u1), a2 = e4m3_of_odd(u0), a3 = e4m3_of_odd(u1);
            const float e0 = float_of(scale[m][0], b), e1 = float_of(scale[m][1], b);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              if (n == 0 || n * 8 < count) {
                float part[4] = {0, 0, 0, 0};
                mma_e4m3(part, a0, a1, a2, a3, even[n], odd[n]);
                acc[m][n][0] = fmaf(e0, part[0], acc[m][n][0]);
                acc[m][n][1] = fmaf(e0, part[1], acc[m][n][1]);
                acc[m][n][2] = fmaf(e1, part[2], acc[m][n][2]);
                acc[m][n][3] = fmaf(e1, part[3], acc[m][n][3]);
              }
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = sxt[n][i][g * a.T];
#pragma unroll
            for (int m = 0; m < kM; ++m) {
              sum[m][n][i] = fmaf(t, acc[m][n][i], sum[m][n][i]);
              sum[m][n][2 + i] = fmaf(t, acc[m][n][2 + i], sum[m][n][2 + i]);
            }
          }
      }
      at = at + C::kStage == ring + kStages * C::kStage ? ring : at + C::kStage;
    }
    // column blk * kBlock + (warp * kM + m) * 8 + g8 of h for tokens 2 q4, 2 q4 + 1 of each eight: gate in
    // sum[0..1], up in sum[2..3]
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
          const float gate = sum[m][n][i];
          hv[m][n][i] = col < count ? w * (gate / (1.0f + expf(-gate)) * sum[m][n][2 + i]) : 0.0f;
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
        for (int w = 0; w < kUpWarps; ++w) top = fmaxf(top, block_max[flip][w][col]);
        // the largest to [2^14, 2^15); both powers stay normal
        const int ex = min(max(static_cast<int>(__float_as_uint(top) >> 23), 27), 254) - 127 - 14;
        const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23), down = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
        uint8_t* row = a.h + (static_cast<long long>(slot + col) * (a.I / 128) + blk * C::kBlock / 128) * kHBytes;
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          // where the second kernel's lanes find this column of the 128: E4M3 as 16-byte pieces of two loads,
          // each of 64 bytes over four lanes; E2M1 in order
          const int cc = blk * C::kBlock % 128 + (warp * kM + m) * 8 + g8;
          const int place = kFp4 ? cc * 2 : cc / 64 * 128 + cc % 16 / 8 * 64 + cc % 64 / 16 * 16 + cc % 8 * 2;
          *reinterpret_cast<__half*>(row + place) = __float2half_rn(hv[m][n][i] * up);
        }
        if (warp == 0 && g8 == 0) {
          float* to = reinterpret_cast<float*>(row + 256);
          if (kM == 2) to[0] = to[1] = down;
          else to[blk & 1] = down;
        }
      }
  }
  cp_async_wait<0>();
}

// -------------------------------------------------------------------------------------------
// Second kernel: y = c + W2 h
// -------------------------------------------------------------------------------------------

template <bool kFp4, bool kBig>
__global__ void __launch_bounds__(32 * Down<kFp4, kBig>::kWarps, 1) moe_down_kernel(const MoeArgs a) {
  using C = Down<kFp4, kBig>;
  using P = typename C::P;
  constexpr int kM = C::kM, NT = C::kCols / 8, kStages = C::kStages, kWarps = C::kWarps;
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Routing r;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3;
  // The first kernel let this one start only after its own wait: ids and weights are there, h is not yet.
  build_routing<C::kCols, 32 * kWarps>(a, r, *reinterpret_cast<RoutingScratch*>(dyn), false);

  const int groups = a.I / 128, items = r.jobs * groups, tiles = a.H / C::kRows;
  const uint32_t row_bytes = kFp4 ? a.I / 2 : a.I;
  const int n4 = kFp4 ? a.H : (a.H / 128 + 3) / 4 * 4;
  const uint32_t ring = dg::smem_addr(dyn) + warp * kStages * C::kStage;
  float* expanded = reinterpret_cast<float*>(dyn + C::kRing) + warp * 64 * kM;
  // every warp's sums of a tile, [2][warps][T][kRows]: the tile before is being added up meanwhile
  float* sums = reinterpret_cast<float*>(dyn + C::kRing + C::kExpanded);
  const int tile_sums = kWarps * a.T * C::kRows;
  for (int i = threadIdx.x; i < 2 * tile_sums; i += 32 * kWarps) sums[i] = 0;

  // a warp takes a run of the tile's (job, K-group) items
  const int begin = warp * items / kWarps, end = (warp + 1) * items / kWarps, begin_job = begin / groups, begin_g = begin % groups;
  int ft = begin < end ? blockIdx.x : tiles, fi = begin, fjob = begin_job, fg = begin_g;
  uint32_t fto = ring;
  const uint8_t* w_from = nullptr;
  const int32_t* scale_from = nullptr;
  const int scale_row = kFp4 ? n4 : 0;
  auto aim = [&] {
    const int e = r.job_expert[fjob];
    w_from = a.w2 + (static_cast<long long>(e) * a.H + ft * C::kRows + P::row(lane)) * row_bytes + fg * P::kRowBytes + P::column(lane);
    scale_from = kFp4 ? a.sf2 + (static_cast<long long>(e) * groups + fg) * n4 + ft * C::kRows + 4 * lane
                      : a.sf2 + static_cast<long long>(e) * ((groups + 3) / 4) * n4 + (ft * C::kRows / 128 & ~3);
  };
  if (ft < tiles) aim();
  auto fetch = [&] {
    if (ft < tiles) {
      const uint32_t to = fto + P::place(lane);
#pragma unroll
      for (int i = 0; i < P::kCopies; ++i) dg::cp_async_16(to + i * 512, w_from + i * P::kCopyRows * row_bytes);
      if (lane < P::kScaleBytes / 16) dg::cp_async_16(fto + P::kBytes + 16 * lane, kFp4 ? scale_from : scale_from + fg / 4 * n4);
      w_from += P::kRowBytes;
      scale_from += scale_row;
      ++fg;
      if (++fi == end) {
        fi = begin, fjob = begin_job, fg = begin_g, ft += gridDim.x;
        if (ft < tiles) aim();
      } else if (fg == groups) {
        fg = 0, ++fjob;
        aim();
      }
    }
    fto = fto + C::kStage == ring + kStages * C::kStage ? ring : fto + C::kStage;
    cp_async_commit();
  };
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();

  // this lane's fragments of an item's tokens (as FP16 pairs) and the scales of its two columns, one item ahead
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
  if (begin < end && static_cast<int>(blockIdx.x) < tiles) load_h(begin_job, begin_g);

  uint32_t at = ring;
  int flip = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, flip ^= 1) {
    float* mine = sums + flip * tile_sums + warp * a.T * C::kRows;
    float sum[kM][NT][4];
#pragma unroll
    for (int m = 0; m < kM; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) sum[m][n][0] = sum[m][n][1] = sum[m][n][2] = sum[m][n][3] = 0;
    int job = begin_job, g = begin_g;
    for (int it = begin; it < end; ++it) {
      const int slot = r.job_slot[job], count = r.job_count[job];
      uint4 hc[NT][4];
      float sc[NT][2][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) hc[n][i] = hr[n][i];
#pragma unroll
        for (int i = 0; i < 2; ++i) sc[n][i][0] = __uint_as_float(hs[n][i].x), sc[n][i][1] = __uint_as_float(hs[n][i].y);
      }
      const bool last = it + 1 == end, turn = g + 1 == groups;
      if (!last) load_h(turn ? job + 1 : job, turn ? 0 : g + 1);
      else if (tile + static_cast<int>(gridDim.x) < tiles) load_h(begin_job, begin_g);
      cp_async_wait<kStages - 2>();
      __syncwarp();
      fetch();
      if constexpr (!kFp4) {
        const float s = dg::ue8m0_value(lds32(at + P::kBytes + (tile * C::kRows / 128 & 3) * 4) >> (8 * (g & 3)) & 255);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          float t[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n) t[n][0] = s * sc[n][0][p], t[n][1] = s * sc[n][1][p];
#pragma unroll
          for (int m = 0; m < kM; ++m) {
            const uint4 w0 = lds128(at + P::chunk(16 * m + g8, 4 * p + q4)), w1 = lds128(at + P::chunk(16 * m + 8 + g8, 4 * p + q4));
            float acc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t u0 = word_of(w0, i), u1 = word_of(w1, i);
              const uint32_t a0 = half2_of_e4m3(u0), a2 = half2_of_e4m3(u0 >> 16), a1 = half2_of_e4m3(u1), a3 = half2_of_e4m3(u1 >> 16);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                if (n == 0 || n * 8 < count)
                  mma_f16(acc[n], a0, a1, a2, a3, word_of(hc[n][2 * p + i / 2], i % 2 * 2), word_of(hc[n][2 * p + i / 2], i % 2 * 2 + 1));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                sum[m][n][i] = fmaf(t[n][i], acc[n][i], sum[m][n][i]);
                sum[m][n][2 + i] = fmaf(t[n][i], acc[n][2 + i], sum[m][n][2 + i]);
              }
          }
        }
      } else {
        P::expand_scales(at + P::kBytes, expanded, lane, 1.0f);
#pragma unroll
        for (int m = 0; m < kM; ++m) {
          const uint4 s0 = reinterpret_cast<const uint4*>(expanded)[16 * m + g8], s1 = reinterpret_cast<const uint4*>(expanded)[16 * m + 8 + g8];
          float half[NT][4];
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const uint32_t u0 = lds32(at + P::chunk(16 * m + g8, b) + 4 * q4), u1 = lds32(at + P::chunk(16 * m + 8 + g8, b) + 4 * q4);
            const float e0 = float_of(s0, b), e1 = float_of(s1, b);
            float part[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t v0 = u0 >> (16 * i), v1 = u1 >> (16 * i);
              const uint32_t a0 = half2_of_e2m1(v0 & 255), a1 = half2_of_e2m1(v1 & 255), a2 = half2_of_e2m1(v0 >> 8 & 255), a3 = half2_of_e2m1(v1 >> 8 & 255);
#pragma unroll
              for (int n = 0; n < NT; ++n)
                if (n == 0 || n * 8 < count) mma_f16(part[n], a0, a1, a2, a3, word_of(hc[n][b], 2 * i), word_of(hc[n][b], 2 * i + 1));
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float e = i < 2 ? e0 : e1;
                half[n][i] = b % 2 == 0 ? e * part[n][i] : fmaf(e, part[n][i], half[n][i]);
                if (b % 2 == 1) sum[m][n][i] = fmaf(sc[n][i % 2][b / 2], half[n][i], sum[m][n][i]);
              }
          }
        }
      }
      at = at + C::kStage == ring + kStages * C::kStage ? ring : at + C::kStage;
      if (last || turn) {
        // rows g8 and g8 + 8 of each 16 for the job's tokens, into the warp's sums
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = n * 8 + 2 * q4 + i;
            if (col < count) {
              float* to = mine + r.token[slot + col] * C::kRows + g8;
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
    float* all = sums + flip * tile_sums;
    for (int i = threadIdx.x; i < a.T * C::kRows; i += 32 * kWarps) {
      const long long to = static_cast<long long>(i / C::kRows) * a.H + tile * C::kRows + i % C::kRows;
      float v = a.c ? __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(a.c) + to))) : 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v += all[w * a.T * C::kRows + i];
        all[w * a.T * C::kRows + i] = 0;
      }
      a.y[to] = __float2bfloat16_rn(v);
    }
  }
  cp_async_wait<0>();
}

// -------------------------------------------------------------------------------------------

template <bool kFp4, bool kBig>
dg_status run_layer(const MoeArgs& a, const LaunchContext& ctx, cudaStream_t stream) {
  using U = Up<kFp4, kBig>;
  using D = Down<kFp4, kBig>;
  static_assert(sizeof(RoutingScratch) <= U::kRing && sizeof(RoutingScratch) <= D::kRing, "scratch in the rings");
  const int up_smem = U::smem(a.H / 128, a.T), down_smem = D::smem(a.T);
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
  const unsigned up_grid = static_cast<unsigned>(U::kBlocksPerSm * ctx.sms), down_grid = static_cast<unsigned>(std::min(ctx.sms, a.H / D::kRows));
  if (dg_status s = dg::launch(moe_up_kernel<kFp4, kBig>, up_grid, 32 * kUpWarps, static_cast<size_t>(up_smem), stream, ctx.pdl, a); s != DG_OK) return s;
  return dg::launch(moe_down_kernel<kFp4, kBig>, down_grid, 32 * D::kWarps, static_cast<size_t>(down_smem), stream, ctx.pdl, a);
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
                  ctx.status, T, topk, E, H, I};
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
