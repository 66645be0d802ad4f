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
// The tokens' side is small, shared by all blocks and stays in L2: a warp reads its fragments of it
// straight into registers, one piece ahead. A warp multiplies 16 weight rows by up to 8 * NT tokens with
// m16n8k16 MMAs: the weights are the M operand, an expert's tokens the N columns. Operands are FP16,
// which holds E4M3 and E2M1 exactly; accumulation is FP32, and the scales are applied to FP32 partial sums.
//
// An expert's tokens are compacted into jobs of at most 8 * NT columns; each distinct (expert, token)
// pair is a slot. The first kernel writes h = weight * silu(g) * u of every slot to the workspace, in
// FP16 with one power-of-two scale per 64 columns (11 bits of every value within 2^-29 of the
// largest of its 64; the plain FP32 would double what the second kernel reads). The second kernel
// owns output rows: a block sums all experts for its 16 rows of W2 and every token, in an order
// that depends on the sizes alone, and writes each output once. No atomics on values.
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
constexpr int kDownWarps = 16;
constexpr int kUpStages = 4;            // of a warp's ring
constexpr int kDownStages = 4;
constexpr int kHBlock = 8 * kUpWarps;   // columns of h that share a scale: one block's rows in the first kernel
static_assert(kHBlock == 64, "h's layout has two scales per 128 columns");
constexpr int kHBytes = 272;            // 128 columns of h of a slot: 256 bytes of FP16, two FP32 scales, padding
constexpr uint32_t kAll = 0xFFFFFFFFu;

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
// A warp's 16 x 128 piece of the weights
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

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t p) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(p));
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

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// The K order of a product is free. Within 128 columns, lane 4 g + q (g the row or column of the MMA
// fragment) takes, in the E4M3 form, columns 64 p + 16 q .. + 15 of half p: one 128-bit load of E4M3
// holds four MMAs' fragments of a row. In the E2M1 form it takes columns 32 b + 8 q .. + 7 of block b:
// the columns of an MMA then share a scale.
//
// A ring stage: the weights' 16 rows, then their scales. Chunk c (16 bytes) of a 128-byte row has the
// halves of odd rows exchanged, so that the eight lanes of a 128-bit shared load (two rows, four chunks)
// cover every bank once; 64-byte rows of E2M1, read 4 bytes per lane (eight rows, one chunk), are
// permuted over four rows pairs for the same reason.
template <bool kFp4>
struct Piece {
  static constexpr int kRowBytes = kFp4 ? 64 : 128;
  static constexpr int kBytes = 16 * kRowBytes;
  static constexpr int kCopies = kBytes / 512;              // 16 bytes per lane each
  static constexpr int kCopyRows = 16 / kCopies;
  // E4M3: the four packed words of neighbouring 128-row blocks that hold the rows'; E2M1: a word per row
  static constexpr int kScaleBytes = kFp4 ? 64 : 32;
  static constexpr int kStage = kBytes + kScaleBytes;

  static __device__ __forceinline__ int chunk(int row, int c) {
    return kFp4 ? row * 64 + ((c ^ ((row >> 1) & 3)) << 4) : row * 128 + ((c ^ ((row & 1) << 2)) << 4);
  }
  // this lane's row (of the first copy), chunk and place in a stage; copy i is kCopyRows rows further
  static __device__ __forceinline__ int row(int lane) { return lane / (kRowBytes / 16); }
  static __device__ __forceinline__ int column(int lane) { return lane % (kRowBytes / 16) * 16; }
  static __device__ __forceinline__ int place(int lane) { return chunk(row(lane), lane % (kRowBytes / 16)); }
};
static_assert(Piece<true>::kCopyRows == 8 && Piece<false>::kCopyRows == 4, "the swizzles repeat every 2 and 8 rows");

// -------------------------------------------------------------------------------------------
// First kernel: h = weight * silu(G x) * (U x)
// -------------------------------------------------------------------------------------------

template <bool kFp4>
__host__ __device__ constexpr int up_ring_bytes() { return kUpWarps * kUpStages * Piece<kFp4>::kStage; }

template <bool kFp4, int NT>
__global__ void __launch_bounds__(32 * kUpWarps, 2) moe_up_kernel(const MoeArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Routing r;
  __shared__ float block_max[2][kUpWarps][NT * 8];
  using P = Piece<kFp4>;
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3;
  const int t4 = (a.T + 3) / 4 * 4;
  const int groups = a.H / 128, blocks = a.I / kHBlock;
  build_routing<NT * 8, 32 * kUpWarps>(a, r, *reinterpret_cast<RoutingScratch*>(dyn), blockIdx.x == 0);
  // after the rings: the tokens' scales [groups, T], and per warp the weights' two scales of every group
  float* sx = reinterpret_cast<float*>(dyn + up_ring_bytes<kFp4>());
  float2* sw = reinterpret_cast<float2*>(sx + (groups * a.T + 1) / 2 * 2) + warp * groups;
  for (int i = threadIdx.x; i < (groups + 3) / 4 * a.T; i += 32 * kUpWarps) {
    const int w = i / a.T, t = i % a.T;
    const uint32_t v = dg::ld_cg_s32(a.sfx + w * t4 + t);
    for (int b = 0; b < 4 && 4 * w + b < groups; ++b) sx[(4 * w + b) * a.T + t] = dg::ue8m0_value(v >> (8 * b) & 255);
  }
  __syncthreads();

  const int units = r.jobs * blocks;
  const uint32_t ring = dg::smem_addr(dyn) + warp * kUpStages * P::kStage;
  const long long row_bytes = kFp4 ? a.H / 2 : a.H;
  const int n4 = kFp4 ? 2 * a.I : (a.I / 64 + 3) / 4 * 4;           // words of a scale row (2 I is a multiple of 4)
  // the copies run kUpStages - 1 pieces ahead of the products, over the block's units one after another
  int fu = blockIdx.x, fg = 0;
  uint32_t fto = ring;
  const uint8_t* gate_from = nullptr;
  const uint8_t* up_from = nullptr;
  const int32_t* scale_from = nullptr;
  uint32_t next_gate = 0, next_up = 0;                              // E4M3: packed scale word `lane` of the unit
  auto load_scales = [&](int u) {
    const int e = r.job_expert[u / blocks], i0 = u % blocks * kHBlock;
    if (lane < (groups + 3) / 4) {
      const int32_t* sf = a.sf13 + (static_cast<long long>(e) * ((groups + 3) / 4) + lane) * n4;
      next_gate = dg::ld_cg_s32(sf + i0 / 128);
      next_up = dg::ld_cg_s32(sf + (a.I + i0) / 128);
    }
  };
  auto fetch = [&] {
    if (fu < units) {
      if (fg == 0) {
        const int e = r.job_expert[fu / blocks], i0 = fu % blocks * kHBlock + warp * 8;
        const uint8_t* w = a.w13 + static_cast<long long>(e) * 2 * a.I * row_bytes;
        const int row = P::row(lane);
        gate_from = w + (i0 + row) * row_bytes + P::column(lane);
        up_from = gate_from + a.I * row_bytes;
        if (kFp4) {
          scale_from = a.sf13 + static_cast<long long>(e) * groups * n4 + (lane < 2 ? i0 : a.I + i0 - 8) + 4 * lane;
        } else if (groups >= kUpStages - 1) {
          load_scales(fu);
        }
      }
      const uint32_t to = fto + P::place(lane);
#pragma unroll
      for (int i = 0; i < P::kCopies; ++i) {
        const uint8_t* from = i < P::kCopies / 2 ? gate_from + i * P::kCopyRows * row_bytes
                                                 : up_from + (i - P::kCopies / 2) * P::kCopyRows * row_bytes;
        dg::cp_async_16(to + i * 512, from);
      }
      gate_from += P::kRowBytes;
      up_from += P::kRowBytes;
      if (kFp4) {
        if (lane < 4) dg::cp_async_16(fto + P::kBytes + 16 * lane, scale_from);
        scale_from += n4;
      }
      if (++fg == groups) fg = 0, fu += gridDim.x;
    }
    fto = fto + P::kStage == ring + kUpStages * P::kStage ? ring : fto + P::kStage;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kUpStages - 1; ++i) fetch();

  int flip = 0;
  uint32_t at = ring;
  for (int u = blockIdx.x; u < units; u += gridDim.x, flip ^= 1) {
    const int job = u / blocks, blk = u % blocks, slot = r.job_slot[job], count = r.job_count[job];
    float sum[NT][4];
    const float* sxt[NT][2];
    const uint8_t* xt[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        sxt[n][i] = sx + (col < count ? r.token[slot + col] : 0);
      }
      const int col = n * 8 + g8;                                   // its fragments: null past the job's tokens
      xt[n] = col < count ? a.x + static_cast<long long>(r.token[slot + col]) * a.H + (kFp4 ? 8 * q4 : 16 * q4) : nullptr;
    }
    if constexpr (!kFp4) {
      // the unit's scales as FP32, read while the unit before was computed (unless the copies, kUpStages - 1
      // pieces ahead, are then past the next unit's start)
      if (groups < kUpStages - 1) load_scales(u);
      __syncwarp();
      if (lane < (groups + 3) / 4)
        for (int b = 0; b < 4 && 4 * lane + b < groups; ++b)
          sw[4 * lane + b] = make_float2(dg::ue8m0_value(next_gate >> (8 * b) & 255), dg::ue8m0_value(next_up >> (8 * b) & 255));
      __syncwarp();
    }
    // E4M3: two 16-byte loads per eight tokens and 128 columns; E2M1: four of 8 bytes
    uint32_t xr[NT][8];
    auto load_x = [&](int g) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (xt[n]) {
          if constexpr (kFp4) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              const uint2 v = ld_cg_v2(xt[n] + g * 128 + b * 32);
              xr[n][2 * b] = v.x, xr[n][2 * b + 1] = v.y;
            }
          } else {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const uint4 v = dg::ld_cg_v4(xt[n] + g * 128 + p * 64);
              xr[n][4 * p] = v.x, xr[n][4 * p + 1] = v.y, xr[n][4 * p + 2] = v.z, xr[n][4 * p + 3] = v.w;
            }
          }
        }
    };
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 8; ++i) xr[n][i] = 0;
    load_x(0);
    for (int g = 0; g < groups; ++g) {
      uint32_t xn[NT][8];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) xn[n][i] = xr[n][i];
      if (g + 1 < groups) load_x(g + 1);
      cp_async_wait<kUpStages - 2>();
      __syncwarp();
      fetch();
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0;
      if constexpr (!kFp4) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w0 = lds128(at + P::chunk(g8, 4 * p + q4)), w1 = lds128(at + P::chunk(g8 + 8, 4 * p + q4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u0 = word_of(w0, i), u1 = word_of(w1, i);
            const uint32_t a0 = half2_of_e4m3(u0), a2 = half2_of_e4m3(u0 >> 16), a1 = half2_of_e4m3(u1), a3 = half2_of_e4m3(u1 >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t x = xn[n][4 * p + i];
              mma_16816(acc[n], a0, a1, a2, a3, half2_of_e4m3(x), half2_of_e4m3(x >> 16));
            }
          }
        }
        const float2 s = sw[g];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = sxt[n][i][g * a.T];
            sum[n][i] = fmaf(t * s.x, acc[n][i], sum[n][i]);
            sum[n][2 + i] = fmaf(t * s.y, acc[n][2 + i], sum[n][2 + i]);
          }
      } else {
        const uint32_t z0 = lds32(at + P::kBytes + 4 * g8), z1 = lds32(at + P::kBytes + 32 + 4 * g8);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t u0 = lds32(at + P::chunk(g8, b) + 4 * q4), u1 = lds32(at + P::chunk(g8 + 8, b) + 4 * q4);
          const float e0 = dg::ue8m0_value(z0 >> (8 * b) & 255), e1 = dg::ue8m0_value(z1 >> (8 * b) & 255);
          float part[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v0 = u0 >> (16 * i), v1 = u1 >> (16 * i);
            const uint32_t a0 = half2_of_e2m1(v0 & 255), a1 = half2_of_e2m1(v1 & 255), a2 = half2_of_e2m1(v0 >> 8 & 255), a3 = half2_of_e2m1(v1 >> 8 & 255);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t x = xn[n][2 * b + i];
              mma_16816(part[n], a0, a1, a2, a3, half2_of_e4m3(x), half2_of_e4m3(x >> 16));
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[n][0] = fmaf(e0, part[n][0], acc[n][0]);
            acc[n][1] = fmaf(e0, part[n][1], acc[n][1]);
            acc[n][2] = fmaf(e1, part[n][2], acc[n][2]);
            acc[n][3] = fmaf(e1, part[n][3], acc[n][3]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float t = sxt[n][i][g * a.T];
            sum[n][i] = fmaf(t, acc[n][i], sum[n][i]);
            sum[n][2 + i] = fmaf(t, acc[n][2 + i], sum[n][2 + i]);
          }
      }
      at = at + P::kStage == ring + kUpStages * P::kStage ? ring : at + P::kStage;
    }
    // column blk * 64 + warp * 8 + g8 of h for tokens 2 q4, 2 q4 + 1 of each eight: gate in sum[0..1], up in sum[2..3]
    float hv[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        const float gate = sum[n][i];
        hv[n][i] = col < count ? r.coef[slot + col] * (gate / (1.0f + expf(-gate)) * sum[n][2 + i]) : 0.0f;
        float m = fabsf(hv[n][i]);
        m = m < INFINITY ? m : 0.0f;
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
        if (g8 == 0) block_max[flip][warp][col] = m;
      }
    __syncthreads();
    // where the second kernel's lanes find this column in the 64: E4M3 as 16-byte pieces of two loads, each
    // of 64 bytes over four lanes; E2M1 in order
    const int cc = warp * 8 + g8;
    const int place = kFp4 ? cc * 2 : (cc % 16) / 8 * 64 + cc / 16 * 16 + cc % 8 * 2;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        if (col >= count) continue;
        float m = 0;
#pragma unroll
        for (int w = 0; w < kUpWarps; ++w) m = fmaxf(m, block_max[flip][w][col]);
        // the largest to [2^14, 2^15); both powers stay normal
        const int ex = min(max(static_cast<int>(__float_as_uint(m) >> 23), 27), 254) - 127 - 14;
        const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        uint8_t* row = a.h + (static_cast<long long>(slot + col) * (a.I / 128) + blk / 2) * kHBytes;
        *reinterpret_cast<__half*>(row + (blk & 1) * 128 + place) = __float2half_rn(hv[n][i] * up);
        if (warp == 0 && g8 == 0)
          reinterpret_cast<float*>(row + 256)[blk & 1] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      }
  }
  cp_async_wait<0>();
}

// -------------------------------------------------------------------------------------------
// Second kernel: y = c + W2 h
// -------------------------------------------------------------------------------------------

template <bool kFp4>
__host__ __device__ constexpr int down_ring_bytes() { return kDownWarps * kDownStages * Piece<kFp4>::kStage; }

template <bool kFp4, int NT>
__global__ void __launch_bounds__(32 * kDownWarps, 1) moe_down_kernel(const MoeArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Routing r;
  using P = Piece<kFp4>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3;
  // The first kernel let this one start only after its own wait: ids and weights are there, h is not yet.
  build_routing<NT * 8, 32 * kDownWarps>(a, r, *reinterpret_cast<RoutingScratch*>(dyn), false);

  const int groups = a.I / 128, items = r.jobs * groups, tiles = a.H / 16;
  const long long row_bytes = kFp4 ? a.I / 2 : a.I;
  const int n4 = kFp4 ? a.H : (a.H / 128 + 3) / 4 * 4;
  const uint32_t ring = dg::smem_addr(dyn) + warp * kDownStages * P::kStage;
  // every warp's sums of a tile, [2][warps][T][16]: the tile before is being added up meanwhile
  float* sums = reinterpret_cast<float*>(dyn + down_ring_bytes<kFp4>());
  const int tile_sums = kDownWarps * a.T * 16;
  for (int i = threadIdx.x; i < 2 * tile_sums; i += 32 * kDownWarps) sums[i] = 0;

  // a warp takes every sixteenth of the tile's (job, K-group) items
  const bool busy = warp < items;
  int ft = busy ? blockIdx.x : tiles, fjob = warp / groups, fg = warp % groups;
  uint32_t fto = ring;
  auto fetch = [&] {
    if (ft < tiles) {
      const int e = r.job_expert[fjob], row = P::row(lane);
      const uint8_t* from = a.w2 + (static_cast<long long>(e) * a.H + ft * 16 + row) * row_bytes + fg * P::kRowBytes + P::column(lane);
      const uint32_t to = fto + P::place(lane);
#pragma unroll
      for (int i = 0; i < P::kCopies; ++i) dg::cp_async_16(to + i * 512, from + i * P::kCopyRows * row_bytes);
      if (kFp4) {
        if (lane < 4) dg::cp_async_16(fto + P::kBytes + 16 * lane, a.sf2 + (static_cast<long long>(e) * groups + fg) * n4 + ft * 16 + 4 * lane);
      } else if (lane == 0) {
        dg::cp_async_16(fto + P::kBytes, a.sf2 + (static_cast<long long>(e) * ((groups + 3) / 4) + fg / 4) * n4 + (ft / 8 & ~3));
      }
      for (fg += kDownWarps; fg >= groups; fg -= groups) ++fjob;
      if (fjob >= r.jobs) fjob = warp / groups, fg = warp % groups, ft += gridDim.x;
    }
    fto = fto + P::kStage == ring + kDownStages * P::kStage ? ring : fto + P::kStage;
    cp_async_commit();
  };
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kDownStages - 1; ++i) fetch();
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();

  // this lane's fragments of an item's tokens (as FP16 pairs) and the scales of its two columns
  uint32_t hr[NT][16];
  uint2 hs[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    hs[n][0] = hs[n][1] = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 16; ++i) hr[n][i] = 0;
  }
  auto load_h = [&](int job, int g) {
    const int slot = r.job_slot[job], count = r.job_count[job];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint8_t* base = a.h + (static_cast<long long>(slot + n * 8) * groups + g) * kHBytes;
      if (n * 8 + g8 < count) {
        const uint8_t* from = base + static_cast<long long>(g8) * groups * kHBytes + q4 * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = dg::ld_cg_v4(from + i * 64);
          hr[n][4 * i] = v.x, hr[n][4 * i + 1] = v.y, hr[n][4 * i + 2] = v.z, hr[n][4 * i + 3] = v.w;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (n * 8 + 2 * q4 + i < count) hs[n][i] = ld_cg_v2(base + static_cast<long long>(2 * q4 + i) * groups * kHBytes + 256);
    }
  };
  if (busy && static_cast<int>(blockIdx.x) < tiles) load_h(warp / groups, warp % groups);

  uint32_t at = ring;
  int flip = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, flip ^= 1) {
    float* mine = sums + flip * tile_sums + warp * a.T * 16;
    float sum[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0;
    int job = warp / groups, g = warp % groups;
    while (job < r.jobs) {
      int next_job = job, next_g = g + kDownWarps;
      for (; next_g >= groups; next_g -= groups) ++next_job;
      auto load_next = [&] {
        if (next_job < r.jobs) load_h(next_job, next_g);
        else if (tile + static_cast<int>(gridDim.x) < tiles) load_h(warp / groups, warp % groups);
      };
      // sixteen tokens' fragments take the registers that a second set would need: they are loaded after use
      constexpr bool kAhead = NT == 1;
      uint32_t hc[NT][16];
      float sc[NT][2][2];
      if constexpr (kAhead) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 16; ++i) hc[n][i] = hr[n][i];
#pragma unroll
          for (int i = 0; i < 2; ++i) sc[n][i][0] = __uint_as_float(hs[n][i].x), sc[n][i][1] = __uint_as_float(hs[n][i].y);
        }
        load_next();
      }
      auto frag = [&](int n, int i) { return kAhead ? hc[n][i] : hr[n][i]; };
      auto col_scale = [&](int n, int i, int p) { return kAhead ? sc[n][i][p] : __uint_as_float(p ? hs[n][i].y : hs[n][i].x); };
      cp_async_wait<kDownStages - 2>();
      __syncwarp();
      fetch();
      if constexpr (!kFp4) {
        const float s = dg::ue8m0_value(lds32(at + P::kBytes + (tile / 8 & 3) * 4) >> (8 * (g & 3)) & 255);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w0 = lds128(at + P::chunk(g8, 4 * p + q4)), w1 = lds128(at + P::chunk(g8 + 8, 4 * p + q4));
          float acc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u0 = word_of(w0, i), u1 = word_of(w1, i);
            const uint32_t a0 = half2_of_e4m3(u0), a2 = half2_of_e4m3(u0 >> 16), a1 = half2_of_e4m3(u1), a3 = half2_of_e4m3(u1 >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(acc[n], a0, a1, a2, a3, frag(n, 8 * p + 2 * i), frag(n, 8 * p + 2 * i + 1));
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float t = s * col_scale(n, i, p);
              sum[n][i] = fmaf(t, acc[n][i], sum[n][i]);
              sum[n][2 + i] = fmaf(t, acc[n][2 + i], sum[n][2 + i]);
            }
        }
      } else {
        const uint32_t z0 = lds32(at + P::kBytes + 4 * g8), z1 = lds32(at + P::kBytes + 32 + 4 * g8);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t u0 = lds32(at + P::chunk(g8, b) + 4 * q4), u1 = lds32(at + P::chunk(g8 + 8, b) + 4 * q4);
          const float e0 = dg::ue8m0_value(z0 >> (8 * b) & 255), e1 = dg::ue8m0_value(z1 >> (8 * b) & 255);
          float part[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) part[n][0] = part[n][1] = part[n][2] = part[n][3] = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t v0 = u0 >> (16 * i), v1 = u1 >> (16 * i);
            const uint32_t a0 = half2_of_e2m1(v0 & 255), a1 = half2_of_e2m1(v1 & 255), a2 = half2_of_e2m1(v0 >> 8 & 255), a3 = half2_of_e2m1(v1 >> 8 & 255);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_16816(part[n], a0, a1, a2, a3, frag(n, 4 * b + 2 * i), frag(n, 4 * b + 2 * i + 1));
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float t = col_scale(n, i, b / 2);
              sum[n][i] = fmaf(t * e0, part[n][i], sum[n][i]);
              sum[n][2 + i] = fmaf(t * e1, part[n][2 + i], sum[n][2 + i]);
            }
        }
      }
      if constexpr (!kAhead) load_next();
      at = at + P::kStage == ring + kDownStages * P::kStage ? ring : at + P::kStage;
      if (next_job != job) {
        // rows g8 and g8 + 8 of the job's tokens, into the warp's sums
        const int slot = r.job_slot[job], count = r.job_count[job];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int col = n * 8 + 2 * q4 + i;
            if (col < count) {
              float* to = mine + r.token[slot + col] * 16;
              to[g8] += sum[n][i];
              to[g8 + 8] += sum[n][2 + i];
            }
            sum[n][i] = sum[n][2 + i] = 0;
          }
        __syncwarp();
      }
      job = next_job, g = next_g;
    }
    __syncthreads();
    float* all = sums + flip * tile_sums;
    for (int i = threadIdx.x; i < a.T * 16; i += 32 * kDownWarps) {
      const long long to = static_cast<long long>(i / 16) * a.H + tile * 16 + i % 16;
      float v = a.c ? __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(a.c) + to))) : 0.0f;
#pragma unroll
      for (int w = 0; w < kDownWarps; ++w) {
        v += all[w * a.T * 16 + i];
        all[w * a.T * 16 + i] = 0;
      }
      a.y[to] = __float2bfloat16_rn(v);
    }
  }
  cp_async_wait<0>();
}

// -------------------------------------------------------------------------------------------

template <bool kFp4, int NT>
dg_status run_layer(const MoeArgs& a, const LaunchContext& ctx, cudaStream_t stream) {
  constexpr int kMaxSmem = 200 * 1024;
  // once per thread and device: the limit, above what any shape needs
  static thread_local int ready = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && ready != dev) {
    e = cudaFuncSetAttribute(moe_up_kernel<kFp4, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(moe_down_kernel<kFp4, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e == cudaSuccess) ready = dev;
  }
  if (e != cudaSuccess) return dg::record_cuda_error(e);
  const int groups = a.H / 128;
  const int up_smem = up_ring_bytes<kFp4>() + (groups * a.T + 1) / 2 * 8 + (kFp4 ? 0 : kUpWarps * groups * 8);
  const int down_smem = down_ring_bytes<kFp4>() + 2 * kDownWarps * a.T * 16 * 4;
  static_assert(up_ring_bytes<kFp4>() + (kMaxH / 128) * (kMaxTokens * 4 + kUpWarps * 8) <= kMaxSmem &&
                down_ring_bytes<kFp4>() + 2 * kDownWarps * kMaxTokens * 16 * 4 <= kMaxSmem, "shared memory");
  static_assert(sizeof(RoutingScratch) <= up_ring_bytes<kFp4>() && sizeof(RoutingScratch) <= down_ring_bytes<kFp4>(), "scratch in the rings");
  const unsigned up_grid = static_cast<unsigned>(2 * ctx.sms), down_grid = static_cast<unsigned>(std::min(ctx.sms, a.H / 16));
  if (dg_status s = dg::launch(moe_up_kernel<kFp4, NT>, up_grid, 32 * kUpWarps, static_cast<size_t>(up_smem), stream, ctx.pdl, a); s != DG_OK) return s;
  return dg::launch(moe_down_kernel<kFp4, NT>, down_grid, 32 * kDownWarps, static_cast<size_t>(down_smem), stream, ctx.pdl, a);
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
  return T <= 8 ? run_layer<kFp4, 1>(a, ctx, stream) : run_layer<kFp4, 2>(a, ctx, stream);
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
