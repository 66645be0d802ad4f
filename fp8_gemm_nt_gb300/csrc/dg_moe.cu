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
// A warp multiplies 16 weight rows by up to 8 * NT tokens with m16n8k16 MMAs: the weights are the M
// operand, an expert's tokens the N columns. Operands are FP16, which holds E4M3 and E2M1 exactly;
// accumulation is FP32, and the scales are applied to FP32 partial sums.
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
constexpr int kMaxExperts = 1024;       // four per thread in the prologue
constexpr int kMaxH = 16384;
constexpr int kMaxSlots = kMaxTokens * kMaxTopk;
constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kStages = 4;              // of a warp's ring in the first kernel
constexpr int kHBlock = 64;             // columns of h that share a scale: one block's rows in the first kernel
constexpr int kHBytes = 272;            // 128 columns of h of a slot: 256 bytes of FP16, two FP32 scales, padding

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
  uint32_t mask[kMaxExperts];           // tokens of an expert
  int first_slot[kMaxExperts];
  int job_expert[kMaxSlots];
  int job_slot[kMaxSlots];              // first slot of a job; a job's slots are consecutive
  int job_count[kMaxSlots];
  float coef[kMaxSlots];                // weight of a slot (the sum, where a token names an expert twice)
  uint8_t token[kMaxSlots];
  int warp_sum[kWarps];
  int jobs;
};

// Builds the routing of the block from the ids, in the order of experts and tokens: the same in
// every block of both kernels. `kCols`: columns of a job.
template <int kCols>
__device__ void build_routing(const MoeArgs& a, Routing& r, bool report) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
  for (int e = tid; e < a.E; e += kThreads) r.mask[e] = 0;
  __syncthreads();
  for (int i = tid; i < a.T * a.k; i += kThreads) {
    const int e = dg::ld_cg_s32(a.ids + i);
    if (e >= 0 && e < a.E) atomicOr(&r.mask[e], 1u << (i / a.k));
    else if (e != -1 && report) atomicOr(a.status, dg::kBadIndexBit);
  }
  __syncthreads();
  // jobs and slots before each expert: four experts per thread, jobs in the upper half of a word
  int n[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * tid + i;
    const int tokens = e < a.E ? __popc(r.mask[e]) : 0;
    n[i] = ((tokens + kCols - 1) / kCols) << 16 | tokens;
    sum += n[i];
  }
  int before = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, before, o);
    if (lane >= o) before += v;
  }
  if (lane == 31) r.warp_sum[warp] = before;
  before -= sum;
  __syncthreads();
  for (int w = 0; w < warp; ++w) before += r.warp_sum[w];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = 4 * tid + i;
    if (e < a.E) {
      const int slot = before & 0xFFFF, tokens = n[i] & 0xFFFF;
      r.first_slot[e] = slot;
      int job = before >> 16;
      for (int c = 0; c < tokens; c += kCols, ++job) {
        r.job_expert[job] = e;
        r.job_slot[job] = slot + c;
        r.job_count[job] = min(kCols, tokens - c);
      }
      before += n[i];
    }
  }
  if (tid == kThreads - 1) r.jobs = before >> 16;
  __syncthreads();
  for (int i = tid; i < a.T * a.k; i += kThreads) {
    const int e = dg::ld_cg_s32(a.ids + i);
    if (e < 0 || e >= a.E) continue;
    const int t = i / a.k;
    bool first = true;
    float w = 0;
    for (int j = t * a.k; j < (t + 1) * a.k; ++j)
      if (dg::ld_cg_s32(a.ids + j) == e) {
        first = first && j >= i;
        w += __ldcg(a.weights + j);
      }
    if (first) {
      const int slot = r.first_slot[e] + __popc(r.mask[e] & ((1u << t) - 1));
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

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Where 16-byte chunk `c` of a 128-byte row lies: odd rows have their halves exchanged, so that the
// eight lanes of a 128-bit shared load (two rows, four chunks) cover every bank once.
__device__ __forceinline__ int chunk128(int row, int c) { return row * 128 + ((c ^ ((row & 1) << 2)) << 4); }
// The same for the 64-byte rows of E2M1, read 4 bytes per lane (eight rows, one chunk).
__device__ __forceinline__ int chunk64(int row, int c) { return row * 64 + ((c ^ ((row >> 1) & 3)) << 4); }

// The K order of a product is free. Within 128 columns, lane 4 g + q (g the row or column of the MMA
// fragment) takes, in the E4M3 form, columns 64 i + 16 q .. + 15 of half i: one 128-bit load of E4M3
// holds four MMAs' fragments of a row. In the E2M1 form it takes columns 32 b + 8 q .. + 7 of block b:
// the columns of an MMA then share a scale.

// Stage: the weights' 16 rows, their scales, then the tokens.
template <bool kFp4>
struct Piece {
  static constexpr int kRowBytes = kFp4 ? 64 : 128;
  static constexpr int kBytes = 16 * kRowBytes;
  // E4M3: for the upper and the lower eight rows, the four packed words of neighbouring 128-row blocks
  // that hold theirs; E2M1: a packed word per row
  static constexpr int kScaleBytes = kFp4 ? 64 : 32;

  // Copies rows r0 .. r0 + 7 and r1 .. r1 + 7 of expert e at K-group g of a [E, N, K] operand.
  static __device__ __forceinline__ void copy(uint32_t to, const uint8_t* w, const int32_t* sf, int e, int r0, int r1,
                                              int g, int N, int K, int lane) {
    const long long row_bytes = kFp4 ? K / 2 : K;
    const uint8_t* from = w + static_cast<long long>(e) * N * row_bytes + g * kRowBytes;
    constexpr int kChunks = kRowBytes / 16;
#pragma unroll
    for (int i = 0; i < 16 * kChunks / 32; ++i) {
      const int row = (i * 32 + lane) / kChunks, c = (i * 32 + lane) % kChunks;
      const int at = row < 8 ? r0 + row : r1 + row - 8;
      dg::cp_async_16(to + (kFp4 ? chunk64(row, c) : chunk128(row, c)), from + at * row_bytes + c * 16);
    }
    if (kFp4) {
      if (lane < 4) {
        const int n4 = (N + 3) / 4 * 4;
        const int at = (lane < 2 ? r0 : r1 - 8) + 4 * lane;
        dg::cp_async_16(to + kBytes + 16 * lane, sf + (static_cast<long long>(e) * (K / 128) + g) * n4 + at);
      }
    } else if (lane < 2) {
      const int n4 = ((N + 127) / 128 + 3) / 4 * 4, kp = (K / 128 + 3) / 4;
      const int at = (lane ? r1 : r0) / 128 & ~3;
      dg::cp_async_16(to + kBytes + 16 * lane, sf + (static_cast<long long>(e) * kp + g / 4) * n4 + at);
    }
  }
};

// The A fragments of one MMA of the E4M3 form: word i of half `p` (row g) and `q` (row g + 8).
__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// -------------------------------------------------------------------------------------------
// First kernel: h = weight * silu(G x) * (U x)
// -------------------------------------------------------------------------------------------

template <bool kFp4, int NT>
__host__ __device__ constexpr int up_stage_bytes() { return Piece<kFp4>::kBytes + Piece<kFp4>::kScaleBytes + NT * 8 * 128; }

template <bool kFp4, int NT>
__global__ void __launch_bounds__(kThreads) moe_up_kernel(const MoeArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Routing r;
  __shared__ float block_max[2][kWarps][NT * 8];
  using P = Piece<kFp4>;
  constexpr int kStage = up_stage_bytes<kFp4, NT>();
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3;
  const int t4 = (a.T + 3) / 4 * 4;
  const int groups = a.H / 128, blocks = a.I / kHBlock;
  uint32_t* sx = reinterpret_cast<uint32_t*>(dyn + kWarps * kStages * kStage);   // [KP, t4]
  for (int i = threadIdx.x; i < (groups + 3) / 4 * t4; i += kThreads) sx[i] = dg::ld_cg_s32(a.sfx + i);
  build_routing<NT * 8>(a, r, blockIdx.x == 0);

  const int units = r.jobs * blocks;
  const uint32_t ring = dg::smem_addr(dyn) + warp * kStages * kStage;
  // the copies run kStages - 1 pieces ahead of the products, over the block's units one after another
  int fu = blockIdx.x, fg = 0, fs = 0;
  auto fetch = [&] {
    if (fu < units) {
      const int job = fu / blocks, i0 = fu % blocks * kHBlock + warp * 8;
      const uint32_t to = ring + fs * kStage;
      P::copy(to, a.w13, a.sf13, r.job_expert[job], i0, a.I + i0, fg, 2 * a.I, a.H, lane);
      const int slot = r.job_slot[job], count = r.job_count[job];
#pragma unroll
      for (int i = 0; i < NT * 2; ++i) {
        const int col = i * 4 + lane / 8, c = lane & 7;
        if (col < count)
          dg::cp_async_16(to + P::kBytes + P::kScaleBytes + chunk128(col, c),
                          a.x + static_cast<long long>(r.token[slot + col]) * a.H + fg * 128 + c * 16);
      }
      if (++fg == groups) fg = 0, fu += gridDim.x;
    }
    fs = fs + 1 == kStages ? 0 : fs + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  int stage = 0, flip = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x, flip ^= 1) {
    const int job = u / blocks, blk = u % blocks, slot = r.job_slot[job], count = r.job_count[job];
    const int i0 = blk * kHBlock + warp * 8;
    float sum[NT][4];
    int tok[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[n][i] = 0;
        if (i < 2) tok[n][i] = n * 8 + 2 * q4 + i < count ? r.token[slot + n * 8 + 2 * q4 + i] : 0;
      }
    for (int g = 0; g < groups; ++g) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      fetch();
      const uint32_t at = ring + stage * kStage, bt = at + P::kBytes + P::kScaleBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      float acc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0;
      float s0 = 1, s1 = 1;
      if constexpr (!kFp4) {
        s0 = dg::ue8m0_value(lds32(at + P::kBytes + (i0 / 128 & 3) * 4) >> (8 * (g & 3)) & 255);
        s1 = dg::ue8m0_value(lds32(at + P::kBytes + 16 + ((a.I + i0) / 128 & 3) * 4) >> (8 * (g & 3)) & 255);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w0 = lds128(at + chunk128(g8, 4 * p + q4)), w1 = lds128(at + chunk128(g8 + 8, 4 * p + q4));
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n) b[n] = lds128(bt + chunk128(8 * n + g8, 4 * p + q4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u0 = word_of(w0, i), u1 = word_of(w1, i);
            const uint32_t a0 = half2_of_e4m3(u0), a2 = half2_of_e4m3(u0 >> 16), a1 = half2_of_e4m3(u1), a3 = half2_of_e4m3(u1 >> 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint32_t x = word_of(b[n], i);
              mma_16816(acc[n], a0, a1, a2, a3, half2_of_e4m3(x), half2_of_e4m3(x >> 16));
            }
          }
        }
      } else {
        const uint32_t z0 = lds32(at + P::kBytes + 4 * g8), z1 = lds32(at + P::kBytes + 32 + 4 * g8);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t u0 = lds32(at + chunk64(g8, b) + 4 * q4), u1 = lds32(at + chunk64(g8 + 8, b) + 4 * q4);
          const float e0 = dg::ue8m0_value(z0 >> (8 * b) & 255), e1 = dg::ue8m0_value(z1 >> (8 * b) & 255);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int col = 8 * n + g8;
            const uint32_t xa = bt + chunk128(col, 2 * b + q4 / 2) + 8 * (q4 & 1);
            float part[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t x = lds32(xa + 4 * i), v0 = u0 >> (16 * i), v1 = u1 >> (16 * i);
              mma_16816(part, half2_of_e2m1(v0 & 255), half2_of_e2m1(v1 & 255), half2_of_e2m1(v0 >> 8 & 255),
                        half2_of_e2m1(v1 >> 8 & 255), half2_of_e4m3(x), half2_of_e4m3(x >> 16));
            }
            acc[n][0] = fmaf(e0, part[0], acc[n][0]);
            acc[n][1] = fmaf(e0, part[1], acc[n][1]);
            acc[n][2] = fmaf(e1, part[2], acc[n][2]);
            acc[n][3] = fmaf(e1, part[3], acc[n][3]);
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float s = dg::ue8m0_value(sx[(g / 4) * t4 + tok[n][i]] >> (8 * (g & 3)) & 255);
          sum[n][i] = fmaf(s * s0, acc[n][i], sum[n][i]);
          sum[n][2 + i] = fmaf(s * s1, acc[n][2 + i], sum[n][2 + i]);
        }
    }
    // column i0 + g8 of h for tokens 2 q4, 2 q4 + 1 of each eight: gate in sum[0..1], up in sum[2..3]
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
        for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (g8 == 0) block_max[flip][warp][col] = m;
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int col = n * 8 + 2 * q4 + i;
        if (col >= count) continue;
        float m = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, block_max[flip][w][col]);
        // the largest to [2^14, 2^15); both powers stay normal
        const int ex = min(max(static_cast<int>(__float_as_uint(m) >> 23), 27), 254) - 127 - 14;
        const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        uint8_t* row = a.h + (static_cast<long long>(slot + col) * (a.I / 128) + blk / 2) * kHBytes;
        reinterpret_cast<__half*>(row)[(blk & 1) * kHBlock + warp * 8 + g8] = __float2half_rn(hv[n][i] * up);
        if (warp == 0 && g8 == 0)
          reinterpret_cast<float*>(row + 256)[blk & 1] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      }
  }
  cp_async_wait<0>();
}

// -------------------------------------------------------------------------------------------
// Second kernel: y = c + W2 h
// -------------------------------------------------------------------------------------------

template <bool kFp4, int NT>
__host__ __device__ constexpr int down_stage_bytes() { return Piece<kFp4>::kBytes + Piece<kFp4>::kScaleBytes + NT * 8 * kHBytes; }
// 16 columns of h a stage leave room for three
template <int NT>
__host__ __device__ constexpr int down_stages() { return NT == 1 ? 4 : 3; }

template <bool kFp4, int NT>
__global__ void __launch_bounds__(kThreads) moe_down_kernel(const MoeArgs a) {
  extern __shared__ __align__(128) uint8_t dyn[];
  __shared__ Routing r;
  using P = Piece<kFp4>;
  constexpr int kStage = down_stage_bytes<kFp4, NT>(), kStages = down_stages<NT>();
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g8 = lane / 4, q4 = lane & 3;
  build_routing<NT * 8>(a, r, false);

  const int groups = a.I / 128, items = r.jobs * groups, tiles = a.H / 16;
  const uint32_t ring = dg::smem_addr(dyn) + warp * kStages * kStage;
  float* total = reinterpret_cast<float*>(dyn + kWarps * kStages * kStage);   // [kWarps, T, 16]
  float* mine = total + warp * a.T * 16;
  for (int i = lane; i < a.T * 16; i += 32) mine[i] = 0;

  // a warp takes every eighth of the tile's (job, K-group) items
  int ft = blockIdx.x, fi = warp, fs = 0;
  auto fetch = [&] {
    while (fi >= items && ft < tiles) {
      ft += gridDim.x;
      fi = warp < items ? warp : items;
      if (items == 0) ft = tiles;
      if (fi >= items) ft = tiles;
    }
    if (ft < tiles) {
      const int job = fi / groups, g = fi % groups;
      const uint32_t to = ring + fs * kStage;
      P::copy(to, a.w2, a.sf2, r.job_expert[job], ft * 16, ft * 16 + 8, g, a.H, a.I, lane);
      const int slot = r.job_slot[job], count = r.job_count[job];
      for (int i = lane; i < count * (kHBytes / 16); i += 32) {
        const int col = i / (kHBytes / 16), c = i % (kHBytes / 16);
        dg::cp_async_16(to + P::kBytes + P::kScaleBytes + col * kHBytes + c * 16,
                        a.h + (static_cast<long long>(slot + col) * groups + g) * kHBytes + c * 16);
      }
      fi += kWarps;
    }
    fs = fs + 1 == kStages ? 0 : fs + 1;
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch();

  int stage = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    for (int it = warp; it < items; it += kWarps) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      fetch();
      const int job = it / groups, g = it % groups, slot = r.job_slot[job], count = r.job_count[job];
      const uint32_t at = ring + stage * kStage, bt = at + P::kBytes + P::kScaleBytes;
      stage = stage + 1 == kStages ? 0 : stage + 1;
      float sum[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) sum[n][0] = sum[n][1] = sum[n][2] = sum[n][3] = 0;
      if constexpr (!kFp4) {
        const float s = dg::ue8m0_value(lds32(at + P::kBytes + (tile / 8 & 3) * 4) >> (8 * (g & 3)) & 255);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const uint4 w0 = lds128(at + chunk128(g8, 4 * p + q4)), w1 = lds128(at + chunk128(g8 + 8, 4 * p + q4));
          float acc[NT][4];
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0;
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            uint4 b[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) b[n] = lds128(bt + (8 * n + g8) * kHBytes + p * 128 + q4 * 32 + i * 8);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t u0 = word_of(w0, i + k), u1 = word_of(w1, i + k);
              const uint32_t a0 = half2_of_e4m3(u0), a2 = half2_of_e4m3(u0 >> 16), a1 = half2_of_e4m3(u1), a3 = half2_of_e4m3(u1 >> 16);
#pragma unroll
              for (int n = 0; n < NT; ++n) mma_16816(acc[n], a0, a1, a2, a3, word_of(b[n], 2 * k), word_of(b[n], 2 * k + 1));
            }
          }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float hs = s * __uint_as_float(lds32(bt + (8 * n + 2 * q4 + i) * kHBytes + 256 + 4 * p));
              sum[n][i] = fmaf(hs, acc[n][i], sum[n][i]);
              sum[n][2 + i] = fmaf(hs, acc[n][2 + i], sum[n][2 + i]);
            }
        }
      } else {
        const uint32_t z0 = lds32(at + P::kBytes + 4 * g8), z1 = lds32(at + P::kBytes + 32 + 4 * g8);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const uint32_t u0 = lds32(at + chunk64(g8, b) + 4 * q4), u1 = lds32(at + chunk64(g8 + 8, b) + 4 * q4);
          const float e0 = dg::ue8m0_value(z0 >> (8 * b) & 255), e1 = dg::ue8m0_value(z1 >> (8 * b) & 255);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = lds128(bt + (8 * n + g8) * kHBytes + b * 64 + q4 * 16);
            float part[4] = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t v0 = u0 >> (16 * i), v1 = u1 >> (16 * i);
              mma_16816(part, half2_of_e2m1(v0 & 255), half2_of_e2m1(v1 & 255), half2_of_e2m1(v0 >> 8 & 255),
                        half2_of_e2m1(v1 >> 8 & 255), word_of(x, 2 * i), word_of(x, 2 * i + 1));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float hs = __uint_as_float(lds32(bt + (8 * n + 2 * q4 + i) * kHBytes + 256 + 4 * (b / 2)));
              sum[n][i] = fmaf(hs * e0, part[i], sum[n][i]);
              sum[n][2 + i] = fmaf(hs * e1, part[2 + i], sum[n][2 + i]);
            }
          }
        }
      }
      // rows g8 and g8 + 8 of the job's tokens, into the warp's own sums
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
        }
      __syncwarp();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.T * 16; i += kThreads) {
      const long long at = static_cast<long long>(i / 16) * a.H + tile * 16 + i % 16;
      float v = a.c ? __bfloat162float(__ushort_as_bfloat16(__ldcg(reinterpret_cast<const unsigned short*>(a.c) + at))) : 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        v += total[w * a.T * 16 + i];
        total[w * a.T * 16 + i] = 0;
      }
      a.y[at] = __float2bfloat16_rn(v);
    }
    __syncthreads();
  }
  cp_async_wait<0>();
}

// -------------------------------------------------------------------------------------------

template <bool kFp4, int NT>
dg_status run_layer(const MoeArgs& a, const LaunchContext& ctx, cudaStream_t stream) {
  const int t4 = (a.T + 3) / 4 * 4;
  const size_t up_smem = static_cast<size_t>(kWarps) * kStages * up_stage_bytes<kFp4, NT>() + static_cast<size_t>((a.H / 128 + 3) / 4) * t4 * 4;
  const size_t down_smem = static_cast<size_t>(kWarps) * down_stages<NT>() * down_stage_bytes<kFp4, NT>() + static_cast<size_t>(kWarps) * a.T * 16 * 4;
  cudaError_t e = cudaFuncSetAttribute(moe_up_kernel<kFp4, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(up_smem));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(moe_down_kernel<kFp4, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(down_smem));
  if (e != cudaSuccess) return dg::record_cuda_error(e);
  if (dg_status s = dg::launch(moe_up_kernel<kFp4, NT>, static_cast<unsigned>(ctx.sms), kThreads, up_smem, stream, ctx.pdl, a); s != DG_OK) return s;
  return dg::launch(moe_down_kernel<kFp4, NT>, static_cast<unsigned>(std::min(ctx.sms, a.H / 16)), kThreads, down_smem, stream, ctx.pdl, a);
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
