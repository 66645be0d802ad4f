// Products of two FP4 operands for sm_103a: D = C + A @ B.T with A and B in packed E2M1, one UE8M0 scale per row per
// 32 K, on block-scaled tcgen05.mma.kind::mxf4 (K = 64 an instruction, FP32 accumulation in TMEM).
//
// A pipeline stage holds 256 K: rows of 128 bytes in the 128-byte swizzle, and two packed scale words per row. The MMA
// reads the scales of 128 rows from four TMEM columns, row r's word in lane r % 32 of column r / 32, an order that the words
// as they are packed do not have.
//
// Two kernels: fp4_pair_kernel, persistent, a CTA pair to a 256 x BN tile (many rows, and the grouped forms), and
// fp4_split_kernel, a 128 x BN tile to a cluster whose CTAs share out K (few tiles).
//
// Measured on one GB300 (nodes of a CUDA graph, inputs larger than L2): 8 experts, 32768 x 4096 x 7168 282 us (6.8 PFLOP/s,
// 74 % of the tensor pipe, bound by the 36 KB that a stage brings an SM from L2: 52 bytes a clock); 8192 x 8192 x 8192 154 us
// (7.2); 4096 x 24576 x 1536 72 us (4.3; its output, 3.3 us a tile, holds it); masked 32 experts of 0 to 256 rows x 7168 x 2048
// 60 us (5.2 TB/s); 128 x 7168 x 16384 with C 16.9 us (4.0 TB/s).
#pragma once

#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "ptx.cuh"
#include "ue8m0.cuh"

namespace dg {
namespace fp4 {

enum class Form { Dense, Contiguous, Masked };

constexpr int kRows = 128;                 // rows of A of a CTA
constexpr int kStageK = 256;               // K of a stage: 128 bytes of a row, two scale words
constexpr int kCountCache = 1024;          // masked form: counts held in shared memory (more are read at L2)
constexpr unsigned long long kDrainNs = 50000000ull;
enum : int { kFaultProducerSilent = 1 };

struct Params {
  int M, N, K, G;                          // M: rows of A, of each group in the masked form
  const int32_t* m_indices;                // contiguous form
  const int32_t* masked_m;                 // masked form
  const __nv_bfloat16* c;
  __nv_bfloat16* d;
  uint32_t a_bytes;                        // split kernel: bytes of A that a stage loads
  uint32_t* status;
  unsigned long long timeout_ns;
  int fault;
};

__host__ __device__ constexpr int up(int a, int b) { return (a + b - 1) / b; }

// Instruction descriptor of kind::mxf4: A and B E2M1 (1 in bits 7 and 10), N / 8 in bits 17 on, UE8M0 scales (bit 23),
// M / 128 in bits 27 on; bits 4 and 29 take the first of the two scale bytes (0 or 2) that B and A use of their words.
__host__ __device__ constexpr uint32_t instruction(uint32_t M, uint32_t N) {
  return 1u << 7 | 1u << 10 | (N >> 3) << 17 | 1u << 23 | (M >> 7) << 27;
}

template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (kPair)
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
  else
    asm volatile(
        "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%5], [%6], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
        : "memory");
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint64_t timeout_ns, volatile uint32_t* abort_flag) {
  return __all_sync(0xffffffffu, *abort_flag == 0 && mbar_wait(bar, parity, timeout_ns));
}

// Turns kChunks x 128 scale words from the order of their rows into the order of tcgen05.cp, in place, by a warp: the
// words of rows l, l + 32, l + 64 and l + 96 to the 16 bytes of lane l. The split kernel's way, whose tiles need not be 128
// columns wide and whose CTAs each have their own words: about a fifth of a stage, in a warp of its own.
template <int kChunks>
__device__ __forceinline__ void arrange_scales(uint32_t at, uint32_t lane) {
  uint32_t w[kChunks][4];
#pragma unroll
  for (int c = 0; c < kChunks; ++c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[c][i] = ld_shared_u32(at + 512 * c + 4 * (lane + 32 * i));
  }
  __syncwarp();
#pragma unroll
  for (int c = 0; c < kChunks; ++c) st_shared_v4(at + 512 * c + 16 * lane, w[c][0], w[c][1], w[c][2], w[c][3]);
}

// A warp's pieces of D, of 32 rows of 32 columns, a row of the accumulator in each lane. A piece goes through 2 KB of
// shared memory, from where it leaves by TMA, or, where not all of its rows are written, in runs of 64 bytes, eight rows
// at a time. C comes the same way, in runs, the copies of two pieces on their way at once. Row i of a piece is row kStep i
// of D from d0's; lane l reads and writes 16 bytes of rows l / 4 + 8 r.
constexpr int kPieceBytes = 32 * 64;
template <int kStep, bool kHasC>
struct Pieces {
  static constexpr int kBytes = (kHasC ? 3 : 1) * kPieceBytes;
  const Params& p;
  uint32_t smem, lane, live;               // live: rows that are written
  int n0;                                  // first column of the tile
  size_t d0;                               // of row lane / 4, at column n0 + 8 (lane % 4)

  __device__ __forceinline__ size_t at(int r, int col) const { return d0 + static_cast<size_t>(8 * kStep * r) * p.N + col; }
  __device__ __forceinline__ bool mine(int r, int col) const {
    return (live >> (lane / 4 + 8 * r) & 1) && n0 + col + 8 * static_cast<int>(lane % 4) < p.N;
  }
  // 16-byte unit u of row r of a buffer (0: D's), in the 64-byte swizzle
  __device__ __forceinline__ uint32_t unit(int buffer, int r, int u) const {
    return smem + buffer * kPieceBytes + r * 64 + ((u ^ (r >> 1 & 3)) << 4);
  }
  // Begins to copy C of a piece of the i-th's parity, at column col of the tile: of the first two before the first is
  // written, of piece i + 2 after piece i is.
  __device__ __forceinline__ void fetch(int i, int col) const {
    if constexpr (kHasC) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (mine(r, col)) cp_async_16(unit(1 + (i & 1), lane / 4 + 8 * r, lane % 4), p.c + at(r, col));
      cp_async_commit();
    }
  }
  // Writes the i-th of `count` pieces, at column col. value(j): column j of this lane's row. tma(): sends the piece, if `whole`.
  template <class Value, class Tma>
  __device__ __forceinline__ void write(int i, int count, int col, bool whole, Value value, Tma tma) const {
    const int row = lane, own = lane % 4, first = lane / 4;
    if (lane == 0) bulk_wait_group_read<0>();      // the last piece has left
    if constexpr (kHasC) {
      if (i + 1 < count)
        cp_async_wait<1>();
      else
        cp_async_wait<0>();
    }
    __syncwarp();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(value(8 * u + e));
      if constexpr (kHasC) {
        const uint4 cv = ld_shared_v4(unit(1 + (i & 1), row, u));
        const uint32_t cw[4] = {cv.x, cv.y, cv.z, cv.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x, y;
          unpack_bf16(cw[e], x, y);
          f[2 * e] += x, f[2 * e + 1] += y;
        }
      }
      st_shared_v4(unit(0, row, u), pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
    if (whole) fence_proxy_async_smem();
    __syncwarp();
    if (whole) {
      if (lane == 0) {
        tma();
        bulk_commit_group();
      }
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint4 w = ld_shared_v4(unit(0, first + 8 * r, own));
        if (mine(r, col)) st_global_v4(p.d + at(r, col), w.x, w.y, w.z, w.w);
      }
      __syncwarp();
    }
  }
};

// ------------------------------------------------------------------------------------
// CTA pairs
// ------------------------------------------------------------------------------------
// The scales go from global memory to TMEM as they are: 128 words of consecutive rows, of which tcgen05.cp gives lane j
// the four of rows 4 j .. 4 j + 3. So the rows are put where their scales are: row 32 c + j of an MMA's operand is row
// 4 j + c of the tile. TMA loads them in that order, through a map that takes four rows apart ([rows / 4] of every
// fourth row, then the four); a lane of the accumulator is row 4 lane + quadrant, and its columns 32 c + j, c = 0 .. 3,
// are columns 4 j + c of D. Rows of A past the last whole four go by a second map, of every fourth row from a given one.
template <int kBN, int kAccums, int kStages_, bool kHasC>
struct PairShape {
  static constexpr int BN = kBN, kAccum = kAccums, kStages = kStages_;
  static constexpr int kEpilogueWarps = 8, kThreads = (4 + kEpilogueWarps) * 32;
  static constexpr int kChunks = BN / 128;                          // of 128 scale words of B
  static constexpr int A_BYTES = kRows * 128, B_BYTES = BN / 2 * 128;
  static constexpr int SFA_BYTES = 2 * 512, SFB_BYTES = 2 * kChunks * 512, SF_BYTES = SFA_BYTES + SFB_BYTES;
  static constexpr int EPI_BYTES = Pieces<4, kHasC>::kBytes;        // of a warp
  static constexpr int OFF_B = kStages * A_BYTES, OFF_SF = OFF_B + kStages * B_BYTES, OFF_EPI = OFF_SF + kStages * SF_BYTES;
  static constexpr int OFF_BAR = OFF_EPI + kEpilogueWarps * EPI_BYTES;
  // TMEM: the accumulators, then a buffer of scales for each stage
  static constexpr int kSfCols = 8 + 8 * kChunks;
  static_assert(BN % 128 == 0 && BN <= 384 && kAccum * BN + kStages * kSfCols <= 512, "TMEM columns");
  // B's columns by MMAs of 256, of which a CTA loads 128 rows, and a last one of 128 where BN has it, of which it loads 64
  static constexpr int kWide = BN / 256;
  static constexpr bool kNarrow = BN % 256 != 0;
  // scale words of B: a copy has both words of up to 256 rows
  static constexpr int kSfBox = BN <= 256 ? BN : 128;
  static constexpr int kBars = 3 * kStages + 2 * kAccum + 2;
  static constexpr int OFF_COUNTS = OFF_BAR + kBars * 8 + 16;
  static constexpr int smem(Form f) { return OFF_COUNTS + (f == Form::Masked ? kCountCache * 4 : 0); }
};

// A tile: the pair's rows from m0 in its group's rows of A, `valid` of them (may be more than the tile has); its columns
// from n0; the group of A and D, and of B.
struct Tile {
  int m0, valid, n0, ga, gb;
};

// The tiles of cluster `t`, t + step, ...: every role of a CTA, a whole warp each, walks the same ones.
template <Form kForm, int BN>
struct Walk {
  int t, step, total, num_n;
  int g = 0, first = 0, tiles = 0;         // masked form: the group that t is in, its first tile and its tiles
  // contiguous form, of the 32 blocks of 128 rows from `chunk`: a lane's block's expert, and how many of it and the next
  // are its expert's; the blocks that begin a tile, and how many do before the chunk; the expert before the chunk, and
  // whether an odd number of blocks of its run are before it
  int chunk = -32, expert_of = -1, own = 0, before = 0, last = -1, odd = 0;
  uint32_t begins = 0;
  const int* counts;

  __device__ __forceinline__ Walk(const Params& p, const int* counts_) : counts(counts_) {
    t = blockIdx.x / 2;
    step = gridDim.x / 2;
    num_n = up(p.N, BN);
    total = up(p.M, 2 * kRows) * num_n;
    if (kForm == Form::Masked) tiles = tiles_of(p, 0);
  }
  __device__ __forceinline__ int count(const Params& p, int group) const {
    return group < kCountCache ? counts[group] : min(max(ld_cg_s32(p.masked_m + group), 0), p.M);
  }
  __device__ __forceinline__ int tiles_of(const Params& p, int group) const { return up(count(p, group), 2 * kRows) * num_n; }
  // The expert of a block of 128 rows, by its first row; -1 where it is to be skipped.
  __device__ __forceinline__ int expert(const Params& p, int block) const {
    const int e = block < up(p.M, kRows) ? ld_cg_s32(p.m_indices + block * kRows) : -1;
    if (e < -1 || e >= p.G) atomicOr(p.status, kBadIndexBit);
    return e < p.G ? e : -1;
  }
  // Looks at the next 32 blocks. Two neighbouring blocks of an expert are a tile, counted from the first block of its run.
  __device__ __forceinline__ void next_chunk(const Params& p) {
    const int lane = static_cast<int>(lane_id());
    before += __popc(begins);
    chunk += 32;
    expert_of = expert(p, chunk + lane);
    int prev = __shfl_up_sync(0xffffffffu, expert_of, 1), after = __shfl_down_sync(0xffffffffu, expert_of, 1);
    if (lane == 0) prev = last;
    if (lane == 31) after = expert(p, chunk + 32);
    own = after == expert_of ? 2 : 1;
    const uint32_t runs = __ballot_sync(0xffffffffu, expert_of >= 0 && expert_of != prev) & (0xffffffffu >> (31 - lane));
    const int place = runs ? lane - (31 - __clz(runs)) : lane + odd;       // in its run
    begins = __ballot_sync(0xffffffffu, expert_of >= 0 && place % 2 == 0);
    last = __shfl_sync(0xffffffffu, expert_of, 31);
    odd = (__shfl_sync(0xffffffffu, place, 31) + 1) & 1;
  }

  __device__ __forceinline__ bool next(const Params& p, Tile& s) {
    if constexpr (kForm == Form::Masked) {
      while (t - first >= tiles) {
        first += tiles;
        if (++g >= p.G) return false;
        tiles = tiles_of(p, g);
      }
      // pair rows of the same columns one after the other: they share B's rows
      const int local = t - first, pairs = tiles / num_n;
      s = {local % pairs * 2 * kRows, 0, local / pairs * BN, g, g};
      s.valid = count(p, g) - s.m0;
    } else if constexpr (kForm == Form::Dense) {
      if (t >= total) return false;
      s = {t / num_n * 2 * kRows, 0, t % num_n * BN, 0, 0};
      s.valid = p.M - s.m0;
    } else {
      const int want = t / num_n;
      while (before + __popc(begins) <= want) {
        if (chunk + 32 >= up(p.M, kRows)) return false;
        next_chunk(p);
      }
      uint32_t left = begins;
      for (int i = before; i < want; ++i) left &= left - 1;
      const int at = __ffs(left) - 1;
      s = {(chunk + at) * kRows, __shfl_sync(0xffffffffu, own, at) * kRows, t % num_n * BN, 0, __shfl_sync(0xffffffffu, expert_of, at)};
    }
    t += step;
    return true;
  }
};

// Roles of a CTA (both of a pair run the same code; a warp's loop stays converged and one elected thread issues):
//   warp 0     TMA: its 128 rows of A and their scales, its half of B's rows and all of the tile's scales of B, all counted
//              by the leader's barrier
//   warp 1     (leader) issues the MMAs; allocates TMEM
//   warp 2     (leader) copies both CTAs' scales to TMEM once a stage has arrived, which keeps copies and waits out of
//              the MMA thread's stream
//   warps 4..  epilogue: half of the tile's columns of 32 rows each, from TMEM to registers, and in pieces to D
template <Form kForm, int BN, int kAccum, int kStages, bool kHasC>
__global__ void __launch_bounds__(PairShape<BN, kAccum, kStages, kHasC>::kThreads, 1)
    fp4_pair_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a_edge,
                    const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_b_narrow,
                    const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb,
                    const __grid_constant__ CUtensorMap tm_d, const Params p) {
  using S = PairShape<BN, kAccum, kStages, kHasC>;
  extern __shared__ __align__(1024) uint8_t smem[];   // at a multiple of 1024: nothing static lies before it
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);   // leader: the stage of both CTAs
  uint64_t* const ready = full + kStages;          // leader: its scales are in TMEM
  uint64_t* const empty = ready + kStages;         // both CTAs: its MMAs are done
  uint64_t* const acc_full = empty + kStages;      // both CTAs
  uint64_t* const acc_empty = acc_full + kAccum;   // leader: epilogue warps of both CTAs
  uint64_t* const drain = acc_empty + kAccum;      // MMA thread, copying thread
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile uint32_t* const abort_flag = tmem_slot + 1;
  int* const counts = reinterpret_cast<int*>(smem + S::OFF_COUNTS);

  const int warp = threadIdx.x / 32;
  const uint32_t lane = threadIdx.x % 32;
  const uint32_t rank = cluster_cta_rank() & 1u;
  const bool leader = rank == 0;
  const int stages_k = up(p.K, kStageK);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < kAccum; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * S::kEpilogueWarps);
    }
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_sfa);
    tma_prefetch_desc(&tm_sfb);
    tma_prefetch_desc(&tm_d);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  grid_dependency_wait();   // programmatic dependent launch: no global access before this
  if constexpr (kForm == Form::Masked) {
    for (int g = threadIdx.x; g < p.G; g += S::kThreads) {
      const int c = ld_cg_s32(p.masked_m + g), in = min(max(c, 0), p.M);
      if (c != in && blockIdx.x == 0) atomicOr(p.status, kBadIndexBit);
      if (g < kCountCache) counts[g] = in;
    }
  }
  __syncthreads();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto on_timeout = [&]() {
    atomicOr(p.status, kTimeoutBit);
    *abort_flag = 1;
  };
  Walk<kForm, BN> walk(p, counts);
  Tile tile;
  uint32_t stage = 0, phase = 0;
  auto advance = [&]() {
    if (++stage == kStages) stage = 0, phase ^= 1;
  };

  if (warp == 0) {
    if (p.fault != kFaultProducerSilent) {
      uint32_t issued = 0;
      bool ok = true;
      while (ok && walk.next(p, tile)) {
        const int m0 = tile.m0 + static_cast<int>(rank) * kRows, n0 = tile.n0;
        const bool rows = tile.valid > static_cast<int>(rank) * kRows;      // this CTA has rows of the tile
        const bool inner = m0 + kRows <= (p.M & ~3);
        const uint32_t bytes = (tile.valid > kRows ? 2 : 1) * (S::A_BYTES + S::SFA_BYTES) + 2 * (S::B_BYTES + S::SFB_BYTES);
        for (int kb = 0; kb < stages_k; ++kb) {
          if (!warp_wait(&empty[stage], phase ^ 1, p.timeout_ns, abort_flag)) {
            if (lane == 0) on_timeout();
            ok = false;
            break;
          }
          if (elect_one()) {
            uint8_t* const a = smem + stage * S::A_BYTES;
            uint8_t* const sf = smem + S::OFF_SF + stage * S::SF_BYTES;
            const uint32_t bar = map_to_rank(&full[stage], 0);
            if (leader) mbar_arrive_expect_tx(&full[stage], bytes);
            uint8_t* const b = smem + S::OFF_B + stage * S::B_BYTES;
#pragma unroll
            for (int w = 0; w < S::kWide; ++w)
              tma_load_4d_pair(b + w * 128 * 128, &tm_b, bar, kb * 128, (n0 + 256 * w) / 4 + 32 * static_cast<int>(rank), 0, tile.gb);
            if constexpr (S::kNarrow)
              tma_load_4d_pair(b + S::kWide * 128 * 128, &tm_b_narrow, bar, kb * 128, (n0 + 256 * S::kWide) / 4, 2 * static_cast<int>(rank), tile.gb);
            if (rows) {
              if (inner) {
                tma_load_4d_pair(a, &tm_a, bar, kb * 128, m0 / 4, 0, tile.ga);
              } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) tma_load_3d_pair(a + c * 32 * 128, &tm_a_edge, bar, kb * 128, m0 + c, tile.ga);
              }
              tma_load_3d_pair(sf, &tm_sfa, bar, m0, 2 * kb, tile.ga);
            }
#pragma unroll
            for (int c = 0; c < BN / S::kSfBox; ++c)
              tma_load_3d_pair(sf + S::SFA_BYTES + c * S::kSfBox * 8, &tm_sfb, bar, n0 + c * S::kSfBox, 2 * kb, tile.gb);
          }
          __syncwarp();
          ++issued;
          advance();
        }
      }
      if (lane == 0) {
        grid_launch_dependents();
        // no copy is in flight when the pair leaves
        if (leader)
          for (uint32_t s = 0; s < kStages && s < issued; ++s) mbar_wait(&full[s], (issued - 1 - s) / kStages & 1, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      constexpr uint32_t kWideMma = instruction(2 * kRows, 256), kNarrowMma = instruction(2 * kRows, 128);
      const uint64_t a0 = make_smem_desc(smem_addr(smem), 16, 1024, kLayoutSwizzle128B);
      const uint64_t b0 = make_smem_desc(smem_addr(smem + S::OFF_B), 16, 1024, kLayoutSwizzle128B);
      uint32_t tiles = 0;
      bool ok = true;
      while (ok && walk.next(p, tile)) {
        const uint32_t acc = tiles % kAccum;
        if (!warp_wait(&acc_empty[acc], (tiles / kAccum & 1) ^ 1, p.timeout_ns, abort_flag)) {
          if (lane == 0) on_timeout();
          break;
        }
        const uint32_t d = tmem + acc * BN;
        for (int kb = 0; kb < stages_k; ++kb) {
          if (!warp_wait(&ready[stage], phase, p.timeout_ns, abort_flag)) {
            if (lane == 0) on_timeout();
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint64_t a = a0 + (stage * S::A_BYTES >> 4), b = b0 + (stage * S::B_BYTES >> 4);
            const uint32_t sfa = tmem + kAccum * BN + stage * S::kSfCols, sfb = sfa + 8;
            const bool whole = p.K - kb * kStageK >= kStageK;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= 2 && !whole) break;
              const uint32_t id = 2u * (k & 1), ids = id << 4 | id << 29, sa = sfa + 4 * (k / 2), sb = sfb + 4 * S::kChunks * (k / 2);
#pragma unroll
              for (int w = 0; w < S::kWide; ++w)
                mma<true>(d + 256 * w, a + 2 * k, b + (w * 128 * 128 >> 4) + 2 * k, kWideMma | ids, sa, sb + 8 * w, (kb | k) != 0);
              if constexpr (S::kNarrow)
                mma<true>(d + 256 * S::kWide, a + 2 * k, b + (S::kWide * 128 * 128 >> 4) + 2 * k, kNarrowMma | ids, sa, sb + 8 * S::kWide, (kb | k) != 0);
            }
            tc_commit_pair(&empty[stage]);
            if (kb == stages_k - 1) tc_commit_pair(&acc_full[acc]);
          }
          __syncwarp();
          advance();
        }
        ++tiles;
      }
      // what the elected thread has issued is done before TMEM is handed back
      if (elect_one()) {
        tc_commit_pair(&drain[0]);
        mbar_wait(&drain[0], 0, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 2) {
    if (leader) {
      const uint64_t sf0 = make_smem_desc(smem_addr(smem + S::OFF_SF), 0, 128, kLayoutNone);
      bool ok = true;
      while (ok && walk.next(p, tile)) {
        for (int kb = 0; kb < stages_k; ++kb) {
          // (the stage's TMEM buffer is free: what is in the stage now was loaded after the MMAs that read it)
          if (!warp_wait(&full[stage], phase, p.timeout_ns, abort_flag)) {
            if (lane == 0) on_timeout();
            ok = false;
            break;
          }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t to = tmem + kAccum * BN + stage * S::kSfCols;
            const uint64_t from = sf0 + (stage * S::SF_BYTES >> 4);
#pragma unroll
            for (int c = 0; c < S::SF_BYTES / 512; ++c) {
              // A's two words; then of B, for each copy, the first words of its chunks and the second ones
              constexpr int kIn = S::kSfBox / 128;
              const int x = c - 2, word = x / kIn % 2, chunk = x / (2 * kIn) * kIn + x % kIn;
              tmem_copy_32x128b_warpx4_pair(to + (c < 2 ? 4 * c : 8 + 4 * (word * S::kChunks + chunk)), from + 32 * c);
            }
            tc_commit_pair(&ready[stage]);
          }
          __syncwarp();
          advance();
        }
      }
      if (elect_one()) {
        tc_commit_pair(&drain[1]);
        mbar_wait(&drain[1], 0, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    const int quad = warp % 4, half = (warp - 4) / 4;
    const uint32_t staging = smem_addr(smem + S::OFF_EPI + (warp - 4) * S::EPI_BYTES);
    constexpr int kPieces = BN / 64;                                         // of 32 columns, for each of the two halves
    uint32_t tiles = 0;
    while (walk.next(p, tile)) {
      const int m0 = tile.m0 + static_cast<int>(rank) * kRows;
      const int mine = 4 * static_cast<int>(lane) + quad, r = static_cast<int>(rank) * kRows + mine;   // the row of this lane's accumulators
      bool live = r < tile.valid;
      if constexpr (kForm == Form::Contiguous) {
        if (live) {
          const int expert = m0 + mine < p.M ? ld_cg_s32(p.m_indices + m0 + mine) : -1;
          if (expert != tile.gb && expert != -1 && tile.n0 == 0 && half == 0) atomicOr(p.status, kBadIndexBit);
          live = expert == tile.gb;
        }
      }
      const uint32_t live_rows = __ballot_sync(0xffffffffu, live);
      // (rows past the last whole four are in no four of the map)
      const bool whole = live_rows == 0xffffffffu && m0 + kRows <= (p.M & ~3);
      const Pieces<4, kHasC> d{p, staging, lane, live_rows, tile.n0,
                               (static_cast<size_t>(tile.ga) * p.M + m0 + 4 * (lane / 4) + quad) * p.N + tile.n0 + 8 * (lane % 4)};
      const int col0 = half * kPieces * 32;
      d.fetch(0, col0);
      d.fetch(1, col0 + 32);
      const uint32_t acc = tiles % kAccum;
      if (!warp_wait(&acc_full[acc], tiles / kAccum & 1, p.timeout_ns, abort_flag)) {
        if (lane == 0) on_timeout();
        break;
      }
      ++tiles;
      tc_fence_after();
      const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + acc * BN;
      // one accumulator: all of the warp's share at once (of a 384-wide tile half of it), then it is free; two: piece by piece
      constexpr int kHeld = kAccum > 1 ? 1 : kPieces > 4 ? kPieces / 2 : kPieces;
      static_assert(kPieces % kHeld == 0, "rounds of pieces");
#pragma unroll
      for (int begin = 0; begin < kPieces; begin += kHeld) {
        uint32_t held[kHeld][4][8];
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int col = col0 + 32 * (begin + i);                             // 8 j of each c: columns 128 x + 8 (col / 32 % 4) + j + 32 c
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_load_32x32b_x8(from + col / 128 * 128 + col % 128 / 4 + 32 * c, held[i][c]);
        }
        tmem_load_wait();
        if (begin + kHeld == kPieces) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(map_to_rank(&acc_empty[acc], 0));
        }
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
          const int piece = begin + i, col = col0 + 32 * piece;
          // column n of the piece: j = n / 4 of the eight, c = n % 4
          d.write(piece, kPieces, col, whole, [&](int n) { return held[i][n & 3][n >> 2]; },
                  [&]() { tma_store_4d(&tm_d, staging, tile.n0 + col, m0 / 4, quad, tile.ga); });
          if (piece + 2 < kPieces) d.fetch(piece, col + 64);
        }
      }
    }
    if constexpr (kHasC) cp_async_wait<0>();
    if (lane == 0) bulk_wait_group_all();
  }

  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (*abort_flag) {
    // a peer's copy may still be in flight towards this CTA: let it land
    for (int i = 0; i < 1000; ++i) nanosleep_ns(1000);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------
// few tiles: K shared out over the CTAs of a cluster
// ------------------------------------------------------------------------------------
template <int kBN, int kStages_>
struct SplitShape {
  static constexpr int BN = kBN, kStages = kStages_, kThreads = 256;
  static constexpr int kChunks = up(BN, 128);
  static constexpr int A_BYTES = kRows * 128, B_BYTES = BN * 128;
  static constexpr int SFA_BYTES = 2 * 512, SFB_BYTES = 2 * kChunks * 512, SF_BYTES = SFA_BYTES + SFB_BYTES;
  static constexpr int OFF_B = kStages * A_BYTES, OFF_SF = OFF_B + kStages * B_BYTES, OFF_BAR = OFF_SF + kStages * SF_BYTES;
  static constexpr int kSfCols = 8 + 8 * kChunks, kAccCols = BN <= 128 ? 128 : 256;
  static constexpr int kTmemCols = kAccCols + kStages * kSfCols <= 256 ? 256 : 512;
  static_assert(kAccCols + kStages * kSfCols <= 512, "a TMEM buffer of scales for each stage");
  static constexpr int OFF_MISC = OFF_BAR + (3 * kStages + 1) * 8;
  static constexpr int kLd = BN + 4;                        // floats between the rows of a partial sum
  static_assert(kRows * kLd * 4 <= OFF_SF, "the ring holds a partial sum");
  static constexpr int SMEM = OFF_MISC + 16 + 1024;
};

// A cluster's tile: 128 rows x BN columns, CTA r taking its r-th share of K's stages. The partial sums meet in
// shared memory: CTA r adds up, in the order of ranks, and stores columns [r, r + 1) * BN / kWays.
//   warp 0     TMA      warp 1     copies scales to TMEM and issues the MMAs     warp 2     arranges the scale words
//   warps 4..  TMEM to D (kWays = 1) or to the partial sum
template <int BN, int kStages, int kWays>
__global__ void __launch_bounds__(256, 1)
    fp4_split_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const __grid_constant__ CUtensorMap tm_sfa, const __grid_constant__ CUtensorMap tm_sfb, const Params p) {
  using S = SplitShape<BN, kStages>;
  extern __shared__ uint8_t raw[];
  uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint64_t* const full = reinterpret_cast<uint64_t*>(smem + S::OFF_BAR);
  uint64_t* const ready = full + kStages;          // the scale words are arranged
  uint64_t* const empty = ready + kStages;
  uint64_t* const acc_full = empty + kStages;
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(smem + S::OFF_MISC);
  volatile uint32_t* const abort_flag = tmem_slot + 1;

  const int warp = threadIdx.x / 32;
  const uint32_t lane = threadIdx.x % 32;
  const int rank = static_cast<int>(cluster_cta_rank());
  const int m_tiles = up(p.M, kRows), of = blockIdx.x / kWays;
  const int m0 = of % m_tiles * kRows, n0 = of / m_tiles * BN;
  const int stages_k = up(p.K, kStageK);
  const int k_begin = static_cast<int>(static_cast<long long>(rank) * stages_k / kWays), k_end = static_cast<int>(static_cast<long long>(rank + 1) * stages_k / kWays);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&ready[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
    fence_proxy_async_smem();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_sfa);
    tma_prefetch_desc(&tm_sfb);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  auto on_timeout = [&]() {
    atomicOr(p.status, kTimeoutBit);
    *abort_flag = 1;
  };
  uint32_t stage = 0, phase = 0;
  auto advance = [&]() {
    if (++stage == kStages) stage = 0, phase ^= 1;
  };

  if (warp == 0) {
    if (p.fault != kFaultProducerSilent) {
      uint32_t issued = 0;
      for (int kb = k_begin; kb < k_end; ++kb) {
        if (!warp_wait(&empty[stage], phase ^ 1, p.timeout_ns, abort_flag)) {
          if (lane == 0) on_timeout();
          break;
        }
        if (elect_one()) {
          uint8_t* const sf = smem + S::OFF_SF + stage * S::SF_BYTES;
          mbar_arrive_expect_tx(&full[stage], p.a_bytes + S::B_BYTES + S::SF_BYTES);
          tma_load_3d(smem + S::OFF_B + stage * S::B_BYTES, &tm_b, &full[stage], kb * 128, n0, 0);
          tma_load_3d(smem + stage * S::A_BYTES, &tm_a, &full[stage], kb * 128, m0, 0);
          tma_load_3d(sf + S::SFA_BYTES, &tm_sfb, &full[stage], n0, 2 * kb, 0);
          tma_load_3d(sf, &tm_sfa, &full[stage], m0, 2 * kb, 0);
        }
        __syncwarp();
        ++issued;
        advance();
      }
      if (lane == 0) {
        grid_launch_dependents();
        for (uint32_t s = 0; s < kStages && s < issued; ++s) mbar_wait(&full[s], (issued - 1 - s) / kStages & 1, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t kIdesc = instruction(kRows, BN);
    const uint64_t a0 = make_smem_desc(smem_addr(smem), 16, 1024, kLayoutSwizzle128B);
    const uint64_t b0 = make_smem_desc(smem_addr(smem + S::OFF_B), 16, 1024, kLayoutSwizzle128B);
    const uint64_t sf0 = make_smem_desc(smem_addr(smem + S::OFF_SF), 0, 128, kLayoutNone);
    for (int kb = k_begin; kb < k_end; ++kb) {
      // (the stage's TMEM buffer of scales is free: what is in the stage now was loaded after the MMAs that read it)
      if (!warp_wait(&full[stage], phase, p.timeout_ns, abort_flag) || !warp_wait(&ready[stage], phase, p.timeout_ns, abort_flag)) {
        if (lane == 0) on_timeout();
        break;
      }
      tc_fence_after();
      if (elect_one()) {
        const uint32_t sfa = tmem + S::kAccCols + stage * S::kSfCols, sfb = sfa + 8;
        const uint64_t from = sf0 + (stage * S::SF_BYTES >> 4);
#pragma unroll
        for (int c = 0; c < S::SF_BYTES / 512; ++c) tmem_copy_32x128b_warpx4(sfa + 4 * c, from + 32 * c);
        const uint64_t a = a0 + (stage * S::A_BYTES >> 4), b = b0 + (stage * S::B_BYTES >> 4);
        const bool whole = p.K - kb * kStageK >= kStageK;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t id = 2u * (k & 1);
          if (k < 2 || whole)
            mma<false>(tmem, a + 2 * k, b + 2 * k, kIdesc | id << 4 | id << 29, sfa + 4 * (k / 2), sfb + 4 * S::kChunks * (k / 2), kb != k_begin || k != 0);
        }
        tc_commit(&empty[stage]);
      }
      __syncwarp();
      advance();
    }
    if (elect_one()) {
      tc_commit(acc_full);
      mbar_wait(acc_full, 0, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 2) {
    for (int kb = k_begin; kb < k_end; ++kb) {
      if (!warp_wait(&full[stage], phase, p.timeout_ns, abort_flag)) {
        if (lane == 0) on_timeout();
        break;
      }
      arrange_scales<S::SF_BYTES / 512>(smem_addr(smem + S::OFF_SF + stage * S::SF_BYTES), lane);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ready[stage]);
      advance();
    }
  } else if (warp >= 4) {
    const int quad = warp - 4, row = quad * 32 + static_cast<int>(lane);
    // the MMA thread commits on every path; a wait that ran out elsewhere leaves no whole sum
    const bool ok = warp_wait(acc_full, 0, p.timeout_ns, abort_flag) && __all_sync(0xffffffffu, *abort_flag == 0);
    if (!ok) {
      if (lane == 0) on_timeout();
    } else if (m0 + quad * 32 < p.M) {
      tc_fence_after();
      const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16);
      if constexpr (kWays == 1) {
        // (the ring is idle)
        auto write = [&](auto has_c) {
          const Pieces<1, decltype(has_c)::value> d{p, smem_addr(smem) + quad * Pieces<1, true>::kBytes, lane, __ballot_sync(0xffffffffu, m0 + row < p.M), n0,
                                                    static_cast<size_t>(m0 + quad * 32 + lane / 4) * p.N + n0 + 8 * (lane % 4)};
          d.fetch(0, 0);
          d.fetch(1, 32);
#pragma unroll
          for (int piece = 0; piece < BN / 32; ++piece) {
            uint32_t v[32];
            tmem_load_32x32b_x32(from + 32 * piece, v);
            tmem_load_wait();
            d.write(piece, BN / 32, 32 * piece, false, [&](int at) { return v[at]; }, []() {});
            if (piece + 2 < BN / 32) d.fetch(piece, 32 * piece + 64);
          }
        };
        if (p.c)
          write(std::true_type());
        else
          write(std::false_type());
      } else {
        float* const partial = reinterpret_cast<float*>(smem) + row * S::kLd;
#pragma unroll
        for (int piece = 0; piece < BN / 32; ++piece) {
          uint32_t v[32];
          tmem_load_32x32b_x32(from + 32 * piece, v);
          tmem_load_wait();
          // (rows past the last are sums of whatever lay in shared memory: no one reads them)
#pragma unroll
          for (int i = 0; i < 32; i += 4) st_shared_v4(smem_addr(partial + 32 * piece + i), v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  if constexpr (kWays > 1) {
    cluster_sync();
    constexpr int kWidth = BN / kWays, kPer = kWidth / 8, kItems = up(kRows * kPer, S::kThreads);
    static_assert(kWidth % 8 == 0, "columns of a CTA");
    const int rows = min(p.M - m0, kRows);
    if (*abort_flag == 0) {
      // every load is in flight before the first sum
      uint4 part[kItems][kWays][2], c[kItems];
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int item = i * S::kThreads + static_cast<int>(threadIdx.x), r = item / kPer, col = rank * kWidth + item % kPer * 8;
        if (r >= rows || n0 + col >= p.N) continue;
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
          const uint32_t from = map_to_rank(reinterpret_cast<float*>(smem) + r * S::kLd + col, w);
          part[i][w][0] = ld_shared_cluster_v4(from), part[i][w][1] = ld_shared_cluster_v4(from + 16);
        }
        if (p.c) c[i] = ld_cg_v4(p.c + static_cast<size_t>(m0 + r) * p.N + n0 + col);
      }
#pragma unroll
      for (int i = 0; i < kItems; ++i) {
        const int item = i * S::kThreads + static_cast<int>(threadIdx.x), r = item / kPer, col = rank * kWidth + item % kPer * 8;
        if (r >= rows || n0 + col >= p.N) continue;
        float v[8] = {};
#pragma unroll
        for (int w = 0; w < kWays; ++w) {
          const uint4 lo = part[i][w][0], hi = part[i][w][1];
          v[0] += __uint_as_float(lo.x), v[1] += __uint_as_float(lo.y), v[2] += __uint_as_float(lo.z), v[3] += __uint_as_float(lo.w);
          v[4] += __uint_as_float(hi.x), v[5] += __uint_as_float(hi.y), v[6] += __uint_as_float(hi.z), v[7] += __uint_as_float(hi.w);
        }
        if (p.c) {
          const uint32_t cw[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x, y;
            unpack_bf16(cw[j], x, y);
            v[2 * j] += x, v[2 * j + 1] += y;
          }
        }
        st_global_v4(p.d + static_cast<size_t>(m0 + r) * p.N + n0 + col, pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                     pack_bf16(v[6], v[7]));
      }
    }
    cluster_sync();     // no CTA leaves while another reads its sums
  } else {
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

}  // namespace fp4
}  // namespace dg
