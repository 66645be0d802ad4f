// Host side of the FP4 x FP4 GEMMs: checks, tensor maps and launches. The kernels are in fp4_gemm.cuh, the choice between
// them in fp4_ways.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "debug_state.h"
#include "dg.h"
#include "fp4_gemm.cuh"
#include "fp4_ways.h"
#include "runtime.h"

namespace {

using dg::LaunchContext;
using dg::fp4::Form;
using dg::fp4::Params;
using dg::fp4::up;

constexpr int kRowBox = dg::fp4::kRows;
static_assert(dg::fp4::kWayStageK == dg::fp4::kStageK, "the estimates' stage");
constexpr int kMaxSize = 1 << 30;          // of a row count, N or K

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Packed codes [G, rows, K / 2], in boxes of 128 bytes of box_rows rows.
bool codes_map(CUtensorMap* m, const void* base, int G, int rows, int K, int box_rows) {
  const uint64_t bytes = static_cast<uint64_t>(K) / 2;
  const uint64_t dims[3] = {bytes, static_cast<uint64_t>(rows), static_cast<uint64_t>(G)}, strides[2] = {bytes, bytes * rows};
  const uint32_t box[3] = {128, static_cast<uint32_t>(box_rows), 1};
  return dg::tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Rows of packed codes four apart: [rows / 4] of every fourth row, then the four, then the groups; in boxes of 32 rows of
// each of `of_four`. Row 4 j + c of a box comes at its row 32 c + j. Rows past the last whole four are not in it.
bool apart_map(CUtensorMap* m, const void* base, int G, int rows, int K, int of_four) {
  const uint64_t bytes = static_cast<uint64_t>(K) / 2;
  const uint64_t dims[4] = {bytes, static_cast<uint64_t>(rows / 4), 4, static_cast<uint64_t>(G)}, strides[3] = {4 * bytes, bytes, bytes * rows};
  const uint32_t box[4] = {128, 32, static_cast<uint32_t>(of_four), 1};
  return dg::tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// D [G, rows, N] the same way, in boxes of 32 columns of 32 rows four apart.
bool out_map(CUtensorMap* m, void* base, int G, int rows, int N) {
  const uint64_t bytes = static_cast<uint64_t>(N) * 2;
  const uint64_t dims[4] = {static_cast<uint64_t>(N), static_cast<uint64_t>(rows / 4), 4, static_cast<uint64_t>(G)}, strides[3] = {4 * bytes, bytes, bytes * rows};
  const uint32_t box[4] = {32, 32, 1, 1};
  return dg::tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B);
}
// All rows, in boxes of every fourth of 128.
bool every_fourth_map(CUtensorMap* m, const void* base, int G, int rows, int K) {
  const uint64_t bytes = static_cast<uint64_t>(K) / 2;
  const uint64_t dims[3] = {bytes, static_cast<uint64_t>(rows), static_cast<uint64_t>(G)}, strides[2] = {bytes, bytes * rows};
  const uint32_t box[3] = {128, 128, 1}, steps[3] = {1, 4, 1};
  return dg::tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B, steps);
}

// Scale words [G, K / 128, ceil4(rows)], in boxes of box_rows rows' two words.
bool scales_map(CUtensorMap* m, const int32_t* base, int G, int rows, int K, int box_rows) {
  const uint64_t w = 4 * ((static_cast<uint64_t>(rows) + 3) / 4), k = static_cast<uint64_t>(K) / 128;
  const uint64_t dims[3] = {w, k, static_cast<uint64_t>(G)}, strides[2] = {4 * w, 4 * w * k};
  const uint32_t box[3] = {static_cast<uint32_t>(box_rows), 2, 1};
  return dg::tensor_map(m, CU_TENSOR_MAP_DATA_TYPE_INT32, 3, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct Operands {
  const void* a;
  const int32_t* sfa;
  const void* b;
  const int32_t* sfb;
};

// kKernel's shared memory is set once per device and host thread.
template <auto kKernel, class... Args>
dg_status launch(int smem, int grid, int threads, int cluster, cudaStream_t stream, bool pdl, const Args&... args) {
  static thread_local int set_on = -1;
  int device = 0;
  if (cudaError_t e = cudaGetDevice(&device); e != cudaSuccess) return dg::record_cuda_error(e);
  if (set_on != device) {
    if (cudaError_t e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); e != cudaSuccess)
      return dg::record_cuda_error(e);
    set_on = device;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kKernel, args...);
  return e == cudaSuccess ? DG_OK : dg::record_cuda_error(e);
}

// pair_rows: 256-row strips of all groups, or a bound of their number.
template <Form kForm, int BN, int kAccum, int kStages, bool kHasC>
dg_status run_pair(const LaunchContext& ctx, const Operands& o, const Params& p, long long pair_rows, cudaStream_t stream) {
  using S = dg::fp4::PairShape<BN, kAccum, kStages, kHasC>;
  const int ga = kForm == Form::Masked ? p.G : 1, gb = kForm == Form::Dense ? 1 : p.G;
  // Only maps that a tile goes by: a host thread keeps 32, which a few products use up. Whole blocks of 128 rows of A and D go
  // by the first and the last of these, A's rows past them by the second.
  CUtensorMap ta, ta_edge, tb, tb_narrow, tsa, tsb, td;
  const bool inner = p.M >= kRowBox, edge = p.M % kRowBox != 0;
  if (inner && (!apart_map(&ta, o.a, ga, p.M, p.K, 4) || !out_map(&td, p.d, ga, p.M, p.N))) return DG_ERR_CUDA;
  if (edge && !every_fourth_map(&ta_edge, o.a, ga, p.M, p.K)) return DG_ERR_CUDA;
  if (!inner) ta = td = ta_edge;
  if (!edge) ta_edge = ta;
  if (S::kWide > 0 && !apart_map(&tb, o.b, gb, p.N, p.K, 4)) return DG_ERR_CUDA;
  if (S::kNarrow && !apart_map(&tb_narrow, o.b, gb, p.N, p.K, 2)) return DG_ERR_CUDA;
  if (S::kWide == 0) tb = tb_narrow;
  if (!S::kNarrow) tb_narrow = tb;
  if (!scales_map(&tsa, o.sfa, ga, p.M, p.K, kRowBox) || !scales_map(&tsb, o.sfb, gb, p.N, p.K, S::kSfBox)) return DG_ERR_CUDA;
  const long long tiles = pair_rows * up(p.N, BN);
  if (tiles > (1ll << 30)) return DG_ERR_UNSUPPORTED;
  const int clusters = static_cast<int>(std::min<long long>(std::max(1, ctx.sms / 2), tiles));
  return launch<dg::fp4::fp4_pair_kernel<kForm, BN, kAccum, kStages, kHasC>>(S::smem(kForm), 2 * clusters, S::kThreads, 2, stream, ctx.pdl, ta,
                ta_edge, tb, tb_narrow, tsa, tsb, td, p);
}

template <int BN, int kStages, int kWays>
dg_status run_split(const LaunchContext& ctx, const Operands& o, Params p, cudaStream_t stream) {
  using S = dg::fp4::SplitShape<BN, kStages>;
  // no more rows of A than there are, in whole swizzle atoms of eight
  const int rows = std::min(kRowBox, 8 * up(std::min(p.M, kRowBox), 8));
  p.a_bytes = static_cast<uint32_t>(rows) * 128;
  CUtensorMap ta, tb, tsa, tsb;
  if (!codes_map(&ta, o.a, 1, p.M, p.K, rows) || !codes_map(&tb, o.b, 1, p.N, p.K, BN) || !scales_map(&tsa, o.sfa, 1, p.M, p.K, kRowBox) ||
      !scales_map(&tsb, o.sfb, 1, p.N, p.K, 128 * S::kChunks))
    return DG_ERR_CUDA;
  const long long grid = static_cast<long long>(up(p.M, kRowBox)) * up(p.N, BN) * kWays;
  if (grid > (1ll << 30)) return DG_ERR_UNSUPPORTED;
  return launch<dg::fp4::fp4_split_kernel<BN, kStages, kWays>>(S::SMEM, static_cast<int>(grid), S::kThreads, kWays, stream, ctx.pdl, ta, tb, tsa, tsb, p);
}

// rows: of A, in each group.
dg_status check(const Operands& o, const void* c, const void* d, int rows, int N, int K) {
  if (rows < 0 || K <= 0 || K % 128 != 0 || N <= 0 || N % 16 != 0) return DG_ERR_INVALID_ARG;
  if (rows > kMaxSize || N > kMaxSize || K > kMaxSize) return DG_ERR_UNSUPPORTED;
  if (rows == 0) return DG_OK;
  if (!o.a || !o.sfa || !o.b || !o.sfb || !d) return DG_ERR_INVALID_ARG;
  if (misaligned(o.a, 16) || misaligned(o.sfa, 16) || misaligned(o.b, 16) || misaligned(o.sfb, 16) || misaligned(c, 16) || misaligned(d, 16))
    return DG_ERR_MISALIGNED;
  return DG_OK;
}

Params params(const LaunchContext& ctx, const void* c, void* d, int M, int N, int K, int G) {
  Params p{};
  p.M = M, p.N = N, p.K = K, p.G = G;
  p.c = static_cast<const __nv_bfloat16*>(c), p.d = static_cast<__nv_bfloat16*>(d);
  p.status = ctx.status, p.timeout_ns = dg::pipeline_wait_timeout_ns(), p.fault = dg::debug_fault_mode();
  return p;
}

// By width; stages as many as shared memory and, of the widest, TMEM hold.
template <Form kForm, bool kHasC>
dg_status run_pair_width(int bn, const LaunchContext& ctx, const Operands& o, const Params& p, long long pair_rows, cudaStream_t stream) {
  constexpr bool kFew = kForm == Form::Masked;      // (its counts take a stage's room)
  if (bn == 384) return run_pair<kForm, 384, 1, 4, kHasC>(ctx, o, p, pair_rows, stream);
  if (bn == 128) return run_pair<kForm, 128, 2, kHasC ? 6 : kFew ? 7 : 8, kHasC>(ctx, o, p, pair_rows, stream);
  return run_pair<kForm, 256, 1, kHasC || kFew ? 5 : 6, kHasC>(ctx, o, p, pair_rows, stream);
}

template <bool kHasC>
dg_status dense(const LaunchContext& ctx, const Operands& o, const Params& p, cudaStream_t stream) {
  const dg::fp4::Way way = dg::fp4::dense_way(p.M, p.N, p.K, ctx.sms);
  if (way.ways == 0) return run_pair_width<Form::Dense, kHasC>(way.bn, ctx, o, p, up(p.M, 256), stream);
  switch (way.bn * 10 + way.ways) {
    case 641: return run_split<64, 6, 1>(ctx, o, p, stream);
    case 642: return run_split<64, 6, 2>(ctx, o, p, stream);
    case 644: return run_split<64, 6, 4>(ctx, o, p, stream);
    case 962: return run_split<96, 6, 2>(ctx, o, p, stream);
    case 1281: return run_split<128, 6, 1>(ctx, o, p, stream);
    case 1282: return run_split<128, 6, 2>(ctx, o, p, stream);
    default: return run_split<192, 5, 1>(ctx, o, p, stream);
  }
}

}  // namespace

extern "C" {

dg_status dg_fp4_gemm_nt(const void* a, const int32_t* sfa, const void* b, const int32_t* sfb, const void* c, void* d, int M, int N, int K,
                         cudaStream_t stream) {
  const Operands o{a, sfa, b, sfb};
  if (dg_status s = check(o, c, d, M, N, K); s != DG_OK || M == 0) return s;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const Params p = params(ctx, c, d, M, N, K, 1);
  return c ? dense<true>(ctx, o, p, stream) : dense<false>(ctx, o, p, stream);
}

dg_status dg_m_grouped_fp4_gemm_nt_contiguous(const void* a, const int32_t* sfa, const void* b, const int32_t* sfb, void* d,
                                              const int32_t* m_indices, int M_total, int N, int K, int G, cudaStream_t stream) {
  const Operands o{a, sfa, b, sfb};
  if (G <= 0) return DG_ERR_INVALID_ARG;
  if (dg_status s = check(o, nullptr, d, M_total, N, K); s != DG_OK || M_total == 0) return s;
  if (!m_indices) return DG_ERR_INVALID_ARG;
  if (misaligned(m_indices, 4)) return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  Params p = params(ctx, nullptr, d, M_total, N, K, G);
  p.m_indices = m_indices;
  // (a bound of the strips' number sizes the grid)
  return run_pair_width<Form::Contiguous, false>(dg::fp4::contiguous_width(M_total, N, K, G, ctx.sms), ctx, o, p, up(M_total, kRowBox), stream);
}

dg_status dg_m_grouped_fp4_gemm_nt_masked(const void* a, const int32_t* sfa, const void* b, const int32_t* sfb, void* d, const int32_t* masked_m,
                                          int G, int max_m, int N, int K, cudaStream_t stream) {
  const Operands o{a, sfa, b, sfb};
  if (G <= 0) return DG_ERR_INVALID_ARG;
  if (dg_status s = check(o, nullptr, d, max_m, N, K); s != DG_OK || max_m == 0) return s;
  if (!masked_m) return DG_ERR_INVALID_ARG;
  if (misaligned(masked_m, 4)) return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  Params p = params(ctx, nullptr, d, max_m, N, K, G);
  p.masked_m = masked_m;
  return run_pair_width<Form::Masked, false>(dg::fp4::masked_width(G, max_m, N, K, ctx.sms), ctx, o, p, static_cast<long long>(G) * up(max_m, 256), stream);
}

}  // extern "C"
