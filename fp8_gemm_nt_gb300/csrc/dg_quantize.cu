// Quantisation to E2M1 with one UE8M0 scale per row per 32 columns, alone and behind the gate of a
// SwiGLU, and the gate's gradient.
//
//   y   = x, or silu(gate) * up of rows (gate | up),          silu(v) = v / (1 + exp(-v))
//   e_b = the least code in [1, 254] with max|y_b| <= 6 * 2^(e_b - 127) in block b of 32 columns; 127 for zeros
//   q   = E2M1(y * 2^(127 - e_b)), to nearest, ties to the even code
//
// E2M1 has no NaN and no infinity: a block that holds one gets the scale code 255 (NaN) and codes 0.
//
// Bound by HBM where there are many rows: 32768 x 7168 BF16 take 100 us (5.9 TB/s), 32768 x 4096 gated ones 96 (6.3), the
// gradient of 8192 x 2048 26 (6.5). Fewer are gone before the loads of enough warps overlap: 8192 x 7168 28 us (5.3), 8192 x
// 2048 gated 15 (5.1). A warp takes a tile of 256 columns: every access of x is 512 contiguous bytes, all of them are in
// flight before the first is used, and the tile's scale words leave together, by column. The largest magnitude of a block
// is found among the bits of x, two BF16 values at once (124 us with float maxima, scale words joined by shuffles and 512
// columns a warp, which left half as many warps room).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "dg.h"
#include "ptx.cuh"
#include "runtime.h"
#include "ue8m0.cuh"

namespace {

using dg::LaunchContext;

constexpr int kWarps = 4;                    // tiles per block
constexpr int kTileCols = 256;
// Rows of a tile: 8, whose scale words are whole 32-byte sectors, where that leaves registers for 32 warps an SM (plain BF16
// rows: 100 us against 111 with 4, at 32768 x 7168), else 4 (FP32 rows: 21.7 us against 26.8, at 4096 x 7168; gated ones: 14.9
// against 17.5, at 8192 x 2048, and 96 against 99, at 32768 x 4096).
template <class T, bool kGate>
constexpr int kRowsOf = kGate || sizeof(T) == 4 ? 4 : 8;
constexpr uint32_t kAll = 0xFFFFFFFFu;

struct QuantArgs {
  const void* x;
  const int32_t* masked_m;
  uint8_t* q;
  int32_t* sf;
  uint32_t* status;
  uint32_t tiles, row_tiles, col_tiles;
  int M, K, sf_rows;
  size_t ldx, ldg;
};

// Rows of expert g that count, as the masked GEMMs take them.
__device__ __forceinline__ int rows_of(const int32_t* masked_m, int g, int M, uint32_t* status) {
  if (!masked_m) return M;
  const int c = __ldcg(masked_m + g);
  if (c < 0 || c > M) atomicOr(status, dg::kBadIndexBit);
  return min(max(c, 0), M);
}

// Least code e in [1, 254] with amax <= 6 * 2^(e - 127): 6 = 1.5 * 2^2, so the exponent of amax less 2, one more if
// the mantissa is above 0.5 = 0x400000 / 2^23, which is when adding 0x3FFFFF carries into the exponent. 127 for 0,
// 255 for an infinity or NaN.
__device__ __forceinline__ int code_for(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return 255;
  const int e = static_cast<int>((amax_bits + 0x3FFFFFu) >> 23) - 2;
  return amax_bits == 0 ? 127 : max(e, 1);
}

// Four floats -> four E2M1 codes, the first in the low four bits; to nearest, ties to the even code.
__device__ __forceinline__ uint32_t pack_e2m1(float a, float b, float c, float d) {
  uint16_t w;
  asm("{\n.reg .b8 lo, hi;\ncvt.rn.satfinite.e2m1x2.f32 lo, %2, %1;\ncvt.rn.satfinite.e2m1x2.f32 hi, %4, %3;\nmov.b16 %0, {lo, hi};\n}"
      : "=h"(w)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return w;
}

// 2^7 / (1 + exp(-g)) of two gates, and 0 where exp(-g) passes 2^133 (g < -92.2, where silu is below FP32's normal numbers):
// the reciprocal of 1 + exp(-g) itself would be flushed from 2^126 on, gates of -87.5, where silu is not small yet. Off by the
// exponent's rounding: 2^-18 of itself at the farthest gates, 2^-21 at gates within 10, which FP4 and BF16 do not see.
// Sums and products of two floats to an instruction: 32768 x 4096 gated rows 96.1 us, by single ones 105.7, and 102.5 without
// the shift.
constexpr float kUnshift = 1.0f / 128;
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 sigmoid_shifted(float2 g) {
  const float2 e = __ffma2_rn(g, both(-dg::kLog2e), both(-7.0f));
  const float2 d = __fadd2_rn(make_float2(dg::exp2_fast(e.x), dg::exp2_fast(e.y)), both(kUnshift));
  return make_float2(dg::reciprocal(d.x), dg::reciprocal(d.y));
}
// (a BF16 gate times 2^-7 is exact)
__device__ __forceinline__ float2 silu(float2 g) { return __fmul2_rn(__fmul2_rn(g, both(kUnshift)), sigmoid_shifted(g)); }

// The columns of 16 bytes of x.
template <class T>
constexpr int kPiece = 16 / sizeof(T);

__device__ __forceinline__ void unpack(const uint4& u, float (&v)[8]) {
  dg::unpack_bf16(u.x, v[0], v[1]);
  dg::unpack_bf16(u.y, v[2], v[3]);
  dg::unpack_bf16(u.z, v[4], v[5]);
  dg::unpack_bf16(u.w, v[6], v[7]);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[4]) {
  v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
}

// A warp's tile: of group g, rows from row0 and columns from col0.
struct Tile {
  int g, row0, col0;
};
__device__ __forceinline__ Tile tile_of(uint32_t tile, uint32_t row_tiles, uint32_t col_tiles, int rows, int cols) {
  const uint32_t rest = tile / col_tiles;
  return {static_cast<int>(rest / row_tiles), static_cast<int>(rest % row_tiles) * rows, static_cast<int>(tile % col_tiles) * cols};
}

// The largest magnitude of 16 bytes, as bits that a block's are compared by: NaN above infinity above the rest.
__device__ __forceinline__ uint32_t magnitude(const uint4& u, const float (&)[8]) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu), __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}
template <int V>
__device__ __forceinline__ uint32_t magnitude(const float (&v)[V]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

// T: type of x. kGate: x has 2 K columns, and y = silu(gate) * up.
template <class T, bool kGate>
__global__ void __launch_bounds__(kWarps * 32) quantize_kernel(const QuantArgs a) {
  constexpr int V = kPiece<T>, kChunk = 32 * V, kChunks = kTileCols / kChunk;   // a chunk: one access of the warp
  constexpr int kBlockLanes = 32 / V, kTileRows = kRowsOf<T, kGate>;            // lanes of a scale
  __shared__ __align__(8) uint8_t codes_of[kWarps][kTileRows][kTileCols / 32];  // the tile's scale codes
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const uint32_t tile = blockIdx.x * kWarps + warp;
  if (tile >= a.tiles) return;
  const Tile t = tile_of(tile, a.row_tiles, a.col_tiles, kTileRows, kTileCols);
  const int valid = rows_of(a.masked_m, t.g, a.M, a.status), rows = valid - t.row0;
  const T* const x = static_cast<const T*>(a.x) + t.g * a.ldg + t.row0 * a.ldx + t.col0 + lane * V;
  uint8_t* const q = a.q + ((static_cast<size_t>(t.g) * a.M + t.row0) * a.K + t.col0 + lane * V) / 2;
  uint4 in[kChunks][kTileRows], up[kGate ? kChunks : 1][kGate ? kTileRows : 1];
#pragma unroll
  for (int r = 0; r < kTileRows; ++r) {
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (r < rows && t.col0 + c * kChunk + lane * V < a.K) {
        const T* at = x + r * a.ldx + c * kChunk;
        in[c][r] = __ldcg(reinterpret_cast<const uint4*>(at));
        if constexpr (kGate) up[c][r] = __ldcg(reinterpret_cast<const uint4*>(at + a.K));
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kTileRows; ++r) {
    if (r >= rows) break;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const bool live = t.col0 + c * kChunk + lane * V < a.K;
      float v[V];
      uint32_t top;
      unpack(in[c][r], v);
      if constexpr (kGate) {
        float u[V];
        unpack(up[c][r], u);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
          const float2 y = __fmul2_rn(silu(make_float2(v[i], v[i + 1])), make_float2(u[i], u[i + 1]));
          v[i] = y.x, v[i + 1] = y.y;
        }
      }
      if constexpr (V == 8 && !kGate)
        top = magnitude(in[c][r], v);
      else
        top = magnitude(v);
      if (!live) top = 0;
#pragma unroll
      for (int o = 1; o < kBlockLanes; o <<= 1) top = max(top, __shfl_xor_sync(kAll, top, o));
      const int e = code_for(top);
      const float by = dg::ue8m0_inverse(min(e, 254));
      uint32_t codes = 0;
#pragma unroll
      for (int i = 0; i < V; i += 4) codes |= pack_e2m1(v[i] * by, v[i + 1] * by, v[i + 2] * by, v[i + 3] * by) << (4 * i);
      if (e == 255) codes = 0;
      if (live) {
        uint8_t* const to = q + (static_cast<size_t>(r) * a.K + c * kChunk) / 2;
        if constexpr (V == 8)
          *reinterpret_cast<uint32_t*>(to) = codes;
        else
          *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(codes);
      }
      if (lane % kBlockLanes == 0) codes_of[warp][r][c * (kChunk / 32) + lane / kBlockLanes] = static_cast<uint8_t>(e);
    }
  }
  __syncwarp();
  // lane l: the word of row l % 8 and the l / 8-th 128 columns, so that words leave in whole sectors
  const int row = t.row0 + lane % kTileRows, group = lane / kTileRows;
  const bool padding = row >= a.M;
  if (group < kTileCols / 128 && t.col0 / 128 + group < a.K / 128 && row < a.sf_rows && (row < valid || padding))
    a.sf[(static_cast<size_t>(t.g) * (a.K / 128) + t.col0 / 128 + group) * a.sf_rows + row] =
        padding ? 0 : *reinterpret_cast<const int32_t*>(&codes_of[warp][lane % kTileRows][4 * group]);
}

struct SwigluGradArgs {
  const __nv_bfloat16* x;
  const __nv_bfloat16* dy;
  __nv_bfloat16* dx;
  const int32_t* masked_m;
  uint32_t* status;
  uint32_t tiles, row_tiles, col_tiles;
  int M, K;
  size_t ldx, ldg;
};
constexpr int kGradRows = 4, kGradCols = 256;

// With s = 1 / (1 + exp(-g)): dgate = dy * up * s * (1 + g * (1 - s)), dup = dy * g * s. A warp takes 4 rows of 256
// columns, a lane 16 bytes of each; it writes what it alone has read, so dx may be x.
__global__ void __launch_bounds__(kWarps * 32) swiglu_grad_kernel(const SwigluGradArgs a) {
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const uint32_t tile = blockIdx.x * kWarps + threadIdx.x / 32;
  if (tile >= a.tiles) return;
  const Tile t = tile_of(tile, a.row_tiles, a.col_tiles, kGradRows, kGradCols);
  const int col = t.col0 + (threadIdx.x & 31) * 8;
  const int rows = min(rows_of(a.masked_m, t.g, a.M, a.status) - t.row0, kGradRows);
  if (col >= a.K) return;
  const __nv_bfloat16* const x = a.x + t.g * a.ldg + t.row0 * a.ldx + col;
  const size_t row0 = static_cast<size_t>(t.g) * a.M + t.row0;
  uint4 wg[kGradRows], wu[kGradRows], wd[kGradRows];
#pragma unroll
  for (int r = 0; r < kGradRows; ++r) {
    if (r < rows) {
      wg[r] = __ldcg(reinterpret_cast<const uint4*>(x + r * a.ldx));
      wu[r] = __ldcg(reinterpret_cast<const uint4*>(x + r * a.ldx + a.K));
      wd[r] = __ldcg(reinterpret_cast<const uint4*>(a.dy + (row0 + r) * a.K + col));
    }
  }
#pragma unroll
  for (int r = 0; r < kGradRows; ++r) {
    if (r >= rows) break;
    float gate[8], up[8], d[8];
    unpack(wg[r], gate);
    unpack(wu[r], up);
    unpack(wd[r], d);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      // (dy times the gate or up first would pass FP32's range where the gradient does not: 0 times infinity at a gate that
      // is masked by its type's lowest value)
      const float2 g = make_float2(gate[i], gate[i + 1]), u = make_float2(up[i], up[i + 1]), dy = make_float2(d[i], d[i + 1]);
      const float2 s = sigmoid_shifted(g), rest = __ffma2_rn(s, both(-kUnshift), both(1.0f));
      const float2 slope = __fmul2_rn(__fmul2_rn(__ffma2_rn(g, rest, both(1.0f)), both(kUnshift)), s);
      const float2 dgate = __fmul2_rn(__fmul2_rn(dy, slope), u), dup = __fmul2_rn(dy, __fmul2_rn(__fmul2_rn(g, both(kUnshift)), s));
      gate[i] = dgate.x, gate[i + 1] = dgate.y;
      up[i] = dup.x, up[i + 1] = dup.y;
    }
    __nv_bfloat16* const to = a.dx + (row0 + r) * 2 * a.K + col;
    *reinterpret_cast<uint4*>(to) = make_uint4(dg::pack_bf16(gate[0], gate[1]), dg::pack_bf16(gate[2], gate[3]),
                                               dg::pack_bf16(gate[4], gate[5]), dg::pack_bf16(gate[6], gate[7]));
    *reinterpret_cast<uint4*>(to + a.K) = make_uint4(dg::pack_bf16(up[0], up[1]), dg::pack_bf16(up[2], up[3]),
                                                     dg::pack_bf16(up[4], up[5]), dg::pack_bf16(up[6], up[7]));
  }
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Strides that an extent of one leaves unread.
size_t row_stride(const dg_rows_desc& d, int per_row) { return d.M > 1 ? d.ldx : static_cast<size_t>(d.K) * per_row; }
size_t group_stride(const dg_rows_desc& d) { return d.G > 1 ? d.ldg : 0; }

// per_row: columns of x for each one of the result.
dg_status check(const void* x, const int32_t* masked_m, const void* q, const int32_t* sf, const dg_rows_desc* desc, int per_row) {
  if (!desc) return DG_ERR_INVALID_ARG;
  const auto [G, M, K, ldx, ldg, x_type] = *desc;
  if (G <= 0 || M < 0 || K <= 0 || K % 128 != 0 || (x_type != DG_BF16 && x_type != DG_F32)) return DG_ERR_INVALID_ARG;
  if (per_row == 2 && x_type != DG_BF16) return DG_ERR_INVALID_ARG;
  if (K > (1 << 30) / per_row || M > 0x7FFFFFF0) return DG_ERR_UNSUPPORTED;
  if (M == 0) return DG_OK;
  if (row_stride(*desc, per_row) < static_cast<size_t>(K) * per_row) return DG_ERR_INVALID_ARG;
  if (!x || !q || !sf) return DG_ERR_INVALID_ARG;
  const size_t size = x_type == DG_BF16 ? 2 : 4;
  if (misaligned(x, 16) || misaligned(q, 16) || misaligned(sf, 16) || misaligned(masked_m, 4)) return DG_ERR_MISALIGNED;
  if (row_stride(*desc, per_row) * size % 16 != 0 || group_stride(*desc) * size % 16 != 0) return DG_ERR_MISALIGNED;
  return DG_OK;
}

// The warps' tiles of G x M rows of K columns.
struct Tiles {
  uint32_t all, row, col;
  bool count(const dg_rows_desc& d, int rows, int cols) {
    row = static_cast<uint32_t>((d.M - 1) / rows + 1);
    col = static_cast<uint32_t>((d.K - 1) / cols + 1);
    const unsigned long long n = static_cast<unsigned long long>(row) * col;      // below 2^32 * 2^22
    all = static_cast<uint32_t>(n * d.G);
    return n <= (1ull << 32) && n * d.G <= 0xFFFFFF00ull;
  }
  unsigned blocks() const { return static_cast<unsigned>((static_cast<unsigned long long>(all) + kWarps - 1) / kWarps); }
};

template <bool kGate>
dg_status quantize(const void* x, const int32_t* masked_m, void* q, int32_t* sf, const dg_rows_desc* desc, cudaStream_t stream) {
  constexpr int kPerRow = kGate ? 2 : 1;
  if (dg_status s = check(x, masked_m, q, sf, desc, kPerRow); s != DG_OK) return s;
  if (desc->M == 0) return DG_OK;
  auto run = [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    // (4 divides the tile's rows, so the padding rows of sf are within the last tile)
    Tiles n;
    if (!n.count(*desc, kRowsOf<T, kGate>, kTileCols)) return DG_ERR_UNSUPPORTED;
    LaunchContext ctx;
    if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
    const QuantArgs a{x, masked_m, static_cast<uint8_t*>(q), sf, ctx.status, n.all, n.row, n.col, desc->M, desc->K,
                      desc->M + (4 - desc->M % 4) % 4, row_stride(*desc, kPerRow), group_stride(*desc)};
    return dg::launch(quantize_kernel<T, kGate>, n.blocks(), kWarps * 32, 0, stream, ctx.pdl, a);
  };
  if constexpr (!kGate)
    if (desc->x_type == DG_F32) return run(static_cast<float*>(nullptr));
  return run(static_cast<__nv_bfloat16*>(nullptr));
}

}  // namespace

extern "C" {

dg_status dg_quantize_fp4(const void* x, const int32_t* masked_m, void* q, int32_t* sf, const dg_rows_desc* desc,
                          cudaStream_t stream) {
  return quantize<false>(x, masked_m, q, sf, desc, stream);
}

dg_status dg_swiglu_quantize_fp4(const void* x, const int32_t* masked_m, void* q, int32_t* sf, const dg_rows_desc* desc,
                                 cudaStream_t stream) {
  return quantize<true>(x, masked_m, q, sf, desc, stream);
}

dg_status dg_swiglu_backward(const void* x, const void* dy, const int32_t* masked_m, void* dx, const dg_rows_desc* desc,
                             cudaStream_t stream) {
  if (dg_status s = check(x, masked_m, dy, static_cast<const int32_t*>(dx), desc, 2); s != DG_OK) return s;
  if (desc->M == 0) return DG_OK;
  Tiles n;
  if (!n.count(*desc, kGradRows, kGradCols)) return DG_ERR_UNSUPPORTED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const SwigluGradArgs a{static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(dy), static_cast<__nv_bfloat16*>(dx),
                         masked_m, ctx.status, n.all, n.row, n.col, desc->M, desc->K, row_stride(*desc, 2), group_stride(*desc)};
  return dg::launch(swiglu_grad_kernel, n.blocks(), kWarps * 32, 0, stream, ctx.pdl, a);
}

}  // extern "C"
