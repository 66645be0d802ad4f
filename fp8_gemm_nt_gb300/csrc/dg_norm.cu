// Residual addition + RMS norm with BF16 and E4M3 outputs, and its gradient.
//
//   s = x + r        rstd = (mean(s^2) + eps)^(-1/2)        y = s * rstd * w
//   q = e4m3(y * 2^-n_g), n_g the least integer with max|y_g| * 2^-n_g <= 448, per group g of 128 columns
//
//   g = dy * w       dx = rstd * (g - s rstd * mean(g * s rstd)) + ds        dw = sum_t dy * s rstd
//
// Every sum and statistic is FP32; s, y and dx are rounded once, where they are stored, and q is
// rounded from the FP32 y.
//
// Both are bound by memory: a row is read once and written once. A team of warps owns a row; a thread
// copies its own columns of the row after it asynchronously to shared memory while it works on one, so
// that loads stay in flight through the row's reduction and stores, and no thread waits for another's
// copies. Blocks are persistent: weight (and the gradient's share of dw) stay in registers over the rows.
// 32768 rows of 7168 in BF16 to E4M3: 240 us, 6.9 TB/s, as fast as a copy (321 us with scalar arithmetic, which
// bounded it; 361 us with a block per row). Gradient of 16384 rows: 137 us, 6.9 TB/s (373 us with a block per row).
// Over 256 to 8192 columns, calls that move 0.5 to 3.5 GB, as shares of a copy's rate: BF16 0.74 to 1.0 forward (0.74 and 0.75 at
// 1152 and 2176 columns to E4M3, where 44 and 29 % of the lanes have no column, and at 256) and 0.88 to 1.0 backward; with
// an FP32 stream 0.73 to 0.81 and 0.65 to 0.71, for a reason not found (no unit is saturated).
#include <cuda_bf16.h>
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

constexpr int kVec = 8;                 // elements a thread takes at once
constexpr int kMaxH = 16384;
constexpr int kMaxV = 4;                // vectors of a row per thread
constexpr int kMaxTeam = 512;           // threads of a row
constexpr int kMaxSmem = 200 * 1024;    // of a block's rows in shared memory

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Two FP32 values in a register pair, and the two-lane instructions on them.
struct Two {
  float x, y;
};
__device__ __forceinline__ unsigned long long bits(Two a) {
  unsigned long long v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a.x), "f"(a.y));
  return v;
}
__device__ __forceinline__ Two two(unsigned long long v) {
  Two a;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(v));
  return a;
}
__device__ __forceinline__ Two operator+(Two a, Two b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return two(d);
}
__device__ __forceinline__ Two operator*(Two a, Two b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return two(d);
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return two(d);
}
__device__ __forceinline__ Two both(float v) { return {v, v}; }

// Eight consecutive elements as they are stored, and their FP32 values.
template <class T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int kChunks = 1;     // of 16 bytes
  uint4 u[1];
  __device__ __forceinline__ Two pair(int i) const {
    Two t;
    dg::unpack_bf16(i == 0 ? u[0].x : i == 1 ? u[0].y : i == 2 ? u[0].z : u[0].w, t.x, t.y);
    return t;
  }
};
template <>
struct Raw<float> {
  static constexpr int kChunks = 2;
  uint4 u[2];
  __device__ __forceinline__ Two pair(int i) const {
    const uint4& v = u[i / 2];
    return i % 2 ? Two{__uint_as_float(v.z), __uint_as_float(v.w)} : Two{__uint_as_float(v.x), __uint_as_float(v.y)};
  }
};

// Loads at L2: what a kernel reads may have been written by the one before it in the stream, whose end
// this one overlaps.
template <class T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < Raw<T>::kChunks; ++i) r.u[i] = dg::ld_cg_v4(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

// Columns: a warp owns V * 256 consecutive ones of its row (whole words of packed scales for V >= 2), of
// which vector j of a lane is columns 256 j + 8 lane .. + 7. In shared memory chunk i of that vector lies at
// [(j * kChunks + i) * 32 + lane] of the warp's region.
template <class T>
__device__ __forceinline__ void copy_piece(uint4* to, const T* from, int j, int lane) {
#pragma unroll
  for (int i = 0; i < Raw<T>::kChunks; ++i)
    dg::cp_async_16(dg::smem_addr(to + (j * Raw<T>::kChunks + i) * 32 + lane), reinterpret_cast<const uint4*>(from) + i);
}
template <class T>
__device__ __forceinline__ Raw<T> piece(const uint4* at, int j, int lane) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < Raw<T>::kChunks; ++i) r.u[i] = at[(j * Raw<T>::kChunks + i) * 32 + lane];
  return r;
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const Two (&v)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(dg::pack_bf16(v[0].x, v[0].y), dg::pack_bf16(v[1].x, v[1].y),
                                            dg::pack_bf16(v[2].x, v[2].y), dg::pack_bf16(v[3].x, v[3].y));
}
__device__ __forceinline__ void store8(float* p, const Two (&v)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
}

// Sum over a team's threads, the same value in each; `part`: one float per warp of the block. Teams of
// several warps meet at the barrier of their own number.
__device__ __forceinline__ float team_sum(float v, float* part, int team, int team_index) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (team == 32) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x / 32] = v;
  asm volatile("bar.sync %0, %1;" ::"r"(team_index + 1), "r"(team) : "memory");
  const float* mine = part + team_index * (team / 32);
  float s = 0;
  for (int i = 0; i < team / 32; ++i) s += mine[i];
  return s;
}

template <class R, class W>
struct NormArgs {
  const __nv_bfloat16* x;
  const R* residual;       // or null
  const W* weight;
  __nv_bfloat16* y;        // or null
  uint8_t* q;              // or null, then sf too
  int32_t* sf;
  R* residual_out;         // or null
  float* rstd;             // or null
  int T, H, team, depth;   // threads and rows of shared memory of a team: the row worked on and, if they fit, the next
  size_t ldx, ldr, ldo;
  float eps, inv_h;
};

template <class R>
__host__ __device__ constexpr int norm_row_chunks(int V) { return V * (1 + Raw<R>::kChunks); }

template <class R, class W, int V>
__global__ void __launch_bounds__(kMaxTeam) norm_kernel(const NormArgs<R, W> a) {
  extern __shared__ uint4 ring[];
  __shared__ float part[2][kMaxTeam / 32];
  const int team_index = threadIdx.x / a.team, tid = threadIdx.x % a.team, teams = blockDim.x / a.team;
  const int lane = threadIdx.x & 31, column = (tid / 32 * V * 32 + lane) * kVec;     // of vector 0; vector j is 256 j further
  constexpr int kApart = 32 * kVec, kRow = norm_row_chunks<R>(V) * 32;
  uint4* mine = ring + threadIdx.x / 32 * a.depth * kRow;                            // the warp's region
  const long long t0 = static_cast<long long>(blockIdx.x) * teams + team_index, step = static_cast<long long>(gridDim.x) * teams;
  const long long t4 = (static_cast<long long>(a.T) + 3) / 4 * 4;
  bool in[V];
#pragma unroll
  for (int j = 0; j < V; ++j) in[j] = column + j * kApart < a.H;
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  // this thread's first column in the row to copy, then in the row worked on: advanced row by row
  const __nv_bfloat16* xf = a.x + t0 * a.ldx + column;
  const R* rf = a.residual ? a.residual + t0 * a.ldr + column : nullptr;
  long long tf = t0;
  auto fetch = [&](int stage) {
    if (tf < a.T) {
      uint4* xs = mine + stage * kRow;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (in[j]) {
          copy_piece(xs, xf + j * kApart, j, lane);
          if (rf) copy_piece(xs + V * 32, rf + j * kApart, j, lane);
        }
    }
    tf += step;
    xf += step * a.ldx;
    if (rf) rf += step * a.ldr;
    cp_async_commit();
  };
  fetch(0);
  Raw<W> w[V];
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (in[j]) w[j] = load_raw(a.weight + column + j * kApart);
  R* so = a.residual_out ? a.residual_out + t0 * a.ldo + column : nullptr;
  const long long first = t0 * a.H + column;
  __nv_bfloat16* yo = a.y ? a.y + first : nullptr;
  uint8_t* qo = a.q ? a.q + first : nullptr;
  // a group is 16 neighbouring lanes' vector (H % 128 == 0: all 16 have one, or none has), so a warp's 2 V
  // codes fill V / 2 words, which lane 0 writes; V = 1 is a row of at most two groups
  const int groups = a.H / 128, word = column / 512, words = (groups + 3) / 4;
  int32_t* sfo = a.sf + word * t4 + t0;
  int flip = 0;
  for (long long t = t0; t < a.T; t += step, flip ^= 1) {
    if (a.depth == 2) {
      fetch(flip ^ 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    const uint4* xs = mine + (a.depth == 2 ? flip * kRow : 0);
    Two v[V][4];
    Two sum = both(0);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (in[j]) {
        const Raw<__nv_bfloat16> x = piece<__nv_bfloat16>(xs, j, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = x.pair(i);
        if (a.residual) {
          const Raw<R> r = piece<R>(xs + V * 32, j, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] = v[j][i] + r.pair(i);
        }
        if (so) store8(so + j * kApart, v[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(v[j][i], v[j][i], sum);
      }
    // each thread's share of the mean: a sum over the whole row could leave FP32's range before its mean does
    const float rstd = 1.0f / sqrtf(team_sum((sum.x + sum.y) * a.inv_h, part[flip], a.team, team_index) + a.eps);
    if (a.rstd && tid == 0) a.rstd[t] = rstd;
    float m[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      m[j] = 0;
      if (in[j]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[j][i] = v[j][i] * both(rstd) * w[j].pair(i);
          m[j] = fmaxf(m[j], fmaxf(fabsf(v[j][i].x), fabsf(v[j][i].y)));   // passes NaN over
        }
        if (yo) store8(yo + j * kApart, v[j]);
      }
    }
    if (qo) {
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
      float top = m[0];
#pragma unroll
      for (int j = 1; j < V; ++j) top = fmaxf(top, m[j]);
      if (__any_sync(0xFFFFFFFFu, top == INFINITY)) {
        // an infinity becomes the NaN code (as a NaN does by itself) and does not count for the scale
#pragma unroll
        for (int j = 0; j < V; ++j) {
          m[j] = 0;
          if (in[j])
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (!(fabsf(v[j][i].x) < INFINITY)) v[j][i].x = NAN;
              if (!(fabsf(v[j][i].y) < INFINITY)) v[j][i].y = NAN;
              m[j] = fmaxf(m[j], fmaxf(fabsf(v[j][i].x), fabsf(v[j][i].y)));
            }
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
        }
      }
      uint32_t codes = 0;      // of this half of the warp: vector j's in byte j
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (in[j]) {
          const int e = dg::ue8m0_for_amax(m[j]);
          const Two k = both(dg::ue8m0_inverse(e));
          Two z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) z[i] = v[j][i] * k;
          *reinterpret_cast<uint2*>(qo + j * kApart) =
              make_uint2(dg::pack_e4m3(z[0].x, z[0].y, z[1].x, z[1].y), dg::pack_e4m3(z[2].x, z[2].y, z[3].x, z[3].y));
          codes |= static_cast<uint32_t>(m[j] == 0 ? 127 : e) << (8 * j);
        }
      const uint32_t upper = __shfl_down_sync(0xFFFFFFFFu, codes, 16);
      if (lane == 0) {
        // bytes of the groups that are there, and 0 after them
        if (word < words) sfo[0] = static_cast<int32_t>(__byte_perm(codes, upper, 0x5140));
        if (V > 2 && word + 1 < words) sfo[t4] = static_cast<int32_t>(__byte_perm(codes, upper, 0x7362));
      }
      if (t == a.T - 1) {
        // and the words of the padding rows
        const int pad = static_cast<int>(t4 - a.T);
        for (int i = tid; i < words * pad; i += a.team) a.sf[i / pad * t4 + a.T + i % pad] = 0;
      }
      qo += step * a.H;
      sfo += step;
    }
    if (so) so += step * a.ldo;
    if (yo) yo += step * a.H;
    if (a.depth == 1) fetch(0);
  }
  cp_async_wait<0>();
}

template <class R, class W>
struct NormGradArgs {
  const __nv_bfloat16* dy;
  const R* s;
  const W* weight;
  const float* rstd;
  const R* ds;             // or null
  __nv_bfloat16* dx;       // or null
  R* dresidual;            // or null
  float* partial;          // [gridDim.x, H]
  int T, H, team, depth;
  float inv_h;
};

template <class R>
__host__ __device__ constexpr int grad_row_chunks(int V) { return V * (1 + 2 * Raw<R>::kChunks); }

// A thread keeps its columns' share of dw in registers over all of its team's rows, so dw costs one row
// of partial sums per block. The row's values are read from shared memory twice, before and after the
// reduction, rather than held.
template <class R, class W, int V>
__global__ void __launch_bounds__(kMaxTeam) norm_grad_kernel(const NormGradArgs<R, W> a) {
  extern __shared__ uint4 ring[];
  __shared__ float part[2][kMaxTeam / 32];
  const int team_index = threadIdx.x / a.team, tid = threadIdx.x % a.team, teams = blockDim.x / a.team;
  const int lane = threadIdx.x & 31, column = (tid / 32 * V * 32 + lane) * kVec;     // as in the forward kernel
  constexpr int kApart = 32 * kVec, kRow = grad_row_chunks<R>(V) * 32;
  uint4* mine = ring + threadIdx.x / 32 * a.depth * kRow;
  const long long t0 = static_cast<long long>(blockIdx.x) * teams + team_index, step = static_cast<long long>(gridDim.x) * teams;
  bool in[V];
#pragma unroll
  for (int j = 0; j < V; ++j) in[j] = column + j * kApart < a.H;
  constexpr int kS = V * 32, kDs = V * (1 + Raw<R>::kChunks) * 32;                   // where s and ds begin in a row's region
  dg::grid_dependency_wait();
  long long tf = t0, at_f = t0 * a.H + column;      // the row to copy, and this thread's first element of it
  auto fetch = [&](int stage) {
    if (tf < a.T) {
      uint4* to = mine + stage * kRow;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (in[j]) {
          copy_piece(to, a.dy + at_f + j * kApart, j, lane);
          copy_piece(to + kS, a.s + at_f + j * kApart, j, lane);
          if (a.ds) copy_piece(to + kDs, a.ds + at_f + j * kApart, j, lane);
        }
    }
    tf += step;
    at_f += step * a.H;
    cp_async_commit();
  };
  fetch(0);
  Raw<W> w[V];
  Two dw[V][4];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    if (in[j]) w[j] = load_raw(a.weight + column + j * kApart);
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = both(0);
  }
  long long at_o = t0 * a.H + column;
  int flip = 0;
  for (long long t = t0; t < a.T; t += step, flip ^= 1) {
    const float rstd = __ldcg(a.rstd + t);
    if (a.depth == 2) {
      fetch(flip ^ 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    const uint4* at = mine + (a.depth == 2 ? flip * kRow : 0);
    Two sum = both(0);
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (in[j]) {
        const Raw<__nv_bfloat16> dy = piece<__nv_bfloat16>(at, j, lane);
        const Raw<R> s = piece<R>(at + kS, j, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const Two p = dy.pair(i) * (s.pair(i) * both(rstd));
          dw[j][i] = dw[j][i] + p;
          sum = fma2(p, w[j].pair(i), sum);
        }
      }
    const float mean = team_sum((sum.x + sum.y) * a.inv_h, part[flip], a.team, team_index);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (in[j]) {
        const Raw<__nv_bfloat16> dy = piece<__nv_bfloat16>(at, j, lane);
        const Raw<R> s = piece<R>(at + kS, j, lane);
        Two d[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = both(0);
        if (a.ds) {
          const Raw<R> ds = piece<R>(at + kDs, j, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = ds.pair(i);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          d[i] = fma2(both(rstd), fma2(s.pair(i) * both(rstd), both(-mean), dy.pair(i) * w[j].pair(i)), d[i]);
        if (a.dx) store8(a.dx + at_o + j * kApart, d);
        if (a.dresidual) store8(a.dresidual + at_o + j * kApart, d);
      }
    }
    at_o += step * a.H;
    if (a.depth == 1) fetch(0);
  }
  cp_async_wait<0>();
  dg::grid_launch_dependents();
  // the teams' shares, one after another, through shared memory
  float* total = reinterpret_cast<float*>(ring);
  for (int k = 0; k < teams; ++k) {
    if (teams > 1) __syncthreads();
    if (team_index != k) continue;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      if (!in[j]) continue;
      const int c = column + j * kApart;
      if (k > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[j][i] = dw[j][i] + Two{total[c + 2 * i], total[c + 2 * i + 1]};
      }
      store8(k == teams - 1 ? a.partial + static_cast<long long>(blockIdx.x) * a.H + c : total + c, dw[j]);
    }
  }
}

// dw[c] = sum over the blocks' partial sums, in a fixed order: 32 columns per block, each of its 32 warps
// every 32nd row of them.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* partial, float* dw, int rows, int H) {
  __shared__ float part[32][33];
  dg::grid_dependency_wait();
  dg::grid_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float sum = 0;
  if (c < H)
#pragma unroll 4
    for (int r = warp; r < rows; r += 32) sum += __ldcg(partial + static_cast<long long>(r) * H + c);
  part[warp][lane] = sum;
  __syncthreads();
  sum = part[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (lane == 0 && blockIdx.x * 32 + warp < static_cast<unsigned>(H)) dw[blockIdx.x * 32 + warp] = sum;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Vectors per thread, threads of a row, and rows that a block works on at a time. Up to 32 threads'
// vectors a row is one warp's; longer ones are spread over as few warps as four vectors each allow, and
// blocks of short rows hold several teams to have 256 threads.
struct Shape {
  int v, team, teams;
  int threads() const { return team * teams; }
};
Shape row_shape(int H) {
  const int nvec = H / kVec;
  const int v = nvec <= 32 ? 1 : nvec <= 64 ? 2 : kMaxV;
  const int team = (nvec + 32 * v - 1) / (32 * v) * 32;
  return {v, team, std::max(1, 256 / team)};
}

template <class F>
dg_status with_v(int v, F f) {
  switch (v) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, kMaxV>());
  }
}

// Blocks for T rows: those that are resident together, at most one per team of rows. `row`: bytes of a
// block's rows in shared memory, two of which per team are taken if they fit.
struct Resident {
  unsigned blocks = 0;
  size_t smem = 0;
  int depth = 0;
};
template <auto kKernel>
dg_status resident_blocks(const Shape& shape, size_t row, int T, int sms, Resident* out) {
  static thread_local struct { int dev = -1, threads = 0; size_t smem = 0; int per_sm = 0; } last;
  out->depth = 2 * row <= kMaxSmem ? 2 : 1;
  out->smem = out->depth * row;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess && last.dev != dev) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e == cudaSuccess && (last.dev != dev || last.threads != shape.threads() || last.smem != out->smem)) {
    int n = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kKernel, shape.threads(), out->smem);
    if (e == cudaSuccess && n < 1) e = cudaErrorInvalidConfiguration;
    if (e == cudaSuccess) last = {dev, shape.threads(), out->smem, n};
  }
  if (e != cudaSuccess) return dg::record_cuda_error(e);
  const long long wanted = (static_cast<long long>(T) + shape.teams - 1) / shape.teams;
  out->blocks = static_cast<unsigned>(std::min(wanted, static_cast<long long>(last.per_sm) * sms));
  return DG_OK;
}

// Calls f with null pointers of the residual stream's type and the weight's.
template <class F>
dg_status with_types(int residual_type, int weight_type, F f) {
  const __nv_bfloat16* b = nullptr;
  const float* s = nullptr;
  if (residual_type == DG_BF16) return weight_type == DG_BF16 ? f(b, b) : f(b, s);
  return weight_type == DG_BF16 ? f(s, b) : f(s, s);
}

bool known_type(int t) { return t == DG_BF16 || t == DG_F32; }
size_t row_bytes(size_t ld, int type) { return ld * (type == DG_BF16 ? 2 : 4); }

}  // namespace

extern "C" {

dg_status dg_add_rms_norm(const void* x, const void* residual, const void* weight, void* residual_out, void* y, void* q,
                          int32_t* sf, float* rstd, const dg_norm_desc* desc, cudaStream_t stream) {
  if (!desc) return DG_ERR_INVALID_ARG;
  const int T = desc->T, H = desc->H, residual_type = desc->residual_type, weight_type = desc->weight_type;
  // a stride matters where there is a next row
  const size_t cols = H > 0 ? static_cast<size_t>(H) : 0;
  const size_t ldx = T > 1 ? desc->ldx : cols, ldr = T > 1 ? desc->ldr : cols, ldo = T > 1 ? desc->ldo : cols;
  const float eps = desc->eps;
  if (T < 0 || H <= 0 || H % kVec != 0 || !known_type(residual_type) || !known_type(weight_type)) return DG_ERR_INVALID_ARG;
  if (!(eps >= 0.0f) || !(eps < INFINITY)) return DG_ERR_INVALID_ARG;
  if ((q != nullptr) != (sf != nullptr) || (T > 0 && !q && !y && !residual_out) || (q && H % 128 != 0)) return DG_ERR_INVALID_ARG;
  if (H > kMaxH) return DG_ERR_UNSUPPORTED;
  if (T == 0) return DG_OK;
  if (!x || !weight || ldx < cols || (residual && ldr < cols) || (residual_out && ldo < cols)) return DG_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(residual) || !aligned16(weight) || !aligned16(residual_out) || !aligned16(y) ||
      !aligned16(q) || !aligned16(sf) || (reinterpret_cast<uintptr_t>(rstd) & 3u) || row_bytes(ldx, DG_BF16) % 16 ||
      (residual && row_bytes(ldr, residual_type) % 16) || (residual_out && row_bytes(ldo, residual_type) % 16))
    return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status s = dg::launch_context(&ctx); s != DG_OK) return s;
  const Shape shape = row_shape(H);
  return with_types(residual_type, weight_type, [&](auto* r, auto* w) {
    using R = std::remove_const_t<std::remove_pointer_t<decltype(r)>>;
    using W = std::remove_const_t<std::remove_pointer_t<decltype(w)>>;
    return with_v(shape.v, [&](auto v) {
      constexpr int V = decltype(v)::value;
      Resident at;
      if (dg_status s = resident_blocks<norm_kernel<R, W, V>>(shape, sizeof(uint4) * norm_row_chunks<R>(V) * shape.threads(), T, ctx.sms, &at); s != DG_OK) return s;
      const NormArgs<R, W> a{static_cast<const __nv_bfloat16*>(x), static_cast<const R*>(residual), static_cast<const W*>(weight),
                             static_cast<__nv_bfloat16*>(y), static_cast<uint8_t*>(q), sf,
                             static_cast<R*>(residual_out), rstd, T, H, shape.team, at.depth, ldx, ldr, ldo, eps, 1.0f / static_cast<float>(H)};
      return dg::launch(norm_kernel<R, W, V>, at.blocks, static_cast<unsigned>(shape.threads()), at.smem, stream, ctx.pdl, a);
    });
  });
}

dg_status dg_add_rms_norm_backward(const void* dy, const void* s, const void* weight, const float* rstd, const void* ds,
                                   void* dx, void* dresidual, float* dw, int T, int H, int residual_type,
                                   int weight_type, cudaStream_t stream) {
  if (T < 0 || H <= 0 || H % kVec != 0 || !known_type(residual_type) || !known_type(weight_type) || !dw) return DG_ERR_INVALID_ARG;
  if (H > kMaxH) return DG_ERR_UNSUPPORTED;
  if (T > 0 && (!dy || !s || !weight || !rstd || (!dx && !dresidual))) return DG_ERR_INVALID_ARG;
  if (!aligned16(dy) || !aligned16(s) || !aligned16(weight) || !aligned16(ds) || !aligned16(dx) || !aligned16(dresidual) ||
      !aligned16(dw) || (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return DG_ERR_MISALIGNED;
  LaunchContext ctx;
  if (dg_status e = dg::launch_context(&ctx); e != DG_OK) return e;
  const unsigned dw_blocks = static_cast<unsigned>((H + 31) / 32);
  if (T == 0)   // the sum over no rows
    return dg::launch(norm_dw_kernel, dw_blocks, 1024, 0, stream, ctx.pdl, static_cast<const float*>(nullptr), dw, 0, H);
  const Shape shape = row_shape(H);
  return with_types(residual_type, weight_type, [&](auto* r, auto* w) {
    using R = std::remove_const_t<std::remove_pointer_t<decltype(r)>>;
    using W = std::remove_const_t<std::remove_pointer_t<decltype(w)>>;
    return with_v(shape.v, [&](auto v) {
      constexpr int V = decltype(v)::value;
      Resident at;
      if (dg_status e = resident_blocks<norm_grad_kernel<R, W, V>>(shape, sizeof(uint4) * grad_row_chunks<R>(V) * shape.threads(), T, ctx.sms, &at); e != DG_OK) return e;
      dg::StreamWorkspace ws;
      void* partial = nullptr;
      if (dg_status e = ws.acquire(stream, static_cast<size_t>(at.blocks) * H * sizeof(float), &partial); e != DG_OK) return e;
      const NormGradArgs<R, W> a{static_cast<const __nv_bfloat16*>(dy), static_cast<const R*>(s), static_cast<const W*>(weight), rstd,
                                 static_cast<const R*>(ds), static_cast<__nv_bfloat16*>(dx), static_cast<R*>(dresidual),
                                 static_cast<float*>(partial), T, H, shape.team, at.depth, 1.0f / static_cast<float>(H)};
      if (dg_status e = dg::launch(norm_grad_kernel<R, W, V>, at.blocks, static_cast<unsigned>(shape.threads()), at.smem, stream, ctx.pdl, a); e != DG_OK) return e;
      return dg::launch(norm_dw_kernel, dw_blocks, 1024, 0, stream, ctx.pdl, static_cast<const float*>(partial), dw, static_cast<int>(at.blocks), H);
    });
  });
}

}  // extern "C"
