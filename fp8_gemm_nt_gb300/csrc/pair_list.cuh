// The pair rows of the contiguous layout, listed once per call for the CTA-pair kernels.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "ue8m0.cuh"

namespace dg {

struct PairListArgs {
  // contiguous form: the pair rows (built by one block of 256 threads), else null
  const int32_t* m_indices;
  int num_mb, groups_g;
  int* pair_list;       // [num_mb][3]: first block, expert, own blocks (1 or 2)
  int* pair_count;
  uint32_t* status;
};

// Pair rows of the contiguous layout, by one block: block b (of 128 rows) belongs to the
// expert in m_indices[128 b] (outside [0, G): not computed, and reported unless it is -1);
// runs of consecutive blocks of one expert are cut into pairs from the run's first block. A
// block starts a pair iff it is valid and an even distance from its run's first block; pair
// rows are numbered by an exclusive prefix sum of those starts (two block-wide scans per
// chunk of blockDim.x blocks, carried across chunks).
__device__ inline void build_pair_list(const PairListArgs& a) {
  __shared__ int s_g[256 + 1];
  __shared__ int s_scan[256];
  const int tid = threadIdx.x;
  const int nt = blockDim.x;   // 256
  int run_start_carry = -1;    // first block of the run the previous chunk ended in
  int prev_g = -2;             // expert of the block before this chunk
  int count_carry = 0;
  auto expert = [&](int b) {
    const int g = ld_cg_s32(a.m_indices + static_cast<long long>(b) * 128);
    return (g >= 0 && g < a.groups_g) ? g : -1;
  };
  for (int base = 0; base < a.num_mb; base += nt) {
    const int b = base + tid;
    const bool in = b < a.num_mb;
    int raw = -1;
    if (in) {
      raw = ld_cg_s32(a.m_indices + static_cast<long long>(b) * 128);
      if (raw < -1 || raw >= a.groups_g) atomicOr(a.status, kBadIndexBit);
    }
    const int g = in && raw >= 0 && raw < a.groups_g ? raw : -1;
    s_g[tid + 1] = g;
    if (tid == 0) s_g[0] = prev_g;
    __syncthreads();
    // run starts: a valid block whose predecessor has another expert
    int rs = (g >= 0 && s_g[tid] != g) ? b : -1;
    s_scan[tid] = rs;
    __syncthreads();
    for (int off = 1; off < nt; off <<= 1) {           // inclusive prefix max
      const int v = tid >= off ? s_scan[tid - off] : -1;
      __syncthreads();
      s_scan[tid] = max(s_scan[tid], v);
      __syncthreads();
    }
    const int run_start = max(s_scan[tid], run_start_carry);
    const bool start = g >= 0 && ((b - run_start) % 2 == 0);
    const int last_rs = s_scan[nt - 1];
    __syncthreads();
    s_scan[tid] = start ? 1 : 0;
    __syncthreads();
    for (int off = 1; off < nt; off <<= 1) {           // inclusive prefix sum
      const int v = tid >= off ? s_scan[tid - off] : 0;
      __syncthreads();
      s_scan[tid] += v;
      __syncthreads();
    }
    if (start) {
      const int idx = count_carry + s_scan[tid] - 1;
      const int own = (b + 1 < a.num_mb && expert(b + 1) == g) ? 2 : 1;
      a.pair_list[3 * idx + 0] = b;
      a.pair_list[3 * idx + 1] = g;
      a.pair_list[3 * idx + 2] = own;
    }
    const int chunk_count = s_scan[nt - 1];
    run_start_carry = max(run_start_carry, last_rs);
    prev_g = s_g[nt];
    __syncthreads();
    count_carry += chunk_count;
    // a run that ended inside this chunk must not leak into the next one: the next chunk's
    // first valid block restarts its run whenever its expert differs from prev_g, which the
    // run-start flags above take care of; run_start_carry only matters for a continuing run
  }
  if (tid == 0) *a.pair_count = count_carry;
}

}  // namespace dg
