// Which way a product of two FP4 operands runs: tiles of CTA pairs, by width, or tiles of 128 rows with K shared out in a
// cluster. Host code alone: tests/fp4_ways_check.cpp prints the ways that sizes take.
#pragma once

#include <algorithm>
#include <cmath>

namespace dg {
namespace fp4 {

// Columns of a tile, and the CTAs that share out its K; ways = 0: CTA pairs.
struct Way {
  int bn, ways;
};
constexpr Way kSplits[] = {{64, 1}, {64, 2}, {64, 4}, {96, 2}, {128, 1}, {128, 2}, {192, 1}};

constexpr int kWayStageK = 256;            // K of a pipeline stage
inline int parts(int a, int b) { return (a + b - 1) / b; }

// Estimated microseconds of a product by CTA pairs with tiles of bn columns, from what the kernel was measured at: a launch
// 4.5, then for each tile of a pair a start and a time for each stage of 256 K, no less than its output takes, and no less
// than its share of B takes from HBM. pair_rows: 256-row strips; sharing: how many of them read the same of B. Widths 256,
// 384 and 128 in us: 8 experts, 32768 x 4096 x 7168 283, 308, 440; of K = 512 89, 78, 120; masked 32 x 256 x 7168 x 2048 67,
// 61, 69; 4096 x 24576 x 1536 74, 79, 92; 512 x 4096 x 7168 13.9, 19.9, 12.2. Over 28 shapes of all forms, from 1 to 32768
// rows, its choice is within 6 % of the best.
inline double pair_time(int bn, int N, int K, double pair_rows, double sharing, int sms) {
  const int stages = parts(K, kWayStageK), clusters = std::max(1, sms / 2);
  const double tiles = pair_rows * parts(N, bn), waves = std::ceil(tiles / clusters);
  const double tile = bn == 256 ? std::max(3.3, 1.4 + 0.3 * stages) : bn == 384 ? 2.6 + 0.47 * stages : std::max(2.0, 1.0 + 0.25 * stages);
  const double bytes = std::min<double>(tiles, clusters) / sharing * bn * (K * 0.53125);
  return 4.5 + waves * std::max(tile, 1.6 + bytes / 6.2e6);
}

inline int pair_width(int N, int K, double pair_rows, double sharing, int sms) {
  int best = 256;
  for (int bn : {384, 128})
    if (pair_time(bn, N, K, pair_rows, sharing, sms) < pair_time(best, N, K, pair_rows, sharing, sms)) best = bn;
  return best;
}

// Estimated microseconds of one of kSplits: a stage of 256 K costs an SM 0.19 us or the time of its bytes from L2 (91 GB/s an
// SM; rows of 128 bytes and 8 of scales) or, all CTAs' together, of B's from HBM (6 TB/s); a launch 3 us, a cluster's sums 0.3
// us and 20 KB a microsecond. Its choice against every way on its own, in us (128 x 7168 x 16384: 16.9, others 17.2 to 37; 128 x
// 256 x 512: 2.5, 2.9 to 6.3; 128 x 2048 x 16384: 11.3, 13.9 to 36): the best at 19 of 20 shapes, 3 % off at the other.
inline double split_time(const Way& w, int M, int N, int K, int sms) {
  const int stages = parts(K, kWayStageK), rows = std::min(M, 128);
  const double m_tiles = parts(M, 128), ctas = m_tiles * parts(N, w.bn) * w.ways;
  // one wave; of clusters of four, 152 SMs hold 36
  if (stages < w.ways || ctas > (w.ways == 4 ? 18 * (sms / 19) : sms / w.ways * w.ways)) return HUGE_VAL;
  const double stage = std::max({0.19, (rows + w.bn) * 136.0 / 91e3, ctas / m_tiles * w.bn * 136.0 / 6e6});
  return 3.0 + parts(stages, w.ways) * stage + (w.ways > 1 ? 0.3 + rows * w.bn * 4.0 / 20e3 : 0.0);
}

inline Way dense_way(int M, int N, int K, int sms) {
  const int strips = parts(M, 256);
  Way best{pair_width(N, K, strips, strips, sms), 0};
  double least = pair_time(best.bn, N, K, strips, strips, sms);
  for (const Way& w : kSplits)
    if (const double t = split_time(w, M, N, K, sms); t < least) best = w, least = t;
  return best;
}

// (strips as they are if every expert's rows fill them)
inline int contiguous_width(int M_total, int N, int K, int G, int sms) {
  const double strips = parts(M_total, 256);
  return pair_width(N, K, strips, std::max(1.0, strips / G), sms);
}

// (the counts are on the device: half of the rows, say)
inline int masked_width(int G, int max_m, int N, int K, int sms) {
  const double strips = parts(parts(max_m, 2), 256);
  return pair_width(N, K, G * strips, strips, sms);
}

}  // namespace fp4
}  // namespace dg
