// Prints the way that each product of the arguments takes: "dense:M,N,K", "contiguous:M_total,N,K,G" or
// "masked:G,max_m,N,K" after the number of SMs; a line each of columns and ways (0: CTA pairs).
#include <cstdio>
#include <cstdlib>

#include "fp4_ways.h"

int main(int argc, char** argv) {
  const int sms = std::atoi(argv[1]);
  for (int i = 2; i < argc; ++i) {
    int a, b, c, d;
    dg::fp4::Way way{0, 0};
    if (std::sscanf(argv[i], "dense:%d,%d,%d", &a, &b, &c) == 3)
      way = dg::fp4::dense_way(a, b, c, sms);
    else if (std::sscanf(argv[i], "contiguous:%d,%d,%d,%d", &a, &b, &c, &d) == 4)
      way.bn = dg::fp4::contiguous_width(a, b, c, d, sms);
    else if (std::sscanf(argv[i], "masked:%d,%d,%d,%d", &a, &b, &c, &d) == 4)
      way.bn = dg::fp4::masked_width(a, b, c, d, sms);
    else
      return 1;
    std::printf("%d %d\n", way.bn, way.ways);
  }
  return 0;
}
