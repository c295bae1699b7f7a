// The room that fp8_exchange.cuh counts for a cluster's sums: every row, split and rank lies inside, no
// two of a CTA at one place, and no area is larger than its fullest split. Prints the number of
// violations.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <utility>

#include "fp8_exchange.cuh"

int main(int argc, char** argv) {
  long bad = 0;
  for (int i = 1; i < argc; ++i) {
    const int rows = atoi(argv[i]), room = gptq::exchange_rows(rows);
    int last = -1;
    for (int split = 1; split <= gptq::kMaxSplit; ++split) {
      std::set<std::pair<int, int>> taken;  // CTA, place
      for (int r = 0; r < rows; ++r)
        for (int rank = 0; rank < split; ++rank) {
          const int at = r / split * split + rank;
          bad += at < 0 || at >= room;
          bad += !taken.insert({r % split, at}).second;
          if (at > last) last = at;
        }
    }
    bad += last != room - 1;
  }
  printf("%ld\n", bad);
  return 0;
}
