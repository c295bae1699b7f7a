// fp8_exchange.cuh — room for the sums of a cluster along K (fp8_skinny.cu). Counted through on the CPU by
// the tests.
#pragma once

namespace gptq {

constexpr int kMaxSplit = 8;  // CTAs along K

// Rows are dealt out to the `split` CTAs, row r to CTA r % split, which holds the sums of all of them side by
// side: the sum of CTA `rank` at place r / split * split + rank. The places that the area has room for,
// whatever the split: 21 for 16 rows (at seven CTAs), 36 for 32 (at six), 70 for 64 (at seven).
constexpr int exchange_rows(int rows) {
  int most = 0;
  for (int s = 1; s <= kMaxSplit; ++s) {
    const int need = (rows + s - 1) / s * s;
    if (need > most) most = need;
  }
  return most;
}

}  // namespace gptq
