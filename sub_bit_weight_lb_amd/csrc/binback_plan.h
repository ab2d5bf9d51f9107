// Sizes, workspace layout and launch rules of the packed layer's gradient
// (binback.hip). Host code alone, without HIP: tests compile it by itself.
#pragma once

#include <algorithm>

#include "sizes.h"

namespace nq {
namespace binback {

constexpr int kDigit = 2048;      // bytes of a digit per 16 rows and 128 columns
constexpr int kThinMax = 64;      // rows of a thin launch
constexpr int kMaxSplit = 8;      // slices of the columns (few tiles)
// 16-row tiles of a thin launch: its kernel reads the digits of all of them,
// rows past T included
constexpr int thin_tiles(int64_t T) { return T <= 16 ? 1 : T <= 32 ? 2 : 4; }

// 128-column blocks of a row of digits: whole groups of four
constexpr int64_t blocks(int64_t cols) { return (cols + 511) / 512 * 4; }

enum Epi : int {
  kProj = 0,   // out: p or dp (fp32, or fp64 partials when the columns are split)
  kGrad = 1,   // column sums of dy q; or dx = s2 da and column sums of da x^
};
constexpr int digits(int epi) { return epi == kProj ? 4 : 3; }
// A wide wave's tile in units of 16 rows and 16 signs: 128 and 120 registers of
// sums (kGrad of 1 x 8 484 us where 2 x 5 takes 453)
constexpr int row_tiles(int epi) { return epi == kProj ? 1 : 2; }
constexpr int sign_tiles(int epi) { return epi == kProj ? 8 : 5; }
// Slices of the columns of a chain's first product: enough tiles for two
// workgroups on each of the 256 CUs (one of a thin launch, which has eight
// waves; the two chains run together), at least 512 columns each.
constexpr int64_t tiles_of(int epi, int64_t T, int64_t N) {
  const int64_t rows = 32 * row_tiles(epi), signs = 32 * sign_tiles(epi);
  return ((T + rows - 1) / rows) * ((N + signs - 1) / signs);
}
inline int proj_split(int64_t T, int64_t r, int64_t K) {
  const int64_t most = T <= kThinMax ? 256 / (2 * ((r + 15) / 16)) : 512 / (2 * tiles_of(kProj, T, r));
  return (int)std::max<int64_t>(1, std::min({(int64_t)kMaxSplit, most, blocks(K) / 4}));
}
// rows per partial column sum
constexpr int64_t kSumRows = 32 * row_tiles(kGrad);
// rows of the digit planes: as many as a launch reads
constexpr int64_t digit_rows(int64_t T) {
  return T <= kThinMax ? 16 * thin_tiles(T) : (T + kSumRows - 1) / kSumRows * kSumRows;
}

struct Plan {
  int split[2];                                   // proj_split of the two chains
  // byte offsets, of the chains' and of the column sums'
  int64_t planes[2], steps[2], sums[2], P[2], cp1, cp2, bytes;
};
inline Plan plan_for(int64_t m, int64_t n, int64_t r, int64_t T) {
  Plan p{};
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  const int64_t nt = (T + kSumRows - 1) / kSumRows;
  for (int c = 0; c < 2; ++c) {
    const int64_t K = c ? m : n;
    const int sp = p.split[c] = proj_split(T, r, K);
    p.planes[c] = take(digit_rows(T) * 128 *
                       std::max(digits(kProj) * blocks(K), digits(kGrad) * blocks(r)));
    p.steps[c] = take(4 * T);
    p.sums[c] = take(16 * T);
    p.P[c] = take(sp == 1 ? 4 * T * r : 8 * T * r * sp);
  }
  p.cp1 = take(4 * nt * m);
  p.cp2 = take(4 * nt * n);
  p.bytes = off;
  return p;
}

}  // namespace binback
}  // namespace nq
