// Sizes, workspace layout and launch rules of the loss over a vocabulary
// (vocab.hip). Host code alone, without HIP: tests compile it by itself.
#pragma once

#include <algorithm>

#include "sizes.h"

namespace nq {
namespace vocab {

constexpr int BK = 64;            // k per stage of a product
// 16-bit terms of an operand of type D
constexpr int terms(int D) { return D == kF32 ? 2 : 1; }
constexpr int kAmaxParts = 1024;
// Factors of a call, read by the kernels that follow.
struct Factors {
  float mw;              // power of two that W is scaled by (fp32, else 1)
  float post_w;          // of dW
};
// copies of H that a gradient takes: for z and for dW (bf16: one for both)
constexpr int forms(int D) { return D == kBF16 ? 1 : 2; }

// Whether score_kernel takes a call. With more tokens mma_kernel reads W at a
// higher rate although half of a tile is empty (4096 x 32000 bf16, 64 tokens: 94
// us, score_kernel 104; 32 tokens: 72 in score_kernel), but fp32 would be copied
// for it (2048 x 32000, 64 tokens: 309 us, score_kernel 90). The gradient's logits
// come from the same kernel; its time is much the same with either (4096 x 32000
// bf16, 1 and 32 tokens, one term of G: 262 and 276 us, with mma_kernel 266 and 274;
// fp32 790 and 810, 829 and 848).
inline bool few(int64_t T, int64_t d, int dtype) { return d >= 8 && T <= (dtype == kF32 ? 64 : 32); }

// Rows of G per token: terms of a 16-bit G that the products take as tokens of their
// own (fp32's two terms lie in one row, for its passes over k). One value of G, the
// label's or a likely word's, carries most of a token's gradient, and a 16-bit G's
// rounding of it is common to the token's row of dH and to dW's row of the word. Over
// many tokens that is a second rounding like the outputs' own, 2^0.5 of their error
// at most (1.05 to 1.25 measured with 2048 tokens, a few 1.4 with 64); the gradient of
// one token can be twice, of 32 tokens 1.5 times as far off as rounding its results
// alone. So 16-bit G of few tokens has a second term, as good as exact, in rows of the
// products' tiles that would be empty.
constexpr int kFewTerms = 2;
inline int g_rows(int64_t T, int64_t d, int dtype) {
  return dtype != kF32 && few(T, d, dtype) ? kFewTerms : 1;
}

struct Plan {
  int64_t dp, tp;              // d to 64, T to 256 (few tokens: to 64)
  int64_t piece, npieces;      // words of a piece, to 256; pieces
  int nz;                      // slices of dH, each with a share of the first piece
  int64_t kz;                  // words per slice, to 64
  // byte offsets
  int64_t hp, wp, top, sum, hit, hm, rows, fac, amax, G, part, bytes;
};
inline int64_t tiles_of(int64_t M, int64_t N, int64_t tile) {
  return ((M + tile - 1) / tile) * ((N + tile - 1) / tile);
}
// Tiles of 256 x 256 (one workgroup of eight waves per CU) or of 128 x 128 (two
// of four per CU, which lose about a fifth of the rate to twice the copies):
// whichever needs less time in whole rounds over the 256 CUs (512 tokens, 32000
// x 2048 bf16: the loss 66 us in big tiles, 90 in small ones; 300 tokens, 20000 x
// 1024: 42 and 32).
inline bool big_tiles(int64_t M, int64_t N, int64_t slices) {
  const int64_t big = tiles_of(M, N, 256) * slices, small = tiles_of(M, N, 128) * slices;
  return (big + 255) / 256 * 4.0 <= (small + 255) / 256 * 1.25;
}
// Of 64 x 64 where 128 x 128 leave half of the CUs idle (loss and gradient in us:
// 128 tokens, 8192 x 4096 bf16 34 and 102, else 48 and 118; 74 tokens, 1115 x 2368
// fp32 74 and 105, else 97 and 128).
inline int tile_for(int64_t M, int64_t N) {
  return tiles_of(M, N, 128) <= 128 ? 64 : big_tiles(M, N, 1) ? 256 : 128;
}
// Slices of the contraction of dH: a workgroup for every CU (two in small
// tiles), 256 words at least. Big tiles need more slices, each with its share of
// fp32 sums to write and join: taken where they fill most CUs, have 1024 words
// each and a clear lead in products per CU (1024 tokens, 32000 x 2048 fp32: 404
// us in 8 slices of big tiles, 550 in 4 of small ones; 1500 tokens, 4000 x 1500
// bf16, 571 words each: dH 106 us in big tiles, 91 in small ones; 600 tokens, 10000
// x 3000 fp16, no lead: 154 and 129).
inline int dh_slices(int64_t T, int64_t d, int64_t piece) {
  const int64_t big = tiles_of(d, T, 256), most = std::max<int64_t>(1, std::min<int64_t>(piece / 256, 64));
  const int64_t nb = std::max<int64_t>(1, std::min(256 / big, most));
  const int64_t ns = std::max<int64_t>(1, std::min(512 / tiles_of(d, T, 128), most));
  const bool lead = 4.0 / nb <= 0.85 * 2.5 / ns;
  return (int)(big * nb >= 192 && piece / nb >= 1024 && lead ? nb : ns);
}
// Words per piece: G, and a copy of W's piece where one is needed, hold at most
// 2^26 values each (two thousand words at least), which leaves the fp32 sums of
// dH, read and written once per piece, a few percent of the piece's products.
inline Plan plan_for(int64_t T, int64_t V, int64_t d, int dtype, bool grad) {
  Plan p{};
  const int nt = terms(dtype);
  p.dp = round_up(d, BK);
  p.tp = round_up(T, few(T, d, dtype) ? BK : 256);
  const int64_t most = std::max<int64_t>(2048, (int64_t(1) << 26) / std::max(p.tp, p.dp) / 256 * 256);
  p.npieces = (V + most - 1) / most;
  p.piece = round_up((V + p.npieces - 1) / p.npieces, 256);
  p.npieces = (V + p.piece - 1) / p.piece;
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  if (!grad) {
    // partials per token: one per 64 words, or two per tile's words (W in place or
    // in pieces)
    const bool tiny = !few(T, d, dtype) && (tile_for(V, T) == 64 || tile_for(p.piece, T) == 64);
    const int64_t np = (tiny ? 2 : 1) * ((V + 63) / 64) + 4;
    p.top = take(4 * np * T);
    p.sum = take(4 * np * T);
    p.hit = take(4 * T);
    if (few(T, d, dtype)) {
      p.bytes = off;
      return p;
    }
  }
  p.fac = take(sizeof(Factors));
  p.amax = take(4 * kAmaxParts);
  p.hm = take(4 * T);
  p.rows = take(4 * 5 * T);
  p.hp = take(2 * nt * p.tp * p.dp * (grad ? forms(dtype) : 1));
  p.wp = take(2 * nt * p.piece * p.dp);
  if (grad) {
    // (the first piece, which may be V itself, writes every slice that is joined)
    const int64_t words = round_up(std::min(p.piece, V), BK), nz = dh_slices(T, d, p.piece);
    p.kz = round_up((words + nz - 1) / nz, BK);
    p.nz = (int)((words + p.kz - 1) / p.kz);
    // (few tokens: their two rows each are 64 at most)
    p.G = take(2 * nt * p.tp * p.piece);
    p.part = take(4 * p.nz * T * g_rows(T, d, dtype) * round_up(d, 4));
  }
  p.bytes = off;
  return p;
}

}  // namespace vocab
}  // namespace nq
