// Sizes, workspace layout and launch rules of the operators over a vocabulary
// (vocab.hip, vocab_top.hip). Host code alone, without HIP: tests compile it by
// itself.
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
// for it (2048 x 32000, 64 tokens: 309 us, score_kernel 79). The gradient's logits
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

// Of a divergence's gradient, from kept logits or from its own: of up to 192 tokens, where W is
// most of what takes the time; and of short products, whose second term costs tens of microseconds
// (loss and gradient in us, two terms and one: 301 tokens, 4999 x 515 92 and 81; 1024 tokens, 8000 x 512
// 128 and 98; 300 tokens, 8000 x 1024 122 and 86; 1000 tokens, 32000 x 128 194 and 146). (One term's error
// of dH and dW, over that of rounding the exact ones: up to 1.7 with 33 to 65 tokens, 1.56 with 200; with
// more it nears 2^0.5, so very many tokens have two only where that is next to nothing: 131072 tokens,
// 128 x 256 2200 and 1500.)
inline int distill_rows(int64_t T, int64_t V, int64_t d, int dtype) {
  const double n = (double)T * V * d;
  return dtype != kF32 && (T <= 192 || n <= (T <= 4096 ? 4294967296.0 : 536870912.0)) ? kFewTerms : 1;
}

struct Plan {
  int64_t dp, tp;              // d to 64, rows of G to 256 (few tokens: T to 64)
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
// Whether dH's and dW's products, of so many 128 x 128 tiles (slices counted), go in one launch: where
// both are taken in such tiles, or dW in smaller ones, and two rounds of two per CU hold them (the
// loss's gradient of 700 tokens, 3000 x 512 bf16: 51 -> 44 us; 300 tokens, 5000 x 300 fp32: 80 -> 66).
// The results are the same.
inline bool pairs(int tile_h, int64_t nh, int tile_w, int64_t nw) {
  return tile_h == 128 && tile_w <= 128 && nh + nw <= 1024;
}
// Words per piece: G, and a copy of W's piece where one is needed, hold at most
// 2^26 values each (two thousand words at least), which leaves the fp32 sums of
// dH, read and written once per piece, a few percent of the piece's products.
// (kept: the operands of a product whose results have their place in a KeepPlan; rows: of G per
// token.)
inline Plan plan_for(int64_t T, int64_t V, int64_t d, int dtype, bool grad, bool kept, int rows) {
  Plan p{};
  const int nt = terms(dtype);
  p.dp = round_up(d, BK);
  p.tp = few(T, d, dtype) ? round_up(T, BK) : round_up(rows * T, 256);
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
  if (!grad && !kept) {
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
    p.part = take(4 * p.nz * T * rows * round_up(d, 4));
  }
  p.bytes = off;
  return p;
}

inline Plan plan_for(int64_t T, int64_t V, int64_t d, int dtype, bool grad) {
  return plan_for(T, V, d, dtype, grad, false, g_rows(T, d, dtype));
}

// ---------------------------------------------------------------- single logits (vocab_top.hip)
// Words of a token's row of logits that are kept for a gradient: whole groups
inline int64_t row_of(int64_t V) { return round_up(V, 128); }
constexpr int64_t kMaxListed = 128;   // words that a token can list, and its best words
constexpr int64_t kKeep = int64_t(1) << 27;   // values of one kind that are kept at most

constexpr int64_t kFirst = 8192;              // words of the first step at least
constexpr int64_t kWhole = int64_t(1) << 26;  // logits of a block that are kept whole, in one step

// What a call keeps of the logits of `block` tokens at a time: the sums of every group of
// words, without listed words or with them; the z of those; and, to find the best words, the largest z
// of each part of a group and the parts that may hold one of them, of a step of the
// vocabulary at a time.
struct KeepPlan {
  Plan p;                     // of the operands
  bool few;                   // score_kernel's: all logits are kept, in one step
  int tile;
  int64_t group, groups;      // words of a group, groups of a token
  int64_t block;              // tokens at a time
  int64_t first, step;        // words of the first step and of the largest (0: no best words)
  bool marked;                // listed words have marks (else their z is found in the row of kept logits)
  int64_t lds, ldz;           // bytes of a token's slots, its row of kept logits
  int64_t zs, ws;             // fp32: factors of tokens and of a piece's words
  int64_t stat, tops, slot, marks, places, zl, z, best, thr, bytes;
};
inline KeepPlan keep_plan(int64_t T, int64_t V, int64_t d, int dtype, int64_t listed, int64_t top) {
  KeepPlan k{};
  k.few = few(T, d, dtype);
  if (!k.few) k.p = plan_for(T, V, d, dtype, false, true, 1);
  k.tile = k.few ? 128 : tile_for(V, T);
  k.group = k.tile / 2;
  k.groups = (V + k.group - 1) / k.group;
  k.block = T;
  // (twice as many groups as best words, so that few of their words are above a group's best)
  const int64_t all = round_up(V, 256), first = std::min(all, std::max(kFirst, round_up(2 * top * k.group, 256)));
  if (!k.few) {
    int64_t most = std::min(kKeep / std::max<int64_t>(8 * listed, 1), kKeep / (4 * k.groups));
    if (top) most = std::min(most, kKeep / first);
    k.block = std::min(T, std::max<int64_t>(256, most / 256 * 256));
  }
  k.marked = listed && !k.few;
  if (k.few) {
    k.ldz = row_of(V);
  } else if (top) {
    k.step = std::min(all, std::max(first, kKeep / k.block / 256 * 256));
    k.first = k.block * all <= kWhole ? all : first;
    k.ldz = k.step;
  }
  k.lds = round_up(k.groups, 16);
  int64_t off = round_up(k.p.bytes, 256);
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  if (dtype == kF32 && !k.few) {
    k.zs = take(4 * T);
    k.ws = take(4 * k.p.piece);
  }
  k.stat = take(16 * k.block * k.groups);
  if (top) k.tops = take(4 * 4 * k.block * k.groups);
  k.z = take(4 * k.block * k.ldz);
  if (k.marked) {
    k.slot = take(k.block * k.lds);
    k.marks = take(32 * k.block * listed);
    k.places = take(k.block * listed);
    k.zl = take(4 * k.block * listed);
  }
  k.best = take(8 * k.block * top);
  k.thr = take(4 * k.block);
  k.bytes = off;
  return k;
}

// ---------------------------------------------------------------- few tokens' gradient (vocab_few.hip)
struct FewPlan {
  int64_t ldz;               // of a token's row of z and of G
  int64_t columns;           // workgroups that share a slice of dH
  int64_t blocks, slices;    // of dH: blocks of 16 words in a slice
  int64_t G, z, part, bytes;
};
// Slices of dH: a round of workgroups of four waves, four per CU (three where a wave has 17 or more
// tokens' sums of a 16-bit W, 33 of an fp32 one), with 64 words or more each.
inline FewPlan few_plan(int64_t T, int64_t V, int64_t d, int dtype) {
  FewPlan p{};
  const int64_t all = (V + 15) / 16;
  p.ldz = row_of(V);
  p.columns = (d * dtype_bytes(dtype) + 255) / 256;
  const int64_t want = std::min(std::max<int64_t>(1, (T <= (dtype == kF32 ? 32 : 16) ? 1024 : 768) / p.columns), (all + 3) / 4);
  p.blocks = round_up((all + want - 1) / want, 4);
  p.slices = (all + p.blocks - 1) / p.blocks;
  p.G = 0;
  p.z = round_up(4 * T * p.ldz, 256);
  p.part = 2 * p.z;
  p.bytes = p.part + round_up(4 * p.slices * T * round_up(d, 4), 256);
  return p;
}
// Whether a divergence keeps its logits for the gradient, which need not compute them once more: 4
// GiB of them at most, and where the hidden size is so large that computing costs more than a store
// and a load (loss and gradient in us, kept and not: 4096 tokens, 131072 words of bf16, d = 4096
// 11634 and 14254, 1024 4137 and 4245, 512 3092 and 2724; logits that stay in the last-level cache,
// 1024 tokens, 32000 words, d = 1024 323 and 328, 512 220 and 223, 128 164 and 157; fp32, 4096
// tokens, 32000 words, d = 512 1652 and 1845, 256 1198 and 1239); or, of 16 bits, where there are few of
// them (150 tokens, 32000 words, d = 128 88 and 93).
inline bool keeps(int64_t T, int64_t V, int64_t d, int dtype) {
  const int64_t n = T * row_of(V);
  const bool pays = d >= (n <= int64_t(1) << 25 || dtype == kF32 ? 256 : 1024);
  return (few(T, d, dtype) || (dtype != kF32 && (T <= 192 || (double)T * V * d <= 536870912.0)) || pays) && n <= int64_t(1) << 30;
}

// Of a divergence's gradient. One plan with and without kept logits: its pieces, and so its bytes,
// depend on the rows of G, of which more can need less (shorter pieces of W).
inline Plan distill_plan(int64_t T, int64_t V, int64_t d, int dtype) {
  return plan_for(T, V, d, dtype, true, false, distill_rows(T, V, d, dtype));
}
// What such a gradient needs beside its products' workspace
struct SharePlan {
  int64_t labels, share, wr, val, bytes;
};
inline SharePlan share_plan(int64_t T, int64_t V, int64_t d, int dtype, int64_t K) {
  SharePlan p;
  p.labels = round_up(few(T, d, dtype) ? few_plan(T, V, d, dtype).bytes : distill_plan(T, V, d, dtype).bytes, 256);
  p.share = p.labels + round_up(4 * T, 256);
  p.wr = p.share + round_up(4 * T, 256);
  p.val = p.wr + round_up(4 * T, 256);
  p.bytes = p.val + round_up(4 * T * K, 256);
  return p;
}

}  // namespace vocab
}  // namespace nq
