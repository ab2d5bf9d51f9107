// The products of the operators over a large vocabulary (vocab.hip, vocab_top.hip):
// z = scale H W^T a tile at a time with an epilogue each, the operands' layouts
// and scales. Device and host code of the files that include it.
#pragma once

#include "tune.h"

#include <algorithm>
#include <type_traits>

#include "vocab_plan.h"

namespace nq {
using namespace vocab;
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_tr_t;

constexpr float kNegInf = -__builtin_inff();

// one 16 x 16 x 32 product of 16-bit operands
template <bool F16>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Passes over k of an operand of type D
constexpr int passes(int D) { return D == kF32 ? 3 : 1; }

// x (already scaled) as N terms of the 16-bit type that the products of D's take.
// Not finite: the first term alone.
template <int D, int N>
__device__ __forceinline__ void split(float x, uint16_t (&t)[N]) {
  typedef Elem<D == kBF16 ? kBF16 : kF16> E;
  const typename E::type h = E::from(x);
  t[0] = __builtin_bit_cast(uint16_t, h);
  if constexpr (N == 2) {
    const float r = x - E::to(h);
    const bool fin = (__float_as_uint(r) & 0x7fffffffu) < 0x7f800000u;
    t[1] = fin ? __builtin_bit_cast(uint16_t, E::from(r)) : (uint16_t)0;
  }
}

// A 16-bit operand of the products, `ld` apart, its terms `plane` apart within
// a row. k-contiguous: `rows` rows of k values. k-major: k runs down the rows
// and `rows` counts the columns. kv: the k that exist (past them
// an operand reads zeros).
struct Opnd {
  const uint16_t* p;
  int64_t ld, plane, rows, kv;
};

// What the operators that look at single logits (vocab_top.hip) keep of them. The words
// of a token lie in groups: half a tile's, or 64 of score_kernel's. The distinct words that a
// token lists have places in its row of zl; a group with any has a mark.
struct Mark {
  u32x4 words;              // which of the group's words are listed
  uint32_t place;           // of the first of them; the others follow
};
struct Kept {
  f32x4* stat;              // [token][groups]: largest z; sum e - 1, e = exp(z - largest), which is
                            // summed without that 1 and so keeps the digits of a small rest; sum e (z - largest)
  int64_t groups;
  const uint8_t* slot;      // [token][lds], nullable: a group's mark, 255: none
  int64_t lds, listed;
  const Mark* marks;        // [token][listed]
  float* zl;                // [token][listed]
  int without;              // stat leaves listed words out
  float* tops;              // [token][parts of groups], nullable: the largest z of each part of a group
  float* z;                 // [token][ldz], nullable: z of the call's words,
  int64_t ldz;
  const float* thr;         // of parts with one above the token's thr (nullable: all)
  int flip;                 // kPick, 16-bit: z's factor is below zero
};
// The place of listed word `in` of a group
__device__ __forceinline__ uint32_t place_of(u32x4 words, uint32_t place, int in) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = in - 32 * i;
    place += __popc(words[i] & (n >= 32 ? ~0u : n > 0 ? (1u << n) - 1 : 0u));
  }
  return place;
}

// Words of a part: a group has four (of 32 words two).
constexpr int part_of(int group) { return group == 128 ? 32 : 16; }

// x of the lanes l, l ^ 16, l ^ 32 and l ^ 48 joined by f, in all of them
template <typename F>
__device__ __forceinline__ float across(float x, F f) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

enum Epi : int { kStat = 0, kGrad = 1, kDh = 2, kDw = 3, kPick = 4, kGradTwo = 5 };
struct Mma {
  Opnd A, B;                // C (M x N), M = A.rows, N = B.rows
  int64_t K;                // a multiple of 64
  int64_t k_slice;          // k per slice (grid y), a multiple of 64
  const float* zs;          // kStat, kGrad, kPick: the factor of the products (fp32: of each token;
  float z0;                 // 16-bit: z0)
  const float* ws;          // kPick, fp32: and of each word (to the next multiple of 256)
  // kStat, kGrad, kGradTwo: rows are words v0 .., columns tokens
  int64_t v0;
  const int32_t* labels;
  float *top, *sum, *hit;   // kStat: partials [half tiles of words][N], target logits
  const float *lse, *wn;    // kGrad: lse and normalised dloss per token
  uint16_t* G;              // kGrad: [token][term][gld]; kGradTwo: two terms of 16 bits, for
  int64_t gld, lines;       // tokens below lines
  // kDh, kDw: rows are the d columns, columns tokens or words
  float* part;              // kDh: slices of N x ldo fp32
  int64_t slice, ldo;
  int add;                  // kDh: add to what part holds
  const float* post;        // kDw: the factor of the results (one float)
  void* out;                // kDw
  Kept kept;                // kPick
};
constexpr bool a_major(int epi) { return epi == kDh || epi == kDw; }
constexpr bool b_major(int epi) { return epi == kDw; }

// Tile order: workgroup b runs on XCD b % 8, which takes consecutive indices;
// indices run down bands of 4 tile rows, so that the 32 tiles an XCD holds at
// once form a 4 x 8 block and share operands in its L2.
__device__ __forceinline__ bool tile_of(uint32_t bx, uint32_t ntm, uint32_t ntn, int64_t& tm, int64_t& tn) {
  const uint32_t nt = ntm * ntn, per = (nt + 7) / 8;   // (< 2^31: 2^24 x 2^20 outputs at most)
  const uint32_t t = (bx & 7) * per + (bx >> 3);
  if ((bx >> 3) >= per || t >= nt) return false;
  const uint32_t band = t / (4 * ntn), idx = t - band * 4 * ntn;
  const uint32_t h = min(4u, ntm - 4 * band);
  tm = 4 * band + idx % h;
  tn = idx / h;
  return true;
}

// One operand's tile: R rows (k-contiguous) or columns (k-major) of 64 k, R *
// 128 bytes per stage, brought from memory to LDS by NC copies of 1 KB per
// wave.
//   k-contiguous: LDS rows of 64 k (128 bytes, eight 16-byte slots); row r
//   keeps k-octet q in slot q ^ ((r >> 1) & 7), so that the 16 lanes that read
//   one octet of 16 consecutive rows hit distinct banks.
//   k-major: LDS rows of R columns (2 R bytes, 32-byte chunks); row k keeps
//   chunk c in place c ^ ((k & 3) + 4 ((k >> 3) & 1)), or for R = 64, where two
//   rows fill the banks, c ^ (((k >> 1) & 1) + 2 ((k >> 3) & 1)), so that the
//   eight rows that half a wave reads at once hit distinct banks.
// A fragment is 16 rows or columns of 32 k: lane (li, g) holds row li, k 8 g ..
// 8 g + 7. In the k-major form two transposing reads of 4 k each fill it: in
// each 16 lanes, lane i addresses row i / 4, columns 4 (i % 4) .., and receives
// column i.
template <int R>
__device__ __forceinline__ int place(int k) {
  return R == 64 ? ((k >> 1) & 1) + 2 * ((k >> 3) & 1) : (k & 3) + 4 * ((k >> 3) & 1);
}
template <int R, int NC, bool MAJOR>
struct Tile {
  static constexpr int kRowsPer = MAJOR ? 512 / R : 8;   // LDS rows per copy
  const uint16_t* base;
  int64_t ld, kv, left;   // left: bytes from base to the operand's end
  // Copies c of a wave come in two kinds, by the swizzle of their rows: even
  // and odd ones, or (k-major, four rows each) the first and the last two.
  static constexpr int kind(int c) { return MAJOR && R == 128 ? c >> 1 : c & 1; }
  static constexpr int first(int q) { return MAJOR && R == 128 ? 2 * q : q; }
  uint32_t off[2];        // byte offset of the lane in the copies of a kind, from their first row
  int koct[2];            // k-contiguous: the lane's octet in them

  __device__ __forceinline__ void init(const Opnd& o, int64_t r0, int wave, int lane) {
    ld = o.ld;
    kv = o.kv;
    const int64_t end = o.plane ? o.ld : MAJOR ? (o.rows + 7) / 8 * 8 : o.kv;   // of the last row
    if constexpr (MAJOR) {
      static_assert(NC % 2 == 0 && NC * kRowsPer % 8 == 0, "rows of a wave");
      const int k0 = wave * NC * kRowsPer;
      base = o.p + r0 + k0 * o.ld;
      left = ((o.kv - 1 - k0) * o.ld + end - r0) * 2;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int k = k0 + first(c) * kRowsPer + lane * 16 / (2 * R), slot = lane * 16 % (2 * R) / 16;
        const int chunk = (slot >> 1) ^ place<R>(k);
        off[c] = (uint32_t)(((int64_t)(lane * 16 / (2 * R)) * o.ld + 16 * chunk + 8 * (slot & 1)) * 2);
      }
    } else {
      const int64_t r = r0 + wave * NC * 8;
      base = o.p + r * o.ld;
      left = ((o.rows - 1 - r) * o.ld + end) * 2;
      static_assert(NC % 2 == 0, "copies in pairs");
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        koct[c] = (lane & 7) ^ (4 * c + (lane >> 4));
        off[c] = (uint32_t)(((lane >> 3) * o.ld + 8 * koct[c]) * 2);
      }
    }
  }
  // The copies of a stage of 64 k: start() and next() say which, aim() makes them ready, put()
  // sends one. What lies past the operand's end reads as zero (the descriptor's range, which
  // counts the vector offset alone: all of an address below its base is in it).
  uint64_t at;            // address of the stage
  int64_t rest;           // bytes from there to the operand's end
  int more;               // k from there to kv
  // the stage from k on, of the term `plane` elements into the rows
  __device__ __forceinline__ void start(int64_t k, int64_t plane) {
    const int64_t skip = 2 * ((MAJOR ? k * ld : k) + plane);
    at = (uint64_t)(uintptr_t)base + skip;
    rest = left - skip;
    more = (int)(kv - k);
  }
  __device__ __forceinline__ void next() {
    const int64_t skip = 2 * (MAJOR ? BK * ld : BK);
    at += skip;
    rest -= skip;
    more -= BK;
  }
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  i32x4 range;            // the descriptor
  int to;
  uint32_t o[2], step;
  // To LDS offset st. (!live: copies of zeros, which read nothing.) In 32-bit steps and without a
  // branch: it runs between products.
  __device__ __forceinline__ void aim(bool live, uint32_t st, int wave) {
    const int high = (int)(rest >> 32);
    const uint32_t low = (uint32_t)rest;
    const int n = high < 0 ? 0 : high > 0 || low > 0x7fffffffu ? 0x7fffffff : (int)low;
    range = i32x4{(int)at, (int)(at >> 32) & 0xffff, live ? n : 0, 0x20000};
    to = (int)st + wave * NC * 1024;
    step = (uint32_t)(kRowsPer * ld * 2);
    // (octets past kv: past any descriptor's range)
#pragma unroll
    for (int c = 0; c < 2; ++c) o[c] = !MAJOR && 8 * koct[c] >= more ? 0x80000000u : off[c];
  }
  // Copy c. Written out: after a builtin's every transposing read would wait
  // for it, though it is for the next stage. It writes no register, sync()
  // waits for it, and it keeps its place among the reads and sync()s. (Five states from
  // whatever wrote the descriptor, as a vector instruction's result would need.)
  __device__ __forceinline__ void put(int c) const {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // (m0 is reserved: nothing is kept in it across)
    asm volatile(
        "s_add_u32 m0, %1, %2\n\t"
        "s_nop 3\n\t"
        "buffer_load_dwordx4 %3, %0, 0 offen lds"
        :
        : "s"(range), "s"(to), "i"(c * 1024), "v"(o[kind(c)] + c * step)
        : "m0", "scc");
#pragma clang diagnostic pop
  }
};
// Fragments of the N 16-row groups from group g0 on, half h (32 k) of a stage.
template <int R, int N, bool MAJOR>
struct Reader {
  int at[MAJOR ? N : 2];

  __device__ __forceinline__ void init(int g0, int g, int li) {
    if constexpr (MAJOR) {
      const int f = place<R>(8 * g + (li >> 2));
#pragma unroll
      for (int j = 0; j < N; ++j)
        at[j] = (8 * g + (li >> 2)) * 2 * R + (((g0 + j) ^ f) << 5) + (li & 3) * 8;
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) at[h] = (g0 * 16 + li) * 128 + (((4 * h + g) ^ (li >> 1)) << 4);
    }
  }
  __device__ __forceinline__ u32x4 read(uint8_t* st, int j, int h) const {
    if constexpr (MAJOR) {
      uint8_t* p = st + at[j] + 32 * h * 2 * R;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_tr_t)(p + 4 * 2 * R));
      const u32x2 a = __builtin_bit_cast(u32x2, lo), b = __builtin_bit_cast(u32x2, hi);
      return u32x4{a[0], a[1], b[0], b[1]};
    } else {
      return *(const u32x4*)(st + at[h] + j * 2048);
    }
  }
};

// WM x WN waves of 16 MI x 16 NI (MI >= NI). NS stages of 64 k in LDS; a
// stage's copies go out as soon as everyone has read the stage that they
// replace, NS - 2 stages, a half-stage of products and more before they are
// waited for. (NS: mma_launch.)
// Bound by how the copies and the products share a CU: 4096 tokens, 131072 words,
// d = 4096 in bf16, kStat 3.26 ms and, in eight pieces, kGrad, kDh and kDw 3.3 to
// 3.5: 1.25 to 1.35 PFLOP/s (a large bf16 product of the library 1.27, one of 8192^3
// 1.62; matrix instructions alone 2.2; under this load the clock is 1.94 GHz, at
// which the matrix cores work 63 to 68 % of the time). fp32, 1024 tokens, 32000
// words, d = 2048: 0.37 to 0.44 ms each, 305 to 360 TFLOP/s. What a stage needs beside
// products, reads and copies is kept off their way: its addresses go on by steps, in
// 32-bit scalar operations between the products of the half before, and the compiler knows
// which reads have come (all of it after the barrier, and a wait for every read at the
// loop's head: kStat 3.56 ms, fp32 0.49 for 0.46). Four waves of 128 x 128, which read a
// third less from LDS but have nobody to work while they wait: 3.8.
template <int D, int EPI, int WM, int WN, int MI, int NI, int NS>
__device__ __forceinline__ void mma_body(const Mma a, uint32_t bx, uint32_t by, uint8_t* lds) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NI * WN, W = WM * WN;
  constexpr int kStage = (BM + BN) * 128;
  constexpr int CA = BM / 8 / W, CB = BN / 8 / W;
  static_assert(CA * 8 * W == BM && CB * 8 * W == BN, "copies");
  constexpr bool AM = a_major(EPI), BM_ = b_major(EPI), F16 = D != kBF16;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int wm = wave / WN, wn = wave % WN;
  const int64_t M = a.A.rows, N = a.B.rows;
  int64_t tm, tn;
  if (!tile_of(bx, (uint32_t)((M + BM - 1) / BM), (uint32_t)((N + BN - 1) / BN), tm, tn)) return;
  const int64_t m0 = tm * BM, n0 = tn * BN;
  const int64_t k_lo = (int64_t)by * a.k_slice;
  const int nk = (int)((lmin(a.K, k_lo + a.k_slice) - k_lo) / BK);
  const int steps = nk * passes(D);

  Tile<BM, CA, AM> ta;
  Tile<BN, CB, BM_> tb;
  ta.init(a.A, m0, wave, lane);
  tb.init(a.B, n0, wave, lane);
  Reader<BM, MI, AM> ra;
  Reader<BN, NI, BM_> rb;
  ra.init(wm * MI, g, li);
  rb.init(wn * NI, g, li);
  // passes: h l, l h, h h (the small ones first: what they round is 2^-11 of a
  // sum with h h in it)
  int pass = 0, kt = 0;
  ta.start(k_lo, 0);
  tb.start(k_lo, D == kF32 ? a.B.plane : 0);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  // the next stage's copies, ready to go to `stage`
  auto aim_a = [&](int stage, bool live) {
    ta.aim(live, lds0 + stage * kStage, wave);
    ta.next();
  };
  auto aim_b = [&](int stage, bool live) {
    tb.aim(live, lds0 + stage * kStage + BM * 128, wave);
    tb.next();
    if constexpr (D == kF32) {
      if (++kt == nk) {
        kt = 0;
        ++pass;
        ta.start(k_lo, pass == 1 ? a.A.plane : 0);
        tb.start(k_lo, 0);
      }
    }
  };
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  u32x4 fa[2][MI], fb[2][NI];
  // Multiplies half h while the other half's fragments come from stage st, and
  // with COPY the copies made ready go out: a row of products, its reads and
  // copies at a time (a run of copies would hold up the products behind it), and with(row).
  auto phase = [&](auto half, auto copies, uint8_t* st, auto with) {
    constexpr int h = decltype(half)::value;
    constexpr bool COPY = decltype(copies)::value;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i < NI) fb[h ^ 1][i] = rb.read(st + BM * 128, i, h ^ 1);
      fa[h ^ 1][i] = ra.read(st, i, h ^ 1);
      with(i);
#pragma unroll
      for (int j = 0; j < NI; ++j) acc[i][j] = mma<F16>(fa[h][i], fb[h][j], acc[i][j]);
      if constexpr (COPY) {
#pragma unroll
        for (int c = i * (CA + CB) / MI; c < (i + 1) * (CA + CB) / MI; ++c) {
          if (c < CA)
            ta.put(c);
          else
            tb.put(c - CA);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // each wave waits for its reads and for its own copies, but for those of the
  // last `ahead` stages, then for the other waves
  auto sync = [&](auto ahead) {
    __builtin_amdgcn_sched_barrier(0);    // (products before it stay before it)
    __builtin_amdgcn_s_waitcnt(0xc07f);   // lgkmcnt(0) once more, for the compiler's own count of reads
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(decltype(ahead)::value * (CA + CB))
                 : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // (copies of stages past the last bring zeros and read nothing: a branch
  // around them would cost more, and every wait counts the same)
#pragma unroll 1
  for (int st = 0; st < NS; ++st) {
    aim_a(st, st < steps);
    aim_b(st, st < steps);
#pragma unroll
    for (int c = 0; c < CA; ++c) ta.put(c);
#pragma unroll
    for (int c = 0; c < CB; ++c) tb.put(c);
  }
  sync(std::integral_constant<int, NS - 1>{});
#pragma unroll
  for (int j = 0; j < NI; ++j) fb[0][j] = rb.read(lds + BM * 128, j, 0);
#pragma unroll
  for (int i = 0; i < MI; ++i) fa[0][i] = ra.read(lds, i, 0);
  typedef std::integral_constant<int, 0> H0;
  typedef std::integral_constant<int, 1> H1;
  int cur = 0;
  for (int s = 0; s < steps; ++s) {
    const int next = cur + 1 == NS ? 0 : cur + 1;
    phase(H0{}, std::false_type{}, lds + cur * kStage, [&](int i) {
      if (i == MI / 2 - 1) aim_a(cur, s + NS < steps);
      if (i == MI / 2) aim_b(cur, s + NS < steps);
    });
    // the next stage has landed; everyone has read this one
    sync(std::integral_constant<int, NS - 2>{});
    // (after the last stage this reads what is there, for nothing)
    phase(H1{}, std::true_type{}, lds + next * kStage, [](int) {});
    cur = next;
  }
  // the last copies must land before this workgroup's LDS is given away
  sync(std::integral_constant<int, 0>{});

  // lane (g, li), element v of tile (i, j): row 16 i + 4 g + v, column 16 j + li
  const int64_t r0 = m0 + wm * MI * 16 + 4 * g, c0 = n0 + wn * NI * 16 + li;
  // kStat, kGrad: element (i, v) is a word if 16 i + v < left, a token's label if
  // it is own() (-1: not one of the lane's)
  const int left = (int)lmax(lmin(M - r0, 16 * MI), 0);
  auto own = [&](int32_t label) {
    const int64_t at = label - a.v0 - r0;
    return label >= 0 && at >= 0 && at < 16 * MI && (at & 15) < 4 ? (int)at : -1;
  };
  if constexpr (EPI == kStat) {
    const int64_t half = a.v0 / (16 * MI) + tm * WM + wm;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const int32_t label = t < N ? a.labels[t] : -1;
      const float zs = D == kF32 ? (t < N ? a.zs[t] : 0.0f) : a.z0;
      float top = kNegInf, low = 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          acc[i][j][v] *= zs;
          if (16 * i + v < left) top = fmaxf(top, acc[i][j][v]);
          low = fminf(low, acc[i][j][v]);   // (0 for rows past the last word)
        }
      const int at = own(label);
      if (at >= 0 && at < left) {   // (one lane of all tiles: no branch per element)
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) z = 16 * i + v == at ? acc[i][j][v] : z;
        a.hit[t] = z;
      }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          sum += 16 * i + v < left ? __expf(acc[i][j][v] - top) : 0.0f;
      sum = low == kNegInf ? __uint_as_float(0x7fc00000u) : sum;   // (an infinity in W: exp makes it 0)
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0 && t < N) {
        a.top[half * N + t] = top;
        a.sum[half * N + t] = sum;
      }
    }
  } else if constexpr (EPI == kPick) {
    // z = acc zs with zs made positive, so that the largest acc is the largest z, e = 2^((acc
    // - largest) zs log2 e) without a scaled z, and dot is NaN where an acc is not finite
    // (0 times infinity, too). 777 tokens, 50021 x 1000 fp16, in us: with kStat the kernel takes 142,
    // with this 147 to 151, with 100 listed words of each token 164.
    const Kept& o = a.kept;
    const int64_t group = a.v0 / (16 * MI) + tm * WM + wm;
    if constexpr (D == kF32) {   // (factors of words differ: z itself)
      float zs[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) zs[j] = c0 + 16 * j < N ? a.zs[c0 + 16 * j] : 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const f32x4 ws = *(const f32x4*)(a.ws + r0 + 16 * i);
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] *= ws * zs[j];
      }
    } else if (o.flip) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = -acc[i][j];
    }
    // what the tokens need from memory, all of it before the first use
    float zsj[NI], thrj[NI];
    uint32_t minej[NI];   // bit 4 i + v: a listed word
    int slotj[NI];
    // bit 4 i + v: past the last word
    uint32_t past = 0;
    if (m0 + (wm + 1) * MI * 16 > M) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) past |= (uint32_t)(16 * i + v >= left) << (4 * i + v);
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const bool used = t < N && group < o.groups;
      zsj[j] = D == kF32 ? 1.0f : fabsf(a.z0);
      thrj[j] = used && o.thr ? o.thr[t] : kNegInf;
      slotj[j] = used && o.slot ? o.slot[t * o.lds + group] : 255;
    }
    u32x4 words[NI];
    uint32_t place[NI];
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      words[j] = u32x4{0, 0, 0, 0};
      place[j] = 0;
      if (slotj[j] != 255) {
        const Mark& m = o.marks[(c0 + 16 * j) * o.listed + slotj[j]];
        words[j] = m.words;
        place[j] = m.place;
      }
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      minej[j] = 0;
      if (!__ballot(slotj[j] != 255)) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const uint32_t four = words[j][i / 2] >> (16 * (i & 1) + 4 * g) & 15u;
        minej[j] |= four << (4 * i);
        if (__ballot(four)) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (four >> v & 1u)
              o.zl[(c0 + 16 * j) * o.listed + place_of(words[j], place[j], 16 * i + 4 * g + v)] = acc[i][j][v] * zsj[j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const bool used = t < N && group < o.groups;
      const float zs = zsj[j], thr = thrj[j];
      const uint32_t mine = minej[j];
      const uint32_t off = past | (o.without ? mine : 0u);   // bits of words that are left out
      // all ones for a word that is not
      auto on = [&](int bit) { return (uint32_t)((int)(~off << (31 - bit)) >> 31); };
      // parts of the group: PI row tiles each
      constexpr int PARTS = 16 * MI / part_of(16 * MI), PI = MI / PARTS;
      float tops[PARTS], top = kNegInf, sum = 0.0f, dot = 0.0f, r;
      const float by = zs * 1.44269504f;
      auto add = [](float x, float y) { return x + y; };
      auto sums = [&](auto whole) {   // (whole: no word is left out)
        constexpr bool ALL = decltype(whole)::value;
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          float x = kNegInf;
#pragma unroll
          for (int i = q * PI; i < (q + 1) * PI; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v)
              x = fmaxf(x, ALL ? acc[i][j][v]
                               : __uint_as_float((__float_as_uint(acc[i][j][v]) & on(4 * i + v)) |
                                                 (0xff800000u & ~on(4 * i + v))));
          tops[q] = across(x, [](float x, float y) { return fmaxf(x, y); });
          top = fmaxf(top, tops[q]);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const float y = (acc[i][j][v] - top) * by;
            float e = __builtin_amdgcn_exp2f(y);
            if (!ALL) e = __uint_as_float(__float_as_uint(e) & on(4 * i + v));
            sum += e;
            dot = fmaf(e, y, dot);
          }
        sum = across(sum, add);
        dot = across(dot, add);
        r = sum - 1.0f;
        // a group that is all but one word: what r leaves out of 2^-4 of it is summed by itself
        if (__ballot(sum < 1.0625f)) {
          float ones = 0.0f, rest = 0.0f;
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              const float y = acc[i][j][v] - top;
              const bool in = ALL || !(off >> (4 * i + v) & 1u);
              ones += in && y == 0.0f ? 1.0f : 0.0f;
              rest += in && y != 0.0f ? __builtin_amdgcn_exp2f(y * by) : 0.0f;
            }
          r = across(rest, add) + (across(ones, add) - 1.0f);
        }
        // (no word left: a sum of 0)
        constexpr uint32_t every = MI == 8 ? ~0u : (1u << (4 * MI & 31)) - 1;
        if (!ALL && across(off == every ? 0.0f : 1.0f, add) == 0.0f) dot = 0.0f;
      };
      if (!__ballot(off))
        sums(std::true_type{});
      else
        sums(std::false_type{});
      if (!used) continue;
      if (g == 0) {
        // (the largest z past fp32's range, of a finite acc: not finite either, unless there is no word)
        const bool fine = dot == dot && (fabsf(top * zs) < __builtin_inff() || r == -1.0f);
        o.stat[t * o.groups + group] = f32x4{top * zs, fine ? r : __uint_as_float(0x7fc00000u), dot * 0.69314718f, 0.0f};
        if (o.tops) {
          float* p = o.tops + (t * o.groups + group) * PARTS;
#pragma unroll
          for (int q = 0; q < PARTS; q += 2) *(u32x2*)(p + q) = u32x2{__float_as_uint(tops[q] * zs), __float_as_uint(tops[q + 1] * zs)};
        }
      }
      auto put = [&](float* p, int i) {   // (of words past the last too: rows hold whole groups)
        *(f32x4*)(p + 16 * i + 4 * g) = acc[i][j] * zs;
      };
      if (o.z) {
        float* p = o.z + t * o.ldz + (tm * WM + wm) * (16 * MI);
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
          if (!o.thr || !(tops[q] * zs <= thr)) {
#pragma unroll
            for (int i = q * PI; i < (q + 1) * PI; ++i) put(p, i);
          }
      }
    }
  } else if constexpr (EPI == kGrad || EPI == kGradTwo) {
    constexpr int P = EPI == kGradTwo ? kFewTerms : terms(D);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const int32_t label = t < N ? a.labels[t] : -1;
      const float lse = label >= 0 ? a.lse[t] : 0.0f, wn_t = label >= 0 ? a.wn[t] : 0.0f;
      const float zs = D == kF32 ? (label >= 0 ? a.zs[t] : 0.0f) : a.z0;
      const int at = own(label), used = label >= 0 ? left : 0;
      uint16_t* row = a.G + t * a.gld * P;
      if (EPI == kGradTwo && t >= a.lines) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        uint16_t q[4][P];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float y = zs * acc[i][j][v] - lse;
          float x = D == kF32 ? expf(y) : __expf(y);
          if (16 * i + v == at) x -= 1.0f;
          x = 16 * i + v < used ? x * wn_t : 0.0f;
          split<D>(x, q[v]);
        }
#pragma unroll
        for (int p = 0; p < P; ++p)
          *(u32x2*)(row + p * a.gld + r0 + 16 * i) =
              u32x2{(uint32_t)q[0][p] | (uint32_t)q[1][p] << 16,
                    (uint32_t)q[2][p] | (uint32_t)q[3][p] << 16};
      }
    }
  } else if constexpr (EPI == kDh) {
    float* part = a.part + (int64_t)by * a.slice;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      if (t >= N) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int64_t c = r0 + 16 * i;   // (ldo is a multiple of 4 and covers c + 3)
        if (c >= M) continue;
        f32x4* p = (f32x4*)(part + t * a.ldo + c);
        *p = a.add ? *p + acc[i][j] : acc[i][j];
      }
    }
  } else {
    typedef typename Elem<D>::type E;
    const float post = *a.post;
    E* out = (E*)a.out;
    const bool vec = a.ldo % 4 == 0 && (uintptr_t)out % (4 * sizeof(E)) == 0;
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t w = c0 + 16 * j;
      if (w >= N) continue;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int64_t c = r0 + 16 * i;
        E e[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) e[v] = Elem<D>::from(acc[i][j][v] * post);
        E* p = out + w * a.ldo + c;
        if (vec && c + 4 <= M) {
          __builtin_memcpy(__builtin_assume_aligned(p, 4 * sizeof(E)), e, sizeof(e));
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (c + v < M) p[v] = e[v];
        }
      }
    }
  }
}

template <int D, int EPI, int WM, int WN, int MI, int NI, int NS>
__global__ __launch_bounds__(64 * WM * WN) void mma_kernel(Mma a) {
  __shared__ __align__(16) uint8_t lds[NS * 16 * (MI * WM + NI * WN) * 128];
  mma_body<D, EPI, WM, WN, MI, NI, NS>(a, blockIdx.x, blockIdx.y, lds);
}
// Two products in one launch, dH's and dW's, in 128 x 128 tiles: where neither fills the chip. nh
// workgroups are dH's, nx to a slice.
template <int D, int NS>
__global__ __launch_bounds__(256) void pair_kernel(Mma h, Mma w, uint32_t nh, uint32_t nx) {
  __shared__ __align__(16) uint8_t lds[NS * 256 * 128];
  if (blockIdx.x < nh)
    mma_body<D, kDh, 2, 2, 4, 4, NS>(h, blockIdx.x % nx, blockIdx.x / nx, lds);
  else
    mma_body<D, kDw, 2, 2, 4, 4, NS>(w, blockIdx.x - nh, 0, lds);
}

// ---------------------------------------------------------------- few tokens
// 64 words and all T <= 16 NT tokens per workgroup of 16 / NT waves, which take
// 32 columns each in turn: neighbours read neighbouring 64 bytes of a row, and
// many waves with one load per row each keep HBM busiest (4096 x 32000 bf16, 16
// tokens, in us with the join: 16 waves 59 (4.4 TB/s), 8 waves 63, 4 waves 96;
// 8 waves of 64 columns 71, 4 waves of 128 columns 80, of two such runs in
// registers 84). Eight values are loaded together from any address (rows that are
// not 16-byte aligned: 3 tokens, 6673 x 68774 fp16 296 us, one by one 727). At the
// end of a row the last eight are loaded, and of H those that came before are
// zeroed (d >= 8).
template <int D>
struct __attribute__((packed)) Raw8 {
  typename Elem<D>::type e[8];
};
// x = h + m + l in bf16, exact, of two values at a time (which is how they are converted: 7.5
// operations a value, 13 one by one: 33 tokens, 27271 x 7872, 244 us and 293); not finite: the first term alone
__device__ __forceinline__ void split3(float x, float y, uint32_t (&t)[3]) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    t[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), bf16x2));
    if (p == 2) break;
    x -= __uint_as_float(t[p] << 16);
    y -= __uint_as_float(t[p] & 0xffff0000u);
    if (p == 0) {
      x = fabsf(x) < __builtin_inff() ? x : 0.0f;
      y = fabsf(y) < __builtin_inff() ? y : 0.0f;
    }
  }
}
constexpr int score_terms(int D) { return D == kF32 ? 3 : 1; }
template <int D>
struct Frag {
  u32x4 t[score_terms(D)];
};
template <int D>
__device__ __forceinline__ Frag<D> frag_of(const Raw8<D>& r) {
  Frag<D> f;
  if constexpr (D == kF32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t q[3];
      split3(r.e[2 * i], r.e[2 * i + 1], q);
#pragma unroll
      for (int p = 0; p < 3; ++p) f.t[p][i] = q[p];
    }
  } else {
    __builtin_memcpy(&f.t[0], &r, 16);
  }
  return f;
}
// the six products of bf16 terms: term of A and of B (2 bits each)
__device__ __forceinline__ int term_a(int s) { return (0x250 >> (2 * s)) & 3; }   // 0 0 1 1 2 0
__device__ __forceinline__ int term_b(int s) { return (0x844 >> (2 * s)) & 3; }   // 0 1 0 1 0 2

// What score_kernel gives: per token and 64 words the largest z and the sum of
// exponentials, and the label's z; or G of the words from v0 on, zero up to the
// next multiple of 64, [token][term][gld]; or (Kept) all z and the groups' sums.
struct ScoreStat {
  float *top, *sum, *hit;
};
struct ScoreGrad {
  const float *lse, *wn;
  uint16_t* G;
  int64_t gld, v0;
};
// Eight 16-bit values from an address that may not be a multiple of 4: words of 4 bytes are loaded
// and shifted (`at`: bytes from `base`, which is such a multiple). Each word loaded holds a byte
// that is asked for. Loads of 16 bytes from such addresses take twice the time where a row has 64 bytes
// of a load (4 tokens, 34797 x 5825 bf16: 239 us, shifted 151; 20 tokens 294 and 233; rows of 5826,
// at multiples of 4, 115 as they are). The values are the same.
template <int D>
__device__ __forceinline__ Raw8<D> shifted(const char* base, uint32_t at) {
  struct __attribute__((packed, aligned(4))) Words { uint32_t v[4]; } w;
  const char* p = base + (at & ~3u);
  __builtin_memcpy(&w, __builtin_assume_aligned(p, 4), 16);
  const uint32_t by = (at & 2u) * 8;
  const uint32_t more = *(const uint32_t*)(p + (by ? 16 : 12));
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __builtin_amdgcn_alignbit(i < 3 ? w.v[i + 1] : more, w.v[i], by);
  Raw8<D> r;
  __builtin_memcpy(&r, o, 16);
  return r;
}
// (64 registers or fewer: two workgroups of 1024 threads per CU. ODD: rows of W, or of H, that do not
// start at multiples of 4 bytes)
template <int D, int NT, bool ODD, typename OUT>
__global__ __launch_bounds__(1024 / NT)
    __attribute__((amdgpu_waves_per_eu(D != kF32 && NT == 1 ? 8 : 1))) void score_kernel(
        const typename Elem<D>::type* __restrict__ H, int64_t ldh,
        const typename Elem<D>::type* __restrict__ W, int64_t ldw, int64_t T, int64_t V, int64_t d,
        const int32_t* __restrict__ labels, float scale, OUT o) {
  constexpr int NW = 16 / NT;
  constexpr bool GRAD = std::is_same_v<OUT, ScoreGrad>, PICK = std::is_same_v<OUT, Kept>;
  __shared__ f32x4 red[NW][4 * NT][64];
  __shared__ float st[PICK ? 4 : 2][4][GRAD ? 1 : 16 * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t v0 = (int64_t)blockIdx.x * 64;
  // byte offsets of the rows (64 rows of 2^21 values at most: 32 bits)
  constexpr int kSize = sizeof(typename Elem<D>::type);
  const char *Wb = (const char*)(W + v0 * ldw), *Hb = (const char*)H;
  const uint32_t in = ODD ? (uint32_t)(uintptr_t)Wb & 2u : 0u, inh = ODD ? (uint32_t)(uintptr_t)Hb & 2u : 0u;
  Wb -= in;
  Hb -= inh;
  uint32_t wr[4], hr[NT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wr[i] = (uint32_t)lmin(16 * i + li, V - 1 - v0) * (uint32_t)(ldw * kSize);
#pragma unroll
  for (int j = 0; j < NT; ++j) hr[j] = (uint32_t)lmin(16 * j + li, T - 1) * (uint32_t)(ldh * kSize);
  f32x4 acc[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave * 32; k0 < d; k0 += 32 * NW) {
    const int k = min(k0 + 8 * g, (int)d - 8);
    const uint32_t at = k * kSize;
    Raw8<D> w[4], h[NT];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (ODD)
        w[i] = shifted<D>(Wb, wr[i] + at + in);
      else
        __builtin_memcpy(&w[i], Wb + (wr[i] + at), sizeof(w[i]));
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if constexpr (ODD)
        h[j] = shifted<D>(Hb, hr[j] + at + inh);
      else
        __builtin_memcpy(&h[j], Hb + (hr[j] + at), sizeof(h[j]));
    }
    __builtin_amdgcn_sched_barrier(0);   // (all loads before the first product)
    if (k0 + 32 > d) {
      const int before = k0 + 8 * g - k;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j].e[i] = i < before ? (typename Elem<D>::type)0 : h[j].e[i];
    }
    Frag<D> b[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) b[j] = frag_of<D>(h[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const Frag<D> f = frag_of<D>(w[i]);
#pragma unroll
      for (int q = 0; q < (D == kF32 ? 6 : 1); ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = mma<D == kF16>(f.t[D == kF32 ? term_a(q) : 0],
                                     b[j].t[D == kF32 ? term_b(q) : 0], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[wave][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  // wave i joins the 16 words of row tile i
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    if (wave >= 4) break;
    const int e = wave * NT + j;
    f32x4 z = red[0][e][lane];
#pragma unroll 4
    for (int n = 1; n < NW; ++n) z += red[n][e][lane];
    const int64_t t = 16 * j + li, w = v0 + 16 * wave + 4 * g;
    const int32_t label = !PICK && t < T ? labels[t] : -1;
    if constexpr (GRAD) {
      if (t >= T) continue;
      const float lse = label >= 0 ? o.lse[t] : 0.0f, wn = label >= 0 ? o.wn[t] : 0.0f;
      uint16_t q[4][kFewTerms];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float y = scale * z[v] - lse;
        float x = D == kF32 ? expf(y) : __expf(y);
        if (o.v0 + w + v == label) x -= 1.0f;
        x = label >= 0 && w + v < V ? x * wn : 0.0f;
        split<D>(x, q[v]);
      }
#pragma unroll
      for (int p = 0; p < kFewTerms; ++p)
        *(u32x2*)(o.G + (t * kFewTerms + p) * o.gld + w) =
            u32x2{(uint32_t)q[0][p] | (uint32_t)q[1][p] << 16,
                  (uint32_t)q[2][p] | (uint32_t)q[3][p] << 16};
    } else {
      float m = kNegInf, x[4];
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x[v] = scale * z[v];
        if (w + v < V) m = fmaxf(m, x[v]);
        if constexpr (!PICK)
          if (w + v < V && w + v == label) o.hit[t] = x[v];
      }
      if constexpr (PICK)
        if (t < T) *(f32x4*)(o.z + t * o.ldz + w) = f32x4{x[0], x[1], x[2], x[3]};
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      float s = 0.0f;
      if constexpr (PICK) {   // (s: without the ones; what Kept says)
        float y = 0.0f, ones = 0.0f;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float a = x[v] - m, e = __expf(a);
          const bool on = w + v < V;
          ones += on && a == 0.0f ? 1.0f : 0.0f;
          s += !on || a == 0.0f ? 0.0f : x[v] == kNegInf ? __uint_as_float(0x7fc00000u) : e;
          y += on ? e * a : 0.0f;
        }
        ones += __shfl_xor(ones, 16);
        ones += __shfl_xor(ones, 32);
        y += __shfl_xor(y, 16);
        y += __shfl_xor(y, 32);
        if (g == 0) {
          st[2][wave][16 * j + li] = y;
          st[3][wave][16 * j + li] = ones - 1.0f;
        }
      } else {
#pragma unroll
        for (int v = 0; v < 4; ++v)   // (-infinity, of an infinity in W, is no zero but NaN)
          s += w + v >= V ? 0.0f : x[v] == kNegInf ? __uint_as_float(0x7fc00000u) : __expf(x[v] - m);
      }
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (g == 0) {
        st[0][wave][16 * j + li] = m;
        st[1][wave][16 * j + li] = s;
      }
    }
  }
  if constexpr (!GRAD) {
    __syncthreads();
    const int t = threadIdx.x;
    if (t < 16 * NT && t < T) {
      float m = kNegInf, s = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = fmaxf(m, st[0][i][t]);
      if constexpr (PICK) {
        float y = 0.0f, ones = -1.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = st[0][i][t] - m, e = __expf(a), r = st[1][i][t] + st[3][i][t];
          if (v0 + 16 * i < V) {
            ones += a == 0.0f ? 1.0f : 0.0f;
            s += a == 0.0f ? r : e * (1.0f + r);
            y += (st[2][i][t] + a * (1.0f + r)) * e;
          }
        }
        if (o.stat) o.stat[t * o.groups + blockIdx.x] = f32x4{m, s + ones, y, 0.0f};
        if (o.tops)
          *(f32x4*)(o.tops + (t * o.groups + blockIdx.x) * 4) = f32x4{st[0][0][t], st[0][1][t], st[0][2][t], st[0][3][t]};
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (v0 + 16 * i < V) s += st[1][i][t] * __expf(st[0][i][t] - m);
        o.top[(int64_t)blockIdx.x * T + t] = m;
        o.sum[(int64_t)blockIdx.x * T + t] = s;
      }
    }
  }
}

// ---------------------------------------------------------------- scales
// Factors of each token, read by the kernels that follow.
struct Rows {
  float *hz, *hw;        // powers of two that its row of H is scaled by, for z and for dW
  float *zs;             // scale / (hz mw): of its products (fp32)
  float *wn, *pt;        // of G, of its row of dH
  float *wr;             // wn times the token's share, where the call has shares
};
Rows rows_of(char* work, const Plan& p, int64_t T) {
  float* f = (float*)(work + p.rows);
  return {f, f + T, f + 2 * T, f + 3 * T, f + 4 * T, nullptr};
}
// The largest finite magnitudes: hm[t] of each row of H (y = 0; 0 for an ignored
// token, labels nullable), parts[x] of a share of W's rows (y = 1).
__global__ __launch_bounds__(256) void amax_kernel(const float* __restrict__ H, int64_t T,
                                                   int64_t ldh, const float* __restrict__ W,
                                                   int64_t V, int64_t ldw, int64_t d,
                                                   const int32_t* __restrict__ labels,
                                                   float* __restrict__ hm,
                                                   float* __restrict__ parts) {
  __shared__ float sm[256];
  struct __attribute__((packed)) Four { float v[4]; };
  float m = 0.0f;
  auto take = [&](float x) {
    const float v = fabsf(x);
    m = v < __builtin_inff() ? fmaxf(m, v) : m;
  };
  // four times 16 bytes at a time, from any address; rows and columns past the end
  // are clamped (a maximum may see a value twice), so that no branch parts the loads
  if (blockIdx.y == 0) {   // a wave per row
    const int lane = threadIdx.x & 63;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < T; t += 4 * (int64_t)gridDim.x) {
      const float* x = H + t * ldh;
      m = 0.0f;
      if (!labels || labels[t] >= 0) {
        if (d < 4) {
          for (int64_t c = lane; c < d; c += 64) take(x[c]);
        } else {
          for (int64_t c = 4 * lane; c < d; c += 1024) {
            Four q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) __builtin_memcpy(&q[u], x + lmin(c + 256 * u, d - 4), 16);
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) take(q[u].v[i]);
          }
        }
      }
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
      if (lane == 0) hm[t] = m;
    }
    return;
  }
  for (int64_t r0 = blockIdx.x; r0 < V; r0 += 4 * (int64_t)gridDim.x) {
    const float* x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) x[u] = W + lmin(r0 + u * (int64_t)gridDim.x, V - 1) * ldw;
    if (d < 4) {
      for (int64_t c = threadIdx.x; c < d; c += 256)
#pragma unroll
        for (int u = 0; u < 4; ++u) take(x[u][c]);
      continue;
    }
    for (int64_t c = 4 * threadIdx.x; c < d; c += 1024) {
      Four q[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) __builtin_memcpy(&q[u], x[u] + lmin(c, d - 4), 16);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) take(q[u].v[i]);
    }
  }
  sm[threadIdx.x] = m;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) sm[threadIdx.x] = fmaxf(sm[threadIdx.x], sm[threadIdx.x + o]);
    __syncthreads();
  }
  if (threadIdx.x == 0) parts[blockIdx.x] = sm[0];
}
// the largest of v over the workgroup's 1024 threads
__device__ __forceinline__ float max_of(float v, float* sm) {
  __syncthreads();
  sm[threadIdx.x] = v;
  __syncthreads();
  for (int o = 512; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) sm[threadIdx.x] = fmaxf(sm[threadIdx.x], sm[threadIdx.x + o]);
    __syncthreads();
  }
  return sm[0];
}
// e with m 2^e in (2^14, 2^15], in -126 .. 126
__device__ __forceinline__ int power_for(float m) {
  const uint32_t b = __float_as_uint(m);
  const int e = 14 - ((int)(b >> 23) - 127) + ((b & 0x7fffffu) == 0);
  return m > 0.0f ? min(max(e, -126), 126) : 0;
}
// The factors. With dloss = f 2^x per token (1/2 <= |f| < 1; x0 of the largest),
//   bf16:       G = (p - [label]) dloss / max|dloss|: its exponents reach far enough;
//   fp32:       G = (p - [label]) f 2^15 whatever the others' dloss are, dH's row
//               takes 2^(x - 15) at its end, and H's copy for dW 2^(x - x0);
//   fp16:       as fp32, but G keeps up to kInG bits of x - x0: it has 29 below its
//               top, of which 11 are asked for, where H, which is not scaled to its
//               type's top, has 14 where it is about 1.
// Where G is a divergence's, of up to Q in place of 1 (rows.wr; 1 for a teacher's probabilities), a
// token of Q >= 1.5 has the power of two above Q in its dloss, not in G.
// (0 for an ignored token; NaN for a label at or past V.) hm and parts (fp32
// operands): the maxima of H's rows and of W. One workgroup.
constexpr int kInG = 10;
template <int D>
__global__ __launch_bounds__(1024) void factors_kernel(const float* __restrict__ hm,
                                                       const float* __restrict__ parts,
                                                       const float* __restrict__ dloss,
                                                       const float* __restrict__ share,
                                                       const int32_t* __restrict__ labels,
                                                       int64_t T, int64_t V, float scale, Rows rows,
                                                       Factors* __restrict__ out) {
  __shared__ float sm[1024];
  int ew = 0;   // (scales are powers of two: factors by ldexp, rounded once at most)
  if (D == kF32) {
    ew = power_for(max_of(parts[threadIdx.x], sm));
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
      const int e = power_for(hm[t]);
      rows.hz[t] = ldexpf(1.0f, e);
      rows.zs[t] = ldexpf(scale, -(e + ew));
    }
  }
  if (!dloss) {
    if (threadIdx.x == 0) out->mw = ldexpf(1.0f, ew);
    return;
  }
  // the power of two that token t's G is taken down by
  auto down = [&](int64_t t) {
    int x = 0;
    if (D != kBF16 && share) {
      const float q = rows.wr[t];
      if (q >= 1.5f && q < __builtin_inff()) frexpf(q, &x);
    }
    return x;
  };
  // the largest of the finite ones
  float m = 0.0f;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const float v = labels[t] >= 0 ? ldexpf(fabsf(dloss[t]), down(t)) : 0.0f;
    m = v < __builtin_inff() ? fmaxf(m, v) : m;
  }
  m = max_of(m, sm);
  int x0 = 0;
  if (m > 0.0f) frexpf(m, &x0);
  // f and x of a token; x = x0 where dloss is 0 or not finite
  auto parted = [&](int64_t t, int& x) {
    x = x0;
    const float l = dloss[t];
    if (l == 0.0f || !(fabsf(l) < __builtin_inff())) return l;
    const float f = frexpf(l, &x);
    x += down(t);
    return f;
  };
  // fp32: H's copy for dW, weighted by 2^(x - x0), to 2^15 at its largest
  int eh = 0;
  if (D == kF32) {
    float e = 0.0f;
    for (int64_t t = threadIdx.x; t < T; t += 1024) {
      int x;
      if (labels[t] >= 0 && parted(t, x) != 0.0f) e = fmaxf(e, ldexpf(hm[t], x - x0));
    }
    eh = power_for(max_of(e, sm));
  }
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const int32_t label = labels[t];
    float wn, pt, hw = 0.0f;
    if (D == kBF16) {
      wn = m == 0.0f ? dloss[t] : dloss[t] / m;   // (none is finite and not zero)
      pt = m == 0.0f ? scale : m * scale;
    } else {
      int x;
      const float f = parted(t, x);
      const int k = D == kF16 ? min(x0 - x, kInG) : 0;
      wn = ldexpf(f, 15 - k - down(t));
      pt = ldexpf(scale, x + k - 15 - ew);
      hw = f == 0.0f ? 0.0f : ldexpf(1.0f, x + k - x0 + eh);
    }
    wn = label < 0 ? 0.0f : label < V ? wn : __uint_as_float(0x7fc00000u);
    rows.wn[t] = wn;
    if (share) rows.wr[t] = label < 0 ? 0.0f : wn * share[t];
    rows.pt[t] = label < 0 ? 0.0f : pt;
    rows.hw[t] = label < 0 ? 0.0f : hw;
    if (D == kF16) rows.hz[t] = 1.0f;
  }
  if (threadIdx.x == 0)
    *out = Factors{ldexpf(1.0f, ew),
                   D == kBF16 ? (m == 0.0f ? 1.0f : m) * scale : ldexpf(scale, x0 - 15 - eh)};
}

// ---------------------------------------------------------------- layout
// out [row][term][kp] = the terms of X (rows x k) times a factor, zero from k to
// kp, for rows past the last up to rp, and for rows whose label is negative (labels
// nullable); with twice, each row two times. Form z of the grid writes the z-th copy
// of out.
enum Mul : int {
  kAsIs = 0,      // 1
  kOne = 1,       // *mul
  kEachRow = 2,   // mul[z * rows + row]
};
template <int D, int M>
__global__ __launch_bounds__(256) void pack_kernel(const typename Elem<D>::type* __restrict__ X,
                                                   int64_t rows, int64_t k, int64_t ld,
                                                   const int32_t* __restrict__ labels,
                                                   const float* __restrict__ mul,
                                                   uint16_t* __restrict__ out, int64_t rp,
                                                   int64_t kp, int twice) {
  typedef typename Elem<D>::type E;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= kp) return;
  out += blockIdx.z * rp * kp * terms(D);
  for (int64_t r = blockIdx.y; r < rp; r += gridDim.y) {
    E e[8];
    const int64_t at = r >> twice;
    const bool row = at < rows && (!labels || labels[at] >= 0);
    const float f = M == kAsIs ? 1.0f : M == kOne ? *mul : row ? mul[blockIdx.z * rows + at] : 0.0f;
    if (row && c + 8 <= k) {
      __builtin_memcpy(e, X + at * ld + c, sizeof(e));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = row && c + i < k ? X[at * ld + c + i] : (E)0;
    }
    uint16_t q[8][terms(D)];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (M != kAsIs)
        split<D>(Elem<D>::to(e[i]) * f, q[i]);
      else
        q[i][0] = __builtin_bit_cast(uint16_t, e[i]);
    }
#pragma unroll
    for (int p = 0; p < terms(D); ++p) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)q[2 * i][p] | (uint32_t)q[2 * i + 1][p] << 16;
      *(u32x4*)(out + (r * terms(D) + p) * kp + c) = w;
    }
  }
}

// The two terms of each row of fp32 X (rows x k), scaled by a power of two of its own to 2^15 at
// their largest, zero from k to kp: out [row][term][kp]; unscale[row] = mul over the power, 0 from
// the last row to unscale[full]. A workgroup per row, which it reads twice where it is long. (512
// tokens, 32000 x 2048: a call of 336 us with a pass for W's largest value and pack_kernel, 295 with
// this, which takes 82: 6.4 TB/s.)
__global__ __launch_bounds__(256) void rowpack_kernel(const float* __restrict__ X, int64_t rows, int64_t k,
                                                      int64_t ld, float mul, uint16_t* __restrict__ out,
                                                      int64_t kp, float* __restrict__ unscale, int64_t full) {
  __shared__ float sm[4];
  if (blockIdx.x == 0)
    for (int64_t i = rows + threadIdx.x; i < full; i += 256) unscale[i] = 0.0f;
  struct __attribute__((packed)) Eight { float v[8]; };
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const float* x = X + r * ld;
    float m = 0.0f;
    auto load = [&](int64_t c, float (&e)[8]) {
      if (c + 8 <= k) {
        Eight q;
        __builtin_memcpy(&q, x + c, 32);
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = q.v[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = c + i < k ? x[c + i] : 0.0f;
      }
    };
    float first[8];
    for (int64_t c = 8 * threadIdx.x; c < kp; c += 2048) {
      float e[8];
      load(c, e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = fabsf(e[i]);
        m = v < __builtin_inff() ? fmaxf(m, v) : m;
        if (c < 2048) first[i] = e[i];
      }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
    __syncthreads();   // (sm of the row before has been read)
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    const int p = power_for(m);
    if (threadIdx.x == 0) unscale[r] = ldexpf(mul, -p);
    const float f = ldexpf(1.0f, p);
    for (int64_t c = 8 * threadIdx.x; c < kp; c += 2048) {
      float e[8];
      if (c < 2048) {
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = first[i];
      } else {
        load(c, e);
      }
      uint16_t q[8][2];
#pragma unroll
      for (int i = 0; i < 8; ++i) split<kF32>(e[i] * f, q[i]);
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)q[2 * i][n] | (uint32_t)q[2 * i + 1][n] << 16;
        *(u32x4*)(out + (r * 2 + n) * kp + c) = w;
      }
    }
  }
}

// ---------------------------------------------------------------- plan
// Whether X's rows can be copied as they are: 16-bit, 16-byte aligned.
bool direct(const void* X, int64_t ld, int64_t k, int dtype) {
  return dtype != kF32 && k % 8 == 0 && ld % 8 == 0 && (uintptr_t)X % 16 == 0;
}

// Four stages where there is one workgroup per CU at most, so that its LDS has
// no other use, and k is long enough to win their start back (301 tokens, 4999
// words of bf16: 8 stages of k 14 us with either, 16 stages 18 v 20, 32 stages
// 27 v 32; 4 stages 19 v 15; 128 tokens, 32000 words, 64 stages: 52 v 80).
template <int D, int EPI>
hipError_t mma_launch(const Mma& a, int tile, int slices, hipStream_t s) {
  const int64_t tiles = tiles_of(a.A.rows, a.B.rows, tile);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)slices);
  if (tile == 256) {
    hipLaunchKernelGGL((mma_kernel<D, EPI, 2, 4, 8, 4, 2>), grid, dim3(512), 0, s, a);
  } else if (tile == 64) {
    if constexpr (EPI != kDh)
      hipLaunchKernelGGL((mma_kernel<D, EPI, 2, 2, 2, 2, 4>), grid, dim3(256), 0, s, a);
  } else if (tiles * slices <= 256 && std::min(a.K, a.k_slice) / BK * passes(D) >= 16) {
    hipLaunchKernelGGL((mma_kernel<D, EPI, 2, 2, 4, 4, 4>), grid, dim3(256), 0, s, a);
  } else {
    hipLaunchKernelGGL((mma_kernel<D, EPI, 2, 2, 4, 4, 2>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

inline hipError_t rowpack(const void* X, int64_t rows, int64_t k, int64_t ld, float mul, uint16_t* out, int64_t kp,
                          float* unscale, int64_t full, hipStream_t s) {
  hipLaunchKernelGGL(rowpack_kernel, dim3((unsigned)std::min<int64_t>(rows, 65536)), dim3(256), 0, s, (const float*)X,
                     rows, k, ld, mul, out, kp, unscale, full);
  return hipGetLastError();
}
// dH's and dW's products at once, in 128 x 128 tiles
template <int D>
hipError_t pair_launch(const Mma& h, int slices, const Mma& w, hipStream_t s) {
  const int64_t nx = (tiles_of(h.A.rows, h.B.rows, 128) + 7) / 8 * 8, nw = (tiles_of(w.A.rows, w.B.rows, 128) + 7) / 8 * 8;
  hipLaunchKernelGGL((pair_kernel<D, 2>), dim3((unsigned)(nx * slices + nw)), dim3(256), 0, s, h, w,
                     (uint32_t)(nx * slices), (uint32_t)nx);
  return hipGetLastError();
}
template <int D, int M>
hipError_t pack(const void* X, int64_t rows, int64_t k, int64_t ld, const int32_t* labels,
                const float* mul, uint16_t* out, int64_t rp, int64_t kp, int forms, bool twice,
                hipStream_t s) {
  const dim3 grid((unsigned)((kp / 8 + 255) / 256), (unsigned)std::min<int64_t>(rp, 16384),
                  (unsigned)forms);
  hipLaunchKernelGGL((pack_kernel<D, M>), grid, dim3(256), 0, s,
                     (const typename Elem<D>::type*)X, rows, k, ld, labels, mul, out, rp, kp, (int)twice);
  return hipGetLastError();
}

// The factors of a call, and H twice: for z, in place where it can be (an ignored
// token's column of products is not used), and with dloss for dW, whose sums over
// the tokens need the rows of ignored ones zeroed and, but for bf16, each token's
// weight in them. Copies that no product of the call reads are not made. rt: rows of G per token.
template <int D>
hipError_t begin(const Vocab& a, const Plan& p, const float* dloss, int rt, Opnd* Hz, Opnd* Hw,
                 hipStream_t s) {
  char* w = (char*)a.work;
  Factors* fac = (Factors*)(w + p.fac);
  float *hm = (float*)(w + p.hm), *amax = (float*)(w + p.amax);
  Rows rows = rows_of(w, p, a.T);
  rows.wr = a.wr;
  hipError_t e;
  if (D == kF32) {
    hipLaunchKernelGGL(amax_kernel, dim3(kAmaxParts, 2), dim3(256), 0, s, (const float*)a.H, a.T,
                       a.ldh, (const float*)a.W, a.V, a.ldw, a.d, a.labels, hm, amax);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (D == kF32 || dloss) {
    hipLaunchKernelGGL(factors_kernel<D>, dim3(1), dim3(1024), 0, s, hm, amax, dloss, a.share, a.labels,
                       a.T, a.V, a.scale, rows, fac);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  // (score: z comes from score_kernel, or has been kept)
  const bool dw = dloss && a.dW, score = dloss && (few(a.T, a.d, D) || a.z);
  // (bf16 has one copy for both)
  const bool z = !score && (!direct(a.H, a.ldh, a.d, D) || (D == kBF16 && dw));
  // (for dW's products with two rows of G per token; z's take every other row)
  const bool twice = dloss && rt == 2;
  uint16_t* out = (uint16_t*)(w + p.hp);
  const int64_t copy = p.tp * p.dp * terms(D);
  *Hz = z ? Opnd{out, p.dp * terms(D) << (int)twice, p.dp, a.T, p.dp}
          : Opnd{(const uint16_t*)a.H, a.ldh, 0, a.T, a.d};
  *Hw = Opnd{out + (forms(D) - 1) * copy, p.dp * terms(D), p.dp, a.d, p.tp};
  if (!z && !dw) return hipSuccess;
  if constexpr (D != kF32) {
    if (D == kBF16 || !dw)
      return pack<D, kAsIs>(a.H, a.T, a.d, a.ldh, a.labels, nullptr, out, p.tp, p.dp, 1, twice, s);
  }
  if constexpr (D != kBF16) {   // the two copies, and their factors, lie behind each other
    const int from = z ? 0 : 1, n = (int)z + (int)dw;
    return pack<D, kEachRow>(a.H, a.T, a.d, a.ldh, a.labels, rows.hz + from * a.T,
                             out + from * copy, p.tp, p.dp, n, twice, s);
  }
}
// nv words of W from v0: in place, or a copy in the workspace
template <int D>
hipError_t words(const Vocab& a, const Plan& p, int64_t v0, int64_t nv, Opnd* o, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const E* W = (const E*)a.W + v0 * a.ldw;
  if (direct(a.W, a.ldw, a.d, D)) {
    *o = Opnd{(const uint16_t*)W, a.ldw, 0, nv, a.d};
    return hipSuccess;
  }
  char* w = (char*)a.work;
  uint16_t* out = (uint16_t*)(w + p.wp);
  *o = Opnd{out, p.dp * terms(D), p.dp, nv, p.dp};
  return pack<D, D == kF32 ? kOne : kAsIs>(W, nv, a.d, a.ldw, nullptr,
                                           &((Factors*)(w + p.fac))->mw, out, nv, p.dp, 1, false, s);
}

// score_kernel over nv words from v0 on
template <int D, typename OUT>
hipError_t score(const Vocab& a, int64_t v0, int64_t nv, const OUT& o, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const dim3 grid((unsigned)((nv + 63) / 64));
  const E *H = (const E*)a.H, *W = (const E*)a.W + v0 * a.ldw;
  auto go = [&](auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    auto* kernel = score_kernel<D, NT, false, OUT>;
    if constexpr (D != kF32)
      if (a.ldw % 2 || a.ldh % 2 || ((uintptr_t)W | (uintptr_t)H) % 4) kernel = score_kernel<D, NT, true, OUT>;
    hipLaunchKernelGGL(kernel, grid, dim3(1024 / NT), 0, s, H, a.ldh, W, a.ldw, a.T, nv, a.d, a.labels,
                       a.scale, o);
  };
  if (a.T <= 16) {
    go(std::integral_constant<int, 1>{});
  } else if (D != kF32 || a.T <= 32) {
    go(std::integral_constant<int, 2>{});
  } else if constexpr (D == kF32) {
    go(std::integral_constant<int, 4>{});
  }
  return hipGetLastError();
}

}  // namespace
}  // namespace nq
