// Softmax cross entropy over a large vocabulary, and its gradient, without
// keeping the logits (the loss that a packed model is tuned and scored with).
// For hidden states H (T x d), the vocabulary's weights W (V x d) and a label
// per token, z_tv = scale h_t . w_v:
//
//   lse_t = log sum_v exp z_tv,  loss_t = lse_t - z_t,label,
//   G_tv = (exp(z_tv - lse_t) - [v = label_t]) dloss_t scale,
//   dH = G W,  dW = G^T H.
//
// A negative label is ignored: loss 0, lse 0, no gradient, and its row of H
// is never used (it may hold NaN).
//
// All products run on the bf16 or fp16 matrix cores from one kernel
// (mma_kernel) with an epilogue each, a piece of the vocabulary at a time:
//   kStat  z of a tile of words x tokens -> per token the largest and the sum
//          of exponentials over each half of the tile; stat_kernel joins them;
//   kGrad  z again, G = exp(z - lse) - [label] rounded to the operands' type,
//          [token][word];
//   kDh    dH += G W over the piece (fp32 sums, slices of the piece when
//          there are few tiles; dh_kernel adds the slices at the end);
//   kDw    dW = G^T H, the piece's rows.
// 8 T V d operations in place of the 6 T V d that keeping T V logits would
// need. Each of H, W and G is read in the one layout it has: an operand whose
// k runs down the rows (W in kDh, H and G in kDw) is transposed on its way from
// LDS to the registers, by ds_read_b64_tr_b16.
//
// Types: bf16 and fp16 operands are exact and sums are fp32. 16-bit G of more than 32
// tokens is rounded to the operands' type once: half a unit, like the results
// (relative to the exact gradient 0.0017 for the plain form, 0.0018 to 0.0019 here in
// bf16); of fewer it has two terms (g_rows). bf16's G holds (p - [label]) dloss of the
// largest dloss 1; fp16's and fp32's hold p - [label] of each token to 2^15,
// whatever the others' dloss (fp16: with dloss to 2^-10 of the largest), so that
// probabilities down to 2^-29 keep all their bits. fp32 operands are scaled by powers
// of two (each row of H, all of H's copy for dW, W: to 2^15 at their largest) and
// split into two fp16 terms x = h + l, which hold x to 2^-24 of itself or 2^-39
// of the largest; x y = h l + l h + h h, three passes over k, leaves out l l, at
// most 2^-24 of the product. (Three bf16 terms and six passes measured 1.9 times
// the time at no smaller error.)
//
// Few tokens (up to 32, fp32 up to 64): score_kernel takes kStat's and kGrad's
// place. It streams W once, 64 words per workgroup, its waves sharing the
// columns; fp32 is split in registers, into three bf16 terms and six products,
// which need no scale.
//
// The gradient's z have to be the very ones that lse came from: each carries an
// error of its sum's rounding, which exp(z - lse) keeps whole in a probability
// near one, and the two mma_kernel epilogues, or score_kernel's two, sum in one
// order. (fp32, 30 tokens, lse from score_kernel and z from mma_kernel: dH up to
// ten times as far off as with the same z for both.)
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

enum Epi : int { kStat = 0, kGrad = 1, kDh = 2, kDw = 3 };
struct Mma {
  Opnd A, B;                // C (M x N), M = A.rows, N = B.rows
  int64_t K;                // a multiple of 64
  int64_t k_slice;          // k per slice (grid y), a multiple of 64
  const float* zs;          // kStat, kGrad: the factor of the products (fp32: of each token;
  float z0;                 // 16-bit: z0)
  // kStat, kGrad: rows are words v0 .., columns tokens
  int64_t v0;
  const int32_t* labels;
  float *top, *sum, *hit;   // kStat: partials [half tiles of words][N], target logits
  const float *lse, *wn;    // kGrad: lse and normalised dloss per token
  uint16_t* G;              // kGrad: [token][term][gld]
  int64_t gld;
  // kDh, kDw: rows are the d columns, columns tokens or words
  float* part;              // kDh: slices of N x ldo fp32
  int64_t slice, ldo;
  int add;                  // kDh: add to what part holds
  const float* post;        // kDw: the factor of the results (one float)
  void* out;                // kDw
};
constexpr bool a_major(int epi) { return epi == kDh || epi == kDw; }
constexpr bool b_major(int epi) { return epi == kDw; }

// Tile order: workgroup b runs on XCD b % 8, which takes consecutive indices;
// indices run down bands of 4 tile rows, so that the 32 tiles an XCD holds at
// once form a 4 x 8 block and share operands in its L2.
__device__ __forceinline__ bool tile_of(uint32_t ntm, uint32_t ntn, int64_t& tm, int64_t& tn) {
  const uint32_t nt = ntm * ntn, per = (nt + 7) / 8;   // (< 2^31: 2^24 x 2^20 outputs at most)
  const uint32_t t = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= per || t >= nt) return false;
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
  // The copies of the 64 k from k on, of the term `plane` elements into the
  // rows, to LDS offset st: made ready here, sent one at a time by put(). What
  // lies past the operand's end reads as zero (the descriptor's range, which
  // counts the vector offset alone: all of an address below its base is in it).
  int lo, hi, n, to;
  uint32_t o[2], step;
  // (!live: copies of zeros, which read nothing.)
  __device__ __forceinline__ void aim(bool live, uint32_t st, int wave, int64_t k, int64_t plane) {
    const int64_t skip = (MAJOR ? k * ld : k) + plane;
    const uint64_t p = (uint64_t)(uintptr_t)(base + skip);
    lo = scalar((int)p);
    hi = scalar((int)(p >> 32) & 0xffff);
    n = scalar(live ? (int)lmin(lmax(left - 2 * skip, 0), 0x7fffffff) : 0);
    to = scalar((int)(st + wave * NC * 1024));
    step = (uint32_t)(kRowsPer * ld * 2);
    o[0] = off[0];
    o[1] = off[1];
    if constexpr (!MAJOR) {
      if (k + BK > kv) {
        // octets past kv: past any descriptor's range
#pragma unroll
        for (int c = 0; c < 2; ++c) o[c] = k + 8 * koct[c] >= kv ? 0x80000000u : o[c];
      }
    }
  }
  // Copy c. Written out: after a builtin's every transposing read would wait
  // for it, though it is for the next stage. It writes no register, sync()
  // waits for it, and it keeps its place among the reads and sync()s.
  __device__ __forceinline__ void put(int c) const {
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // (m0 is reserved: nothing is kept in it across)
    asm volatile(
        "s_mov_b32 s92, %0\n\t"
        "s_mov_b32 s93, %1\n\t"
        "s_mov_b32 s94, %2\n\t"
        "s_mov_b32 s95, 0x20000\n\t"
        "s_add_u32 m0, %3, %4\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %5, s[92:95], 0 offen lds"
        :
        : "s"(lo), "s"(hi), "s"(n), "s"(to), "i"(c * 1024), "v"(o[kind(c)] + c * step)
        : "m0", "s92", "s93", "s94", "s95", "scc");
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
// d = 4096 in bf16, kStat 3.65 ms and, in eight pieces, kGrad 3.7, kDh 3.4, kDw
// 3.5: 1.19 to 1.29 PFLOP/s (a large bf16 product of the library 1.27; this
// kernel without its copies 1.5, matrix instructions alone 2.2). fp32, 1024
// tokens, 32000 words, d = 2048: 0.40 to 0.46 ms each, 290 to 330 TFLOP/s.
template <int D, int EPI, int WM, int WN, int MI, int NI, int NS>
__global__ __launch_bounds__(64 * WM * WN) void mma_kernel(Mma a) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NI * WN, W = WM * WN;
  constexpr int kStage = (BM + BN) * 128;
  constexpr int CA = BM / 8 / W, CB = BN / 8 / W;
  static_assert(CA * 8 * W == BM && CB * 8 * W == BN, "copies");
  constexpr bool AM = a_major(EPI), BM_ = b_major(EPI), F16 = D != kBF16;
  __shared__ __align__(16) uint8_t lds[NS * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int wm = wave / WN, wn = wave % WN;
  const int64_t M = a.A.rows, N = a.B.rows;
  int64_t tm, tn;
  if (!tile_of((uint32_t)((M + BM - 1) / BM), (uint32_t)((N + BN - 1) / BN), tm, tn)) return;
  const int64_t m0 = tm * BM, n0 = tn * BN;
  const int64_t k_lo = (int64_t)blockIdx.y * a.k_slice;
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
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)lds;
  // the next stage's copies, ready to go to `stage`
  auto aim = [&](int stage, bool live) {
    const uint32_t st = lds0 + stage * kStage;
    const int64_t k = k_lo + (int64_t)kt * BK;
    ta.aim(live, st, wave, k, D == kF32 && pass == 1 ? a.A.plane : 0);
    tb.aim(live, st + BM * 128, wave, k, D == kF32 && pass == 0 ? a.B.plane : 0);
    if (++kt == nk) {
      kt = 0;
      ++pass;
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
  // copies at a time (a run of copies would hold up the products behind it).
  auto phase = [&](auto half, auto copies, uint8_t* st) {
    constexpr int h = decltype(half)::value;
    constexpr bool COPY = decltype(copies)::value;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      if (i < NI) fb[h ^ 1][i] = rb.read(st + BM * 128, i, h ^ 1);
      fa[h ^ 1][i] = ra.read(st, i, h ^ 1);
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
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"i"(decltype(ahead)::value * (CA + CB))
                 : "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  // (copies of stages past the last bring zeros and read nothing: a branch
  // around them would cost more, and every wait counts the same)
#pragma unroll 1
  for (int st = 0; st < NS; ++st) {
    aim(st, st < steps);
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
    phase(H0{}, std::false_type{}, lds + cur * kStage);
    // the next stage has landed; everyone has read this one
    sync(std::integral_constant<int, NS - 2>{});
    aim(cur, s + NS < steps);
    // (after the last stage this reads what is there, for nothing)
    phase(H1{}, std::true_type{}, lds + next * kStage);
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
  } else if constexpr (EPI == kGrad) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const int32_t label = t < N ? a.labels[t] : -1;
      const float lse = label >= 0 ? a.lse[t] : 0.0f, wn_t = label >= 0 ? a.wn[t] : 0.0f;
      const float zs = D == kF32 ? (label >= 0 ? a.zs[t] : 0.0f) : a.z0;
      const int at = own(label), used = label >= 0 ? left : 0;
      uint16_t* row = a.G + t * a.gld * terms(D);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        uint16_t q[4][terms(D)];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float y = zs * acc[i][j][v] - lse;
          float x = D == kF32 ? expf(y) : __expf(y);
          if (16 * i + v == at) x -= 1.0f;
          x = 16 * i + v < used ? x * wn_t : 0.0f;
          split<D>(x, q[v]);
        }
#pragma unroll
        for (int p = 0; p < terms(D); ++p)
          *(u32x2*)(row + p * a.gld + r0 + 16 * i) =
              u32x2{(uint32_t)q[0][p] | (uint32_t)q[1][p] << 16,
                    (uint32_t)q[2][p] | (uint32_t)q[3][p] << 16};
      }
    }
  } else if constexpr (EPI == kDh) {
    float* part = a.part + (int64_t)blockIdx.y * a.slice;
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

// ---------------------------------------------------------------- few tokens
// 64 words and all T <= 16 NT tokens per workgroup of 16 / NT waves, which take
// 32 columns each in turn: neighbours read neighbouring 64 bytes of a row, and
// many waves with one load per row each keep HBM busiest (4096 x 32000 bf16, 16
// tokens, in us with the join: 16 waves 59 (4.4 TB/s), 8 waves 63, 4 waves 96;
// 8 waves of 64 columns 71, 4 waves of 128 columns 80, of two such runs in
// registers 84). Eight values are loaded together from any address (rows that are
// not 16-byte aligned: 3 tokens, 6673 x 68774 fp16 350 us, one by one 727). At the
// end of a row the last eight are loaded, and of H those that came before are
// zeroed (d >= 8).
template <int D>
struct __attribute__((packed)) Raw8 {
  typename Elem<D>::type e[8];
};
// x = h + m + l in bf16, exact; not finite: the first term alone
__device__ __forceinline__ void split3(float x, uint16_t (&t)[3]) {
  t[0] = Elem<kBF16>::from(x);
  const float r = x - Elem<kBF16>::to(t[0]);
  const bool fin = (__float_as_uint(r) & 0x7fffffffu) < 0x7f800000u;
  t[1] = fin ? Elem<kBF16>::from(r) : (uint16_t)0;
  t[2] = fin ? Elem<kBF16>::from(r - Elem<kBF16>::to(t[1])) : (uint16_t)0;
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
    uint16_t q[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(r.e[i], q[i]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f.t[p][i] = (uint32_t)q[2 * i][p] | (uint32_t)q[2 * i + 1][p] << 16;
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
// next multiple of 64, [token][term][gld].
struct ScoreStat {
  float *top, *sum, *hit;
};
struct ScoreGrad {
  const float *lse, *wn;
  uint16_t* G;
  int64_t gld, v0;
};
// (64 registers or fewer: two workgroups of 1024 threads per CU)
template <int D, int NT, bool GRAD>
__global__ __launch_bounds__(1024 / NT)
    __attribute__((amdgpu_waves_per_eu(D != kF32 && NT == 1 ? 8 : 1))) void score_kernel(
        const typename Elem<D>::type* __restrict__ H, int64_t ldh,
        const typename Elem<D>::type* __restrict__ W, int64_t ldw, int64_t T, int64_t V, int64_t d,
        const int32_t* __restrict__ labels, float scale, std::conditional_t<GRAD, ScoreGrad, ScoreStat> o) {
  constexpr int NW = 16 / NT;
  __shared__ f32x4 red[NW][4 * NT][64];
  __shared__ float st[2][4][GRAD ? 1 : 16 * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t v0 = (int64_t)blockIdx.x * 64;
  // byte offsets of the rows (64 rows of 2^21 values at most: 32 bits)
  constexpr int kSize = sizeof(typename Elem<D>::type);
  const char *Wb = (const char*)(W + v0 * ldw), *Hb = (const char*)H;
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
    for (int i = 0; i < 4; ++i) __builtin_memcpy(&w[i], Wb + (wr[i] + at), sizeof(w[i]));
#pragma unroll
    for (int j = 0; j < NT; ++j) __builtin_memcpy(&h[j], Hb + (hr[j] + at), sizeof(h[j]));
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
    const int32_t label = t < T ? labels[t] : -1;
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
        if (w + v < V && w + v == label) o.hit[t] = x[v];
      }
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      float s = 0.0f;
#pragma unroll
      for (int v = 0; v < 4; ++v)   // (-infinity, of an infinity in W, is no zero but NaN)
        s += w + v >= V ? 0.0f : x[v] == kNegInf ? __uint_as_float(0x7fc00000u) : __expf(x[v] - m);
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
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (v0 + 16 * i < V) s += st[1][i][t] * __expf(st[0][i][t] - m);
      o.top[(int64_t)blockIdx.x * T + t] = m;
      o.sum[(int64_t)blockIdx.x * T + t] = s;
    }
  }
}

// ---------------------------------------------------------------- joins
// loss and lse of 16 tokens per workgroup from np partials each (64 threads
// per token, the partials of a thread in order, then a fixed tree). A label
// at or past V gives NaN.
__global__ __launch_bounds__(1024) void stat_kernel(const float* __restrict__ top,
                                                    const float* __restrict__ sum, int64_t np,
                                                    int64_t T, int64_t V,
                                                    const int32_t* __restrict__ labels,
                                                    const float* __restrict__ hit,
                                                    float* __restrict__ loss,
                                                    float* __restrict__ lse) {
  __shared__ float sm[64][17], ss[64][17];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t t = (int64_t)blockIdx.x * 16 + tx;
  float m = kNegInf, s = 0.0f;
  auto join = [&](float m2, float s2) {
    const float n = fmaxf(m, m2);
    // (equal: also both -inf, before any partial)
    s = (m == n ? s : s * __expf(m - n)) + (m2 == n ? s2 : s2 * __expf(m2 - n));
    m = n;
  };
  if (t < T)
    for (int64_t p = ty; p < np; p += 64) join(top[p * T + t], sum[p * T + t]);
  sm[ty][tx] = m;
  ss[ty][tx] = s;
  __syncthreads();
  for (int o = 32; o > 0; o >>= 1) {
    if (ty < o) {
      join(sm[ty + o][tx], ss[ty + o][tx]);
      sm[ty][tx] = m;
      ss[ty][tx] = s;
    }
    __syncthreads();
  }
  if (ty || t >= T) return;
  const int32_t label = labels[t];
  const float l = m + logf(s);
  const float h = label < 0 ? 0.0f : label < V ? hit[t] : __uint_as_float(0x7fc00000u);
  lse[t] = label < 0 ? 0.0f : l;
  loss[t] = label < 0 ? 0.0f : l - h;
}

// Factors of each token, read by the kernels that follow.
struct Rows {
  float *hz, *hw;        // powers of two that its row of H is scaled by, for z and for dW
  float *zs;             // scale / (hz mw): of its products (fp32)
  float *wn, *pt;        // of G, of its row of dH
};
Rows rows_of(char* work, const Plan& p, int64_t T) {
  float* f = (float*)(work + p.rows);
  return {f, f + T, f + 2 * T, f + 3 * T, f + 4 * T};
}
// The largest finite magnitudes: hm[t] of each row of H (y = 0; 0 for an ignored
// token), parts[x] of a share of W's rows (y = 1).
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
      if (labels[t] >= 0) {
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
// (0 for an ignored token; NaN for a label at or past V.) hm and parts (fp32
// operands): the maxima of H's rows and of W. One workgroup.
constexpr int kInG = 10;
template <int D>
__global__ __launch_bounds__(1024) void factors_kernel(const float* __restrict__ hm,
                                                       const float* __restrict__ parts,
                                                       const float* __restrict__ dloss,
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
  // the largest of the finite ones
  float m = 0.0f;
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const float v = labels[t] >= 0 ? fabsf(dloss[t]) : 0.0f;
    m = v < __builtin_inff() ? fmaxf(m, v) : m;
  }
  m = max_of(m, sm);
  int x0 = 0;
  if (m > 0.0f) frexpf(m, &x0);
  // f and x of a token; x = x0 where dloss is 0 or not finite
  auto parted = [&](int64_t t, int& x) {
    x = x0;
    const float l = dloss[t];
    return l != 0.0f && fabsf(l) < __builtin_inff() ? frexpf(l, &x) : l;
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
      wn = ldexpf(f, 15 - k);
      pt = ldexpf(scale, x + k - 15 - ew);
      hw = f == 0.0f ? 0.0f : ldexpf(1.0f, x + k - x0 + eh);
    }
    rows.wn[t] = label < 0 ? 0.0f : label < V ? wn : __uint_as_float(0x7fc00000u);
    rows.pt[t] = label < 0 ? 0.0f : pt;
    rows.hw[t] = label < 0 ? 0.0f : hw;
    if (D == kF16) rows.hz[t] = 1.0f;
  }
  if (threadIdx.x == 0)
    *out = Factors{ldexpf(1.0f, ew),
                   D == kBF16 ? (m == 0.0f ? 1.0f : m) * scale : ldexpf(scale, x0 - 15 - eh)};
}

// dH = each token's factor times the sum of nz slices (in order) of its RT rows; zero
// for an ignored token
template <int D, int RT>
__global__ __launch_bounds__(256) void dh_kernel(const float* __restrict__ part, int nz,
                                                 int64_t slice, int64_t ldp, int64_t T, int64_t d,
                                                 const int32_t* __restrict__ labels,
                                                 const float* __restrict__ pt,
                                                 typename Elem<D>::type* __restrict__ out,
                                                 int64_t ldo) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (c >= d) return;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    const bool used = labels[t] >= 0;
    const float f = pt[t];
    f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int z = 0; z < nz; ++z)
#pragma unroll
      for (int p = 0; p < RT; ++p)
        s += *(const f32x4*)(part + z * slice + (t * RT + p) * ldp + c);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (c + v < d) out[t * ldo + c + v] = Elem<D>::from(used ? s[v] * f : 0.0f);
  }
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
// weight in them. Copies that no product of the call reads are not made.
template <int D>
hipError_t begin(const Vocab& a, const Plan& p, const float* dloss, Opnd* Hz, Opnd* Hw,
                 hipStream_t s) {
  char* w = (char*)a.work;
  Factors* fac = (Factors*)(w + p.fac);
  float *hm = (float*)(w + p.hm), *amax = (float*)(w + p.amax);
  const Rows rows = rows_of(w, p, a.T);
  hipError_t e;
  if (D == kF32) {
    hipLaunchKernelGGL(amax_kernel, dim3(kAmaxParts, 2), dim3(256), 0, s, (const float*)a.H, a.T,
                       a.ldh, (const float*)a.W, a.V, a.ldw, a.d, a.labels, hm, amax);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (D == kF32 || dloss) {
    hipLaunchKernelGGL(factors_kernel<D>, dim3(1), dim3(1024), 0, s, hm, amax, dloss, a.labels, a.T,
                       a.V, a.scale, rows, fac);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  const bool dw = dloss && a.dW, score = dloss && few(a.T, a.d, D);
  // (bf16 has one copy for both)
  const bool z = !score && (!direct(a.H, a.ldh, a.d, D) || (D == kBF16 && dw));
  // (for dW's products with two rows of G per token)
  const bool twice = score && g_rows(a.T, a.d, D) == 2;
  uint16_t* out = (uint16_t*)(w + p.hp);
  const int64_t copy = p.tp * p.dp * terms(D);
  *Hz = z ? Opnd{out, p.dp * terms(D), p.dp, a.T, p.dp}
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
template <int D, bool GRAD>
hipError_t score(const Vocab& a, int64_t v0, int64_t nv,
                 const std::conditional_t<GRAD, ScoreGrad, ScoreStat>& o, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const dim3 grid((unsigned)((nv + 63) / 64));
  const E *H = (const E*)a.H, *W = (const E*)a.W + v0 * a.ldw;
  auto go = [&](auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    hipLaunchKernelGGL((score_kernel<D, NT, GRAD>), grid, dim3(1024 / NT), 0, s, H, a.ldh, W, a.ldw,
                       a.T, nv, a.d, a.labels, a.scale, o);
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

template <int D>
hipError_t loss(const Vocab& a, hipStream_t s) {
  const Plan p = plan_for(a.T, a.V, a.d, D, false);
  char* w = (char*)a.work;
  hipError_t e;
  int64_t np;   // partials per token
  if (few(a.T, a.d, D)) {
    np = (a.V + 63) / 64;
    const ScoreStat o{(float*)(w + p.top), (float*)(w + p.sum), (float*)(w + p.hit)};
    if ((e = score<D, false>(a, 0, a.V, o, s)) != hipSuccess) return e;
  } else {
    Mma m{};
    Opnd unused;
    if ((e = begin<D>(a, p, nullptr, &m.B, &unused, s)) != hipSuccess) return e;
    m.K = m.k_slice = p.dp;
    m.zs = rows_of(w, p, a.T).zs;
    m.z0 = a.scale;
    m.labels = a.labels;
    m.top = (float*)(w + p.top); m.sum = (float*)(w + p.sum); m.hit = (float*)(w + p.hit);
    // all words at once where W is used in place
    const int64_t piece = direct(a.W, a.ldw, a.d, D) ? a.V : p.piece;
    const int tile = tile_for(piece, a.T);
    np = 2 * ((a.V + tile - 1) / tile);
    for (int64_t v0 = 0; v0 < a.V; v0 += piece) {
      m.v0 = v0;
      if ((e = words<D>(a, p, v0, std::min(piece, a.V - v0), &m.A, s)) != hipSuccess) return e;
      if ((e = mma_launch<D, kStat>(m, tile, 1, s)) != hipSuccess) return e;
    }
  }
  hipLaunchKernelGGL(stat_kernel, dim3((unsigned)((a.T + 15) / 16)), dim3(1024), 0, s,
                     (const float*)(w + p.top), (const float*)(w + p.sum), np, a.T, a.V, a.labels,
                     (const float*)(w + p.hit), a.loss, a.lse);
  return hipGetLastError();
}

template <int D>
hipError_t backward(const Vocab& a, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const Plan p = plan_for(a.T, a.V, a.d, D, true);
  char* w = (char*)a.work;
  Factors* fac = (Factors*)(w + p.fac);
  uint16_t* G = (uint16_t*)(w + p.G);
  // rows of G, and so of dH's sums, as the products see them: the terms of 16-bit G
  // are rows of their own
  const int rt = g_rows(a.T, a.d, D);
  const int64_t RT = rt * a.T, gld = p.piece * terms(D);
  const int64_t ldp = round_up(a.d, 4), slice = RT * ldp;
  const bool score_g = few(a.T, a.d, D);
  hipError_t e;
  const Rows rows = rows_of(w, p, a.T);
  Opnd Hz, Hw, W;
  if ((e = begin<D>(a, p, a.dloss, &Hz, &Hw, s)) != hipSuccess) return e;
  // every piece uses the same slices of its words for dH; the first writes them
  // all, the last, where it is another, may leave some as they are: those are not
  // launched
  for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
    const int64_t nv = std::min(p.piece, a.V - v0), nvp = round_up(nv, 256);
    if ((e = words<D>(a, p, v0, nv, &W, s)) != hipSuccess) return e;
    if (score_g) {
      const ScoreGrad o{a.lse, rows.wn, G, p.piece, v0};
      if ((e = score<D, true>(a, v0, nv, o, s)) != hipSuccess) return e;
    } else {
      Mma m{};
      m.A = W; m.B = Hz;
      m.K = m.k_slice = p.dp;
      m.zs = rows.zs;
      m.z0 = a.scale;
      m.v0 = v0; m.labels = a.labels; m.lse = a.lse; m.wn = rows.wn;
      m.G = G; m.gld = p.piece;
      if ((e = mma_launch<D, kGrad>(m, tile_for(nv, a.T), 1, s)) != hipSuccess) return e;
    }
    // (G is zero for words past nv to the next multiple of 64, and from
    // mma_kernel for tokens past T to the tile's end)
    if (a.dH) {
      Mma h{};
      h.A = Opnd{W.p, W.ld, W.plane, a.d, nv};
      h.B = Opnd{G, gld, p.piece, RT, nvp};
      h.K = round_up(nv, BK);
      h.k_slice = p.kz;
      h.part = (float*)(w + p.part); h.slice = slice; h.ldo = ldp; h.add = v0 > 0;
      const int n = (int)((h.K + p.kz - 1) / p.kz), tile = big_tiles(a.d, RT, p.nz) ? 256 : 128;
      if ((e = mma_launch<D, kDh>(h, tile, n, s)) != hipSuccess) return e;
    }
    if (a.dW) {
      Mma x{};
      x.A = Hw;
      x.B = Opnd{G, gld, p.piece, nv, score_g ? RT : p.tp};
      x.K = x.k_slice = round_up(RT, BK);
      x.post = &fac->post_w;
      x.out = (E*)a.dW + v0 * a.lddw; x.ldo = a.lddw;
      if ((e = mma_launch<D, kDw>(x, tile_for(a.d, nv), 1, s)) != hipSuccess) return e;
    }
  }
  if (a.dH) {
    const dim3 grid((unsigned)((a.d + 1023) / 1024), (unsigned)std::min<int64_t>(a.T, 16384));
    auto* join = dh_kernel<D, 1>;
    if constexpr (D != kF32) join = rt == 1 ? join : dh_kernel<D, kFewTerms>;
    hipLaunchKernelGGL(join, grid, dim3(256), 0, s, (const float*)(w + p.part), p.nz, slice, ldp,
                       a.T, a.d, a.labels, rows.pt, (E*)a.dH, a.lddh);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t vocab_work_bytes(int64_t T, int64_t V, int64_t d, int dtype, bool grad) {
  return plan_for(T, V, d, dtype, grad).bytes;
}

hipError_t launch_vocab_loss(const Vocab& a, hipStream_t s) {
  if (a.dtype == kF32) return loss<kF32>(a, s);
  return a.dtype == kBF16 ? loss<kBF16>(a, s) : loss<kF16>(a, s);
}

hipError_t launch_vocab_loss_backward(const Vocab& a, hipStream_t s) {
  if (a.dtype == kF32) return backward<kF32>(a, s);
  return a.dtype == kBF16 ? backward<kBF16>(a, s) : backward<kF16>(a, s);
}

}  // namespace nq
