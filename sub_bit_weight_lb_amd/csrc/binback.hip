// Gradient of a packed low-rank binary layer from an 8-bit checkpoint of its
// input (the tuning of scales with the signs held, NanoQuant digest, section
// 方法步骤详情, stage 3). The layer is y = s1 * q, q = S_U p, p = S_V^T a,
// a = s2 * x^; with dy = dL/dy,
//
//   ds1 = sum_t dy * q,   dp = S_U^T (s1 * dy),   da = S_V dp,
//   dx  = s2 * da,        ds2 = sum_t da * x^,
//
// four products with packed signs: a -> p -> q and s1 dy -> dp -> da. q and
// da are never stored: the epilogues of their products form dy q, dx and
// da x^ from the accumulators.
//
// A product's left factor (T rows of fp32 values v) is written in fixed point
// with one power-of-two step per row: v = step D, D = sum_i 256^i d_i, the d's
// ND signed bytes. A sign is a byte 0 or 1 (bit = [+1]): sum_c sign_c v_c =
// step (2 sum_c bit_c D_c - sum_c D_c). Every sum of digits is exact (|d| <=
// 128, so 2^23 columns fit 32 bits) and no order of summing changes a result;
// the digits' sums are joined at the end by ND - 1 fp32 multiply-adds. Against three bf16 terms
// (six v_mfma_f32_16x16x32_bf16 for 64 columns) ND v_mfma_i32_16x16x64_i8 take
// half to two thirds of the matrix cores' time.
// ND = 4 for a and s1 dy: |D| < 2^31, a value is off by at most 2^-31 of its
// row's largest, less than an fp32 rounding of any value within 2^-7 of it;
// activations have channels a hundred times the rest, and with three digits
// (2^-23 of the largest) ds1 measured 2.2e-6 off, three times an fp32 product.
// ND = 3 for p and dp, whose entries are sums over a whole row and alike in
// size: 2^-23 of the largest is then below what the rounding of p to fp32
// and an fp32 sum over r terms lose.
//
// Digit layout, written by rows_kernel: per 16 rows and 128 columns a block
// of 2048 ND bytes, [digit][s][lane][16]: lane (li, g) = row li, word g of the
// block's four 32-column words; byte 4 d + b of half s is column 8 b + 4 s + d
// of the word, so that (w >> (4 s + d)) & 0x01010101 is dword d of the signs'
// operand, one shift and one and for four columns. The signs go from memory
// to registers and never to LDS.
//
// The two chains a -> p -> q and s1 dy -> dp -> da do not depend on each
// other: each launch takes a step of both (grid z, or y).
//
// wide_kernel (more than kThinMax rows): 256 threads, 2 x 2 waves of 16 MI
// rows x 64 signs (MI = 4 for three digits, 2 for four: 192 and 128 registers
// of sums). The digits of 64 columns are copied straight to LDS, double
// buffered; the lanes' fragments are consecutive, so reads have no bank
// conflicts. The digits share one expansion of the signs (32 vector
// instructions against 4 MI ND products per wave and stage). Workgroup b runs
// on XCD b % 8, and an XCD takes consecutive tiles, which share their rows'
// digits in its L2.
// thin_kernel (few rows): a workgroup takes all rows and 16 signs' rows, its
// waves split the columns and add up through LDS.
#include "tune.h"

#include <algorithm>

namespace nq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int kDigit = 2048;      // bytes of a digit per 16 rows and 128 columns
constexpr int kTile = 128;        // signs of a wide tile; its rows with three digits
constexpr int kThinMax = 64;      // rows of a thin launch
constexpr int kThinWaves = 8;
constexpr int kMaxSplit = 8;      // slices of the columns (wide, few tiles)
constexpr int64_t kTeamRows = 1024;   // up to this many rows, a workgroup per row
// the largest magnitude of ND balanced digits, 1.99215...  2^(8 ND - 2): an
// fp32 value with a mantissa up to this is below it
constexpr uint32_t kTopMant = 8322814;

// ---------------------------------------------------------------- rows
// Sources of four columns c, c + 8, c + 16, c + 24 of a row (of one 32-column
// word); columns past the end are 0.
struct SrcAct {      // s2 * x^
  Act8 q;
  const float* scale;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c, float (&x)[4]) const {
    if (c >= cols) {
      x[0] = x[1] = x[2] = x[3] = 0.0f;
      return;
    }
    const float st = act8_step(q.exps[row * q.lde + (c >> 5)]);
    const int8_t* p = q.codes + row * q.ldc + c;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      x[b] = c + 8 * b < cols ? (float)p[8 * b] * st * scale[c + 8 * b] : 0.0f;
  }
};
template <int D>
struct SrcGrad {     // s1 * dy
  const typename Elem<D>::type* p;
  int64_t ld;
  const float* scale;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c, float (&x)[4]) const {
    const typename Elem<D>::type* q = p + row * ld + c;
#pragma unroll
    for (int b = 0; b < 4; ++b)
      x[b] = c + 8 * b < cols ? Elem<D>::to(q[8 * b]) * scale[c + 8 * b] : 0.0f;
  }
};
struct SrcProj {     // p or dp: fp32, or the fp64 partial sums of nsum slices
  const void* p;
  int64_t ld, slice;
  int nsum;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c, float (&x)[4]) const {
    if (nsum == 1) {
      const float* q = (const float*)p + row * ld + c;
#pragma unroll
      for (int b = 0; b < 4; ++b) x[b] = c + 8 * b < cols ? q[8 * b] : 0.0f;
      return;
    }
    const double* q = (const double*)p + row * ld + c;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      double a = 0.0;
      if (c + 8 * b < cols)
        for (int z = 0; z < nsum; ++z) a += q[z * slice + 8 * b];
      x[b] = (float)a;
    }
  }
};

// Digits of T rows, their steps (NaN for a row that holds a NaN or an
// infinity: its results are NaN) and, per row, the sum of each digit.
struct Digits {
  uint8_t* planes;
  float* steps;
  i32x4* sums;
};

// The step of a row whose largest magnitude has the bits mx:
// max|v| = 1.f 2^(E - 127) <= 127.5 256^(ND - 1) 2^e.
template <int ND>
__device__ __forceinline__ int row_exponent(uint32_t mx) {
  return max((int)(mx >> 23) - 127 - (8 * ND - 2) + ((mx & 0x7fffffu) > kTopMant), -126);
}
// Four values of a word as digits: out[p] holds digit p of column b in byte b.
// With 128 added to each digit's place the bytes of an integer are its balanced
// digits plus 128; then a 4 x 4 transpose of bytes.
template <int ND>
__device__ __forceinline__ void to_digits(const float (&x)[4], float inv, uint32_t (&out)[4]) {
  constexpr uint32_t kBias = ND == 4 ? 0x80808080u : 0x00808080u;
  uint32_t u[4];
#pragma unroll
  for (int b = 0; b < 4; ++b) u[b] = ((uint32_t)(int)rintf(x[b] * inv) + kBias) ^ 0x80808080u;
  const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(u[1], u[0], 0x07030602u);
  const uint32_t e = __builtin_amdgcn_perm(u[3], u[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(e, d, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(e, d, 0x07060302u);
}

// Eight rows per workgroup, a wave each (lane = word (lane / 8) of 256
// columns, byte position lane % 8 in it), the digits of 256 columns exchanged
// through LDS so that whole 128-byte lines are stored. TEAM: one row per
// workgroup, its waves taking 256 columns in turn (few rows). blockIdx.y picks
// one of two jobs. Columns past the end up to a multiple of 128 get zeros.
template <int ND, bool TEAM, class S0, class S1>
__global__ __launch_bounds__(512) void rows_kernel(S0 s0, S1 s1, int64_t T, Digits o0, Digits o1) {
  constexpr int kRun = 8 * 16 + 16;   // eight rows of 16 bytes, padded against bank conflicts
  __shared__ __align__(16) uint8_t buf[TEAM ? 16 : 2][TEAM ? 16 : ND * 16 * kRun];
  __shared__ uint32_t wmax[8];
  __shared__ int wsum[8][ND];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = TEAM ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + wave;
  const bool job = blockIdx.y;
  const int64_t cols = job ? s1.cols : s0.cols;
  const Digits o = job ? o1 : o0;
  const bool in = row < T;
  const int64_t nkb = (cols + 127) / 128, nch = (nkb + 1) / 2;
  const int64_t first = TEAM ? wave : 0, stride = TEAM ? 8 : 1;
  const int w8 = lane >> 3, sd = lane & 7;
  auto load = [&](int64_t ch, float (&x)[4]) {
    const int64_t c = ch * 256 + 32 * w8 + sd;
    if (!in) {
      x[0] = x[1] = x[2] = x[3] = 0.0f;
    } else if (job) {
      s1.load(row, c, x);
    } else {
      s0.load(row, c, x);
    }
  };
  uint32_t mx = 0;
  for (int64_t ch = first; ch < nch; ch += stride) {
    float x[4];
    load(ch, x);
#pragma unroll
    for (int b = 0; b < 4; ++b) mx = max(mx, __float_as_uint(x[b]) & 0x7fffffffu);
  }
#pragma unroll
  for (int q = 32; q > 0; q >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, q));
  if (TEAM) {
    if (lane == 0) wmax[wave] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) mx = max(mx, wmax[w]);
  }
  const bool bad = mx >= 0x7f800000u;
  const int e = row_exponent<ND>(mx);
  const float inv = bad ? 0.0f : __uint_as_float((uint32_t)(127 - e) << 23);
  int sum[ND];
#pragma unroll
  for (int p = 0; p < ND; ++p) sum[p] = 0;
  uint8_t* block = o.planes + (row >> 4) * nkb * (ND * kDigit);
  for (int64_t ch = first; ch < nch; ch += stride) {
    float x[4];
    load(ch, x);
    if (bad) x[0] = x[1] = x[2] = x[3] = 0.0f;
    uint32_t dig[4];
    to_digits<ND>(x, inv, dig);
#pragma unroll
    for (int p = 0; p < ND; ++p) sum[p] = __builtin_amdgcn_sdot4((int)dig[p], 0x01010101, sum[p], false);
    if (TEAM) {
      const int64_t kb = 2 * ch + (w8 >> 2);
      if (kb < nkb) {
        uint8_t* dst = block + kb * (ND * kDigit) + (sd >> 2) * 1024 +
                       ((w8 & 3) * 16 + (int)(row & 15)) * 16 + 4 * (sd & 3);
#pragma unroll
        for (int p = 0; p < ND; ++p) *(uint32_t*)(dst + p * kDigit) = dig[p];
      }
    } else {
      // run (kb, digit, s, g) of eight rows, the row's 16 bytes
      uint8_t* b = buf[ch & 1];
#pragma unroll
      for (int p = 0; p < ND; ++p)
        *(uint32_t*)(b + ((((w8 >> 2) * ND + p) * 2 + (sd >> 2)) * 4 + (w8 & 3)) * kRun + wave * 16 +
                     4 * (sd & 3)) = dig[p];
      __syncthreads();   // (the other buffer is free: its readers passed this barrier)
      const int t = threadIdx.x;
      if (t < ND * 128) {
        const int run = t >> 3, g = run & 3, s = (run >> 2) & 1, q = run >> 3;
        const int64_t kb = 2 * ch + q / ND;
        if (kb < nkb)
          *(u32x4*)(o.planes + (((int64_t)blockIdx.x >> 1) * nkb + kb) * (ND * kDigit) +
                    (q % ND) * kDigit + s * 1024 + (g * 16 + (blockIdx.x & 1) * 8 + (t & 7)) * 16) =
              *(const u32x4*)(b + run * kRun + (t & 7) * 16);
      }
    }
  }
#pragma unroll
  for (int p = 0; p < ND; ++p)
#pragma unroll
    for (int q = 32; q > 0; q >>= 1) sum[p] += __shfl_xor(sum[p], q);
  if (TEAM) {
    if (lane == 0)
#pragma unroll
      for (int p = 0; p < ND; ++p) wsum[wave][p] = sum[p];
    __syncthreads();
    if (wave) return;
#pragma unroll
    for (int w = 1; w < 8; ++w)
#pragma unroll
      for (int p = 0; p < ND; ++p) sum[p] += wsum[w][p];
  }
  if (lane == 0 && in) {
    o.steps[row] = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(e + 127) << 23);
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < ND; ++p) v[p] = sum[p];
    o.sums[row] = v;
  }
}

// ---------------------------------------------------------------- products
enum Epi : int {
  kProj = 0,   // out: p or dp (fp32, or fp64 partials when the columns are split)
  kGrad = 1,   // column sums of dy q; or dx = s2 da and column sums of da x^
};
constexpr int digits(int epi) { return epi == kProj ? 4 : 3; }
constexpr int row_tiles(int epi) { return epi == kProj ? 2 : 4; }   // 16-row tiles per wave
struct Prod {
  Digits a;                   // T rows, K columns
  const uint32_t* bits;       // N x K signs
  int64_t ldb, T, N, K;
  // kProj
  void* P;
  int64_t ldp, slice;
  int split;
  int64_t kbs;                // 128-column blocks per slice
  // kGrad
  float* colp;                // row tiles x N partial column sums
  const void* dY;             // null: the second chain
  int64_t lddy;
  Act8 x;
  const float* s2;
  void* dX;                   // nullable
  int64_t lddx;
};

// sum_c sign_c v_c = step sum_p 256^p (2 acc_p - sum_p) from a row's step and
// digit sums: the terms are exact, joined from the largest by fp32
// multiply-adds.
template <int ND>
__device__ __forceinline__ float value(float step, const i32x4& sum, const int (&acc)[ND]) {
  float r = (float)(2 * acc[ND - 1] - sum[ND - 1]);
#pragma unroll
  for (int p = ND - 2; p >= 0; --p) r = fmaf(r, 256.0f, (float)(2 * acc[p] - sum[p]));
  return r * step;
}
// What the sums acc of row t (step, sum) and sign row n give: stored, or
// returned as a share of the column sum.
template <int EPI, int D>
__device__ __forceinline__ float finish(const Prod& a, int64_t t, int64_t n, float step,
                                        const i32x4& sum, const int (&acc)[digits(EPI)], int z) {
  typedef typename Elem<D>::type E;
  constexpr int ND = digits(EPI);
  if (t >= a.T || n >= a.N) return 0.0f;
  if (EPI == kProj) {
    if (a.split == 1) {
      ((float*)a.P)[t * a.ldp + n] = value<ND>(step, sum, acc);
    } else {   // a slice's share, exact; the first takes the digit sums
      double r = 0.0;
#pragma unroll
      for (int p = ND - 1; p >= 0; --p)
        r = fma(r, 256.0, 2.0 * (double)acc[p] - (z == 0 ? (double)sum[p] : 0.0));
      ((double*)a.P)[z * a.slice + t * a.ldp + n] = r * (double)step;
    }
    return 0.0f;
  }
  const float v = value<ND>(step, sum, acc);
  if (a.dY) return Elem<D>::to(((const E*)a.dY)[t * a.lddy + n]) * v;
  if (a.dX) ((E*)a.dX)[t * a.lddx + n] = Elem<D>::from(a.s2[n] * v);
  return v * ((float)a.x.codes[t * a.x.ldc + n] * act8_step(a.x.exps[t * a.x.lde + (n >> 5)]));
}
// dwords of the signs' operand, half s of word w
__device__ __forceinline__ i32x4 spread(uint32_t w, int s) {
  i32x4 r;
#pragma unroll
  for (int d = 0; d < 4; ++d) r[d] = (int)((w >> (4 * s + d)) & 0x01010101u);
  return r;
}

template <int EPI, int D>
__global__ __launch_bounds__(256, 2) void wide_kernel(Prod a0, Prod a1) {
  constexpr int ND = digits(EPI), MI = row_tiles(EPI);
  constexpr int kBlock = ND * kDigit, kRows = 32 * MI;
  constexpr int kStage = 2 * MI * ND * 1024;   // 32 MI rows, 64 columns
  __shared__ __align__(16) uint8_t lds[2 * kStage];
  const Prod& a = blockIdx.z ? a1 : a0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t ntn = (a.N + kTile - 1) / kTile, ntm = (a.T + kRows - 1) / kRows;
  const int64_t per = (ntn * ntm + 7) / 8;
  const int64_t tile = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  const int z = blockIdx.y;
  if ((int64_t)(blockIdx.x >> 3) >= per || tile >= ntn * ntm || z >= a.split) return;
  const int64_t tm = tile / ntn, tn = tile - tm * ntn;
  const int64_t nkb = (a.K + 127) / 128, nw = (a.K + 31) / 32;
  const int64_t kb0 = z * a.kbs, kb1 = min(nkb, kb0 + a.kbs);
  // this tile's digits: 2 MI blocks of 16 rows, nkb blocks apart (rows past
  // T hold no digits of the call: whatever they give is dropped at the end)
  const __amdgpu_buffer_rsrc_t pr = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.a.planes + tm * 2 * MI * nkb * kBlock), (short)0, (int)(2 * MI * nkb * kBlock),
      0x00020000);
  auto copy = [&](int stage, int64_t kb, int s) {
    constexpr int C = 2 * MI * ND / 4;   // copies of 1 KB per wave
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = wave * C + c, rt = i / ND, p = i - ND * rt;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          pr, (lds_ptr_t)(lds + stage * kStage + i * 1024), 16, lane * 16,
          (int)((rt * nkb + kb) * kBlock) + p * kDigit + s * 1024, 0, 0);
    }
  };
  // the lane's sign rows (clamped: rows past N are dropped at the end; words
  // past a row's last meet zero digits)
  const uint32_t* bp[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    bp[j] = a.bits + min<int64_t>(tn * kTile + wn * 64 + j * 16 + li, a.N - 1) * a.ldb;
  uint32_t word[4], next[4];
  auto words = [&](uint32_t (&w)[4], int64_t kb) {
    const int64_t at = min<int64_t>(4 * kb + g, nw - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = bp[j][at];
  };
  i32x4 acc[ND][MI][4];
#pragma unroll
  for (int p = 0; p < ND; ++p)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[p][i][j] = i32x4{0, 0, 0, 0};
  auto mult = [&](int stage, int s) {
    i32x4 b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = spread(word[j], s);
    const uint8_t* st = lds + stage * kStage + lane * 16;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int p = 0; p < ND; ++p) {
        const i32x4 f = *(const i32x4*)(st + ((wm * MI + i) * ND + p) * 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[p][i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f, b[j], acc[p][i][j], 0, 0, 0);
      }
  };
  // each wave waits for its own copies and reads, then for the other waves
  auto sync = [&]() {
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
  };
  copy(0, kb0, 0);
  words(word, kb0);
  for (int64_t kb = kb0; kb < kb1; ++kb) {
    sync();   // stage 0 holds (kb, 0); everyone is done with stage 1
    copy(1, kb, 1);
    words(next, kb + 1);
    mult(0, 0);
    sync();   // stage 1 holds (kb, 1); everyone is done with stage 0
    if (kb + 1 < kb1) copy(0, kb + 1, 0);
    mult(1, 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) word[j] = next[j];
  }
  const int64_t t0 = tm * kRows + wm * 16 * MI, n0 = tn * kTile + wn * 64;
  float cs[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t t = t0 + 16 * i + 4 * g + v;
      const float step = a.a.steps[min(t, a.T - 1)];
      const i32x4 sum = a.a.sums[min(t, a.T - 1)];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        int d[ND];
#pragma unroll
        for (int p = 0; p < ND; ++p) d[p] = acc[p][i][j][v];
        cs[j] += finish<EPI, D>(a, t, n0 + 16 * j + li, step, sum, d, z);
      }
    }
  if (EPI == kProj) return;
  // the tile's column sums: the rows of a lane, then the four lanes of a
  // column, then the two row halves, each in a fixed order
  __syncthreads();
  float* half = (float*)lds;   // [wm][128]
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cs[j] += __shfl_xor(cs[j], 16);
    cs[j] += __shfl_xor(cs[j], 32);
    if (g == 0) half[wm * 128 + wn * 64 + 16 * j + li] = cs[j];
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < 128 && tn * kTile + c < a.N) a.colp[tm * a.N + tn * kTile + c] = half[c] + half[128 + c];
}

// All T <= 16 MT rows and 16 sign rows per workgroup; wave w takes the
// 128-column blocks w, w + 8, ...
template <int EPI, int D, int MT>
__global__ __launch_bounds__(64 * kThinWaves) void thin_kernel(Prod a0, Prod a1) {
  constexpr int ND = digits(EPI), kBlock = ND * kDigit;
  __shared__ i32x4 red[kThinWaves][MT][64];
  const Prod& a = blockIdx.y ? a1 : a0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  if (n0 >= a.N) return;
  const int64_t nkb = (a.K + 127) / 128, nw = (a.K + 31) / 32;
  const uint32_t* bp = a.bits + min<int64_t>(n0 + li, a.N - 1) * a.ldb;
  i32x4 acc[ND][MT];
#pragma unroll
  for (int p = 0; p < ND; ++p)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[p][i] = i32x4{0, 0, 0, 0};
  for (int64_t kb = wave; kb < nkb; kb += kThinWaves) {
    const uint32_t w = bp[min<int64_t>(4 * kb + g, nw - 1)];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const i32x4 b = spread(w, s);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int p = 0; p < ND; ++p) {
          const i32x4 f = *(const i32x4*)(a.a.planes + (i * nkb + kb) * kBlock + p * kDigit +
                                          s * 1024 + lane * 16);
          acc[p][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f, b, acc[p][i], 0, 0, 0);
        }
    }
  }
  // the waves' sums, one digit at a time through LDS
#pragma unroll
  for (int p = 0; p < ND; ++p) {
    if (p) __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[p][i];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int w = 1; w < kThinWaves; ++w) acc[p][i] += red[w][i][lane];
    }
  }
  if (wave) return;
  float cs = 0.0f;
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t t = 16 * i + 4 * g + v;
      int d[ND];
#pragma unroll
      for (int p = 0; p < ND; ++p) d[p] = acc[p][i][v];
      cs += finish<EPI, D>(a, t, n0 + li, a.a.steps[min(t, a.T - 1)], a.a.sums[min(t, a.T - 1)], d, 0);
    }
  if (EPI == kProj) return;
  cs += __shfl_xor(cs, 16);
  cs += __shfl_xor(cs, 32);
  if (g == 0 && n0 + li < a.N) a.colp[n0 + li] = cs;
}

// ds1 and ds2 from the partial column sums of nt row tiles, in fp64: thread
// (c, q) adds the tiles q, q + 8, ... of column c in order, then the eight are
// added in order
__global__ __launch_bounds__(256) void colsum_kernel(const float* __restrict__ p1, int64_t m,
                                                     float* __restrict__ ds1,
                                                     const float* __restrict__ p2, int64_t n,
                                                     float* __restrict__ ds2, int64_t nt) {
  __shared__ double part[8][32];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + tx;
  double s = 0.0;
  if (i < m + n) {
    const float* p = i < m ? p1 + i : p2 + (i - m);
    const int64_t ld = i < m ? m : n;
    for (int64_t t = ty; t < nt; t += 8) s += (double)p[t * ld];
  }
  part[ty][tx] = s;
  __syncthreads();
  if (ty || i >= m + n) return;
#pragma unroll
  for (int q = 1; q < 8; ++q) s += part[q][tx];
  if (i < m)
    ds1[i] = (float)s;
  else
    ds2[i - m] = (float)s;
}

// ---------------------------------------------------------------- launches
struct Work {
  Digits d[2];      // of the two chains
  void* P[2];
  float *cp1, *cp2;
  int64_t bytes;
};
// Slices of the columns of a chain's first product: enough tiles for two
// workgroups on each of the 256 CUs (the two chains run together), at least
// four blocks of 128 each.
int proj_split(int64_t T, int64_t r, int64_t K) {
  if (T <= kThinMax) return 1;
  const int64_t rows = 32 * row_tiles(kProj);
  const int64_t tiles = 2 * ((T + rows - 1) / rows) * ((r + kTile - 1) / kTile);
  const int64_t nkb = (K + 127) / 128;
  return (int)std::max<int64_t>(1, std::min({(int64_t)kMaxSplit, 512 / tiles, nkb / 4}));
}
Work carve(char* base, int64_t m, int64_t n, int64_t r, int64_t T) {
  Work w{};
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    char* p = base ? base + off : nullptr;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t Tp = round_up(T, T <= kThinMax ? 16 : kTile), nt = (T + kTile - 1) / kTile;
  for (int c = 0; c < 2; ++c) {
    const int64_t K = c ? m : n;
    const int sp = proj_split(T, r, K);
    w.d[c].planes = (uint8_t*)take(Tp * std::max(4 * round_up(K, 128), 3 * round_up(r, 128)));
    w.d[c].steps = (float*)take(4 * T);
    w.d[c].sums = (i32x4*)take(16 * T);
    w.P[c] = take(sp == 1 ? 4 * T * r : 8 * T * r * sp);
  }
  w.cp1 = (float*)take(4 * nt * m);
  w.cp2 = (float*)take(4 * nt * n);
  w.bytes = off;
  return w;
}

template <int ND, class S0, class S1>
hipError_t rows(const S0& s0, const S1& s1, int64_t T, const Work& w, hipStream_t s) {
  if (T <= kTeamRows)
    hipLaunchKernelGGL((rows_kernel<ND, true, S0, S1>), dim3((unsigned)T, 2), dim3(512), 0, s, s0,
                       s1, T, w.d[0], w.d[1]);
  else
    hipLaunchKernelGGL((rows_kernel<ND, false, S0, S1>), dim3((unsigned)((T + 7) / 8), 2),
                       dim3(512), 0, s, s0, s1, T, w.d[0], w.d[1]);
  return hipGetLastError();
}
template <int EPI, int D>
hipError_t products(const Prod& a, const Prod& b, hipStream_t s) {
  const int64_t N = std::max(a.N, b.N);
  if (a.T <= kThinMax) {
    const dim3 grid((unsigned)((N + 15) / 16), 2), block(64 * kThinWaves);
    if (a.T <= 16)
      hipLaunchKernelGGL((thin_kernel<EPI, D, 1>), grid, block, 0, s, a, b);
    else if (a.T <= 32)
      hipLaunchKernelGGL((thin_kernel<EPI, D, 2>), grid, block, 0, s, a, b);
    else
      hipLaunchKernelGGL((thin_kernel<EPI, D, 4>), grid, block, 0, s, a, b);
    return hipGetLastError();
  }
  const int64_t rows = 32 * row_tiles(EPI);
  const int64_t tiles = ((a.T + rows - 1) / rows) * ((N + kTile - 1) / kTile);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)std::max(a.split, b.split), 2);
  hipLaunchKernelGGL((wide_kernel<EPI, D>), grid, dim3(256), 0, s, a, b);
  return hipGetLastError();
}

template <int D>
hipError_t run(const BinBack& a, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const Work w = carve((char*)a.work, a.m, a.n, a.r, a.T);
  const bool one = a.T <= kTile;   // a single row tile: its column sums are the result
  hipError_t e;
  // a and s1 dy, then p and dp
  if ((e = rows<digits(kProj)>(SrcAct{a.x, a.s2, a.n},
                               SrcGrad<D>{(const E*)a.dY, a.lddy, a.s1, a.m}, a.T, w, s)) != hipSuccess)
    return e;
  Prod p[2]{};
  for (int c = 0; c < 2; ++c) {
    const int64_t K = c ? a.m : a.n, nkb = (K + 127) / 128;
    p[c].a = w.d[c];
    p[c].bits = c ? a.ut : a.vt;
    p[c].ldb = c ? a.ldut : a.ldvt;
    p[c].T = a.T; p[c].N = a.r; p[c].K = K;
    p[c].P = w.P[c]; p[c].ldp = a.r; p[c].slice = a.T * a.r;
    p[c].split = proj_split(a.T, a.r, K);
    p[c].kbs = (nkb + p[c].split - 1) / p[c].split;
    p[c].split = (int)((nkb + p[c].kbs - 1) / p[c].kbs);   // (no empty slice)
  }
  if ((e = products<kProj, D>(p[0], p[1], s)) != hipSuccess) return e;
  // p -> q: ds1; dp -> da: dx, ds2
  if ((e = rows<digits(kGrad)>(SrcProj{w.P[0], a.r, a.T * a.r, p[0].split, a.r},
                               SrcProj{w.P[1], a.r, a.T * a.r, p[1].split, a.r}, a.T, w, s)) != hipSuccess)
    return e;
  for (int c = 0; c < 2; ++c) {
    p[c].K = a.r; p[c].split = 1; p[c].kbs = (a.r + 127) / 128;
  }
  p[0].bits = a.u; p[0].ldb = a.ldu; p[0].N = a.m;
  p[0].dY = a.dY; p[0].lddy = a.lddy;
  p[0].colp = one ? a.ds1 : w.cp1;
  p[1].bits = a.v; p[1].ldb = a.ldv; p[1].N = a.n;
  p[1].x = a.x; p[1].s2 = a.s2; p[1].dX = a.dX; p[1].lddx = a.lddx;
  p[1].colp = one ? a.ds2 : w.cp2;
  if ((e = products<kGrad, D>(p[0], p[1], s)) != hipSuccess) return e;
  if (one) return hipSuccess;
  hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((a.m + a.n + 31) / 32)), dim3(256), 0, s,
                     w.cp1, a.m, a.ds1, w.cp2, a.n, a.ds2, (a.T + kTile - 1) / kTile);
  return hipGetLastError();
}

}  // namespace

int64_t binback_work_bytes(int64_t m, int64_t n, int64_t r, int64_t T) {
  return carve(nullptr, m, n, r, T).bytes;
}

hipError_t launch_binback(const BinBack& a, hipStream_t s) {
  if (a.dtype == kF32) return run<kF32>(a, s);
  return a.dtype == kBF16 ? run<kBF16>(a, s) : run<kF16>(a, s);
}

}  // namespace nq
