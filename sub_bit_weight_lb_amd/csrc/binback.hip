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
// 128, so 2^24 columns fit 32 bits), no order of summing changes a result,
// and the value is rounded to fp32 once, at the end. Against three bf16 terms
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
// the largest magnitude of ND balanced digits, 1.99215...  2^(8 ND - 2): an
// fp32 value with a mantissa up to this is below it
constexpr uint32_t kTopMant = 8322814;

// ---------------------------------------------------------------- rows
// Sources of 32 consecutive columns of a row (c0 a multiple of 32).
struct SrcAct {      // s2 * x^
  Act8 q;
  const float* scale;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c0, float (&x)[32]) const {
    const int left = (int)min<int64_t>(32, cols - c0);
    const float st = act8_step(q.exps[row * q.lde + (c0 >> 5)]);
    const int8_t* p = q.codes + row * q.ldc + c0;
    if (left == 32) {
      u32x4 v[2];
      __builtin_memcpy(v, p, 32);
#pragma unroll
      for (int i = 0; i < 32; ++i)
        x[i] = (float)(int8_t)(v[i >> 4][(i >> 2) & 3] >> (8 * (i & 3))) * st * scale[c0 + i];
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = i < left ? (float)p[i] * st * scale[c0 + i] : 0.0f;
    }
  }
};
template <int D>
struct SrcGrad {     // s1 * dy
  const typename Elem<D>::type* p;
  int64_t ld;
  const float* scale;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c0, float (&x)[32]) const {
    typedef typename Elem<D>::type E;
    const int left = (int)min<int64_t>(32, cols - c0);
    const E* q = p + row * ld + c0;
    if (left == 32) {
      E r[32];
      __builtin_memcpy(r, q, sizeof(r));
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = Elem<D>::to(r[i]) * scale[c0 + i];
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = i < left ? Elem<D>::to(q[i]) * scale[c0 + i] : 0.0f;
    }
  }
};
struct SrcProj {     // p or dp: fp32, or the fp64 partial sums of nsum slices
  const void* p;
  int64_t ld, slice;
  int nsum;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c0, float (&x)[32]) const {
    const int left = (int)min<int64_t>(32, cols - c0);
    if (nsum == 1) {
      const float* q = (const float*)p + row * ld + c0;
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = i < left ? q[i] : 0.0f;
      return;
    }
    const double* q = (const double*)p + row * ld + c0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      double a = 0.0;
      if (i < left)
        for (int z = 0; z < nsum; ++z) a += q[z * slice + i];
      x[i] = (float)a;
    }
  }
};

// One wave per row: the largest magnitude, then the digits and their sum.
// steps[row] = the row's step (NaN where the row holds a NaN or an
// infinity: its results are NaN), sums[row] = the sum of its integers.
// Columns past `cols` up to a multiple of 128 get zero digits.
template <int ND, class Src>
__global__ __launch_bounds__(512) void rows_kernel(Src src, int64_t T, int64_t cols,
                                                   uint8_t* __restrict__ planes,
                                                   float* __restrict__ steps,
                                                   int64_t* __restrict__ sums) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 6);
  if (row >= T) return;
  const int64_t nkb = (cols + 127) / 128, nw = (cols + 31) / 32;
  uint32_t mx = 0;
  float x[32];
  for (int64_t w = lane; w < nw; w += 64) {
    src.load(row, w * 32, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = max(mx, __float_as_uint(x[i]) & 0x7fffffffu);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
  // max|v| = 1.f 2^(E - 127) <= 127.5 256^(ND - 1) 2^e
  const bool bad = mx >= 0x7f800000u;
  const int e = max((int)(mx >> 23) - 127 - (8 * ND - 2) + ((mx & 0x7fffffu) > kTopMant), -126);
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  int64_t sum = 0;
  for (int64_t w = lane; w < 4 * nkb; w += 64) {
    uint32_t dig[ND][8];
#pragma unroll
    for (int p = 0; p < ND; ++p)
#pragma unroll
      for (int k = 0; k < 8; ++k) dig[p][k] = 0;
    if (w < nw && !bad) {
      src.load(row, w * 32, x);
#pragma unroll
      for (int c = 0; c < 32; ++c) {
        int v = (int)rintf(x[c] * inv);
        sum += v;
        // dword 4 s + d, byte b of the operand: column 8 b + 4 s + d
        const int k = c & 7, sh = 8 * (c >> 3);
#pragma unroll
        for (int p = 0; p < ND; ++p) {
          const int d = (int)(int8_t)v;
          dig[p][k] |= ((uint32_t)d & 0xffu) << sh;
          v = (v - d) >> 8;
        }
      }
    }
    uint8_t* dst = planes + ((row >> 4) * nkb + (w >> 2)) * (ND * kDigit) +
                   (((int)(w & 3) << 4) + (int)(row & 15)) * 16;
#pragma unroll
    for (int p = 0; p < ND; ++p)
#pragma unroll
      for (int s = 0; s < 2; ++s)
        *(u32x4*)(dst + p * kDigit + s * 1024) =
            u32x4{dig[p][4 * s], dig[p][4 * s + 1], dig[p][4 * s + 2], dig[p][4 * s + 3]};
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor((long long)sum, o);
  if (lane == 0) {
    steps[row] = bad ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(e + 127) << 23);
    sums[row] = sum;
  }
}

// ---------------------------------------------------------------- products
enum Epi : int {
  kProj = 0,   // out: p or dp (fp32, or fp64 partials when the columns are split)
  kDs1 = 1,    // column sums of dy q
  kDx = 2,     // dx = s2 da, column sums of da x^
};
constexpr int digits(int epi) { return epi == kProj ? 4 : 3; }
constexpr int row_tiles(int epi) { return epi == kProj ? 2 : 4; }   // 16-row tiles per wave
struct Prod {
  const uint8_t* planes;      // digits of T rows, K columns
  const float* steps;
  const int64_t* sums;
  const uint32_t* bits;       // N x K signs
  int64_t ldb, T, N, K;
  // kProj
  void* P;
  int64_t ldp, slice;
  int split;
  int64_t kbs;                // 128-column blocks per slice
  // kDs1, kDx
  float* colp;                // row tiles x N partial column sums
  const void* dY;             // kDs1
  int64_t lddy;
  Act8 x;                     // kDx
  const float* s2;
  void* dX;                   // nullable
  int64_t lddx;
};

// What one accumulator element D = sum_c bit_c D_c (row t, sign row n) gives:
// stores it, or returns its share of the column sum.
template <int EPI, int D>
__device__ __forceinline__ float finish(const Prod& a, int64_t t, int64_t n, double acc, int z) {
  typedef typename Elem<D>::type E;
  if (t >= a.T || n >= a.N) return 0.0f;
  const double sum = z == 0 ? (double)a.sums[t] : 0.0;
  const double val = (double)a.steps[t] * (2.0 * acc - sum);
  if (EPI == kProj) {
    if (a.split == 1)
      ((float*)a.P)[t * a.ldp + n] = (float)val;
    else
      ((double*)a.P)[z * a.slice + t * a.ldp + n] = val;
    return 0.0f;
  }
  const float v = (float)val;
  if (EPI == kDs1) return Elem<D>::to(((const E*)a.dY)[t * a.lddy + n]) * v;
  if (a.dX) ((E*)a.dX)[t * a.lddx + n] = Elem<D>::from(a.s2[n] * v);
  return v * ((float)a.x.codes[t * a.x.ldc + n] * act8_step(a.x.exps[t * a.x.lde + (n >> 5)]));
}

// sum_i 256^i d_i, exact
template <int ND>
__device__ __forceinline__ double join(const int (&d)[ND]) {
  double r = (double)d[ND - 1];
#pragma unroll
  for (int p = ND - 2; p >= 0; --p) r = fma(r, 256.0, (double)d[p]);
  return r;
}
// dwords of the signs' operand, half s of word w
__device__ __forceinline__ i32x4 spread(uint32_t w, int s) {
  i32x4 r;
#pragma unroll
  for (int d = 0; d < 4; ++d) r[d] = (int)((w >> (4 * s + d)) & 0x01010101u);
  return r;
}

template <int EPI, int D>
__global__ __launch_bounds__(256, 2) void wide_kernel(Prod a) {
  constexpr int ND = digits(EPI), MI = row_tiles(EPI);
  constexpr int kBlock = ND * kDigit, kRows = 32 * MI;
  constexpr int kStage = 2 * MI * ND * 1024;   // 32 MI rows, 64 columns
  __shared__ __align__(16) uint8_t lds[2 * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t ntn = (a.N + kTile - 1) / kTile, ntm = (a.T + kRows - 1) / kRows;
  const int64_t per = (ntn * ntm + 7) / 8;
  const int64_t tile = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || tile >= ntn * ntm) return;
  const int64_t tm = tile / ntn, tn = tile - tm * ntn;
  const int z = blockIdx.y;
  const int64_t nkb = (a.K + 127) / 128, nw = (a.K + 31) / 32;
  const int64_t kb0 = z * a.kbs, kb1 = min(nkb, kb0 + a.kbs);
  // this tile's digits: 2 MI blocks of 16 rows, nkb blocks apart (rows past
  // T hold no digits of the call: whatever they give is dropped at the end)
  const __amdgpu_buffer_rsrc_t pr = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.planes + tm * 2 * MI * nkb * kBlock), (short)0, (int)(2 * MI * nkb * kBlock),
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
  float cs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    cs[j] = 0.0f;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        int d[ND];
#pragma unroll
        for (int p = 0; p < ND; ++p) d[p] = acc[p][i][j][v];
        cs[j] += finish<EPI, D>(a, t0 + 16 * i + 4 * g + v, n0 + 16 * j + li, join<ND>(d), z);
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
__global__ __launch_bounds__(64 * kThinWaves) void thin_kernel(Prod a) {
  constexpr int ND = digits(EPI), kBlock = ND * kDigit;
  __shared__ i32x4 red[kThinWaves][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
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
          const i32x4 f = *(const i32x4*)(a.planes + (i * nkb + kb) * kBlock + p * kDigit +
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
      int d[ND];
#pragma unroll
      for (int p = 0; p < ND; ++p) d[p] = acc[p][i][v];
      cs += finish<EPI, D>(a, 16 * i + 4 * g + v, n0 + li, join<ND>(d), 0);
    }
  if (EPI == kProj) return;
  cs += __shfl_xor(cs, 16);
  cs += __shfl_xor(cs, 32);
  if (g == 0 && n0 + li < a.N) a.colp[n0 + li] = cs;
}

// ds1 and ds2 from the partial column sums of nt row tiles, in fp64, in order
__global__ __launch_bounds__(256) void colsum_kernel(const float* __restrict__ p1, int64_t m,
                                                     float* __restrict__ ds1,
                                                     const float* __restrict__ p2, int64_t n,
                                                     float* __restrict__ ds2, int64_t nt) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= m + n) return;
  const float* p = i < m ? p1 + i : p2 + (i - m);
  const int64_t ld = i < m ? m : n;
  double s = 0.0;
  for (int64_t t = 0; t < nt; ++t) s += (double)p[t * ld];
  if (i < m)
    ds1[i] = (float)s;
  else
    ds2[i - m] = (float)s;
}

// ---------------------------------------------------------------- launches
struct Work {
  uint8_t* planes;
  void* P;
  float* steps;
  int64_t* sums;
  float *cp1, *cp2;
  int split;
  int64_t bytes;
};
// Slices of the columns of the first product of a chain: enough tiles for
// two workgroups on each of the 256 CUs, at least four blocks of 128 each.
int proj_split(int64_t T, int64_t r, int64_t K) {
  if (T <= kThinMax) return 1;
  const int64_t rows = 32 * row_tiles(kProj);
  const int64_t tiles = ((T + rows - 1) / rows) * ((r + kTile - 1) / kTile);
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
  const int sp = std::max(proj_split(T, r, n), proj_split(T, r, m));
  w.planes = (uint8_t*)take(Tp * std::max(4 * round_up(std::max(m, n), 128), 3 * round_up(r, 128)));
  w.P = take(sp == 1 ? 4 * T * r : 8 * T * r * sp);
  w.steps = (float*)take(4 * T);
  w.sums = (int64_t*)take(8 * T);
  w.cp1 = (float*)take(4 * nt * m);
  w.cp2 = (float*)take(4 * nt * n);
  w.bytes = off;
  return w;
}

template <int ND, class Src>
hipError_t rows(const Src& src, int64_t T, int64_t cols, const Work& w, hipStream_t s) {
  hipLaunchKernelGGL((rows_kernel<ND, Src>), dim3((unsigned)((T + 7) / 8)), dim3(512), 0, s, src, T,
                     cols, w.planes, w.steps, w.sums);
  return hipGetLastError();
}
template <int EPI, int D>
hipError_t product(const Prod& a, hipStream_t s) {
  if (a.T <= kThinMax) {
    const dim3 grid((unsigned)((a.N + 15) / 16)), block(64 * kThinWaves);
    if (a.T <= 16)
      hipLaunchKernelGGL((thin_kernel<EPI, D, 1>), grid, block, 0, s, a);
    else if (a.T <= 32)
      hipLaunchKernelGGL((thin_kernel<EPI, D, 2>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((thin_kernel<EPI, D, 4>), grid, block, 0, s, a);
    return hipGetLastError();
  }
  const int64_t rows = 32 * row_tiles(EPI);
  const int64_t tiles = ((a.T + rows - 1) / rows) * ((a.N + kTile - 1) / kTile);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)a.split);
  hipLaunchKernelGGL((wide_kernel<EPI, D>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int D>
hipError_t run(const BinBack& a, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const Work w = carve((char*)a.work, a.m, a.n, a.r, a.T);
  const bool one = a.T <= kTile;   // a single row tile: its column sums are the result
  hipError_t e;
  auto proj = [&](const uint32_t* bits, int64_t ldb, int64_t K) {
    Prod p{};
    p.planes = w.planes; p.steps = w.steps; p.sums = w.sums;
    p.bits = bits; p.ldb = ldb; p.T = a.T; p.N = a.r; p.K = K;
    p.P = w.P; p.ldp = a.r; p.slice = a.T * a.r; p.split = proj_split(a.T, a.r, K);
    const int64_t nkb = (K + 127) / 128;
    p.kbs = (nkb + p.split - 1) / p.split;
    p.split = (int)((nkb + p.kbs - 1) / p.kbs);   // (no empty slice)
    if ((e = product<kProj, D>(p, s)) != hipSuccess) return e;
    return rows<digits(kDs1)>(SrcProj{w.P, a.r, a.T * a.r, p.split, a.r}, a.T, a.r, w, s);
  };
  Prod p{};
  p.planes = w.planes; p.steps = w.steps; p.sums = w.sums;
  p.T = a.T; p.K = a.r; p.split = 1; p.kbs = (a.r + 127) / 128;
  // a -> p -> q: ds1
  if ((e = rows<digits(kProj)>(SrcAct{a.x, a.s2, a.n}, a.T, a.n, w, s)) != hipSuccess) return e;
  if ((e = proj(a.vt, a.ldvt, a.n)) != hipSuccess) return e;
  p.bits = a.u; p.ldb = a.ldu; p.N = a.m;
  p.dY = a.dY; p.lddy = a.lddy;
  p.colp = one ? a.ds1 : w.cp1;
  if ((e = product<kDs1, D>(p, s)) != hipSuccess) return e;
  // s1 dy -> dp -> da: dx, ds2
  if ((e = rows<digits(kProj)>(SrcGrad<D>{(const E*)a.dY, a.lddy, a.s1, a.m}, a.T, a.m, w, s)) != hipSuccess) return e;
  if ((e = proj(a.ut, a.ldut, a.m)) != hipSuccess) return e;
  p.bits = a.v; p.ldb = a.ldv; p.N = a.n;
  p.x = a.x; p.s2 = a.s2; p.dX = a.dX; p.lddx = a.lddx;
  p.colp = one ? a.ds2 : w.cp2;
  if ((e = product<kDx, D>(p, s)) != hipSuccess) return e;
  if (one) return hipSuccess;
  hipLaunchKernelGGL(colsum_kernel, dim3((unsigned)((a.m + a.n + 255) / 256)), dim3(256), 0, s,
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
