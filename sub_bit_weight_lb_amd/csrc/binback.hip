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
// of 2048 ND bytes, [digit][s][lane][16]: lane (li, g) = row li, a 32-column
// word per lane group g; byte 4 d + b of half s is column 8 b + 4 s + d of the
// word, so that (w >> (4 s + d)) & 0x01010101 is dword d of the signs'
// operand, one shift and one and for four columns. Four blocks share 512
// columns, 16 words: block k takes words 4 g + k, so that a lane's signs for
// all four are 16 consecutive bytes.
//
// The two chains a -> p -> q and s1 dy -> dp -> da do not depend on each
// other: each launch takes a step of both (grid z, or y), the one with more
// columns first.
//
// wide_kernel (more than kThinMax rows): 256 threads, 2 x 2 waves of 16 MI
// rows x 16 NJ signs. A wave loads its digits from memory to registers two
// steps of 64 columns ahead (a fragment is 1 KB in a row; the two waves of a
// row share it in the L1). The signs of 512 columns are copied to LDS as they
// are, double buffered, by each wave for itself: with copies shared by the
// workgroup and a barrier per 512 columns the waves wait for each other (8192 x
// 4096 columns of four digits by 2 x 2048 signs' rows 575 us, so 491). The digits
// share one expansion of the signs (8 NJ vector instructions against MI NJ ND
// products per step). Workgroup b runs on XCD b % 8, and an XCD takes
// consecutive tiles, which share their rows' digits in its L2.
// Bound by how well the loads and the expansion hide behind the products: those
// 1100 TOP in 491 us are 2.24 POP/s, kGrad's 825 TOP with their epilogue 453 us,
// 1.82 (products and expansion alone reach 3.7 POP/s, without loads here 2.5; a
// large int8 product of the library 2.16).
// thin_kernel (few rows): a workgroup takes all rows and 16 signs' rows, its
// waves split the columns and add up through LDS. Bound by latency: two launches
// of 7 us for one row of a 4096 x 4096 layer of rank 2048 (2 MB of signs each).
#include "tune.h"

#include <algorithm>

#include "binback_plan.h"

namespace nq {
using namespace binback;
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint32_t* lds_ptr_t;

constexpr int kThinWaves = 8;
// Up to this many rows, a workgroup per row, else eight rows per workgroup
// (whole calls in us, rank 1024: 200 rows of a 4096 x 4096 layer 56 v 77, 512
// rows of 11008 x 4096 117 v 139, 1000 rows of 4096 x 4096 119 v 112).
constexpr int64_t kTeamRows = 512;
// the largest magnitude of ND balanced digits, 1.99215...  2^(8 ND - 2): an
// fp32 value with a mantissa up to this is below it
constexpr uint32_t kTopMant = 8322814;

// ---------------------------------------------------------------- rows
// Sources of four columns c .. c + 3 of a row, c a multiple of 4 (past the end:
// 0), loaded together from any address.
template <class T>
struct __attribute__((packed)) Four {
  T v[4];
};
template <class T>
__device__ __forceinline__ Four<T> load4(const T* p, int64_t left) {
  Four<T> r;
  if (left >= 4) {
    __builtin_memcpy(&r, p, sizeof(r));
  } else {
#pragma unroll
    for (int d = 0; d < 4; ++d) r.v[d] = d < left ? p[d] : (T)0;
  }
  return r;
}
struct SrcAct {      // s2 * x^
  Act8 q;
  const float* scale;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c, float (&x)[4]) const {
    const float st = c < cols ? act8_step(q.exps[row * q.lde + (c >> 5)]) : 0.0f;
    const Four<int8_t> v = load4(q.codes + row * q.ldc + c, cols - c);
    const Four<float> f = load4(scale + c, cols - c);
#pragma unroll
    for (int d = 0; d < 4; ++d) x[d] = c + d < cols ? (float)v.v[d] * st * f.v[d] : 0.0f;
  }
};
template <int D>
struct SrcGrad {     // s1 * dy
  const typename Elem<D>::type* p;
  int64_t ld;
  const float* scale;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c, float (&x)[4]) const {
    const Four<typename Elem<D>::type> v = load4(p + row * ld + c, cols - c);
    const Four<float> f = load4(scale + c, cols - c);
#pragma unroll
    for (int d = 0; d < 4; ++d) x[d] = Elem<D>::to(v.v[d]) * f.v[d];
  }
};
struct SrcProj {     // p or dp: fp32, or the fp64 partial sums of nsum slices
  const void* p;
  int64_t ld, slice;
  int nsum;
  int64_t cols;
  __device__ __forceinline__ void load(int64_t row, int64_t c, float (&x)[4]) const {
    if (nsum == 1) {
      const Four<float> v = load4((const float*)p + row * ld + c, cols - c);
#pragma unroll
      for (int d = 0; d < 4; ++d) x[d] = v.v[d];
      return;
    }
    double a[4] = {0.0, 0.0, 0.0, 0.0};
    for (int z = 0; z < nsum; ++z) {
      const Four<double> v = load4((const double*)p + z * slice + row * ld + c, cols - c);
#pragma unroll
      for (int d = 0; d < 4; ++d) a[d] += v.v[d];
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) x[d] = (float)a[d];
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
// max|v| = 1.f 2^(E - 127) <= 127.5 256^(ND - 1) 2^e; 2^-149, of which every fp32
// value is a multiple, at least.
template <int ND>
__device__ __forceinline__ int row_exponent(uint32_t mx) {
  return max((int)(mx >> 23) - 127 - (8 * ND - 2) + ((mx & 0x7fffffu) > kTopMant), -149);
}
// out[k] = byte k of u[0], u[1], u[2], u[3]
__device__ __forceinline__ void transpose_bytes(const uint32_t (&u)[4], uint32_t (&out)[4]) {
  const uint32_t a = __builtin_amdgcn_perm(u[1], u[0], 0x05010400u);
  const uint32_t c = __builtin_amdgcn_perm(u[3], u[2], 0x05010400u);
  const uint32_t d = __builtin_amdgcn_perm(u[1], u[0], 0x07030602u);
  const uint32_t e = __builtin_amdgcn_perm(u[3], u[2], 0x07030602u);
  out[0] = __builtin_amdgcn_perm(c, a, 0x05040100u);
  out[1] = __builtin_amdgcn_perm(c, a, 0x07060302u);
  out[2] = __builtin_amdgcn_perm(e, d, 0x05040100u);
  out[3] = __builtin_amdgcn_perm(e, d, 0x07060302u);
}
// Four values as digits: out[p] holds digit p of value d in byte d. With 128
// added to each digit's place the bytes of an integer are its balanced digits
// plus 128.
template <int ND>
__device__ __forceinline__ void to_digits(const float (&x)[4], int e, uint32_t (&out)[4]) {
  constexpr uint32_t kBias = ND == 4 ? 0x80808080u : 0x00808080u;
  uint32_t u[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) u[d] = ((uint32_t)(int)rintf(ldexpf(x[d], -e)) + kBias) ^ 0x80808080u;
  transpose_bytes(u, out);
}

// A wave takes 256 columns of a row at a time, four consecutive ones per lane,
// and exchanges digits through LDS: a lane's four columns 8 b + 4 s + d, d = 0
// .. 3, are one byte each of half s's four dwords, so whole halves (16 bytes, b
// = 0 .. 3) are read back and their bytes transposed. Eight rows per workgroup,
// a wave each, so that whole 128-byte lines are stored; TEAM: one row per
// workgroup, its waves taking 256 columns in turn (few rows). blockIdx.y picks
// one of two jobs. Columns past the end up to a multiple of 512 get zeros.
// Bound by its loads and stores: 8192 x 4096 fp32 and as many codes to four
// digits (436 MB) 127 us, 3.4 TB/s (loads of single elements 8 columns apart
// 137; two waves per row 147).
template <int ND, bool TEAM, class S0, class S1>
__global__ __launch_bounds__(512) void rows_kernel(S0 s0, S1 s1, int64_t T, Digits o0, Digits o1) {
  constexpr int kGroup = TEAM ? 1 : 8;                // rows
  constexpr int kRun = 16 * kGroup + (TEAM ? 0 : 16); // a half of each row, padded for the banks
  constexpr int kBuf = ND * 16 * kRun;                // 256 columns
  __shared__ __align__(16) uint8_t buf[TEAM ? 8 : 2][kBuf];
  __shared__ uint32_t wmax[8];
  __shared__ int wsum[8][ND];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = TEAM ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 8 + wave;
  const bool job = blockIdx.y;
  const int64_t cols = job ? s1.cols : s0.cols;
  const Digits o = job ? o1 : o0;
  const bool in = row < T;
  const int64_t nkb = blocks(cols), nch = nkb / 2;
  const int64_t first = TEAM ? wave : 0, stride = TEAM ? 8 : 1;
  const int w8 = lane >> 3, b = (lane >> 1) & 3, s = lane & 1;   // word, and where in it
  auto load = [&](int64_t ch, float (&x)[4]) {
    const int64_t c = ch * 256 + 4 * lane;
    if (!in) {
      x[0] = x[1] = x[2] = x[3] = 0.0f;
    } else if (job) {
      s1.load(row, c, x);
    } else {
      s0.load(row, c, x);
    }
  };
  uint32_t mx = 0;
  auto look = [&](const float (&x)[4]) {
#pragma unroll
    for (int b = 0; b < 4; ++b) mx = max(mx, __float_as_uint(x[b]) & 0x7fffffffu);
  };
  // the first runs of 256 columns stay in registers (4096 columns), the rest
  // are read a second time
  constexpr int kKeep = TEAM ? 2 : 16;
  float keep[kKeep][4];
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (first + k * stride < nch) load(first + k * stride, keep[k]);
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (first + k * stride < nch) look(keep[k]);
  for (int64_t ch = first + kKeep * stride; ch < nch; ch += stride) {
    float x[4];
    load(ch, x);
    look(x);
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
  int sum[ND];
#pragma unroll
  for (int p = 0; p < ND; ++p) sum[p] = 0;
  // run (digit, s, word) of LDS holds that half of the group's rows; it goes to
  // block word % 4 of the 512 columns' four, lane group word / 4, plus two in the
  // second 256
  auto half_of = [&](int64_t ch, int run, int64_t r, const uint8_t* src) {
    const int w = run & 7, h = (run >> 3) & 1, p = run >> 4;
    const u32x4 v = *(const u32x4*)src;
    const uint32_t u[4] = {v[0], v[1], v[2], v[3]};
    uint32_t t[4];
    transpose_bytes(u, t);
    *(u32x4*)(o.planes + ((r >> 4) * nkb + (ch >> 1) * 4 + (w & 3)) * (ND * kDigit) + p * kDigit +
              h * 1024 + (((w >> 2) + 2 * (int)(ch & 1)) * 16 + (int)(r & 15)) * 16) =
        u32x4{t[0], t[1], t[2], t[3]};
  };
  auto write = [&](int64_t ch, float (&x)[4]) {
    if (bad) x[0] = x[1] = x[2] = x[3] = 0.0f;
    uint32_t dig[4];
    to_digits<ND>(x, e, dig);
#pragma unroll
    for (int p = 0; p < ND; ++p)
      sum[p] = __builtin_amdgcn_sdot4((int)dig[p], 0x01010101, sum[p], false);
    uint8_t* to = buf[TEAM ? wave : ch & 1];
#pragma unroll
    for (int p = 0; p < ND; ++p)
      *(uint32_t*)(to + ((p * 2 + s) * 8 + w8) * kRun + (TEAM ? 0 : wave * 16) + 4 * b) = dig[p];
    if (TEAM) {
      // a wave's own 256 columns
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      if (lane < ND * 16) half_of(ch, lane, row, to + lane * kRun);
      __builtin_amdgcn_wave_barrier();
    } else {
      __syncthreads();   // (the other buffer is free: its readers passed this barrier)
      const int t = threadIdx.x;
      if (t < ND * 128)
        half_of(ch, t >> 3, (int64_t)blockIdx.x * 8 + (t & 7), to + (t >> 3) * kRun + (t & 7) * 16);
    }
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k)
    if (first + k * stride < nch) write(first + k * stride, keep[k]);
  for (int64_t ch = first + kKeep * stride; ch < nch; ch += stride) {
    float x[4];
    load(ch, x);
    write(ch, x);
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
    o.steps[row] = bad ? __uint_as_float(0x7fc00000u) : ldexpf(1.0f, e);
    i32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < ND; ++p) v[p] = sum[p];
    o.sums[row] = v;
  }
}

// ---------------------------------------------------------------- products
struct Prod {
  Digits a;                   // T rows, K columns
  const uint32_t* bits;       // N x K signs
  int64_t ldb, T, N, K;
  // kProj
  void* P;
  int64_t ldp, slice;
  int split;
  int64_t kbs;                // blocks per slice, a multiple of 4
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
// The end of a wave's MI x NJ tiles from row t0 and sign row n0: acc[p][i][j]
// of lane (g, li), element v is row 16 i + 4 g + v, sign row 16 j + li. Stores
// kProj's values or dx, and adds the wave's share of the column sums to cs.
// Loads are clamped to the last row and column and what they give dropped, so
// that a row's loads go out together.
template <int EPI, int D, int MI, int NJ>
__device__ __forceinline__ void finish(const Prod& a, int64_t t0, int64_t n0, int g, int li, int z,
                                       const i32x4 (&acc)[digits(EPI)][MI][NJ], float (&cs)[NJ]) {
  typedef typename Elem<D>::type E;
  constexpr int ND = digits(EPI);
  int64_t n[NJ];
  bool in[NJ];
  float s2[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    in[j] = n0 + 16 * j + li < a.N;
    n[j] = in[j] ? n0 + 16 * j + li : a.N - 1;
    s2[j] = EPI == kGrad && !a.dY ? a.s2[n[j]] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const bool row = t0 + 16 * i + 4 * g + v < a.T;
      const int64_t t = row ? t0 + 16 * i + 4 * g + v : a.T - 1;
      const float step = a.a.steps[t];
      const i32x4 sum = a.a.sums[t];
      float val[NJ];
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        int d[ND];
#pragma unroll
        for (int p = 0; p < ND; ++p) d[p] = acc[p][i][j][v];
        val[j] = value<ND>(step, sum, d);
      }
      if (EPI == kProj) {
        if (a.split == 1) {
          float* out = (float*)a.P + t * a.ldp;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            if (row && in[j]) out[n[j]] = val[j];
        } else {   // a slice's share, exact; the first takes the digit sums
          double* out = (double*)a.P + z * a.slice + t * a.ldp;
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            double r = 0.0;
#pragma unroll
            for (int p = ND - 1; p >= 0; --p)
              r = fma(r, 256.0, 2.0 * (double)acc[p][i][j][v] - (z == 0 ? (double)sum[p] : 0.0));
            if (row && in[j]) out[n[j]] = r * (double)step;
          }
        }
      } else if (a.dY) {
        const E* y = (const E*)a.dY + t * a.lddy;
        E e[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) e[j] = y[n[j]];
#pragma unroll
        for (int j = 0; j < NJ; ++j) cs[j] += row && in[j] ? Elem<D>::to(e[j]) * val[j] : 0.0f;
      } else {
        const int8_t* c = a.x.codes + t * a.x.ldc;
        const uint8_t* x = a.x.exps + t * a.x.lde;
        int code[NJ];
        uint32_t ex[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          code[j] = c[n[j]];
          ex[j] = x[n[j] >> 5];
        }
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          cs[j] += row && in[j] ? val[j] * ((float)code[j] * act8_step(ex[j])) : 0.0f;
        if (a.dX) {
          E* out = (E*)a.dX + t * a.lddx;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            if (row && in[j]) out[n[j]] = Elem<D>::from(s2[j] * val[j]);
        }
      }
    }
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
  constexpr int ND = digits(EPI), MI = row_tiles(EPI), NJ = sign_tiles(EPI);
  constexpr int kBlock = ND * kDigit, kRows = 32 * MI, kSigns = 32 * NJ;
  // a wave's own 16 NJ rows of signs of 512 columns, two of these: no wave waits
  // for another. Four rows are 65 words apart, so that 16 rows' words 4 g lie in
  // distinct banks.
  constexpr int kFour = 65;
  __shared__ uint32_t lds[4][2][4 * NJ][kFour];
  const Prod& a = blockIdx.z ? a1 : a0;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t ntn = (a.N + kSigns - 1) / kSigns, ntm = (a.T + kRows - 1) / kRows;
  const int64_t per = (ntn * ntm + 7) / 8;
  const int64_t tile = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  const int z = blockIdx.y;
  if ((int64_t)(blockIdx.x >> 3) >= per || tile >= ntn * ntm || z >= a.split) return;
  const int64_t tm = tile / ntn, tn = tile - tm * ntn;
  const int64_t nkb = blocks(a.K), nw = (a.K + 31) / 32;
  const int64_t kb0 = z * a.kbs, kb1 = lmin(nkb, kb0 + a.kbs);
  // signs of the wave: rows past N are past the descriptor's range (which counts
  // the vector offset alone) and read as zero; words past a row's last read what
  // follows, or nothing past the last row's: they meet zero digits
  const int64_t n0 = tn * kSigns + wn * 16 * NJ, rows = lmin(16 * NJ, a.N - n0);
  const uint64_t at0 = (uint64_t)(uintptr_t)(a.bits + n0 * a.ldb);
  const int lo = scalar((int)at0), hi = scalar((int)(at0 >> 32) & 0xffff);
  const int size = scalar(rows > 0 ? (int)(((rows - 1) * a.ldb + nw) * 4) : 0);
  const int to = scalar((int)(uint32_t)(uintptr_t)(lds_ptr_t)&lds[wave][0][0][0]);
  const uint32_t from = (uint32_t)((lane >> 4) * a.ldb * 4) + (lane & 15) * 4;
  const uint32_t four = (uint32_t)(16 * a.ldb);   // bytes of four rows
  // Copy c, 4 rows x 16 words, of the signs of 512 columns sb (!live: of zeros,
  // which reads nothing). Written out: after a builtin's the compiler waits for
  // all loads at the next use of one. It writes no register and keeps its place
  // among the loads of digits and the waits.
  auto copy = [&](int64_t sb, int c, bool live) {
    const int st = to + (int)(sb & 1) * 16 * NJ * kFour;
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"   // (m0 is reserved: nothing is kept in it across)
    asm volatile(
        "s_mov_b32 s92, %0\n\t"
        "s_mov_b32 s93, %1\n\t"
        "s_mov_b32 s94, %2\n\t"
        "s_mov_b32 s95, 0x20000\n\t"
        "s_add_u32 m0, %3, %4\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %5, s[92:95], 0 offen lds"
        :
        : "s"(lo), "s"(hi), "s"(live ? size : 0), "s"(st), "i"(c * kFour * 4),
          "v"(from + ((uint32_t)sb * 64 + c * four))
        : "m0", "s92", "s93", "s94", "s95", "scc");
#pragma clang diagnostic pop
  };
  // the wave's digits: MI rows of blocks, nkb blocks apart (rows past T hold no
  // digits of the call: whatever they give is dropped at the end)
  const uint8_t* dp = a.a.planes + (tm * 2 + wm) * MI * nkb * kBlock;
  i32x4 fr[2][MI][ND];
  auto digits_of = [&](int64_t kb, int s) {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int p = 0; p < ND; ++p)
        fr[s][i][p] = *(const i32x4*)((dp + (i * nkb + kb) * kBlock + p * kDigit + s * 1024) +
                                      (uint32_t)lane * 16);
  };
  i32x4 acc[ND][MI][NJ];
#pragma unroll
  for (int p = 0; p < ND; ++p)
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[p][i][j] = i32x4{0, 0, 0, 0};
#pragma unroll
  for (int c = 0; c < 4 * NJ; ++c) copy(kb0 >> 2, c, true);
  __builtin_amdgcn_sched_barrier(0);
  digits_of(kb0, 0);
  __builtin_amdgcn_sched_barrier(0);   // (in the order of the loop's, which the waits count)
  digits_of(kb0, 1);
  __builtin_amdgcn_sched_barrier(0);
  // word 4 g + q of row 16 j + li
  const uint32_t* mine = &lds[wave][0][0][0] + (li >> 2) * kFour + (li & 3) * 16 + 4 * g;
  // the copies issued before the last half step's digits have landed
  auto landed = [&]() { asm volatile("s_waitcnt vmcnt(%0)" ::"i"(MI * ND) : "memory"); };
  uint32_t word[2][NJ];
  auto words_of = [&](int64_t sb, int q) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) word[q & 1][j] = mine[((int)(sb & 1) * NJ + j) * 4 * kFour + q];
  };
  landed();
  words_of(kb0 >> 2, 0);
  for (int64_t k0 = kb0; k0 < kb1; k0 += 4) {
    const bool more = k0 + 4 < kb1;
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      const int q = h >> 1, s = h & 1;
      const int64_t ahead = lmin(k0 + q + 1, kb1 - 1);
      i32x4 b = spread(word[q & 1][0], s);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const i32x4 nb = spread(word[q & 1][j + 1 < NJ ? j + 1 : j], s);
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int p = 0; p < ND; ++p)
            acc[p][i][j] =
                __builtin_amdgcn_mfma_i32_16x16x64_i8(fr[s][i][p], b, acc[p][i][j], 0, 0, 0);
        // the next signs are spread between the products
#pragma unroll
        for (int q = 0; q < MI * ND; ++q) {
          __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x2, 2, 0);
        }
        b = nb;
        if (j == 0) {
          // (after this half step's wait for its digits, which counts what is
          // younger)
          __builtin_amdgcn_sched_barrier(0);
          if (s) {
            // the next block's words (after the last block, of what is there)
            if (q == 3) landed();
            words_of((k0 >> 2) + (q == 3), (q + 1) & 3);
          }
          if (h < 4) {
            // a quarter of the next 512's copies (of zeros at the end)
#pragma unroll
            for (int c = h * NJ; c < (h + 1) * NJ; ++c) copy((k0 >> 2) + 1, c, more);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // (kept here: the next step's products must not move above these loads)
      digits_of(ahead, s);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // the last copies must land before LDS is used again or given away
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  float cs[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) cs[j] = 0.0f;
  finish<EPI, D, MI, NJ>(a, tm * kRows + wm * 16 * MI, tn * kSigns + wn * 16 * NJ, g, li, z, acc, cs);
  if (EPI == kProj) return;
  // the tile's column sums: the rows of a lane, then the four lanes of a
  // column, then the two row halves, each in a fixed order
  __syncthreads();
  float* half = (float*)lds;   // [wm][kSigns]
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    cs[j] += __shfl_xor(cs[j], 16);
    cs[j] += __shfl_xor(cs[j], 32);
    if (g == 0) half[wm * kSigns + wn * 16 * NJ + 16 * j + li] = cs[j];
  }
  __syncthreads();
  const int c = threadIdx.x;
  if (c < kSigns && tn * kSigns + c < a.N)
    a.colp[tm * a.N + tn * kSigns + c] = half[c] + half[kSigns + c];
}

// All T <= 16 MT rows and 16 sign rows per workgroup; wave w takes the
// 128-column blocks w, w + 8, ... (rows past T up to 16 MT hold no digits of the
// call, but the planes have room for them: digit_rows)
template <int EPI, int D, int MT>
__global__ __launch_bounds__(64 * kThinWaves) void thin_kernel(Prod a0, Prod a1) {
  constexpr int ND = digits(EPI), kBlock = ND * kDigit;
  __shared__ i32x4 red[kThinWaves][MT][64];
  const Prod& a = blockIdx.y ? a1 : a0;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int z = blockIdx.z;
  if (n0 >= a.N || z >= a.split) return;
  const int64_t nkb = blocks(a.K), nw = (a.K + 31) / 32;
  const int64_t kb1 = lmin(nkb, (z + 1) * a.kbs);
  const uint32_t* bp = a.bits + lmin(n0 + li, a.N - 1) * a.ldb;
  i32x4 acc[ND][MT][1];
#pragma unroll
  for (int p = 0; p < ND; ++p)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[p][i][0] = i32x4{0, 0, 0, 0};
  for (int64_t kb = z * a.kbs + wave; kb < kb1; kb += kThinWaves) {
    const uint32_t w = bp[lmin((kb >> 2) * 16 + 4 * g + (kb & 3), nw - 1)];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const i32x4 b = spread(w, s);
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int p = 0; p < ND; ++p) {
          const i32x4 f = *(const i32x4*)(a.a.planes + (i * nkb + kb) * kBlock + p * kDigit +
                                          s * 1024 + lane * 16);
          acc[p][i][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f, b, acc[p][i][0], 0, 0, 0);
        }
    }
  }
  // the waves' sums, one digit at a time through LDS
#pragma unroll
  for (int p = 0; p < ND; ++p) {
    if (p) __syncthreads();
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[p][i][0];
    __syncthreads();
    if (wave == 0) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int w = 1; w < kThinWaves; ++w) acc[p][i][0] += red[w][i][lane];
    }
  }
  if (wave) return;
  float cs[1] = {0.0f};
  finish<EPI, D, MT, 1>(a, 0, n0, g, li, z, acc, cs);
  if (EPI == kProj) return;
  cs[0] += __shfl_xor(cs[0], 16);
  cs[0] += __shfl_xor(cs[0], 32);
  if (g == 0 && n0 + li < a.N) a.colp[n0 + li] = cs[0];
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
};
Work carve(char* base, const Plan& p) {
  Work w{};
  for (int c = 0; c < 2; ++c) {
    w.d[c] = Digits{(uint8_t*)base + p.planes[c], (float*)(base + p.steps[c]),
                    (i32x4*)(base + p.sums[c])};
    w.P[c] = base + p.P[c];
  }
  w.cp1 = (float*)(base + p.cp1);
  w.cp2 = (float*)(base + p.cp2);
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
    const dim3 grid((unsigned)((N + 15) / 16), 2, (unsigned)std::max(a.split, b.split));
    const dim3 block(64 * kThinWaves);
    const int tiles = thin_tiles(a.T);
    if (tiles == 1)
      hipLaunchKernelGGL((thin_kernel<EPI, D, 1>), grid, block, 0, s, a, b);
    else if (tiles == 2)
      hipLaunchKernelGGL((thin_kernel<EPI, D, 2>), grid, block, 0, s, a, b);
    else
      hipLaunchKernelGGL((thin_kernel<EPI, D, 4>), grid, block, 0, s, a, b);
    return hipGetLastError();
  }
  const int64_t tiles = tiles_of(EPI, a.T, N);
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8), (unsigned)std::max(a.split, b.split), 2);
  // the longer chain's tiles start first
  if (a.K >= b.K)
    hipLaunchKernelGGL((wide_kernel<EPI, D>), grid, dim3(256), 0, s, a, b);
  else
    hipLaunchKernelGGL((wide_kernel<EPI, D>), grid, dim3(256), 0, s, b, a);
  return hipGetLastError();
}

template <int D>
hipError_t run(const BinBack& a, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const Plan plan = plan_for(a.m, a.n, a.r, a.T);
  const Work w = carve((char*)a.work, plan);
  const bool one = a.T <= kSumRows;   // a single row tile: its column sums are the result
  hipError_t e;
  // a and s1 dy, then p and dp
  if ((e = rows<digits(kProj)>(SrcAct{a.x, a.s2, a.n},
                               SrcGrad<D>{(const E*)a.dY, a.lddy, a.s1, a.m}, a.T, w, s)) != hipSuccess)
    return e;
  Prod p[2]{};
  for (int c = 0; c < 2; ++c) {
    const int64_t K = c ? a.m : a.n, nkb = blocks(K);
    p[c].a = w.d[c];
    p[c].bits = c ? a.ut : a.vt;
    p[c].ldb = c ? a.ldut : a.ldvt;
    p[c].T = a.T; p[c].N = a.r; p[c].K = K;
    p[c].P = w.P[c]; p[c].ldp = a.r; p[c].slice = a.T * a.r;
    p[c].split = plan.split[c];
    p[c].kbs = round_up((nkb + p[c].split - 1) / p[c].split, 4);
    p[c].split = (int)((nkb + p[c].kbs - 1) / p[c].kbs);   // (no empty slice)
  }
  if ((e = products<kProj, D>(p[0], p[1], s)) != hipSuccess) return e;
  // p -> q: ds1; dp -> da: dx, ds2
  if ((e = rows<digits(kGrad)>(SrcProj{w.P[0], a.r, a.T * a.r, p[0].split, a.r},
                               SrcProj{w.P[1], a.r, a.T * a.r, p[1].split, a.r}, a.T, w, s)) != hipSuccess)
    return e;
  for (int c = 0; c < 2; ++c) {
    p[c].K = a.r; p[c].split = 1; p[c].kbs = blocks(a.r);
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
                     w.cp1, a.m, a.ds1, w.cp2, a.n, a.ds2, (a.T + kSumRows - 1) / kSumRows);
  return hipGetLastError();
}

}  // namespace

int64_t binback_work_bytes(int64_t m, int64_t n, int64_t r, int64_t T) {
  return plan_for(m, n, r, T).bytes;
}

hipError_t launch_binback(const BinBack& a, hipStream_t s) {
  if (a.dtype == kF32) return run<kF32>(a, s);
  return a.dtype == kBF16 ? run<kBF16>(a, s) : run<kF16>(a, s);
}

}  // namespace nq
