// 8-bit checkpoints of activations. 32 consecutive columns of a row share a
// power-of-two step 2^e, e the least integer with max|x| <= 127 2^e, clamped
// to -126 .. 121 (and at most 9 for fp16 inputs, so that every value stays
// finite in the input's type); a value is kept as code = round-to-even(x /
// 2^e) in -127 .. 127, in 8.25 bits with its share of the exponent. A group
// that holds a NaN or an infinity gets the exponent 255 and reads as NaN.
//
// Why powers of two: x / 2^e and code * 2^e are exact in fp32, so the codes
// do not depend on how a quotient rounds; and a code has at most 7 bits, so
// code * 2^e is exact in bf16 as well. The price is a step up to twice that
// of max|x| / 127; groups of 32 columns in place of whole rows win more than
// that back on activations, whose channel magnitudes differ.
//
// Both directions are bound by HBM: 16 columns per thread (two threads share
// an exponent), 16-byte accesses also where rows are not 16-byte aligned (the
// hardware takes any alignment), a workgroup per 256 / tx rows at a time.
#include "tune.h"

#include <algorithm>

namespace nq {
namespace {

constexpr int kPer = 16;   // columns per thread

template <class T>
struct __attribute__((packed)) Raw16 {
  T v[kPer];
};

// x[i] = p[i], i < cnt (0 beyond); cnt >= 16 reads whole vectors
template <int D>
__device__ __forceinline__ void load16(const typename Elem<D>::type* p, int cnt, float (&x)[kPer]) {
  typedef typename Elem<D>::type E;
  if (cnt >= kPer) {
    Raw16<E> r;
    __builtin_memcpy(&r, p, sizeof(r));
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = Elem<D>::to(r.v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = i < cnt ? Elem<D>::to(p[i]) : 0.0f;
  }
}

// Threads: tx = 2^txs columns of threads (16 columns each), 256 / tx rows.
template <int D>
__global__ __launch_bounds__(256) void act8_quantize_kernel(
    const typename Elem<D>::type* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
    int8_t* __restrict__ codes, int64_t ldc, uint8_t* __restrict__ exps, int64_t lde, int txs) {
  const int64_t unit = ((int64_t)blockIdx.x << txs) + (threadIdx.x & ((1 << txs) - 1));
  const int64_t c0 = unit * kPer;
  const int64_t left = cols - c0;
  const int cnt = left >= kPer ? kPer : left > 0 ? (int)left : 0;
  const int ty = 256 >> txs;
  constexpr uint32_t kTop = D == kF16 ? 9 + 127 : 121 + 127;
  for (int64_t r0 = (int64_t)blockIdx.y * ty; r0 < rows; r0 += (int64_t)gridDim.y * ty) {
    const int64_t row = r0 + (threadIdx.x >> txs);
    const int n = row < rows ? cnt : 0;
    float x[kPer];
    load16<D>(X + (n ? row * ldx + c0 : 0), n, x);
    // magnitudes compare as integers; a NaN or an infinity is the largest
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) mx = max(mx, __float_as_uint(x[i]) & 0x7fffffffu);
    mx = max(mx, (uint32_t)__shfl_xor((int)mx, 1));   // the group's other half
    // max|x| = 1.f 2^(E - 127) <= 127 2^e = 1.984375 2^(e + 6)
    const int ex = (int)(mx >> 23) - 6 + ((mx & 0x7fffffu) > 0x7e0000u);
    const uint32_t be = (uint32_t)min(max(ex, 1), (int)kTop);
    const bool bad = mx >= 0x7f800000u;
    const float inv = __uint_as_float((254u - be) << 23);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float c = fminf(fmaxf(rintf(x[i] * inv), -127.0f), 127.0f);
      w[i >> 2] |= ((uint32_t)(int)(bad ? 0.0f : c) & 0xffu) << (8 * (i & 3));
    }
    int8_t* dst = codes + row * ldc + c0;
    if (n == kPer) {
      const u32x4 v = {w[0], w[1], w[2], w[3]};
      __builtin_memcpy(dst, &v, 16);
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < n) dst[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
    if (n && !(unit & 1)) exps[row * lde + (unit >> 1)] = bad ? 255u : (uint8_t)be;
  }
}

template <int D>
__global__ __launch_bounds__(256) void act8_dequantize_kernel(
    const int8_t* __restrict__ codes, int64_t ldc, const uint8_t* __restrict__ exps, int64_t lde,
    int64_t rows, int64_t cols, typename Elem<D>::type* __restrict__ X, int64_t ldx, int txs) {
  typedef typename Elem<D>::type E;
  const int64_t unit = ((int64_t)blockIdx.x << txs) + (threadIdx.x & ((1 << txs) - 1));
  const int64_t c0 = unit * kPer;
  const int64_t left = cols - c0;
  if (left <= 0) return;
  const int ty = 256 >> txs;
  for (int64_t row = (int64_t)blockIdx.y * ty + (threadIdx.x >> txs); row < rows;
       row += (int64_t)gridDim.y * ty) {
    const float step = act8_step(exps[row * lde + (unit >> 1)]);
    const int8_t* src = codes + row * ldc + c0;
    E* dst = X + row * ldx + c0;
    if (left >= kPer) {
      u32x4 v;
      __builtin_memcpy(&v, src, 16);
      Raw16<E> r;
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        r.v[i] = Elem<D>::from((float)(int8_t)(v[i >> 2] >> (8 * (i & 3))) * step);
      __builtin_memcpy(dst, &r, sizeof(r));
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < (int)left) dst[i] = Elem<D>::from((float)src[i] * step);
    }
  }
}

__global__ __launch_bounds__(256) void act8_steps_kernel(const uint8_t* __restrict__ exps,
                                                         int64_t lde, int64_t rows, int64_t groups,
                                                         float* __restrict__ steps, int64_t lds) {
  const int64_t total = rows * groups;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < total;
       e += (int64_t)gridDim.x * 256) {
    const int64_t row = e / groups, g = e - row * groups;
    steps[row * lds + g] = act8_step(exps[row * lde + g]);
  }
}

// The thread layout for rows of `cols` columns: tx = 2^txs >= 2 threads along
// a row (at most 256), and a grid of about 8192 workgroups that walk the rows.
struct Shape {
  dim3 grid;
  int txs;
};
Shape shape_for(int64_t rows, int64_t cols) {
  const int64_t units = 2 * ((cols + kActGroup - 1) / kActGroup);
  int txs = 1;
  while (txs < 8 && (int64_t(1) << txs) < units) ++txs;
  const int64_t gx = (units + (int64_t(1) << txs) - 1) >> txs;
  const int64_t ty = 256 >> txs;
  const int64_t gy = std::min((rows + ty - 1) / ty, std::max<int64_t>(1, 8192 / gx));
  return {dim3((unsigned)gx, (unsigned)gy), txs};
}

}  // namespace

hipError_t launch_act8_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                                int8_t* codes, int64_t ldc, uint8_t* exps, int64_t lde,
                                hipStream_t s) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const Shape p = shape_for(rows, cols);
  switch (dtype) {
    case kF32:
      hipLaunchKernelGGL(act8_quantize_kernel<kF32>, p.grid, dim3(256), 0, s, (const float*)X,
                         rows, cols, ldx, codes, ldc, exps, lde, p.txs);
      break;
    case kBF16:
      hipLaunchKernelGGL(act8_quantize_kernel<kBF16>, p.grid, dim3(256), 0, s, (const uint16_t*)X,
                         rows, cols, ldx, codes, ldc, exps, lde, p.txs);
      break;
    default:
      hipLaunchKernelGGL(act8_quantize_kernel<kF16>, p.grid, dim3(256), 0, s, (const _Float16*)X,
                         rows, cols, ldx, codes, ldc, exps, lde, p.txs);
  }
  return hipGetLastError();
}

hipError_t launch_act8_dequantize(const Act8& q, int64_t rows, int64_t cols, void* X, int dtype,
                                  int64_t ldx, hipStream_t s) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const Shape p = shape_for(rows, cols);
  switch (dtype) {
    case kF32:
      hipLaunchKernelGGL(act8_dequantize_kernel<kF32>, p.grid, dim3(256), 0, s, q.codes, q.ldc,
                         q.exps, q.lde, rows, cols, (float*)X, ldx, p.txs);
      break;
    case kBF16:
      hipLaunchKernelGGL(act8_dequantize_kernel<kBF16>, p.grid, dim3(256), 0, s, q.codes, q.ldc,
                         q.exps, q.lde, rows, cols, (uint16_t*)X, ldx, p.txs);
      break;
    default:
      hipLaunchKernelGGL(act8_dequantize_kernel<kF16>, p.grid, dim3(256), 0, s, q.codes, q.ldc,
                         q.exps, q.lde, rows, cols, (_Float16*)X, ldx, p.txs);
  }
  return hipGetLastError();
}

hipError_t launch_act8_steps(const uint8_t* exps, int64_t lde, int64_t rows, int64_t groups,
                             float* steps, int64_t lds, hipStream_t s) {
  if (rows <= 0 || groups <= 0) return hipSuccess;
  const int64_t blocks = std::min<int64_t>((rows * groups + 255) / 256, 8192);
  hipLaunchKernelGGL(act8_steps_kernel, dim3((unsigned)blocks), dim3(256), 0, s, exps, lde, rows,
                     groups, steps, lds);
  return hipGetLastError();
}

}  // namespace nq
