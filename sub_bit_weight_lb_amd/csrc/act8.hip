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
// Both directions are bound by HBM: whole lines per wave also where rows are not
// 16-byte aligned (the hardware takes any alignment), a workgroup of 256 / tx
// rows at a time. Values that
// do not fit the last-level cache are read and written past it (nontemporal).
// 65536 x 4096 (3.03 bytes per bf16 value, 5.03 per fp32 value), in us: to codes
// 136 (6.0 TB/s) and 216, from codes 130 (6.2 TB/s) and 229; without the mark
// 141, 239, 142 and 258, but at 64 MB, where the values stay in the last-level
// cache, a chain of producer, both directions and consumer takes 55 without it
// and 61 with it.
#include "tune.h"

#include <algorithm>
#include <type_traits>

namespace nq {
namespace {

template <class T, int N>
struct __attribute__((packed)) Raw {
  T v[N];
};
// columns per thread, of values in and of values out
constexpr int cols_in(int D) { return D == kF32 ? 4 : 16; }
constexpr int cols_out(int D) { return D == kF32 ? 4 : 8; }

constexpr int64_t kFar = int64_t(256) << 20;   // bytes of the last-level cache

// accesses at any address; FAR: past the caches (a template, as the compiler
// merges the two sides of a branch and drops the mark)
typedef u32x4 __attribute__((aligned(1))) wide_t;
typedef uint32_t __attribute__((aligned(1))) word_t;
template <bool FAR>
__device__ __forceinline__ u32x4 stream_in(const void* p) {
  return FAR ? __builtin_nontemporal_load((const wide_t*)p) : *(const wide_t*)p;
}
template <bool FAR, class R>
__device__ __forceinline__ void stream_out(void* p, const R& r) {
  typedef std::conditional_t<sizeof(R) == 16, wide_t, word_t> W;
  static_assert(sizeof(R) == sizeof(W), "one store");
  W w;
  __builtin_memcpy(&w, &r, sizeof(w));
  if constexpr (FAR)
    __builtin_nontemporal_store(w, (W*)p);
  else
    *(W*)p = w;
}

// Threads: tx = 2^txs columns of threads, 256 / tx rows.
template <int D, bool FAR>
__global__ __launch_bounds__(256) void act8_quantize_kernel(
    const typename Elem<D>::type* __restrict__ X, int64_t rows, int64_t cols, int64_t ldx,
    int8_t* __restrict__ codes, int64_t ldc, uint8_t* __restrict__ exps, int64_t lde, int txs) {
  typedef typename Elem<D>::type E;
  constexpr int N = cols_in(D);
  const int64_t c0 = (((int64_t)blockIdx.x << txs) + (threadIdx.x & ((1 << txs) - 1))) * N;
  const int64_t left = cols - c0;
  const int ty = 256 >> txs;
  constexpr uint32_t kTop = D == kF16 ? 9 + 127 : 121 + 127;
  for (int64_t r0 = (int64_t)blockIdx.y * ty; r0 < rows; r0 += (int64_t)gridDim.y * ty) {
    const int64_t row = r0 + (threadIdx.x >> txs);
    const int64_t n = row < rows ? left : 0;   // (every thread joins the shuffles)
    const E* src = X + row * ldx + c0;
    Raw<E, N> r;
    if (n >= N) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(r) / 16; ++i) {
        const u32x4 v = stream_in<FAR>((const char*)src + 16 * i);
        __builtin_memcpy((char*)&r + 16 * i, &v, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) r.v[i] = i < n ? src[i] : (E)0;
    }
    // magnitudes compare as integers; a NaN or an infinity is the largest
    float x[N];
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      x[i] = Elem<D>::to(r.v[i]);
      mx = max(mx, __float_as_uint(x[i]) & 0x7fffffffu);
    }
#pragma unroll
    for (int o = 1; o < kActGroup / N; o *= 2) mx = max(mx, (uint32_t)__shfl_xor((int)mx, o));
    // max|x| = 1.f 2^(E - 127) <= 127 2^e = 1.984375 2^(e + 6)
    const int ex = (int)(mx >> 23) - 6 + ((mx & 0x7fffffu) > 0x7e0000u);
    const uint32_t be = (uint32_t)min(max(ex, 1), (int)kTop);
    const bool bad = mx >= 0x7f800000u;
    const float inv = __uint_as_float((254u - be) << 23);
    Raw<int8_t, N> q;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float c = fminf(fmaxf(rintf(x[i] * inv), -127.0f), 127.0f);
      q.v[i] = (int8_t)(int)(bad ? 0.0f : c);
    }
    int8_t* dst = codes + row * ldc + c0;
    if (n >= N) {
      stream_out<FAR>(dst, q);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < n) dst[i] = q.v[i];
    }
    if (n > 0 && c0 % kActGroup == 0)
      exps[row * lde + c0 / kActGroup] = bad ? 255u : (uint8_t)be;
  }
}

// value = code times step; two rows in flight
template <int D, bool FAR>
__global__ __launch_bounds__(256) void act8_dequantize_kernel(
    const int8_t* __restrict__ codes, int64_t ldc, const uint8_t* __restrict__ exps, int64_t lde,
    int64_t rows, int64_t cols, typename Elem<D>::type* __restrict__ X, int64_t ldx, int txs) {
  typedef typename Elem<D>::type E;
  constexpr int N = cols_out(D);
  const int64_t c0 = (((int64_t)blockIdx.x << txs) + (threadIdx.x & ((1 << txs) - 1))) * N;
  const int64_t left = cols - c0;
  if (left <= 0) return;
  const int64_t hop = (int64_t)gridDim.y * (256 >> txs);
  for (int64_t row = (int64_t)blockIdx.y * (256 >> txs) + (threadIdx.x >> txs); row < rows;
       row += 2 * hop) {
    const bool two = row + hop < rows;
    const int64_t at[2] = {row, two ? row + hop : row};
    float step[2];
    Raw<int8_t, N> v[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      step[u] = act8_step(exps[at[u] * lde + c0 / kActGroup]);
      const int8_t* src = codes + at[u] * ldc + c0;
      if (left >= N) {
        __builtin_memcpy(&v[u], src, N);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) v[u].v[i] = i < left ? src[i] : (int8_t)0;
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (u && !two) break;
      E* dst = X + at[u] * ldx + c0;
      Raw<E, N> r;
#pragma unroll
      for (int i = 0; i < N; ++i) r.v[i] = Elem<D>::from((float)v[u].v[i] * step[u]);
      if (left >= N) {
        stream_out<FAR>(dst, r);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (i < left) dst[i] = r.v[i];
      }
    }
  }
}

// four groups per thread
__global__ __launch_bounds__(256) void act8_steps_kernel(const uint8_t* __restrict__ exps,
                                                         int64_t lde, int64_t rows, int64_t groups,
                                                         float* __restrict__ steps, int64_t lds,
                                                         int txs) {
  const int64_t g = (((int64_t)blockIdx.x << txs) + (threadIdx.x & ((1 << txs) - 1))) * 4;
  const int64_t left = groups - g;
  if (left <= 0) return;
  const int64_t hop = (int64_t)gridDim.y * (256 >> txs);
  for (int64_t row = (int64_t)blockIdx.y * (256 >> txs) + (threadIdx.x >> txs); row < rows;
       row += hop) {
    const uint8_t* src = exps + row * lde + g;
    float* dst = steps + row * lds + g;
    if (left >= 4) {
      Raw<uint8_t, 4> e;
      __builtin_memcpy(&e, src, 4);
      Raw<float, 4> r;
#pragma unroll
      for (int i = 0; i < 4; ++i) r.v[i] = act8_step(e.v[i]);
      __builtin_memcpy(dst, &r, 16);
    } else {
      for (int i = 0; i < left; ++i) dst[i] = act8_step(src[i]);
    }
  }
}

// The thread layout for rows of `units` threads' work: tx = 2^txs threads along
// a row, 256 at most and 2^least at least, and a grid of about 65536 workgroups
// that walk the rows (8192 measured a fifth slower).
struct Shape {
  dim3 grid;
  int txs;
};
Shape shape_for(int64_t rows, int64_t units, int least) {
  int txs = least;
  while (txs < 8 && (int64_t(1) << txs) < units) ++txs;
  const int64_t gx = (units + (int64_t(1) << txs) - 1) >> txs;
  const int64_t ty = 256 >> txs;
  const int64_t gy = std::min((rows + ty - 1) / ty, std::max<int64_t>(1, 65535 / gx));
  return {dim3((unsigned)gx, (unsigned)gy), txs};
}

bool far(int64_t rows, int64_t cols, int dtype) {
  return rows * cols * (dtype == kF32 ? 4 : 2) > kFar;
}

template <int D, bool FAR>
void quantize(const void* X, int64_t rows, int64_t cols, int64_t ldx, int8_t* codes, int64_t ldc,
              uint8_t* exps, int64_t lde, hipStream_t s) {
  // (the threads of a group lie side by side in one row: two, or eight)
  const Shape p = shape_for(rows, (cols + cols_in(D) - 1) / cols_in(D), D == kF32 ? 3 : 1);
  hipLaunchKernelGGL((act8_quantize_kernel<D, FAR>), p.grid, dim3(256), 0, s,
                     (const typename Elem<D>::type*)X, rows, cols, ldx, codes, ldc, exps, lde,
                     p.txs);
}

template <int D, bool FAR>
void dequantize(const Act8& q, int64_t rows, int64_t cols, void* X, int64_t ldx, hipStream_t s) {
  const Shape p = shape_for(rows, (cols + cols_out(D) - 1) / cols_out(D), 0);
  hipLaunchKernelGGL((act8_dequantize_kernel<D, FAR>), p.grid, dim3(256), 0, s, q.codes, q.ldc,
                     q.exps, q.lde, rows, cols, (typename Elem<D>::type*)X, ldx, p.txs);
}

}  // namespace

hipError_t launch_act8_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                                int8_t* codes, int64_t ldc, uint8_t* exps, int64_t lde,
                                hipStream_t s) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const bool f = far(rows, cols, dtype);
  auto* go = dtype == kF32    ? f ? quantize<kF32, true> : quantize<kF32, false>
             : dtype == kBF16 ? f ? quantize<kBF16, true> : quantize<kBF16, false>
                              : f ? quantize<kF16, true> : quantize<kF16, false>;
  go(X, rows, cols, ldx, codes, ldc, exps, lde, s);
  return hipGetLastError();
}

hipError_t launch_act8_dequantize(const Act8& q, int64_t rows, int64_t cols, void* X, int dtype,
                                  int64_t ldx, hipStream_t s) {
  if (rows <= 0 || cols <= 0) return hipSuccess;
  const bool f = far(rows, cols, dtype);
  auto* go = dtype == kF32    ? f ? dequantize<kF32, true> : dequantize<kF32, false>
             : dtype == kBF16 ? f ? dequantize<kBF16, true> : dequantize<kBF16, false>
                              : f ? dequantize<kF16, true> : dequantize<kF16, false>;
  go(q, rows, cols, X, ldx, s);
  return hipGetLastError();
}

hipError_t launch_act8_steps(const uint8_t* exps, int64_t lde, int64_t rows, int64_t groups,
                             float* steps, int64_t lds, hipStream_t s) {
  if (rows <= 0 || groups <= 0) return hipSuccess;
  const Shape p = shape_for(rows, (groups + 3) / 4, 0);
  hipLaunchKernelGGL(act8_steps_kernel, p.grid, dim3(256), 0, s, exps, lde, rows, groups, steps,
                     lds, p.txs);
  return hipGetLastError();
}

}  // namespace nq
