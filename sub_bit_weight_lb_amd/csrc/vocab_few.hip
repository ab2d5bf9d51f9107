// Gradient of a divergence (vocab_top.hip) over few tokens, in fp32 throughout:
//   G_tv = exp(z_tv - ref_t) share_t dl_t, or val dl_t at the token's listed words,
//   dH = G W,  dW = G^T H.
// With up to 64 tokens each product is bound by W, read once, or dW, written once, if
// its operands are taken as they lie: v_mfma_f32_16x16x4_f32 wants four words of a column, or
// four tokens, which are loads of whole lines from row-major W, G and H. So no copies, scales or
// terms (the 16-bit products of vocab_product.h would need W's columns gathered and G in two
// terms), and G keeps all its bits. Its rate, 256 operations per CU and cycle, is the
// bandwidth's with 32 tokens of a 16-bit W or 64 of an fp32 one; there both take their share:
//   32000 x 2048 fp32, us, dH and dW (262 MB each, 53): 16 tokens 44 and 48, 64 tokens 131 and 166
//   (the products alone 55 at the library's fp32 rate).
//   32000 x 4096 bf16, 1 token, loss and gradient: 214 us, 333 with the 16-bit products. dH 54 us and
//   dW 51, 262 MB each: 4.9 and 5.1 TB/s.
#include "tune.h"

#include <algorithm>

#include "vocab_share.h"

namespace nq {
using namespace vocab;
namespace {

// 16 bytes of a row, from any address
template <int D>
struct __attribute__((packed)) Raw {
  static constexpr int N = 16 / sizeof(typename Elem<D>::type);
  typename Elem<D>::type e[N];
};

// G of 1024 words of a token per workgroup, zero past the last word to the next multiple of 64, and
// the token's label. Each workgroup finds the token's share and its entries' val for itself: that is
// a launch less.
__global__ __launch_bounds__(256) void few_g_kernel(Taught a, const float* __restrict__ z, int64_t ldz,
                                                    const float* __restrict__ dloss, float scale,
                                                    int32_t* __restrict__ labels, float* __restrict__ G) {
  __shared__ int word[kList];
  __shared__ double q[kList];
  __shared__ float val[kList], shared;
  __shared__ int32_t tag;
  const int64_t t = blockIdx.y, v0 = (int64_t)blockIdx.x * 1024, v = v0 + 4 * threadIdx.x;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (v < ldz) x = *(const f32x4*)(z + t * ldz + v);
  const float ref = a.tail ? a.rest[t] : a.lse[t], dt = dloss[t];
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const Share s = share_of(a, t, lane, word, q);
    val[lane] = s.val[0];
    val[lane + 64] = s.val[1];
    if (lane == 0) {
      tag = s.label;
      shared = s.share;
      if (blockIdx.x == 0) labels[t] = s.label;
    }
  }
  __syncthreads();
  const int32_t label = tag;
  const float dl = label < 0 ? 0.0f : label < a.V ? dt * scale : __builtin_nanf("");
  if (v < ldz) {
    f32x4 g = {0.0f, 0.0f, 0.0f, 0.0f};
    if (label >= 0) {
      const float s = shared * dl;
#pragma unroll
      for (int i = 0; i < 4; ++i) g[i] = v + i < a.V ? expf(x[i] - ref) * s : 0.0f;
    }
    *(f32x4*)(G + t * ldz + v) = g;
  }
  __syncthreads();
  // (a word listed twice has the same val twice)
  for (int k = threadIdx.x; k < a.K; k += 256) {
    const int64_t id = word[k];
    if (id >= v0 && id < v0 + 1024 && id < a.V) G[t * ldz + id] = val[k] * dl;
  }
}

// dH's sums over a slice of the words (grid y), of 16 columns of 16 bytes. The four waves take
// blocks of 16 words in turn; a lane loads 16 bytes of four rows: row g's words 4 g .. are k of
// four steps, column li's elements are rows of as many tiles. NT: 16 tokens each.
template <int D, int NT>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(NT * Raw<D>::N <= 8 ? 4 : 3))) void few_dh_kernel(const typename Elem<D>::type* __restrict__ W,
                                                     int64_t ldw, int64_t V, int64_t d,
                                                     const float* __restrict__ G, int64_t ldg, int T,
                                                     int64_t blocks, float* __restrict__ part,
                                                     int64_t slice, int64_t ldp) {
  constexpr int C = Raw<D>::N;
  __shared__ f32x4 red[3][C * NT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t c0 = (int64_t)blockIdx.x * 16 * C;
  // (columns past the end: the last ones again, whose results are not written)
  const typename Elem<D>::type* Wc = W + lmin(c0 + C * li, d - C);
  const int64_t all = (V + 15) / 16, b1 = lmin(all, (int64_t)(blockIdx.y + 1) * blocks);
  const float* Gt[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) Gt[j] = G + (int64_t)min(16 * j + li, T - 1) * ldg + 4 * g;
  f32x4 acc[C][NT];
#pragma unroll
  for (int m = 0; m < C; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Raw<D> w[2][4];
  f32x4 q[2][NT];
  // (words past the last: the last one's row again, and G is zero there)
  auto load = [&](int64_t b, Raw<D> (&r)[4], f32x4 (&x)[NT]) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      __builtin_memcpy(&r[s], Wc + lmin(16 * b + 4 * g + s, V - 1) * ldw, 16);
#pragma unroll
    for (int j = 0; j < NT; ++j) x[j] = *(const f32x4*)(Gt[j] + 16 * b);
  };
  auto use = [&](const Raw<D> (&r)[4], const f32x4 (&x)[NT]) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int m = 0; m < C; ++m)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(Elem<D>::to(r[s].e[m]), x[j][s], acc[m][j], 0, 0, 0);
  };
  int64_t b = (int64_t)blockIdx.y * blocks + wave;
  if (b < b1) load(b, w[0], q[0]);
  for (; b < b1; b += 8) {   // the next block's loads before this one's products
    if (b + 4 < b1) load(b + 4, w[1], q[1]);
    __builtin_amdgcn_sched_barrier(0);
    use(w[0], q[0]);
    if (b + 8 < b1) load(b + 8, w[0], q[0]);
    __builtin_amdgcn_sched_barrier(0);
    if (b + 4 < b1) use(w[1], q[1]);
  }
  if (wave) {
#pragma unroll
    for (int m = 0; m < C; ++m)
#pragma unroll
      for (int j = 0; j < NT; ++j) red[wave - 1][m * NT + j][lane] = acc[m][j];
  }
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int m = 0; m < C; ++m)
#pragma unroll
      for (int n = 0; n < 3; ++n) acc[m][j] += red[n][m * NT + j][lane];
    const int t = 16 * j + li;
    if (t >= T) continue;
    float* out = part + (int64_t)blockIdx.y * slice + (int64_t)t * ldp;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t want = c0 + C * (4 * g + v), c = lmin(want, d - C);
#pragma unroll
      for (int m = 0; m < C; ++m)
        if (c + m >= want) out[c + m] = acc[m][j][v];   // (the others are an earlier lane's)
    }
  }
}

// dH = the sum of the slices, in order; zero for an ignored token
template <int D>
__global__ __launch_bounds__(256) void few_join_kernel(const float* __restrict__ part, int n, int64_t slice,
                                                       int64_t ldp, int64_t d,
                                                       const int32_t* __restrict__ labels,
                                                       typename Elem<D>::type* __restrict__ out, int64_t ldo) {
  const int64_t t = blockIdx.y, c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= d) return;
  float s = 0.0f;
#pragma unroll 8
  for (int i = 0; i < n; ++i) s += part[i * slice + t * ldp + c];
  out[t * ldo + c] = Elem<D>::from(labels[t] >= 0 ? s : 0.0f);
}

// dW of `blocks` times 64 words (grid y) and 64 columns per wave, whose part of H stays in
// registers: NS steps of four tokens. Of 64 words a lane loads G of four neighbours: one for each
// of four products, which have every fourth word. It gets 4 columns of a word per tile; the columns
// of a 16-bit row lie so in the tiles that two of them make 16 bytes.
template <int D, int NS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(NS == 16 ? 2 : NS == 8 ? 3 : 4))) void few_dw_kernel(
    const typename Elem<D>::type* __restrict__ H, int64_t ldh, int T, int64_t V, int64_t d,
    const int32_t* __restrict__ labels, const float* __restrict__ G, int64_t ldg, int64_t blocks,
    typename Elem<D>::type* __restrict__ out, int64_t ldo) {
  typedef typename Elem<D>::type E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t c0 = ((int64_t)blockIdx.x * 4 + wave) * 64;
  if (c0 >= d) return;
  float h[NS][4];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    const int t = 4 * s + g;
    const bool used = t < T && labels[t] >= 0;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int64_t c = D == kF32 ? c0 + 16 * m + li
                                  : c0 + 32 * (m >> 1) + 8 * (li >> 2) + 4 * (m & 1) + (li & 3);
      h[s][m] = used && c < d ? Elem<D>::to(H[t * ldh + c]) : 0.0f;   // (tokens past T: G is another's)
    }
  }
  // G of the next 64 words comes before the stores of these: a wait for it is none for them
  // (a wait for loads is one for all that went out before; so no branch either among the stores
  // of 64 whole words and columns). With NS = 16 there are no registers for it.
  constexpr bool AHEAD = NS < 16;
  f32x4 x[AHEAD ? 2 : 1][NS];
  auto load = [&](int64_t b, f32x4 (&y)[NS]) {
#pragma unroll
    for (int s = 0; s < NS; ++s) y[s] = *(const f32x4*)(G + (int64_t)min(4 * s + g, T - 1) * ldg + 64 * b + 4 * li);
  };
  struct __attribute__((packed)) Any { u32x4 v; };   // 16 bytes at any address
  auto block = [&](int64_t b, const f32x4 (&y)[NS], auto whole) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f32x4 acc[4];
#pragma unroll
      for (int m = 0; m < 4; ++m) acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int m = 0; m < 4; ++m)
          acc[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(h[s][m], y[s][q], acc[m], 0, 0, 0);
      const int64_t word = 64 * b + 4 * li + q;
      constexpr int P = 16 / sizeof(E), N = 16 / P;   // elements of 16 bytes, stores
      E* p = out + word * ldo + c0 + P * g;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        E e[P];
#pragma unroll
        for (int i = 0; i < P; ++i) e[i] = Elem<D>::from(acc[n * (P / 4) + i / 4][i % 4]);
        if constexpr (decltype(whole)::value) {
          Any w;
          __builtin_memcpy(&w, e, 16);
          *(Any*)(p + 4 * P * n) = w;
        } else {
#pragma unroll
          for (int i = 0; i < P; ++i)
            if (word < V && c0 + 4 * P * n + P * g + i < d) p[4 * P * n + i] = e[i];
        }
      }
    }
  };
  const int64_t b0 = (int64_t)blockIdx.y * blocks, b1 = lmin((V + 63) / 64, b0 + blocks);
  const int64_t bw = c0 + 64 <= d ? lmin(b1, V / 64) : b0;   // whole ones
  int64_t b = b0;
  if constexpr (AHEAD) {
    if (b < bw) load(b, x[0]);
    for (; b + 1 < bw; b += 2) {
      load(b + 1, x[1]);
      block(b, x[0], std::true_type{});
      load(lmin(b + 2, b1 - 1), x[0]);
      block(b + 1, x[1], std::true_type{});
    }
    if (b < bw) block(b, x[0], std::true_type{});
    b = lmax(b0, bw);
  } else {
    for (; b < bw; ++b) {
      load(b, x[0]);
      block(b, x[0], std::true_type{});
    }
  }
  for (; b < b1; ++b) {
    load(b, x[0]);
    block(b, x[0], std::false_type{});
  }
}

template <int D>
hipError_t gradient(const Few& a, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const Vocab& v = a.a.v;
  const FewPlan p = few_plan(v.T, v.V, v.d, D);
  const int T = (int)v.T;
  hipError_t e;
  const Taught of{a.a.ids, a.a.logq, a.a.lse, a.a.rest, a.a.hit, a.a.ldi, a.a.ldq, v.V, (int)a.a.K, a.a.tail};
  hipLaunchKernelGGL(few_g_kernel, dim3((unsigned)((p.ldz + 1023) / 1024), (unsigned)T), dim3(256), 0, s, of, a.z,
                     p.ldz, v.dloss, v.scale, a.labels, a.G);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  if (v.dH) {
    const int64_t ldp = round_up(v.d, 4), slice = v.T * ldp;
    const dim3 grid((unsigned)p.columns, (unsigned)p.slices);
    auto go = [&](auto tiles) {
      constexpr int NT = decltype(tiles)::value;
      hipLaunchKernelGGL((few_dh_kernel<D, NT>), grid, dim3(256), 0, s, (const E*)v.W, v.ldw, v.V, v.d, a.G,
                         p.ldz, T, p.blocks, a.part, slice, ldp);
    };
    if (T <= 16) go(std::integral_constant<int, 1>{});
    else if (D != kF32 || T <= 32) go(std::integral_constant<int, 2>{});
    else if constexpr (D == kF32) go(std::integral_constant<int, 4>{});
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(few_join_kernel<D>, dim3((unsigned)((v.d + 255) / 256), (unsigned)T), dim3(256), 0, s,
                       a.part, (int)p.slices, slice, ldp, v.d, a.labels, (E*)v.dH, v.lddh);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  if (v.dW) {
    const int64_t x = (v.d + 255) / 256;
    // (a round of workgroups: each has its part of H to fetch)
    const int64_t all = (v.V + 63) / 64, blocks = (all * x + 1023) / 1024;
    const dim3 grid((unsigned)x, (unsigned)((all + blocks - 1) / blocks));
    auto go = [&](auto steps) {
      constexpr int NS = decltype(steps)::value;
      hipLaunchKernelGGL((few_dw_kernel<D, NS>), grid, dim3(256), 0, s, (const E*)v.H, v.ldh, T, v.V, v.d, a.labels,
                         a.G, p.ldz, blocks, (E*)v.dW, v.lddw);
    };
    if (T <= 4) go(std::integral_constant<int, 1>{});
    else if (T <= 8) go(std::integral_constant<int, 2>{});
    else if (T <= 16) go(std::integral_constant<int, 4>{});
    else if (D != kF32 || T <= 32) go(std::integral_constant<int, 8>{});
    else if constexpr (D == kF32) go(std::integral_constant<int, 16>{});
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_few_gradient(const Few& a, hipStream_t s) {
  if (a.a.v.dtype == kF32) return gradient<kF32>(a, s);
  return a.a.v.dtype == kBF16 ? gradient<kBF16>(a, s) : gradient<kF16>(a, s);
}

}  // namespace nq
