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
//          [token][word] (kGradTwo: with a second term in a row of its own);
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
// bf16); of fewer it has two terms (g_rows), and a divergence's of more (distill_rows). bf16's G holds (p - [label]) dloss of the
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
#include "vocab_product.h"

namespace nq {
namespace {

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
#pragma unroll 8
    for (int z = 0; z < nz; ++z)
#pragma unroll
      for (int p = 0; p < RT; ++p)
        s += *(const f32x4*)(part + z * slice + (t * RT + p) * ldp + c);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (c + v < d) out[t * ldo + c + v] = Elem<D>::from(used ? s[v] * f : 0.0f);
  }
}

// G of 2048 words of a token per workgroup from kept logits (z: of the piece's words): what kGrad
// makes of them, in N terms, and val at the words that the token lists; zero to the next multiple
// of 64 words and for tokens past T. Bound by HBM: a piece of 4096 tokens and 16384 words of bf16 72
// us, 5.6 TB/s. (z is read once more and never again: past the caches, loss and gradient of 1024
// tokens, 32000 x 2048, 508 -> 497 us.)
template <int D, int N>
__global__ __launch_bounds__(256) void kept_kernel(const float* __restrict__ z, int64_t ldz, int64_t T,
                                                   int64_t v0, int64_t nv, const int32_t* __restrict__ ids,
                                                   int64_t ldi, int K, const float* __restrict__ val,
                                                   const int32_t* __restrict__ labels,
                                                   const float* __restrict__ lse,
                                                   const float* __restrict__ wr,
                                                   const float* __restrict__ wn, uint16_t* __restrict__ G,
                                                   int64_t gld) {
  const int64_t t = blockIdx.x, w0 = (int64_t)blockIdx.y * 2048, w = w0 + 8 * threadIdx.x;
  const bool used = t < T && labels[t] >= 0;
  uint16_t* row = G + t * N * gld;
  if (w < (nv + 63) / 64 * 64) {
    uint16_t q[8][N];
    const float ref = used ? lse[t] : 0.0f, s = used ? wr[t] : 0.0f;
    f32x4 x[2] = {};
    if (used) {   // (rows hold whole groups of 128 words)
      x[0] = __builtin_nontemporal_load((const f32x4*)(z + t * ldz + w));
      x[1] = __builtin_nontemporal_load((const f32x4*)(z + t * ldz + w + 4));
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float y = x[i / 4][i % 4] - ref;
      split<D>(used && w + i < nv ? (D == kF32 ? expf(y) : __expf(y)) * s : 0.0f, q[i]);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      u32x4 o;
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = (uint32_t)q[2 * i][n] | (uint32_t)q[2 * i + 1][n] << 16;
      *(u32x4*)(row + n * gld + w) = o;
    }
  }
  if (t >= T) return;
  __syncthreads();
  for (int k = threadIdx.x; k < K; k += 256) {
    const int64_t id = ids[t * ldi + k], at = id - v0;
    if (id < 0 || at < w0 || at >= w0 + 2048 || at >= nv) continue;
    uint16_t q[N];
    split<D>(val[t * K + k] * wn[t], q);
#pragma unroll
    for (int n = 0; n < N; ++n) row[n * gld + at] = q[n];
  }
}

// G of the words that a token lists, in its N terms: val, before dloss, in place of what the
// products' epilogue left there (a word listed twice has the same val twice).
template <int D, int N>
__global__ __launch_bounds__(256) void listed_kernel(const int32_t* __restrict__ ids, int64_t ldi,
                                                     int64_t K, const float* __restrict__ val,
                                                     const float* __restrict__ wn, int64_t T,
                                                     int64_t v0, int64_t nv,
                                                     uint16_t* __restrict__ G, int64_t gld) {
  const uint32_t e = blockIdx.x * 256 + threadIdx.x;   // (< 2^27 and a workgroup)
  const uint32_t t = e / (uint32_t)K, k = e - t * (uint32_t)K;
  if (t >= T) return;
  const int64_t at = ids[t * ldi + k] - v0;
  if (ids[t * ldi + k] < 0 || at < 0 || at >= nv) return;
  uint16_t q[N];
  split<D>(val[e] * wn[t], q);
#pragma unroll
  for (int p = 0; p < N; ++p) G[((int64_t)t * N + p) * gld + at] = q[p];
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
    if ((e = score<D>(a, 0, a.V, o, s)) != hipSuccess) return e;
  } else {
    Mma m{};
    Opnd unused;
    if ((e = begin<D>(a, p, nullptr, 1, &m.B, &unused, s)) != hipSuccess) return e;
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
  const Plan p = a.share ? distill_plan(a.T, a.V, a.d, D) : plan_for(a.T, a.V, a.d, D, true);
  char* w = (char*)a.work;
  Factors* fac = (Factors*)(w + p.fac);
  uint16_t* G = (uint16_t*)(w + p.G);
  // rows of G, and so of dH's sums, as the products see them: the terms of 16-bit G
  // are rows of their own
  const int rt = a.share ? distill_rows(a.T, a.V, a.d, D) : g_rows(a.T, a.d, D);
  const int64_t RT = rt * a.T, gld = p.piece * terms(D);
  const int64_t ldp = round_up(a.d, 4), slice = RT * ldp;
  const bool score_g = few(a.T, a.d, D);
  hipError_t e;
  const Rows rows = rows_of(w, p, a.T);
  const float* wn = a.share ? a.wr : rows.wn;
  Opnd Hz, Hw, W;
  if ((e = begin<D>(a, p, a.dloss, rt, &Hz, &Hw, s)) != hipSuccess) return e;
  // every piece uses the same slices of its words for dH; the first writes them
  // all, the last, where it is another, may leave some as they are: those are not
  // launched
  for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
    const int64_t nv = std::min(p.piece, a.V - v0), nvp = round_up(nv, 256);
    if ((e = words<D>(a, p, v0, nv, &W, s)) != hipSuccess) return e;
    if (a.z) {
      const dim3 grid((unsigned)(round_up(RT, BK) / rt), (unsigned)((nv + 2047) / 2048));
      auto* fill = kept_kernel<D, terms(D)>;
      if constexpr (D != kF32) fill = rt == 1 ? fill : kept_kernel<D, kFewTerms>;
      hipLaunchKernelGGL(fill, grid, dim3(256), 0, s, a.z + v0, a.ldz, a.T, v0, nv, a.ids, a.ldi,
                         (int)a.listed, a.val, a.labels, a.lse, wn, rows.wn, G, p.piece);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    } else if (score_g) {
      const ScoreGrad o{a.lse, wn, G, p.piece, v0};
      if ((e = score<D>(a, v0, nv, o, s)) != hipSuccess) return e;
    } else {
      Mma m{};
      m.A = W; m.B = Hz;
      m.K = m.k_slice = p.dp;
      m.zs = rows.zs;
      m.z0 = a.scale;
      m.v0 = v0; m.labels = a.labels; m.lse = a.lse; m.wn = wn;
      m.G = G; m.gld = p.piece;
      m.lines = round_up(RT, BK) / rt;
      const int tile = tile_for(nv, a.T);
      if constexpr (D != kF32)
        e = rt == 1 ? mma_launch<D, kGrad>(m, tile, 1, s) : mma_launch<D, kGradTwo>(m, tile, 1, s);
      else
        e = mma_launch<D, kGrad>(m, tile, 1, s);
      if (e != hipSuccess) return e;
    }
    if (a.listed && !a.z) {
      const dim3 grid((unsigned)((a.T * a.listed + 255) / 256));
      auto* put = listed_kernel<D, terms(D)>;
      if constexpr (D != kF32) put = rt == 1 ? put : listed_kernel<D, kFewTerms>;
      hipLaunchKernelGGL(put, grid, dim3(256), 0, s, a.ids, a.ldi, a.listed, a.val, rows.wn, a.T, v0,
                         nv, G, p.piece);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    // (G is zero for words past nv to the next multiple of 64, and from
    // mma_kernel for tokens past T to the tile's end, or to the products' last 64 rows)
    Mma h{}, x{};
    int slices = 0, tile_h = 0, tile_x = 0;
    if (a.dH) {
      h.A = Opnd{W.p, W.ld, W.plane, a.d, nv};
      h.B = Opnd{G, gld, p.piece, RT, nvp};
      h.K = round_up(nv, BK);
      h.k_slice = p.kz;
      h.part = (float*)(w + p.part); h.slice = slice; h.ldo = ldp; h.add = v0 > 0;
      slices = (int)((h.K + p.kz - 1) / p.kz);
      tile_h = big_tiles(a.d, RT, p.nz) ? 256 : 128;
    }
    if (a.dW) {
      x.A = Hw;
      x.B = Opnd{G, gld, p.piece, nv, score_g ? RT : p.tp};
      x.K = x.k_slice = round_up(RT, BK);
      x.post = &fac->post_w;
      x.out = (E*)a.dW + v0 * a.lddw; x.ldo = a.lddw;
      tile_x = tile_for(a.d, nv);
    }
    if (a.dH && a.dW && pairs(tile_h, tiles_of(a.d, RT, 128) * slices, tile_x, tiles_of(a.d, nv, 128))) {
      if ((e = pair_launch<D>(h, slices, x, s)) != hipSuccess) return e;
      continue;
    }
    if (a.dH && (e = mma_launch<D, kDh>(h, tile_h, slices, s)) != hipSuccess) return e;
    if (a.dW && (e = mma_launch<D, kDw>(x, tile_x, 1, s)) != hipSuccess) return e;
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
