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
// All products run on the bf16 or fp16 matrix cores as C = A B^T with both
// operands k-contiguous, from one kernel (mma_kernel) with an epilogue each:
//   kStat  z of 256 words x 256 tokens -> per token the largest and the sum
//          of exponentials over each half of the tile; stat_kernel joins them;
//   kGrad  z again, G = exp(z - lse) - [label] rounded to the operands' type,
//          written both ways (G and G^T) for a piece of the vocabulary;
//   kDh    dH += G W over the piece (fp32 sums, slices of the piece when
//          there are few tiles; dh_kernel adds the slices at the end);
//   kDw    dW = G^T H, the piece's rows.
// 8 T V d operations in place of the 6 T V d that keeping T V logits would
// need. W^T of the piece and H^T are laid out by transposing copies.
//
// Types: bf16 and fp16 operands are exact and sums are fp32; G is rounded to
// the operands' type once (half a unit, like the results). fp16's G is scaled
// to 2^15 at its largest, so that probabilities down to 2^-29 keep all their
// bits. fp32 operands are split into three bf16 terms x = h + m + l (exact)
// and multiplied as h h + h m + m h + h l + l h + m m, six passes over k: what
// is left out is below 2^-24 of a product.
//
// Few tokens (up to 64, the loss alone): score_kernel streams W once, 64 words
// per workgroup, its waves sharing the columns; fp32 is split in registers.
#include "tune.h"

#include <algorithm>

namespace nq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int BK = 64;            // k per stage: 128-byte rows in LDS
constexpr int kScoreMax = 64;     // tokens of score_kernel
constexpr float kNegInf = -__builtin_inff();

// one 16 x 16 x 32 product; D says how the 16-bit operands read (fp32 tensors
// come as bf16 terms)
template <int D>
__device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (D == kF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Terms of an operand of type D: one, or three for fp32.
constexpr int terms(int D) { return D == kF32 ? 3 : 1; }
constexpr int passes(int D) { return D == kF32 ? 6 : 1; }
// term of A and of B in pass s (2 bits each)
__device__ __forceinline__ int term_a(int s) { return (0x250 >> (2 * s)) & 3; }   // 0 0 1 1 2 0
__device__ __forceinline__ int term_b(int s) { return (0x844 >> (2 * s)) & 3; }   // 0 1 0 1 0 2

// x as its 16-bit terms of type D. Not finite: the first term alone.
template <int D>
__device__ __forceinline__ void split(float x, uint16_t (&t)[terms(D)]) {
  if constexpr (D == kF32) {
    t[0] = Elem<kBF16>::from(x);
    const float r = x - Elem<kBF16>::to(t[0]);
    const bool fin = (__float_as_uint(r) & 0x7fffffffu) < 0x7f800000u;
    t[1] = fin ? Elem<kBF16>::from(r) : (uint16_t)0;
    t[2] = fin ? Elem<kBF16>::from(r - Elem<kBF16>::to(t[1])) : (uint16_t)0;
  } else {
    t[0] = __builtin_bit_cast(uint16_t, Elem<D>::from(x));
  }
}
// an element's own bits as terms (16-bit types pass through)
template <int D>
__device__ __forceinline__ void split_elem(typename Elem<D>::type x, uint16_t (&t)[terms(D)]) {
  if constexpr (D == kF32)
    split<D>(x, t);
  else
    t[0] = __builtin_bit_cast(uint16_t, x);
}

// A k-contiguous operand: `rows` rows of 16-bit values, `ld` apart, whose
// terms are `plane` apart within a row.
struct Opnd {
  const uint16_t* p;
  int64_t ld, plane, rows;
};

enum Epi : int { kStat = 0, kGrad = 1, kDh = 2, kDw = 3 };
struct Mma {
  Opnd A, B;                // C (M x N) = A B^T; M = A.rows, N = B.rows
  int64_t K;                // a multiple of 64
  int64_t k_slice;          // k per slice (grid y), a multiple of 64
  float scale;
  // kStat, kGrad: rows are words v0 .., columns tokens
  int64_t v0;
  const int32_t* labels;
  float *top, *sum, *hit;   // kStat: partials [2 ceil(M / 256)][N], target logits
  const float *lse, *wn;    // kGrad: lse and normalised dloss per token
  uint16_t *G, *Gt;         // kGrad: G [token][term][gld], Gt [word][term][gtld]
  int64_t gld, gtld;
  // kDh, kDw: rows are the d columns, columns tokens or words
  float* part;              // kDh: slices of N x ldo fp32
  int64_t slice, ldo;
  int add;                  // kDh: add to what part holds
  const float* post;        // kDw: the factor taken out of wn (one float)
  void* out;                // kDw
};

// Tile order: workgroup b runs on XCD b % 8, which takes consecutive indices;
// indices run down bands of 4 tile rows, so that the 32 tiles an XCD holds at
// once form a 4 x 8 block and share operands in its L2.
__device__ __forceinline__ bool tile_of(int64_t ntm, int64_t ntn, int64_t& tm, int64_t& tn) {
  const int64_t nt = ntm * ntn, per = (nt + 7) / 8;
  const int64_t t = (int64_t)(blockIdx.x & 7) * per + (blockIdx.x >> 3);
  if ((int64_t)(blockIdx.x >> 3) >= per || t >= nt) return false;
  const int64_t band = t / (4 * ntn), idx = t - band * 4 * ntn;
  const int64_t h = min<int64_t>(4, ntm - 4 * band);
  tm = 4 * band + idx % h;
  tn = idx / h;
  return true;
}

// 512 threads, WM x WN waves of 16 MI x 16 NI. Rows of 64 k (128 bytes, eight
// 16-byte slots) go straight from memory to LDS, double buffered; row r keeps
// k-octet q in slot q ^ ((r >> 1) & 7), so that the 16 lanes that read one
// octet of 16 consecutive rows hit distinct banks.
template <int D, int EPI, int WM, int WN, int MI, int NI>
__global__ __launch_bounds__(64 * WM * WN) void mma_kernel(Mma a) {
  constexpr int BM = 16 * MI * WM, BN = 16 * NI * WN, W = WM * WN;
  constexpr int kStage = (BM + BN) * 128;
  constexpr int CA = BM / 8 / W, CB = BN / 8 / W;   // copies of 8 rows per wave and stage
  static_assert(CA * 8 * W == BM && CB * 8 * W == BN, "copies");
  __shared__ __align__(16) uint8_t lds[2 * kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, li = lane & 15;
  const int wm = wave / WN, wn = wave % WN;
  const int64_t M = a.A.rows, N = a.B.rows;
  int64_t tm, tn;
  if (!tile_of((M + BM - 1) / BM, (N + BN - 1) / BN, tm, tn)) return;
  const int64_t m0 = tm * BM, n0 = tn * BN;
  const int64_t k_lo = (int64_t)blockIdx.y * a.k_slice;
  const int nk = (int)((min(a.K, k_lo + a.k_slice) - k_lo) / BK);
  const int steps = nk * passes(D);

  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.A.p + m0 * a.A.ld), (short)0, 0x7fffffff, 0x00020000);
  const __amdgpu_buffer_rsrc_t rb = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(a.B.p + n0 * a.B.ld), (short)0, 0x7fffffff, 0x00020000);
  // lane -> row lane / 8 of a copy, slot lane % 8; rows past the end are
  // clamped (what they give is dropped)
  uint32_t oa[CA], ob[CB];
#pragma unroll
  for (int c = 0; c < CA; ++c) {
    const int r = (wave * CA + c) * 8 + (lane >> 3);
    const int q = (lane & 7) ^ ((r >> 1) & 7);
    oa[c] = (uint32_t)((min<int64_t>(r, M - 1 - m0) * a.A.ld + 8 * q) * 2);
  }
#pragma unroll
  for (int c = 0; c < CB; ++c) {
    const int r = (wave * CB + c) * 8 + (lane >> 3);
    const int q = (lane & 7) ^ ((r >> 1) & 7);
    ob[c] = (uint32_t)((min<int64_t>(r, N - 1 - n0) * a.B.ld + 8 * q) * 2);
  }
  auto copy = [&](int stage, int pass, int kt) {
    uint8_t* st = lds + stage * kStage;
    const int64_t k = k_lo + (int64_t)kt * BK;
    const int ka = (int)((k + (D == kF32 ? term_a(pass) * a.A.plane : 0)) * 2);
    const int kb = (int)((k + (D == kF32 ? term_b(pass) * a.B.plane : 0)) * 2);
#pragma unroll
    for (int c = 0; c < CA; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(st + (wave * CA + c) * 1024), 16,
                                               (int)oa[c], ka, 0, 0);
#pragma unroll
    for (int c = 0; c < CB; ++c)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rb, (lds_ptr_t)(st + BM * 128 + (wave * CB + c) * 1024), 16, (int)ob[c], kb, 0, 0);
  };
  f32x4 acc[MI][NI];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int fa = (wm * MI * 16 + li) * 128, fb = BM * 128 + (wn * NI * 16 + li) * 128;
  auto mult = [&](int stage) {
    const uint8_t* st = lds + stage * kStage;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int slot = ((4 * h + g) ^ (li >> 1)) * 16;
      u32x4 b[NI];
#pragma unroll
      for (int j = 0; j < NI; ++j) b[j] = *(const u32x4*)(st + fb + slot + j * 2048);
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const u32x4 f = *(const u32x4*)(st + fa + slot + i * 2048);
#pragma unroll
        for (int j = 0; j < NI; ++j) acc[i][j] = mma<D>(f, b[j], acc[i][j]);
      }
    }
  };
  // each wave waits for its own copies and reads, then for the other waves
  auto sync = [&]() {
    __builtin_amdgcn_s_waitcnt(0x0070);   // vmcnt(0) lgkmcnt(0)
    asm volatile("s_barrier" ::: "memory");
  };
  int pass = 0, kt = 0;
  auto advance = [&]() {
    if (++kt == nk) {
      kt = 0;
      ++pass;
    }
  };
  copy(0, 0, 0);
  advance();
  for (int s = 0; s < steps; ++s) {
    sync();   // stage s & 1 has landed; everyone is done with the other
    if (s + 1 < steps) {
      copy((s & 1) ^ 1, pass, kt);
      advance();
    }
    mult(s & 1);
  }

  // lane (g, li), element v of tile (i, j): row 16 i + 4 g + v, column 16 j + li
  const int64_t r0 = m0 + wm * MI * 16 + 4 * g, c0 = n0 + wn * NI * 16 + li;
  if constexpr (EPI == kStat) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const int32_t label = t < N ? a.labels[t] : -1;
      float top = kNegInf;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t w = r0 + 16 * i + v;
          const float z = a.scale * acc[i][j][v];
          acc[i][j][v] = z;
          if (w < M) top = fmaxf(top, z);
          if (w < M && w + a.v0 == label) a.hit[t] = z;
        }
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          sum += r0 + 16 * i + v < M ? __expf(acc[i][j][v] - top) : 0.0f;
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      if (g == 0 && t < N) {
        a.top[(tm * WM + wm) * N + t] = top;
        a.sum[(tm * WM + wm) * N + t] = sum;
      }
    }
  } else if constexpr (EPI == kGrad) {
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int64_t t = c0 + 16 * j;
      const int32_t label = t < N ? a.labels[t] : -1;
      const float lse = label >= 0 ? a.lse[t] : 0.0f, wn_t = label >= 0 ? a.wn[t] : 0.0f;
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        uint16_t q[4][terms(D)];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t w = r0 + 16 * i + v;
          const float y = a.scale * acc[i][j][v] - lse;
          float x = D == kF32 ? expf(y) : __expf(y);
          if (w + a.v0 == label) x -= 1.0f;
          x = label >= 0 && w < M ? x * wn_t : 0.0f;
          split<D>(x, q[v]);
        }
        const int64_t w = r0 + 16 * i;
#pragma unroll
        for (int p = 0; p < terms(D); ++p) {
          *(u32x2*)(a.G + t * a.gld * terms(D) + p * a.gld + w) =
              u32x2{(uint32_t)q[0][p] | (uint32_t)q[1][p] << 16,
                    (uint32_t)q[2][p] | (uint32_t)q[3][p] << 16};
#pragma unroll
          for (int v = 0; v < 4; ++v)
            a.Gt[(w + v) * a.gtld * terms(D) + p * a.gtld + t] = q[v][p];
        }
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
// 64 words and all T <= 16 NT tokens per workgroup; wave w takes the columns
// 128 w .. 128 w + 127 of every 512. Rows are 16-byte aligned and d % 8 == 0
// (VEC), or elements are loaded one by one.
template <int D>
struct Frag {
  u32x4 t[terms(D)];
};
template <int D, bool VEC>
__device__ __forceinline__ Frag<D> load_frag(const typename Elem<D>::type* row, int64_t k,
                                             int64_t d) {
  typedef typename Elem<D>::type E;
  E e[8];
  if constexpr (VEC) {
    if (k < d)
      __builtin_memcpy(e, __builtin_assume_aligned(row + k, 16), sizeof(e));
    else
      __builtin_memset(e, 0, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = k + i < d ? row[k + i] : (E)0;
  }
  Frag<D> f;
  if constexpr (D == kF32) {
    uint16_t q[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) split<kF32>(e[i], q[i]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f.t[p][i] = (uint32_t)q[2 * i][p] | (uint32_t)q[2 * i + 1][p] << 16;
  } else {
    __builtin_memcpy(&f.t[0], e, 16);
  }
  return f;
}

template <int D, int NT, bool VEC>
__global__ __launch_bounds__(256) void score_kernel(const typename Elem<D>::type* __restrict__ H,
                                                    int64_t ldh,
                                                    const typename Elem<D>::type* __restrict__ W,
                                                    int64_t ldw, int64_t T, int64_t V, int64_t d,
                                                    const int32_t* __restrict__ labels,
                                                    float scale, float* __restrict__ top,
                                                    float* __restrict__ sum,
                                                    float* __restrict__ hit) {
  __shared__ f32x4 red[4][4 * NT][64];
  __shared__ float st[2][4][16 * NT];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, li = lane & 15;
  const int64_t v0 = (int64_t)blockIdx.x * 64;
  const typename Elem<D>::type *wr[4], *hr[NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) wr[i] = W + min<int64_t>(v0 + 16 * i + li, V - 1) * ldw;
#pragma unroll
  for (int j = 0; j < NT; ++j) hr[j] = H + min<int64_t>(16 * j + li, T - 1) * ldh;
  f32x4 acc[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k0 = wave * 128; k0 < d; k0 += 512) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t k = k0 + 32 * s + 8 * g;
      Frag<D> b[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) b[j] = load_frag<D, VEC>(hr[j], k, d);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Frag<D> f = load_frag<D, VEC>(wr[i], k, d);
#pragma unroll
        for (int q = 0; q < passes(D); ++q)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[i][j] = mma<D>(f.t[D == kF32 ? term_a(q) : 0], b[j].t[D == kF32 ? term_b(q) : 0],
                               acc[i][j]);
      }
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
    const int e = wave * NT + j;
    const f32x4 z = ((red[0][e][lane] + red[1][e][lane]) + red[2][e][lane]) + red[3][e][lane];
    const int64_t t = 16 * j + li, w = v0 + 16 * wave + 4 * g;
    const int32_t label = t < T ? labels[t] : -1;
    float m = kNegInf, x[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      x[v] = scale * z[v];
      if (w + v < V) m = fmaxf(m, x[v]);
      if (w + v < V && w + v == label) hit[t] = x[v];
    }
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    float s = 0.0f;
#pragma unroll
    for (int v = 0; v < 4; ++v) s += w + v < V ? __expf(x[v] - m) : 0.0f;
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (g == 0) {
      st[0][wave][16 * j + li] = m;
      st[1][wave][16 * j + li] = s;
    }
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < 16 * NT && t < T) {
    float m = kNegInf, s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, st[0][i][t]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (v0 + 16 * i < V) s += st[1][i][t] * __expf(st[0][i][t] - m);
    top[(int64_t)blockIdx.x * T + t] = m;
    sum[(int64_t)blockIdx.x * T + t] = s;
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

// wn[t] = dloss[t] / max|dloss| times gs (0 for an ignored token, NaN for a
// label at or past V); post = max|dloss| scale / gs. One workgroup.
__global__ __launch_bounds__(1024) void weight_kernel(const float* __restrict__ dloss,
                                                      const int32_t* __restrict__ labels,
                                                      int64_t T, int64_t V, float gs, float scale,
                                                      float* __restrict__ wn,
                                                      float* __restrict__ post) {
  __shared__ float sm[1024];
  float m = 0.0f;
  for (int64_t t = threadIdx.x; t < T; t += 1024)
    if (labels[t] >= 0) m = fmaxf(m, fabsf(dloss[t]));
  sm[threadIdx.x] = m;
  __syncthreads();
  for (int o = 512; o > 0; o >>= 1) {
    if ((int)threadIdx.x < o) sm[threadIdx.x] = fmaxf(sm[threadIdx.x], sm[threadIdx.x + o]);
    __syncthreads();
  }
  m = sm[0];
  for (int64_t t = threadIdx.x; t < T; t += 1024) {
    const int32_t label = labels[t];
    const float w = m == 0.0f ? dloss[t] : dloss[t] / m * gs;   // (all zero, or NaN)
    wn[t] = label < 0 ? 0.0f : label < V ? w : __uint_as_float(0x7fc00000u);
  }
  if (threadIdx.x == 0) *post = (m == 0.0f ? 1.0f : m) * scale / gs;
}

// dH = post times the sum of nz slices (in order)
template <int D>
__global__ __launch_bounds__(256) void dh_kernel(const float* __restrict__ part, int nz,
                                                 int64_t slice, int64_t ldp, int64_t T, int64_t d,
                                                 const float* __restrict__ post,
                                                 typename Elem<D>::type* __restrict__ out,
                                                 int64_t ldo) {
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const float f = *post;
  if (c >= d) return;
  for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
    f32x4 s = *(const f32x4*)(part + t * ldp + c);
    for (int z = 1; z < nz; ++z) s += *(const f32x4*)(part + z * slice + t * ldp + c);
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (c + v < d) out[t * ldo + c + v] = Elem<D>::from(s[v] * f);
  }
}

// ---------------------------------------------------------------- layout
// out [row][term][kp] = X (rows x k), zero from k to kp
template <int D>
__global__ __launch_bounds__(256) void pack_kernel(const typename Elem<D>::type* __restrict__ X,
                                                   int64_t rows, int64_t k, int64_t ld,
                                                   uint16_t* __restrict__ out, int64_t kp) {
  typedef typename Elem<D>::type E;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (c >= kp) return;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    E e[8];
    if (c + 8 <= k) {
      __builtin_memcpy(e, X + r * ld + c, sizeof(e));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = c + i < k ? X[r * ld + c + i] : (E)0;
    }
    uint16_t q[8][terms(D)];
#pragma unroll
    for (int i = 0; i < 8; ++i) split_elem<D>(e[i], q[i]);
#pragma unroll
    for (int p = 0; p < terms(D); ++p) {
      u32x4 w;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (uint32_t)q[2 * i][p] | (uint32_t)q[2 * i + 1][p] << 16;
      *(u32x4*)(out + (r * terms(D) + p) * kp + c) = w;
    }
  }
}

// out [col][term][rp] = X^T (X rows x cols), zero from rows to rp and for rows
// whose label is negative (labels nullable). 64 x 64 tiles through LDS.
template <int D>
__global__ __launch_bounds__(256) void pack_t_kernel(const typename Elem<D>::type* __restrict__ X,
                                                     int64_t rows, int64_t cols, int64_t ld,
                                                     const int32_t* __restrict__ labels,
                                                     uint16_t* __restrict__ out, int64_t rp) {
  typedef typename Elem<D>::type E;
  __shared__ E tile[64][64 + (D == kF32 ? 1 : 2)];
  const int64_t c0 = (int64_t)blockIdx.x * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  for (int64_t r0 = (int64_t)blockIdx.y * 64; r0 < rp; r0 += (int64_t)gridDim.y * 64) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int64_t r = r0 + ty + 4 * i, c = c0 + tx;
      const bool ok = r < rows && c < cols && (!labels || labels[r] >= 0);
      tile[ty + 4 * i][tx] = ok ? X[r * ld + c] : (E)0;
    }
    __syncthreads();
    // thread -> column threadIdx / 8 (+ 32), rows 8 (threadIdx % 8) ..
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = (threadIdx.x >> 3) + 32 * h, r = 8 * (threadIdx.x & 7);
      if (c0 + c >= cols) continue;
      uint16_t q[8][terms(D)];
#pragma unroll
      for (int i = 0; i < 8; ++i) split_elem<D>(tile[r + i][c], q[i]);
#pragma unroll
      for (int p = 0; p < terms(D); ++p) {
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)q[2 * i][p] | (uint32_t)q[2 * i + 1][p] << 16;
        *(u32x4*)(out + ((c0 + c) * terms(D) + p) * rp + r0 + r) = w;
      }
    }
  }
}

// ---------------------------------------------------------------- plan
// Whether X's rows can be copied as they are (16-byte aligned, k % 64 == 0).
bool direct(const void* X, int64_t ld, int64_t k, int dtype) {
  return dtype != kF32 && k % BK == 0 && ld % 8 == 0 && (uintptr_t)X % 16 == 0;
}

struct Plan {
  int64_t dp, tp;              // d to 64, T to 256
  int64_t piece, pp, npieces;  // words of a piece, to 256; pieces
  int64_t np;                  // partials per token
  int nz;                      // slices of dH
  // byte offsets
  int64_t hp, wp, top, sum, hit, wn, post, ht, wt, G, Gt, part, bytes;
};
// Words per piece: G and W^T of a piece hold at most 2^26 values each (two
// thousand words at least), which leaves the fp32 sums of dH, read and written
// once per piece, a few percent of the piece's products.
Plan plan_for(int64_t T, int64_t V, int64_t d, int dtype, bool grad) {
  Plan p{};
  const int nt = terms(dtype);
  p.dp = round_up(d, BK);
  p.tp = round_up(T, 256);
  int64_t off = 0;
  auto take = [&](int64_t bytes) {
    const int64_t at = off;
    off += round_up(bytes, 256);
    return at;
  };
  const bool score = !grad && T <= kScoreMax;
  p.np = score ? (V + 63) / 64 : 2 * ((V + 255) / 256);
  if (!grad) {
    p.top = take(4 * p.np * T);
    p.sum = take(4 * p.np * T);
    p.hit = take(4 * T);
  }
  if (!score) {
    p.hp = take(2 * nt * T * p.dp);
    p.wp = take(2 * nt * V * p.dp);
  }
  if (grad) {
    const int64_t most = std::max<int64_t>(2048, (int64_t(1) << 26) / std::max(T, d) / 256 * 256);
    p.npieces = (V + most - 1) / most;
    p.piece = round_up((V + p.npieces - 1) / p.npieces, 256);
    p.npieces = (V + p.piece - 1) / p.piece;
    p.pp = p.piece;
    const int64_t tiles = ((d + 255) / 256) * ((T + 255) / 256);
    p.nz = (int)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, p.pp / 512, 64}));
    p.wn = take(4 * T);
    p.post = take(4);
    p.ht = take(2 * nt * d * p.tp);
    p.wt = take(2 * nt * d * p.pp);
    p.G = take(2 * nt * p.tp * p.pp);
    p.Gt = take(2 * nt * p.tp * p.pp);
    p.part = take(4 * p.nz * T * round_up(d, 4));
  }
  p.bytes = off;
  return p;
}

template <int D, int EPI>
hipError_t mma_launch(const Mma& a, int slices, hipStream_t s) {
  const int64_t tiles = ((a.A.rows + 255) / 256) * ((a.B.rows + 255) / 256);
  hipLaunchKernelGGL((mma_kernel<D, EPI, 2, 4, 8, 4>),
                     dim3((unsigned)((tiles + 7) / 8 * 8), (unsigned)slices), dim3(512), 0, s, a);
  return hipGetLastError();
}

template <int D>
hipError_t pack(const void* X, int64_t rows, int64_t k, int64_t ld, uint16_t* out, int64_t kp,
                hipStream_t s) {
  const dim3 grid((unsigned)((kp / 8 + 255) / 256), (unsigned)std::min<int64_t>(rows, 16384));
  hipLaunchKernelGGL(pack_kernel<D>, grid, dim3(256), 0, s, (const typename Elem<D>::type*)X, rows,
                     k, ld, out, kp);
  return hipGetLastError();
}
template <int D>
hipError_t pack_t(const void* X, int64_t rows, int64_t cols, int64_t ld, const int32_t* labels,
                  uint16_t* out, int64_t rp, hipStream_t s) {
  const dim3 grid((unsigned)((cols + 63) / 64), (unsigned)std::min<int64_t>(rp / 64, 65535));
  hipLaunchKernelGGL(pack_t_kernel<D>, grid, dim3(256), 0, s, (const typename Elem<D>::type*)X,
                     rows, cols, ld, labels, out, rp);
  return hipGetLastError();
}

// H or W as a k-contiguous operand: in place, or a copy in the workspace
template <int D>
hipError_t operand(const void* X, int64_t rows, int64_t ld, const Vocab& a, const Plan& p,
                   int64_t at, Opnd* o, hipStream_t s) {
  if (direct(X, ld, a.d, D)) {
    *o = Opnd{(const uint16_t*)X, ld, 0, rows};
    return hipSuccess;
  }
  uint16_t* out = (uint16_t*)((char*)a.work + at);
  *o = Opnd{out, p.dp * terms(D), p.dp, rows};
  return pack<D>(X, rows, a.d, ld, out, p.dp, s);
}

template <int D, int NT>
void score(const Vocab& a, const Plan& p, hipStream_t s) {
  typedef typename Elem<D>::type E;
  char* w = (char*)a.work;
  const bool vec = a.d % 8 == 0 && a.ldh * sizeof(E) % 16 == 0 && a.ldw * sizeof(E) % 16 == 0 &&
                   ((uintptr_t)a.H | (uintptr_t)a.W) % 16 == 0;
  const dim3 grid((unsigned)p.np);
  if (vec)
    hipLaunchKernelGGL((score_kernel<D, NT, true>), grid, dim3(256), 0, s, (const E*)a.H, a.ldh,
                       (const E*)a.W, a.ldw, a.T, a.V, a.d, a.labels, a.scale,
                       (float*)(w + p.top), (float*)(w + p.sum), (float*)(w + p.hit));
  else
    hipLaunchKernelGGL((score_kernel<D, NT, false>), grid, dim3(256), 0, s, (const E*)a.H, a.ldh,
                       (const E*)a.W, a.ldw, a.T, a.V, a.d, a.labels, a.scale,
                       (float*)(w + p.top), (float*)(w + p.sum), (float*)(w + p.hit));
}

template <int D>
hipError_t loss(const Vocab& a, hipStream_t s) {
  const Plan p = plan_for(a.T, a.V, a.d, D, false);
  char* w = (char*)a.work;
  hipError_t e;
  if (a.T <= kScoreMax) {
    if (a.T <= 16) score<D, 1>(a, p, s);
    else if (a.T <= 32) score<D, 2>(a, p, s);
    else score<D, 4>(a, p, s);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  } else {
    Mma m{};
    if ((e = operand<D>(a.W, a.V, a.ldw, a, p, p.wp, &m.A, s)) != hipSuccess) return e;
    if ((e = operand<D>(a.H, a.T, a.ldh, a, p, p.hp, &m.B, s)) != hipSuccess) return e;
    m.K = m.k_slice = p.dp;
    m.scale = a.scale;
    m.labels = a.labels;
    m.top = (float*)(w + p.top); m.sum = (float*)(w + p.sum); m.hit = (float*)(w + p.hit);
    if ((e = mma_launch<D, kStat>(m, 1, s)) != hipSuccess) return e;
  }
  hipLaunchKernelGGL(stat_kernel, dim3((unsigned)((a.T + 15) / 16)), dim3(1024), 0, s,
                     (const float*)(w + p.top), (const float*)(w + p.sum), p.np, a.T, a.V,
                     a.labels, (const float*)(w + p.hit), a.loss, a.lse);
  return hipGetLastError();
}

template <int D>
hipError_t backward(const Vocab& a, hipStream_t s) {
  typedef typename Elem<D>::type E;
  const Plan p = plan_for(a.T, a.V, a.d, D, true);
  char* w = (char*)a.work;
  float *wn = (float*)(w + p.wn), *post = (float*)(w + p.post);
  const float gs = D == kF16 ? 32768.0f : 1.0f;
  hipError_t e;
  hipLaunchKernelGGL(weight_kernel, dim3(1), dim3(1024), 0, s, a.dloss, a.labels, a.T, a.V, gs,
                     a.scale, wn, post);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  Opnd H, W;
  if ((e = operand<D>(a.W, a.V, a.ldw, a, p, p.wp, &W, s)) != hipSuccess) return e;
  if ((e = operand<D>(a.H, a.T, a.ldh, a, p, p.hp, &H, s)) != hipSuccess) return e;
  uint16_t *Ht = (uint16_t*)(w + p.ht), *Wt = (uint16_t*)(w + p.wt);
  uint16_t *G = (uint16_t*)(w + p.G), *Gt = (uint16_t*)(w + p.Gt);
  constexpr int NTm = terms(D);
  if (a.dW && (e = pack_t<D>(a.H, a.T, a.d, a.ldh, a.labels, Ht, p.tp, s)) != hipSuccess) return e;
  const int64_t ldp = round_up(a.d, 4), slice = a.T * ldp;
  int64_t kz = 0;
  for (int64_t q = 0; q < p.npieces; ++q) {
    const int64_t v0 = q * p.piece, nv = std::min(p.piece, a.V - v0);
    const int64_t nvp = round_up(nv, 256);
    Mma m{};
    m.A = Opnd{W.p + v0 * W.ld, W.ld, W.plane, nv};
    m.B = H;
    m.K = m.k_slice = p.dp;
    m.scale = a.scale;
    m.v0 = v0; m.labels = a.labels; m.lse = a.lse; m.wn = wn;
    m.G = G; m.Gt = Gt; m.gld = p.pp; m.gtld = p.tp;
    if ((e = mma_launch<D, kGrad>(m, 1, s)) != hipSuccess) return e;
    if (a.dH) {
      if ((e = pack_t<D>((const E*)a.W + v0 * a.ldw, nv, a.d, a.ldw, nullptr, Wt, p.pp, s)) != hipSuccess)
        return e;
      Mma h{};
      h.A = Opnd{Wt, p.pp * NTm, p.pp, a.d};
      h.B = Opnd{G, p.pp * NTm, p.pp, a.T};
      h.K = nvp;
      // every piece uses the same slices (the last may leave some of them
      // without a share of its own: those are not launched)
      h.k_slice = kz ? kz : round_up((nvp + p.nz - 1) / p.nz, BK);
      kz = h.k_slice;
      h.part = (float*)(w + p.part); h.slice = slice; h.ldo = ldp; h.add = q > 0;
      if ((e = mma_launch<D, kDh>(h, (int)((nvp + kz - 1) / kz), s)) != hipSuccess) return e;
    }
    if (a.dW) {
      Mma x{};
      x.A = Opnd{Ht, p.tp * NTm, p.tp, a.d};
      x.B = Opnd{Gt, p.tp * NTm, p.tp, nv};
      x.K = x.k_slice = round_up(a.T, BK);
      x.post = post;
      x.out = (E*)a.dW + v0 * a.lddw; x.ldo = a.lddw;
      if ((e = mma_launch<D, kDw>(x, 1, s)) != hipSuccess) return e;
    }
  }
  if (a.dH) {
    const int64_t first = round_up(std::min(p.piece, a.V), 256);
    const int nz = (int)((first + kz - 1) / kz);
    const dim3 grid((unsigned)((a.d + 1023) / 1024), (unsigned)std::min<int64_t>(a.T, 16384));
    hipLaunchKernelGGL(dh_kernel<D>, grid, dim3(256), 0, s, (const float*)(w + p.part), nz, slice,
                       ldp, a.T, a.d, post, (E*)a.dH, a.lddh);
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
