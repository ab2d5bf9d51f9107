// What is asked of single logits of a large vocabulary (z = scale H W^T, the products of
// vocab_product.h; of many tokens they are kept only where a gradient will read them):
//
// Log probabilities, to score a model and to write down what it holds likely:
//   lse_t = log sum_v exp z_tv,  log p = z - lse of the given words,
//   entropy_t = -sum_v p log p = log S - U / S,  S = sum exp(z - m), U = sum
//   exp(z - m) (z - m), m the largest z (both terms are 0 or more; S - 1 is summed by itself),
//   the k largest z, the lower word first among equals.
// Divergence from a teacher's K words with log probabilities logq, KL(q || p):
//   q = exp logq, r = max(0, 1 - sum q), rest = log sum exp z over the words that are
//   not listed, loss = sum q (logq - z + lse) + r (log r - rest + lse)
//   (tail), or q = softmax(logq) over the token's entries, r = 0, rest = lse;
//   its derivative by z_v, with Q = sum q + r: Q p_v - sum q of v's entries where v is
//   listed, exp(z_v - rest) (Q exp(rest - lse) - r) where it is not (with r = 0 and rest
//   = lse: Q p_v). Here rest is a sum of its own: what is left of exp lse without
//   the listed words' part would be rounding where they hold all but 2^-20 of it.
//
// The product's epilogue kPick (up to 32 tokens, fp32 64: score_kernel) leaves, per token and
// group of words, the largest z and the sums S and U about it (for a divergence with a tail
// without the listed words), and the z of
//   listed words: marks_kernel has told where they are;
//   parts of groups that may hold one of the best words: the vocabulary is taken in steps,
//   and from the second on only parts with a z above the k-th best so far are written.
// A workgroup per token (top_kernel, distill_kernel) then joins the groups.
#include "vocab_product.h"
#include "vocab_share.h"

namespace nq {
namespace {

const float kNaN = __builtin_nanf("");

// ---------------------------------------------------------------- joins of sums
// About the largest z of all, m: r = sum e - 1 and u = sum e (z - m), e = exp(z - m).
// r is a sum of its own, so that log(1 + r) keeps the digits of a row that is all but certain.
struct Sums {
  float m, r, u;
};
constexpr Sums kNothing{kNegInf, -1.0f, 0.0f};   // (a sum of 0)
__device__ __forceinline__ void join(Sums& a, Sums b) {
  if (b.r == -1.0f) return;
  if (a.r == -1.0f) {
    a = b;
    return;
  }
  const float n = fmaxf(a.m, b.m);
  const float x = a.m - n, y = b.m - n;
  const float p = __expf(x), q = __expf(y), as = 1.0f + a.r, bs = 1.0f + b.r;
  a.r = x == 0.0f ? a.r + q * bs : b.r + p * as;
  a.u = p * (a.u + x * as) + q * (b.u + y * bs);
  a.m = n;
}
// Joins a lane's sums with those of lane ^ o: both join the lower one's with the upper one's.
__device__ __forceinline__ void pair(Sums& a, int o) {
  const Sums b{__shfl_xor(a.m, o), __shfl_xor(a.r, o), __shfl_xor(a.u, o)};
  const bool up = threadIdx.x & o;
  Sums l = up ? b : a;
  join(l, up ? a : b);
  a = l;
}
// Over the workgroup's NT threads, in a fixed order; all of them get the result. sm: three
// floats per wave.
template <int NT>
__device__ __forceinline__ Sums join_all(Sums a, float* sm) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) pair(a, o);
  constexpr int NW = NT / 64;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  __syncthreads();
  if (lane == 0) {
    sm[3 * wave] = a.m;
    sm[3 * wave + 1] = a.r;
    sm[3 * wave + 2] = a.u;
  }
  __syncthreads();
  const int w = lane & (NW - 1);
  a = Sums{sm[3 * w], sm[3 * w + 1], sm[3 * w + 2]};
#pragma unroll
  for (int o = NW / 2; o > 0; o >>= 1) pair(a, o);
  return a;
}

// ---------------------------------------------------------------- listed words
// slot, marks (Kept) and the place of each of a token's K entries in its row of zl (255: a word
// below 0 or past the last): the distinct words of its list, by groups in the order of their
// first entries. A workgroup per token, a thread per entry, which all look through the whole
// list in LDS (K^2 / 4 reads of 16 bytes: 5 us for 4096 tokens of one word, 11 for 64; 777 tokens
// of 100 words 6). So that the products' epilogue reads a byte per token and group, and a bit
// map where it says so: 12 us of 164 with 100 words of each token (777 tokens, 50021 x 1000 fp16).
struct Marks {
  uint8_t* slot;
  int64_t lds;
  Mark* marks;               // [token][K]
  uint8_t* places;           // [token][K]
};
__global__ __launch_bounds__(kList) void marks_kernel(const int32_t* __restrict__ ids, int64_t ldi,
                                                      int K, int64_t V, int group, Marks o) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  __shared__ __align__(16) int grp[kList], sizes[kList];
  __shared__ u32x4 words[kList];
  __shared__ uint32_t base[kList];
  const int64_t t = blockIdx.x;
  const int k = threadIdx.x;
  const int32_t id = k < K ? ids[t * ldi + k] : -1;
  const bool real = id >= 0 && id < V;
  const int mine = real ? id / group : -1, in = real ? id - mine * group : 0;
  uint8_t* row = o.slot + t * o.lds;
  for (int64_t i = 16 * k; i < o.lds; i += 16 * kList) *(u32x4*)(row + i) = u32x4{~0u, ~0u, ~0u, ~0u};
  grp[k] = mine;
  words[k] = u32x4{0, 0, 0, 0};
  __syncthreads();
  int owner = k;   // the first entry of the same group
#pragma unroll 4
  for (int j = 0; j < K; j += 4) {
    const i32x4 g = *(const i32x4*)(grp + j);
#pragma unroll
    for (int u = 3; u >= 0; --u) owner = g[u] == mine && j + u < owner ? j + u : owner;
  }
  if (real) atomicOr((uint32_t*)&words[owner] + (in >> 5), 1u << (in & 31));
  __syncthreads();
  const u32x4 own = words[k];
  sizes[k] = __popc(own[0]) + __popc(own[1]) + __popc(own[2]) + __popc(own[3]);
  __syncthreads();
  uint32_t place = 0;
#pragma unroll 4
  for (int j = 0; j < K; j += 4) {
    const i32x4 n = *(const i32x4*)(sizes + j);
#pragma unroll
    for (int u = 0; u < 4; ++u) place += j + u < k ? (uint32_t)n[u] : 0u;
  }
  base[k] = place;
  if (real && owner == k) {
    row[mine] = (uint8_t)k;
    o.marks[t * K + k].words = own;
    o.marks[t * K + k].place = place;
  }
  __syncthreads();
  if (k < K) o.places[t * K + k] = real ? (uint8_t)place_of(words[owner], base[owner], in) : (uint8_t)255;
}

// ---------------------------------------------------------------- log probabilities
struct Top {
  Kept kept;
  int group;                 // words of a group
  int64_t V, v0, p0, p1;     // the step's first word, its parts
  int k, have;               // best words; whether `best` holds those of earlier steps
  uint64_t* best;            // [token][k], best first
  float* thr;                // [token]: the k-th best z
  int last;                  // the last step: what follows is written
  const int32_t* tokens;     // [token][ldt]
  const uint8_t* places;     // [token][given], nullable: where their z are in zl (else in z)
  int64_t ldt;
  int given;
  float *logprobs, *entropy, *lse;
  int32_t* top_ids;
  float* top_logprobs;
};
// Order of the words: larger z first, then the lower word. 0: less than any.
__device__ __forceinline__ uint32_t order_of(float z) {
  const uint32_t b = __float_as_uint(z + 0.0f);   // (no zero below zero)
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float z, uint32_t word) {
  return (uint64_t)order_of(z) << 32 | (uint32_t)~word;
}

// how many lanes of `who` come before this one
__device__ __forceinline__ int rank_in(uint64_t who) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
}
// The largest c of the form that bits 31 .. low can write with k of the N values of each lane at
// or above c (0: with none); *n: how many those are. Stops where they are k.
template <int N>
__device__ __forceinline__ uint32_t reached(const uint32_t (&x)[N], int k, int low, int* n) {
  uint32_t c = 0;
  *n = 64 * N;
  for (int b = 31; b >= low; --b) {
    const uint32_t d = c | 1u << b;
    int above = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) above += __popcll(__ballot(x[i] >= d));
    if (above >= k) {
      c = d;
      *n = above;
      if (above == k) break;
    }
  }
  return c;
}

// The best words of a step join those of earlier ones; in the last step the token's outputs
// follow. A workgroup of NT threads per token.
//   Bound: 256 shares of the step's parts have a largest z each; one that k of these reach
//   is one that k words reach. Only parts that reach it are looked at: k, and few more
//   where a share has two.
//   Their words above the bound go to a list in LDS, in any order (an atomic counter gives
//   the places; keys are distinct, so that the order does not show), which one wave cuts to
//   its k best, found bit by bit. If the list is too short for them (many words of one
//   value), as many parts at a time as it has room for, and after each cut, which leaves only
//   words above the k-th best key, twice as many. (One token of 131072 words, 20 best, all z equal: with
//   the k-th best z as the bound, and no more parts than have room, 2640 us; a random row 58.)
// Bound by a token's chain of dependent loads and barriers: 9 us for one token of 32000 words, 20
// best; 4096 tokens of 131072 words, 64 best, five steps of 35 to 47 us each (0.23 ms of 3.3).
template <int NT>
__global__ __launch_bounds__(NT) void top_kernel(Top a) {
  static_assert(NT % 256 == 0, "256 shares");
  constexpr int kCap = 512, NW = NT / 64, kEach = kCap / 64;
  __shared__ uint64_t list[kCap];
  __shared__ uint32_t most[NT];
  __shared__ int todo[4 * NT];
  __shared__ int count, left;
  __shared__ uint32_t lim, low;
  __shared__ float sm[3 * NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t = blockIdx.x;
  const f32x4* stat = a.kept.stat + t * a.kept.groups;
  const int k = a.k;
  int n = 0;   // words in the list
  // what the outputs need, on its way while the best words are found
  f32x4 mine = {kNegInf, -1.0f, 0.0f, 0.0f};
  if (a.last && tid < a.kept.groups) mine = stat[tid];
  int32_t id = -1;
  float zid = kNaN;
  if (a.last && tid < a.given) {
    id = a.tokens[t * a.ldt + tid];
    if (id >= 0 && id < a.V)
      zid = a.places ? a.kept.zl[t * a.given + a.places[t * a.given + tid]] : a.kept.z[t * a.kept.ldz + id];
  }
  if (k) {
    // parts of the token, four at a time (a step's first is a multiple of 4; past its last:
    // -infinity, which is nobody's largest unless nothing is finite)
    const int part = part_of(a.group);
    const float* tops = a.kept.tops + t * a.kept.groups * (a.group / part);
    auto four = [&](int64_t p) {
      f32x4 x;
      if (p + 4 <= a.p1) {
        __builtin_memcpy(&x, tops + p, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p + i < a.p1 ? tops[p + i] : kNegInf;
      }
      return x;
    };
    // (one part at a time where four would leave threads without any, and words where the parts are
    // few for the best words: fewer shares than those bound nothing. 500 tokens of 1000 parts, 128
    // best: 513 us by fours, 20; 2000 tokens, 128 best: of 125 parts 89 us, by words 26, of 250 30
    // and 32)
    const float* z = a.kept.z + t * a.kept.ldz;
    uint32_t m = 0;
    if (2 * (a.p1 - a.p0) < 3 * k && !a.have) {   // (the first step's z are all there)
      const int64_t end = lmin(a.V, a.p1 * part);
#pragma unroll 4
      for (int64_t w = a.v0 + tid; w < end; w += NT) m = max(m, order_of(z[w - a.v0]));
    } else if (a.p1 - a.p0 >= 4 * NT) {
      for (int64_t p = a.p0 + 4 * tid; p < a.p1; p += 4 * NT) {
        const f32x4 x = four(p);
        m = max(m, order_of(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]))));
      }
    } else {
#pragma unroll 4
      for (int64_t p = a.p0 + tid; p < a.p1; p += NT) m = max(m, order_of(tops[p]));
    }
    most[tid] = m;
    if (a.have)
      for (int i = tid; i < k; i += NT) list[i] = a.best[t * k + i];
    if (tid == 0) count = a.have ? k : 0;
    __syncthreads();
    uint64_t bound;   // keys above it are in
    {
      uint32_t x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = most[64 * i + lane];
#pragma unroll
        for (int o = 256; o < NT; o += 256) x[i] = max(x[i], most[o + 64 * i + lane]);
      }
      int n;
      const uint32_t c = reached(x, k, 12, &n);
      bound = c ? ((uint64_t)c << 32) - 1 : 0;
      // (later words lose to earlier ones of the same z)
      if (a.have) bound = max(bound, (uint64_t)order_of(a.thr[t]) << 32 | 0xffffffffu);
    }
    n = a.have ? k : 0;
    // cuts the list to its k best; afterwards lim is what their z reach, low what the words of that z do
    auto cut = [&]() {
      if (wave == 0) {
        uint32_t hi[kEach], lo[kEach];
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const uint64_t key = 64 * i + lane < n ? list[64 * i + lane] : 0;
          hi[i] = (uint32_t)(key >> 32);
          lo[i] = (uint32_t)key;
        }
        int got;
        const uint32_t c = n <= 256 ? reached(reinterpret_cast<const uint32_t(&)[4]>(hi), k, 0, &got)
                                    : reached(hi, k, 0, &got);
        uint32_t d = 0;
        if (got != k) {   // several of the k-th z: the lower words
          uint32_t x[kEach];
          int above = 0;
#pragma unroll
          for (int i = 0; i < kEach; ++i) {
            above += __popcll(__ballot(hi[i] > c));
            x[i] = hi[i] == c ? lo[i] : 0;
          }
          d = reached(x, k - above, 0, &got);
        }
        int at = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const bool in = 64 * i + lane < n && (hi[i] > c || (hi[i] == c && lo[i] >= d));
          const uint64_t who = __ballot(in);
          if (in) list[at + rank_in(who)] = (uint64_t)hi[i] << 32 | lo[i];
          at += __popcll(who);
        }
        if (lane == 0) {
          count = at;
          lim = c;
          low = d;
        }
      }
      __syncthreads();
      n = count;
      __syncthreads();
      bound = max(bound, ((uint64_t)lim << 32 | low) - (lim != 0));
    };
    // words above the bound of the parts todo[b .. end); whether all had room
    auto collect = [&](int b, int end) {
      // a wave reads 64 / part of them at once, eight times before the first use
      constexpr int Q = 8;
      const int each = 64 / part, first = wave * each + lane / part, in = lane % part;
      for (int i = b; i < end; i += Q * NW * each) {
        float x[Q];
        uint32_t w[Q];
        bool on[Q];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int e = i + q * NW * each + first;
          w[q] = (uint32_t)(todo[min(e, end - 1)] * part + in);
          on[q] = e < end && w[q] < a.V;
          x[q] = on[q] ? z[w[q] - a.v0] : 0.0f;
        }
        uint64_t who[Q];
        int some = 0;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          who[q] = __ballot(on[q] && key_of(x[q], w[q]) > bound);
          some += __popcll(who[q]);
        }
        if (!some) continue;
        int at = 0;
        if (lane == 0) at = atomicAdd(&count, some);
        at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int place = at + rank_in(who[q]);
          if (who[q] >> lane & 1 && place < kCap) list[place] = key_of(x[q], w[q]);
          at += __popcll(who[q]);
        }
      }
      __syncthreads();
      const int c = count;
      __syncthreads();   // (nobody changes count before all have read it)
      if (c > kCap) {
        if (tid == 0) count = n;
        __syncthreads();
        return false;
      }
      n = c;
      return true;
    };
    for (int64_t base = a.p0; base < a.p1; base += 4 * NT) {
      if (tid == 0) left = 0;
      __syncthreads();
      const int64_t p = base + 4 * tid;
      if (p < a.p1) {
        const f32x4 x = four(p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p + i < a.p1 && key_of(x[i], (uint32_t)((p + i) * part)) > bound)
            todo[atomicAdd(&left, 1)] = (int)(p + i);
      }
      __syncthreads();
      const int c = left;
      if (c && !collect(0, c)) {
        int more = 0;
        for (int b = 0; b < c;) {
          if (n > k) cut();
          const int sure = (kCap - n) / part, end = min(c, b + max(sure, more));
          if (collect(b, end)) {
            more = 2 * (end - b);
            b = end;
          } else {
            more = 0;
          }
        }
      }
    }
    // (a short list is put in order as it is)
    if (!a.last || n > 256) cut();
    if (!a.last) {
      for (int i = tid; i < k; i += NT) a.best[t * k + i] = i < n ? list[i] : 0;
      if (tid == 0) a.thr[t] = value_of(lim);
      return;
    }
  }
  Sums r{mine[0], mine[1], mine[2]};
  for (int64_t g = tid + NT; g < a.kept.groups; g += NT) {
    const f32x4 x = stat[g];
    join(r, Sums{x[0], x[1], x[2]});
  }
  r = join_all<NT>(r, sm);
  const float log_s = log1pf(r.r);
  const bool fine = r.r == r.r;
  if (tid == 0) {
    a.lse[t] = r.m + log_s;
    a.entropy[t] = log_s - r.u / (1.0f + r.r);
  }
  if (!fine) {
    for (int i = tid; i < k; i += NT) {
      a.top_ids[t * k + i] = -1;
      a.top_logprobs[t * k + i] = kNaN;
    }
  } else if (tid < n) {   // (n <= NT; k of them are at least as good as the others)
    const uint64_t key = list[tid];
    int place = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) place += list[j] > key;
    if (place < k) {
      a.top_ids[t * k + place] = (int32_t)~(uint32_t)key;
      a.top_logprobs[t * k + place] = value_of((uint32_t)(key >> 32)) - r.m - log_s;
    }
  }
  if (tid < a.given) a.logprobs[t * a.given + tid] = id < 0 ? 0.0f : zid - r.m - log_s;
}

// ---------------------------------------------------------------- divergence
struct Near {
  Kept kept;
  int64_t V;
  const int32_t* ids;
  const float* logq;
  int64_t ldi, ldq;
  const uint8_t* places;     // [token][K]
  int K, tail;
  float *loss, *lse, *rest, *hit;
};
// loss, lse, rest and hit of token t, by one wave: r joins the groups' sums (with a tail: without the
// listed words); of entries lane and lane + 64 on: whether they are one, z (NaN for a word past the
// last); the distinct listed words' z are those x that are `part`.
__device__ __forceinline__ void finish(const Near& a, int64_t t, int lane, Sums r, const bool (&on)[2],
                                       const float (&z)[2], const float (&x)[2], const bool (&part)[2]) {
  float l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) l[i] = on[i] ? a.logq[t * a.ldq + lane + 64 * i] : 0.0f;
  const bool used = __ballot(on[0] || on[1]) != 0;
  const Teacher q = teacher(l, on, a.tail);
  double m = r.m, s = 1.0 + (double)r.r;
  const bool all = r.r == -1.0f;   // every word is listed
  if (a.tail) {
    m = wave_max(fmax(part[0] ? (double)x[0] : -INFINITY, part[1] ? (double)x[1] : -INFINITY));
    m = fmax(m, (double)r.m);
    // (a listed z of -infinity is no zero but NaN, as in the groups' sums)
    auto e = [&](int i) { return !part[i] ? 0.0 : x[i] == kNegInf ? (double)kNaN : exp((double)x[i] - m); };
    s = wave_sum(e(0) + e(1));
    if (!all) s += (1.0 + (double)r.r) * exp((double)r.m - m);
  }
  const double log_s = log(s);
  double e = 0.0;
#pragma unroll
  for (int i = 0; i < 2; ++i)   // (a word past the last has its NaN without any mass, too)
    e += q.q[i] == 0.0 ? (z[i] == z[i] ? 0.0 : (double)kNaN) : q.q[i] * (q.logq[i] - ((double)z[i] - m) + log_s);
  double loss = wave_sum(e);
  const double rest = a.tail ? (double)r.m + log1p((double)r.r) : m + log_s;
  // (without a rest there is none to be off from)
  if (!all && q.r != 0.0) loss += q.r * (log(q.r) - (rest - m) + log_s);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64 * i < a.K) a.hit[t * a.K + lane + 64 * i] = z[i];
  if (lane == 0) {
    a.loss[t] = !used ? 0.0f : log_s == log_s ? (float)loss : kNaN;
    a.lse[t] = used ? (float)(m + log_s) : 0.0f;
    a.rest[t] = used ? (float)rest : 0.0f;
  }
}

// A workgroup of NT threads per token; all of it but the join in one wave, in 64 bits. 777 tokens of
// 782 groups 10 us, 4096 tokens of 1024 28 (67 MB of sums: 2.4 TB/s).
template <int NT>
__global__ __launch_bounds__(NT) void distill_kernel(Near a) {
  __shared__ float sm[3 * (NT / 64)];
  const int tid = threadIdx.x, lane = tid & 63;
  const int64_t t = blockIdx.x;
  const Kept& o = a.kept;
  const f32x4* stat = o.stat + t * o.groups;
  const float* zl = o.zl + t * a.K;
  float z[2], x[2];
  bool on[2], part[2];
  int place[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = lane + 64 * i;
    on[i] = k < a.K && a.ids[t * a.ldi + k] >= 0;
    place[i] = on[i] ? a.places[t * a.K + k] : 255;
    z[i] = !on[i] ? 0.0f : place[i] == 255 ? kNaN : zl[place[i]];
  }
  Sums r = kNothing;
  for (int64_t g = tid; g < o.groups; g += NT) {
    const f32x4 q = stat[g];
    join(r, Sums{q[0], q[1], 0.0f});
  }
  r = join_all<NT>(r, sm);
  if (tid >= 64) return;
  // the listed words have the places 0 .. n - 1
  int n = max(place[0] == 255 ? 0 : place[0] + 1, place[1] == 255 ? 0 : place[1] + 1);
#pragma unroll
  for (int i = 32; i > 0; i >>= 1) n = max(n, __shfl_xor(n, i));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    part[i] = lane + 64 * i < n;
    x[i] = part[i] && a.tail ? zl[lane + 64 * i] : 0.0f;
  }
  finish(a, t, lane, r, on, z, x, part);
}

// The same of few tokens, whose logits are all there (without marks: a launch less, 7 tokens, 32000 x
// 4096 bf16 66 -> 62 us). With a tail, groups of 64 words with a listed one are summed again, from
// those logits. 9 us: dependent loads.
template <int NT>
__global__ __launch_bounds__(NT) void distill_few_kernel(Near a) {
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  constexpr int NW = NT / 64;
  __shared__ __align__(16) int word[kList];
  __shared__ int owner[kList];          // the first entry of the same group; -1: none
  __shared__ bool again[kList];         // an earlier entry has the same word
  __shared__ uint32_t out[kList][2];    // of the owner's group: the words that are listed
  __shared__ float sm[3 * NW];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t t = blockIdx.x;
  const Kept& o = a.kept;
  f32x4* stat = o.stat + t * o.groups;
  const float* row = o.z + t * o.ldz;
  float z[2], x[2];
  bool on[2], part[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = lane + 64 * i;
    const int32_t id = k < a.K ? a.ids[t * a.ldi + k] : -1;
    on[i] = id >= 0;
    z[i] = !on[i] ? 0.0f : id < a.V ? row[id] : kNaN;
    if (wave == 0) {
      word[k] = id < a.V ? id : -1;
      out[k][0] = out[k][1] = 0;
    }
  }
  __syncthreads();
  if (a.tail && tid < kList) {
    const int id = word[tid], g = id >> 6;   // (-1 of none: no group's)
    int own = tid;
    bool twice = false;
#pragma unroll 4
    for (int j = 0; j < a.K; j += 4) {
      const i32x4 w = *(const i32x4*)(word + j);
#pragma unroll
      for (int u = 3; u >= 0; --u) {
        own = (w[u] >> 6) == g && j + u < own ? j + u : own;
        twice |= w[u] == id && j + u < tid;
      }
    }
    owner[tid] = id >= 0 ? own : -1;
    again[tid] = twice;
    if (id >= 0) {
      atomicOr(&out[own][id >> 5 & 1], 1u << (id & 31));
      if (own == tid) stat[g] = f32x4{kNegInf, -1.0f, 0.0f, 0.0f};
    }
  }
  __syncthreads();
  Sums r = kNothing;
  for (int64_t g = tid; g < o.groups; g += NT) {
    const f32x4 q = stat[g];
    join(r, Sums{q[0], q[1], 0.0f});
  }
  if (a.tail) {
    // four groups of a wave at a time, all their loads before the first use
    for (int k0 = wave; k0 < a.K; k0 += 4 * NW) {
      float y[4];
      bool in[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = min(k0 + q * NW, a.K - 1);
        const int64_t w = (int64_t)(word[k] >> 6) * 64 + lane;
        in[q] = k0 + q * NW < a.K && owner[k] == k && w < a.V && !(out[k][lane >> 5] >> (lane & 31) & 1);
        y[q] = in[q] ? row[w] : 0.0f;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (in[q]) join(r, Sums{y[q], fabsf(y[q]) < __builtin_inff() ? 0.0f : kNaN, 0.0f});
    }
  }
  r = join_all<NT>(r, sm);
  if (wave) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    part[i] = a.tail && word[lane + 64 * i] >= 0 && !again[lane + 64 * i];
    x[i] = z[i];
  }
  finish(a, t, lane, r, on, z, x, part);
}

// Labels, shares, val (struct Vocab) and Q of the gradient. Four tokens per workgroup, a wave each.
// 4096 tokens of 64 words: 9 us.
__global__ __launch_bounds__(256) void shares_kernel(Taught a, int64_t T, int32_t* __restrict__ labels,
                                                     float* __restrict__ share, float* __restrict__ whole,
                                                     float* __restrict__ val) {
  __shared__ int word[4][kList];
  __shared__ double q[4][kList];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= T) return;
  const Share s = share_of(a, t, lane, word[wave], q[wave]);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 64 * i < a.K) val[t * a.K + lane + 64 * i] = s.val[i];
  if (lane == 0) {
    labels[t] = s.label;
    share[t] = s.share;
    whole[t] = s.whole;
  }
}

// ---------------------------------------------------------------- launches
// H as the products take it
template <int D>
hipError_t tokens(const Vocab& a, const KeepPlan& k, Opnd* H, hipStream_t s) {
  Opnd unused;
  if constexpr (D != kF32) {
    return begin<D>(a, k.p, nullptr, 1, H, &unused, s);
  } else {
    char* w = (char*)a.work;
    uint16_t* out = (uint16_t*)(w + k.p.hp);
    *H = Opnd{out, 2 * k.p.dp, k.p.dp, a.T, k.p.dp};
    return rowpack(a.H, a.T, a.d, a.ldh, a.scale, out, k.p.dp, (float*)(w + k.zs), a.T, s);
  }
}
// The logits of tokens t0 .. t0 + n of the words v0 .. v0 + nv, as `kept` says
template <int D>
hipError_t pick(const Vocab& a, const KeepPlan& k, const Opnd& H, int64_t t0, int64_t n, int64_t v0,
                int64_t nv, const Kept& kept, hipStream_t s) {
  Mma m{};
  m.B = H;
  m.B.p += t0 * H.ld;
  m.B.rows = n;
  m.K = m.k_slice = k.p.dp;
  char* w = (char*)a.work;
  m.zs = (float*)(w + k.zs) + t0;
  m.ws = (float*)(w + k.ws);
  m.z0 = a.scale;
  m.v0 = v0;
  m.kept = kept;
  hipError_t e;
  if constexpr (D != kF32) {
    e = words<D>(a, k.p, v0, nv, &m.A, s);
  } else {   // (every word to the top of the terms' range by itself: no pass over W for its largest)
    uint16_t* out = (uint16_t*)(w + k.p.wp);
    m.A = Opnd{out, 2 * k.p.dp, k.p.dp, nv, k.p.dp};
    e = rowpack((const float*)a.W + v0 * a.ldw, nv, a.d, a.ldw, 1.0f, out, k.p.dp, (float*)(w + k.ws),
                round_up(nv, 256), s);
  }
  if (e != hipSuccess) return e;
  return mma_launch<D, kPick>(m, k.tile, 1, s);
}

// Where what is kept of listed words lies, and the marks of n tokens
hipError_t mark(char* w, const KeepPlan& k, const int32_t* ids, int64_t ldi, int64_t K, int64_t n, int64_t V,
                Kept* o, const uint8_t** places, hipStream_t s) {
  const Marks m{(uint8_t*)(w + k.slot), k.lds, (Mark*)(w + k.marks), (uint8_t*)(w + k.places)};
  o->slot = m.slot;
  o->lds = k.lds;
  o->listed = K;
  o->marks = m.marks;
  o->zl = (float*)(w + k.zl);
  *places = m.places;
  hipLaunchKernelGGL(marks_kernel, dim3((unsigned)n), dim3(kList), 0, s, ids, ldi, (int)K, V, (int)k.group, m);
  return hipGetLastError();
}

template <int NT> void go_top(const Top& t, int64_t rows, hipStream_t s) {
  hipLaunchKernelGGL(top_kernel<NT>, dim3((unsigned)rows), dim3(NT), 0, s, t);
}

template <int D>
hipError_t logprobs(const Logprobs& a, hipStream_t s) {
  const Vocab& v = a.v;
  const KeepPlan k = keep_plan(v.T, v.V, v.d, D, a.given, a.k);
  char* w = (char*)v.work;
  hipError_t e;
  Kept o{};
  o.flip = v.scale < 0.0f;
  o.stat = (f32x4*)(w + k.stat);
  o.groups = k.groups;
  o.ldz = k.ldz;
  Top t{};
  t.group = (int)k.group;
  t.V = v.V;
  t.k = (int)a.k;
  t.best = (uint64_t*)(w + k.best);
  t.thr = (float*)(w + k.thr);
  t.ldt = a.ldt;
  t.given = (int)a.given;
  Opnd H{};
  if (!k.few && (e = tokens<D>(v, k, &H, s)) != hipSuccess) return e;
  for (int64_t t0 = 0; t0 < v.T; t0 += k.block) {
    const int64_t n = std::min(k.block, v.T - t0);
    t.tokens = a.tokens ? a.tokens + t0 * a.ldt : nullptr;
    t.logprobs = a.logprobs + t0 * a.given;
    t.entropy = a.entropy + t0;
    t.lse = a.lse + t0;
    t.top_ids = a.top_ids + t0 * a.k;
    t.top_logprobs = a.top_logprobs + t0 * a.k;
    if (k.marked && (e = mark(w, k, t.tokens, a.ldt, a.given, n, v.V, &o, &t.places, s)) != hipSuccess) return e;
    if (k.few || a.k) o.z = (float*)(w + k.z);
    if (a.k) o.tops = (float*)(w + k.tops);
    // without best words all at once, or a copy of W's at a time
    const int64_t most = k.few ? v.V : direct(v.W, v.ldw, v.d, D) ? v.V : k.p.piece;
    int64_t step = k.few || !a.k ? most : std::min(k.first, most);
    for (int64_t v0 = 0, nv; v0 < v.V; v0 += nv) {
      nv = std::min(step, v.V - v0);
      o.thr = v0 ? t.thr : nullptr;
      if (k.few)
        e = score<D>(v, 0, v.V, o, s);
      else
        e = pick<D>(v, k, H, t0, n, v0, nv, o, s);
      if (e != hipSuccess) return e;
      t.last = v0 + nv >= v.V;
      if (!a.k && !t.last) continue;
      t.kept = o;
      t.v0 = v0;
      t.p0 = v0 / part_of(t.group);
      t.p1 = (v0 + nv + part_of(t.group) - 1) / part_of(t.group);
      t.have = v0 > 0;
      // (512 threads and 256, us a launch: one token of 32000 words 10 and 11, 256 tokens of 131072, 64
      // best, 15 and 21, 509 of 50021 12.8 and 13.1; 1000 of 32000 20 and 14, 4096 80 and 57: more
      // tokens share a CU)
      n <= 512 ? go_top<512>(t, n, s) : go_top<256>(t, n, s);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      if (a.k) step = std::min(std::min(3 * step, k.step), most);
    }
  }
  return hipSuccess;
}

template <int D>
hipError_t distill(const Distill& a, hipStream_t s) {
  const Vocab& v = a.v;
  const KeepPlan k = keep_plan(v.T, v.V, v.d, D, a.K, 0);
  char* w = (char*)v.work;
  hipError_t e;
  Near r{};
  r.kept.flip = v.scale < 0.0f;
  r.kept.stat = (f32x4*)(w + k.stat);
  r.kept.groups = k.groups;
  r.kept.without = a.tail;
  r.V = v.V;
  r.ldi = a.ldi;
  r.ldq = a.ldq;
  r.K = (int)a.K;
  r.tail = a.tail;
  Opnd H{};
  if (!k.few && (e = tokens<D>(v, k, &H, s)) != hipSuccess) return e;
  for (int64_t t0 = 0; t0 < v.T; t0 += k.block) {
    const int64_t n = std::min(k.block, v.T - t0);
    r.ids = a.ids + t0 * a.ldi;
    r.logq = a.logq + t0 * a.ldq;
    r.loss = a.loss + t0;
    r.lse = a.lse + t0;
    r.rest = a.rest + t0;
    r.hit = a.hit + t0 * a.K;
    float* z = a.z && keeps(v.T, v.V, v.d, D) ? a.z + t0 * row_of(v.V) : nullptr;
    r.kept.z = z;
    r.kept.ldz = row_of(v.V);
    if (k.few) {
      if (!z) r.kept.z = (float*)(w + k.z);
      if ((e = score<D>(v, 0, v.V, r.kept, s)) != hipSuccess) return e;
      hipLaunchKernelGGL(distill_few_kernel<512>, dim3((unsigned)n), dim3(512), 0, s, r);
      if ((e = hipGetLastError()) != hipSuccess) return e;
      continue;
    }
    if ((e = mark(w, k, r.ids, a.ldi, a.K, n, v.V, &r.kept, &r.places, s)) != hipSuccess) return e;
    const int64_t step = direct(v.W, v.ldw, v.d, D) ? v.V : k.p.piece;
    for (int64_t v0 = 0; v0 < v.V; v0 += step) {
      r.kept.z = z ? z + v0 : nullptr;
      if ((e = pick<D>(v, k, H, t0, n, v0, std::min(step, v.V - v0), r.kept, s)) != hipSuccess) return e;
    }
    hipLaunchKernelGGL(distill_kernel<256>, dim3((unsigned)n), dim3(256), 0, s, r);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int64_t logprobs_work_bytes(int64_t T, int64_t V, int64_t d, int dtype, int64_t given, int64_t k) {
  return keep_plan(T, V, d, dtype, given, k).bytes;
}
int64_t distill_work_bytes(int64_t T, int64_t V, int64_t d, int dtype, int64_t K, bool grad) {
  return grad ? share_plan(T, V, d, dtype, K).bytes : keep_plan(T, V, d, dtype, K, 0).bytes;
}

hipError_t launch_vocab_logprobs(const Logprobs& a, hipStream_t s) {
  if (a.v.dtype == kF32) return logprobs<kF32>(a, s);
  return a.v.dtype == kBF16 ? logprobs<kBF16>(a, s) : logprobs<kF16>(a, s);
}

hipError_t launch_vocab_distill(const Distill& a, hipStream_t s) {
  if (a.v.dtype == kF32) return distill<kF32>(a, s);
  return a.v.dtype == kBF16 ? distill<kBF16>(a, s) : distill<kF16>(a, s);
}

hipError_t launch_vocab_distill_backward(const Distill& a, hipStream_t s) {
  Vocab v = a.v;
  const SharePlan p = share_plan(v.T, v.V, v.d, v.dtype, a.K);
  char* w = (char*)v.work;
  int32_t* labels = (int32_t*)(w + p.labels);
  const Taught of{a.ids, a.logq, a.lse, a.rest, a.hit, a.ldi, a.ldq, v.V, (int)a.K, a.tail};
  const float* z = keeps(v.T, v.V, v.d, v.dtype) ? a.z : nullptr;
  v.labels = labels;
  v.lse = a.tail ? a.rest : a.lse;
  if (few(v.T, v.d, v.dtype)) {
    const FewPlan f = few_plan(v.T, v.V, v.d, v.dtype);
    Few g{a, z, (float*)(w + f.G), (float*)(w + f.part), labels};
    if (!g.z) {
      Kept o{};
      o.z = (float*)(w + f.z);
      o.ldz = f.ldz;
      const hipError_t e = v.dtype == kF32    ? score<kF32>(v, 0, v.V, o, s)
                           : v.dtype == kBF16 ? score<kBF16>(v, 0, v.V, o, s)
                                              : score<kF16>(v, 0, v.V, o, s);
      if (e != hipSuccess) return e;
      g.z = o.z;
    }
    return launch_few_gradient(g, s);
  }
  float *share = (float*)(w + p.share), *val = (float*)(w + p.val);
  hipLaunchKernelGGL(shares_kernel, dim3((unsigned)((v.T + 3) / 4)), dim3(256), 0, s, of, v.T, labels, share,
                     (float*)(w + p.wr), val);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  v.share = share;
  v.wr = (float*)(w + p.wr);
  v.ids = a.ids;
  v.ldi = a.ldi;
  v.listed = a.K;
  v.val = val;
  v.z = z;
  v.ldz = row_of(v.V);
  return launch_vocab_loss_backward(v, s);
}

}  // namespace nq
