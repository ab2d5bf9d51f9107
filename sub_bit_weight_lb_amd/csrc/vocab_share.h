// A teacher's probabilities of a token, and what the gradient of a divergence from them needs of it
// (vocab_top.hip, vocab_few.hip).
#pragma once

#include "tune.h"
#include "vocab_plan.h"

namespace nq {
namespace {

constexpr int kList = (int)vocab::kMaxListed;

// sum of x over a wave, in a fixed order; all lanes get it
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}
__device__ __forceinline__ double wave_max(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x = fmax(x, __shfl_xor(x, o));
  return x;
}
// A teacher's probabilities of one token: entries lane and lane + 64 of a wave, in 64 bits (r is
// what a sum near one leaves). on: whether the entry is one.
struct Teacher {
  double q[2], logq[2], sum, r;
};
__device__ __forceinline__ Teacher teacher(const float (&l)[2], const bool (&on)[2], bool tail) {
  Teacher t;
  double top = 0.0;
  if (!tail) {
    top = wave_max(fmax(on[0] ? (double)l[0] : -INFINITY, on[1] ? (double)l[1] : -INFINITY));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    t.logq[i] = on[i] ? (double)l[i] - top : 0.0;
    t.q[i] = on[i] ? exp(t.logq[i]) : 0.0;
  }
  t.sum = wave_sum(t.q[0] + t.q[1]);
  if (!tail) {
    const double log_sum = log(t.sum);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      t.q[i] /= t.sum;
      t.logq[i] -= log_sum;
    }
    t.sum = t.sum == t.sum ? 1.0 : t.sum;
  }
  t.r = tail ? 1.0 - t.sum : 0.0;
  t.r = t.r < 0.0 ? 0.0 : t.r;   // (a NaN stays)
  return t;
}

// What the gradient needs of token t: its label (the first word listed; V where one is at or past V;
// -1 without any), its share, its entries' words and val (struct Vocab), Q = sum q + r. By one wave, entries lane and
// lane + 64; word, q: kList each in LDS, of this wave alone.
struct Share {
  int32_t label;
  float share, val[2], whole;   // whole: Q
};
struct Taught {
  const int32_t* ids;
  const float *logq, *lse, *rest, *hit;
  int64_t ldi, ldq, V;
  int K, tail;
};
__device__ __forceinline__ Share share_of(const Taught& a, int64_t t, int lane, int* word, double* q) {
  float l[2];
  bool on[2];
  int id[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = lane + 64 * i;
    id[i] = k < a.K ? a.ids[t * a.ldi + k] : -1;
    on[i] = id[i] >= 0;
    l[i] = on[i] ? a.logq[t * a.ldq + k] : 0.0f;
    word[k] = id[i];
  }
  const Teacher p = teacher(l, on, a.tail);
#pragma unroll
  for (int i = 0; i < 2; ++i) q[lane + 64 * i] = p.q[i];
  __builtin_amdgcn_wave_barrier();
  const double e = a.lse[t], out = a.tail ? (double)a.rest[t] : e;
  const double r = out == -INFINITY ? 0.0 : p.r, whole = p.sum + r;
  Share s;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    double mine = 0.0;
    if (on[i])
#pragma unroll 8
      for (int j = 0; j < a.K; ++j) mine += word[j] == id[i] ? q[j] : 0.0;
    s.val[i] = on[i] ? (float)(whole * exp((double)a.hit[t * a.K + lane + 64 * i] - e) - mine) : 0.0f;
  }
  const uint64_t some[2] = {__ballot(on[0]), __ballot(on[1])};
  const bool past = __ballot(id[0] >= a.V || id[1] >= a.V) != 0;
  const int first = some[0] ? __ffsll((unsigned long long)some[0]) - 1 : 63 + __ffsll((unsigned long long)some[1]);
  const bool used = some[0] || some[1];
  s.label = !used ? -1 : past ? (int32_t)a.V : word[first];
  s.whole = (float)whole;
  s.share = used ? (float)(a.tail ? whole * exp(out - e) - r : whole) : 0.0f;
  return s;
}

}  // namespace
}  // namespace nq
