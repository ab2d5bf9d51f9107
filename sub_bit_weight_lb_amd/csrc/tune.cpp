// C ABI of the operators that tune a packed model (declared in include/nq.h):
// 8-bit activation checkpoints (act8.hip), the gradient of a packed layer from
// such a checkpoint (binback.hip), the loss over a large vocabulary with its
// gradient (vocab.hip), log probabilities and the divergence from a teacher's words
// with its gradient (vocab_top.hip, vocab_few.hip). Each call only checks its arguments and enqueues
// kernels on the caller's stream: no allocation, no wait.
#include <algorithm>
#include <cmath>
#include <string>

#include "abi.h"
#include "tune.h"
#include "vocab_plan.h"

using namespace nq;

namespace {

constexpr int64_t kMaxDim = int64_t(1) << 21;    // layer sizes
constexpr int64_t kMaxRows = int64_t(1) << 31;   // tokens
// of a layer's gradient: every launch stays below 2^32 threads
constexpr int64_t kMaxTuned = int64_t(1) << 24, kMaxValues = int64_t(1) << 36;
constexpr int64_t kMaxWords = int64_t(1) << 20;  // of a row of signs: 256 rows stay below 2^31 bytes

bool dtype_ok(int32_t t) { return t == NQ_F32 || t == NQ_BF16 || t == NQ_F16; }
static_assert((int)NQ_F32 == kF32 && (int)NQ_BF16 == kBF16 && (int)NQ_F16 == kF16, "nq_dtype");

nq_status bad(const char* msg) { return set_error(NQ_ERR_INVALID_ARG, msg); }
bool misaligned(const void* p, int64_t bytes) { return (uintptr_t)p % (uintptr_t)bytes != 0; }

// rows x cols of a checkpoint and its buffers
nq_status check_act8(const int8_t* codes, int64_t ldc, const uint8_t* exps, int64_t lde,
                     int64_t cols) {
  if (!codes || !exps) return bad("codes and exps are required");
  if (ldc < cols) return bad("ldc < cols");
  if (lde < (cols + kActGroup - 1) / kActGroup) return bad("lde < ceil(cols/32)");
  return NQ_OK;
}

// limits of the loss: byte offsets inside a 256-row tile of any operand stay
// below 2^31, and a launch of one tile per 256 x 256 logits below 2^32 threads
constexpr int64_t kMaxTokens = int64_t(1) << 20, kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxHidden = int64_t(1) << 18, kMaxLd = int64_t(1) << 21;
constexpr int64_t kMaxLogits = int64_t(1) << 38;

nq_status check_head(const void* H, int64_t ldh, const void* W, int64_t ldw, int32_t dtype,
                     int64_t T, int64_t V, int64_t d, float scale, const void* work) {
  if (!dtype_ok(dtype)) return bad("dtype must be NQ_F32, NQ_BF16 or NQ_F16");
  if (T < 0 || T > kMaxTokens) return bad("T must be in [0, 2^20]");
  if (V < 1 || V > kMaxVocab) return bad("V must be in [1, 2^24]");
  if (d < 1 || d > kMaxHidden) return bad("d must be in [1, 2^18]");
  if (T * V > kMaxLogits) return bad("T V must be <= 2^38");
  if (!std::isfinite(scale)) return bad("scale must be finite");
  if (T == 0) return NQ_OK;
  if (!H || !W || !work) return bad("H, W and work are required");
  if (ldh < d || ldw < d) return bad("ldh < d or ldw < d");
  if (ldh > kMaxLd || ldw > kMaxLd) return bad("ldh and ldw must be <= 2^21");
  if (misaligned(H, dtype_bytes(dtype)) || misaligned(W, dtype_bytes(dtype)))
    return bad("H or W is not aligned to its type");
  if (misaligned(work, 16)) return bad("work must be 16-byte aligned");
  return NQ_OK;
}
nq_status check_vocab(const void* H, int64_t ldh, const void* W, int64_t ldw, int32_t dtype,
                      int64_t T, int64_t V, int64_t d, const int32_t* labels, float scale,
                      const void* work) {
  const nq_status st = check_head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  return st == NQ_OK && T > 0 && !labels ? bad("labels are required") : st;
}
bool head_ok(int64_t T, int64_t V, int64_t d, int32_t dtype) {
  return dtype_ok(dtype) && T >= 0 && V >= 1 && d >= 1 && T <= kMaxTokens && V <= kMaxVocab &&
         d <= kMaxHidden && T * V <= kMaxLogits;
}
nq_status check_listed(const int32_t* ids, int64_t ldi, const float* logq, int64_t ldq, int64_t K) {
  if (K < 1 || K > vocab::kMaxListed) return bad("K must be in [1, 128]");
  if (!ids || !logq) return bad("ids and logq are required");
  if (ldi < K || ldq < K) return bad("ldi < K or ldq < K");
  if (ldi > kMaxLd || ldq > kMaxLd) return bad("ldi and ldq must be <= 2^21");
  if (misaligned(ids, 4) || misaligned(logq, 4)) return bad("ids or logq is not aligned to its type");
  return NQ_OK;
}
Vocab head(const void* H, int64_t ldh, const void* W, int64_t ldw, int32_t dtype, int64_t T, int64_t V,
           int64_t d, float scale, void* work) {
  Vocab a{};
  a.H = H; a.W = W; a.dtype = dtype; a.ldh = ldh; a.ldw = ldw; a.T = T; a.V = V; a.d = d;
  a.scale = scale; a.work = work;
  return a;
}

}  // namespace

extern "C" {

nq_status nq_act8_quantize(const void* X, int32_t dtype, int64_t rows, int64_t cols, int64_t ldx,
                           int8_t* codes, int64_t ldc, uint8_t* exps, int64_t lde, void* stream) {
  if (!dtype_ok(dtype)) return bad("dtype must be NQ_F32, NQ_BF16 or NQ_F16");
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxRows)
    return bad("rows and cols must be in [0, 2^31]");
  if (rows == 0 || cols == 0) return NQ_OK;
  if (!X) return bad("X is required");
  if (ldx < cols) return bad("ldx < cols");
  if (misaligned(X, dtype_bytes(dtype))) return bad("X is not aligned to its type");
  const nq_status st = check_act8(codes, ldc, exps, lde, cols);
  if (st != NQ_OK) return st;
  NQ_HIPCHK(launch_act8_quantize(X, dtype, rows, cols, ldx, codes, ldc, exps, lde,
                                 (hipStream_t)stream));
  return NQ_OK;
}

nq_status nq_act8_dequantize(const int8_t* codes, int64_t ldc, const uint8_t* exps, int64_t lde,
                             int64_t rows, int64_t cols, void* X, int32_t dtype, int64_t ldx,
                             void* stream) {
  if (!dtype_ok(dtype)) return bad("dtype must be NQ_F32, NQ_BF16 or NQ_F16");
  if (rows < 0 || cols < 0 || rows > kMaxRows || cols > kMaxRows)
    return bad("rows and cols must be in [0, 2^31]");
  if (rows == 0 || cols == 0) return NQ_OK;
  if (!X) return bad("X is required");
  if (ldx < cols) return bad("ldx < cols");
  if (misaligned(X, dtype_bytes(dtype))) return bad("X is not aligned to its type");
  const nq_status st = check_act8(codes, ldc, exps, lde, cols);
  if (st != NQ_OK) return st;
  NQ_HIPCHK(launch_act8_dequantize(Act8{codes, ldc, exps, lde}, rows, cols, X, dtype, ldx,
                                   (hipStream_t)stream));
  return NQ_OK;
}

nq_status nq_act8_steps(const uint8_t* exps, int64_t lde, int64_t rows, int64_t groups,
                        float* steps, int64_t lds, void* stream) {
  if (rows < 0 || groups < 0 || rows > kMaxRows || groups > kMaxRows)
    return bad("rows and groups must be in [0, 2^31]");
  if (rows == 0 || groups == 0) return NQ_OK;
  if (!exps || !steps) return bad("exps and steps are required");
  if (lde < groups || lds < groups) return bad("lde < groups or lds < groups");
  if (misaligned(steps, 4)) return bad("steps is not aligned to its type");
  NQ_HIPCHK(launch_act8_steps(exps, lde, rows, groups, steps, lds, (hipStream_t)stream));
  return NQ_OK;
}

int64_t nq_binary_matmul_backward_work_bytes(int64_t T, int64_t m, int64_t n, int64_t r) {
  if (T < 0 || m < 0 || n < 0 || r < 0 || T > kMaxTuned || m > kMaxDim || n > kMaxDim ||
      r > kMaxDim || T * std::max(std::max(m, n), r) > kMaxValues)
    return -1;
  return T == 0 || m == 0 || n == 0 || r == 0 ? 0 : binback_work_bytes(m, n, r, T);
}

nq_status nq_binary_matmul_backward(const uint32_t* U_bits, int64_t ldu, const uint32_t* Ut_bits,
                                    int64_t ldut, const uint32_t* V_bits, int64_t ldv,
                                    const uint32_t* Vt_bits, int64_t ldvt, int64_t m, int64_t n,
                                    int64_t r, const float* s1, const float* s2,
                                    const int8_t* codes, int64_t ldc, const uint8_t* exps,
                                    int64_t lde, int64_t T, const void* dY, int32_t dtype,
                                    int64_t lddy, void* dX, int64_t lddx, float* ds1, float* ds2,
                                    void* work, void* stream) {
  if (!dtype_ok(dtype)) return bad("dtype must be NQ_F32, NQ_BF16 or NQ_F16");
  if (m < 1 || n < 1 || r < 1 || m > kMaxDim || n > kMaxDim || r > kMaxDim)
    return bad("m, n and r must be in [1, 2^21]");
  if (T < 0 || T > kMaxTuned) return bad("T must be in [0, 2^24]");
  if (T * std::max(std::max(m, n), r) > kMaxValues)
    return bad("T m, T n and T r must be <= 2^36");
  if (!ds1 || !ds2) return bad("ds1 and ds2 are required");
  hipStream_t s = (hipStream_t)stream;
  if (T == 0) {   // no tokens: the sums over them are zero
    NQ_HIPCHK(launch_zero(ds1, (size_t)m, s));
    NQ_HIPCHK(launch_zero(ds2, (size_t)n, s));
    return NQ_OK;
  }
  if (!U_bits || !Ut_bits || !V_bits || !Vt_bits || !s1 || !s2 || !dY || !work)
    return bad("U_bits, Ut_bits, V_bits, Vt_bits, s1, s2, dY and work are required");
  const int64_t rw = (r + 31) / 32, mw = (m + 31) / 32, nw = (n + 31) / 32;
  if (ldu < rw) return bad("ldu < ceil(r/32)");
  if (ldut < mw) return bad("ldut < ceil(m/32)");
  if (ldv < rw) return bad("ldv < ceil(r/32)");
  if (ldvt < nw) return bad("ldvt < ceil(n/32)");
  if (std::max(std::max(ldu, ldut), std::max(ldv, ldvt)) > kMaxWords)
    return bad("the signs' row strides must be <= 2^20 words");
  const nq_status st = check_act8(codes, ldc, exps, lde, n);
  if (st != NQ_OK) return st;
  if (lddy < m) return bad("lddy < m");
  if (dX && lddx < n) return bad("lddx < n");
  if (misaligned(dY, dtype_bytes(dtype)) || misaligned(dX, dtype_bytes(dtype)))
    return bad("dY or dX is not aligned to its type");
  if (misaligned(work, 16)) return bad("work must be 16-byte aligned");
  BinBack a{};
  a.u = U_bits; a.ut = Ut_bits; a.v = V_bits; a.vt = Vt_bits;
  a.ldu = ldu; a.ldut = ldut; a.ldv = ldv; a.ldvt = ldvt;
  a.m = m; a.n = n; a.r = r; a.T = T;
  a.s1 = s1; a.s2 = s2; a.x = Act8{codes, ldc, exps, lde};
  a.dY = dY; a.dtype = dtype; a.lddy = lddy; a.dX = dX; a.lddx = lddx;
  a.ds1 = ds1; a.ds2 = ds2; a.work = work;
  NQ_HIPCHK(launch_binback(a, s));
  return NQ_OK;
}

int64_t nq_vocab_loss_work_bytes(int64_t T, int64_t V, int64_t d, int32_t dtype, int32_t grad) {
  if (!dtype_ok(dtype) || T < 0 || V < 1 || d < 1 || T > kMaxTokens || V > kMaxVocab ||
      d > kMaxHidden || T * V > kMaxLogits)
    return -1;
  return T == 0 ? 0 : vocab_work_bytes(T, V, d, dtype, grad != 0);
}

nq_status nq_vocab_loss(const void* H, int64_t ldh, const void* W, int64_t ldw, int32_t dtype,
                        int64_t T, int64_t V, int64_t d, const int32_t* labels, float scale,
                        float* loss, float* lse, void* work, void* stream) {
  const nq_status st = check_vocab(H, ldh, W, ldw, dtype, T, V, d, labels, scale, work);
  if (st != NQ_OK || T == 0) return st;
  if (!loss || !lse) return bad("loss and lse are required");
  Vocab a{};
  a.H = H; a.W = W; a.dtype = dtype; a.ldh = ldh; a.ldw = ldw; a.T = T; a.V = V; a.d = d;
  a.labels = labels; a.scale = scale; a.loss = loss; a.lse = lse; a.work = work;
  NQ_HIPCHK(launch_vocab_loss(a, (hipStream_t)stream));
  return NQ_OK;
}

nq_status nq_vocab_loss_backward(const void* H, int64_t ldh, const void* W, int64_t ldw,
                                 int32_t dtype, int64_t T, int64_t V, int64_t d,
                                 const int32_t* labels, float scale, const float* lse,
                                 const float* dloss, void* dH, int64_t lddh, void* dW,
                                 int64_t lddw, void* work, void* stream) {
  if (T == 0 && dW && V >= 1 && d >= 1)
    return bad("T == 0: there is no gradient (dW is all zero)");
  const nq_status st = check_vocab(H, ldh, W, ldw, dtype, T, V, d, labels, scale, work);
  if (st != NQ_OK || T == 0) return st;
  if (!lse || !dloss) return bad("lse and dloss are required");
  if (!dH && !dW) return bad("dH or dW is required");
  if ((dH && lddh < d) || (dW && lddw < d)) return bad("lddh < d or lddw < d");
  if (misaligned(dH, dtype_bytes(dtype)) || misaligned(dW, dtype_bytes(dtype)))
    return bad("dH or dW is not aligned to its type");
  Vocab a{};
  a.H = H; a.W = W; a.dtype = dtype; a.ldh = ldh; a.ldw = ldw; a.T = T; a.V = V; a.d = d;
  a.labels = labels; a.scale = scale; a.lse = (float*)lse; a.dloss = dloss;
  a.dH = dH; a.lddh = lddh; a.dW = dW; a.lddw = lddw; a.work = work;
  NQ_HIPCHK(launch_vocab_loss_backward(a, (hipStream_t)stream));
  return NQ_OK;
}

int64_t nq_vocab_logprobs_work_bytes(int64_t T, int64_t V, int64_t d, int32_t dtype, int64_t G,
                                     int64_t k) {
  if (!head_ok(T, V, d, dtype) || G < 0 || k < 0 || G > vocab::kMaxListed || k > vocab::kMaxListed || k > V)
    return -1;
  return T == 0 ? 0 : logprobs_work_bytes(T, V, d, dtype, G, k);
}

nq_status nq_vocab_logprobs(const void* H, int64_t ldh, const void* W, int64_t ldw, int32_t dtype,
                            int64_t T, int64_t V, int64_t d, const int32_t* tokens, int64_t ldt,
                            int64_t G, int64_t k, float scale, float* logprobs, float* entropy,
                            float* lse, int32_t* top_ids, float* top_logprobs, void* work,
                            void* stream) {
  const nq_status st = check_head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  if (st != NQ_OK) return st;
  if (G < 0 || G > vocab::kMaxListed) return bad("G must be in [0, 128]");
  if (k < 0 || k > vocab::kMaxListed) return bad("k must be in [0, 128]");
  if (k > V) return bad("k > V");
  if (T == 0) return NQ_OK;
  if (!entropy || !lse) return bad("entropy and lse are required");
  if (G && (!tokens || !logprobs)) return bad("tokens and logprobs are required");
  if (G && (ldt < G || ldt > kMaxLd)) return bad("ldt must be in [G, 2^21]");
  if (k && (!top_ids || !top_logprobs)) return bad("top_ids and top_logprobs are required");
  if (misaligned(tokens, 4) || misaligned(logprobs, 4) || misaligned(entropy, 4) ||
      misaligned(lse, 4) || misaligned(top_ids, 4) || misaligned(top_logprobs, 4))
    return bad("tokens or an output is not aligned to its type");
  Logprobs a{};
  a.v = head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  a.tokens = tokens; a.given = G; a.ldt = ldt; a.k = k;
  a.logprobs = logprobs; a.entropy = entropy; a.lse = lse;
  a.top_ids = top_ids; a.top_logprobs = top_logprobs;
  NQ_HIPCHK(launch_vocab_logprobs(a, (hipStream_t)stream));
  return NQ_OK;
}

int64_t nq_vocab_distill_work_bytes(int64_t T, int64_t V, int64_t d, int32_t dtype, int64_t K,
                                    int32_t grad) {
  if (!head_ok(T, V, d, dtype) || K < 1 || K > vocab::kMaxListed) return -1;
  return T == 0 ? 0 : distill_work_bytes(T, V, d, dtype, K, grad != 0);
}

int64_t nq_vocab_distill_logits(int64_t T, int64_t V, int64_t d, int32_t dtype) {
  if (!head_ok(T, V, d, dtype)) return -1;
  return T > 0 && vocab::keeps(T, V, d, dtype) ? T * vocab::row_of(V) : 0;
}

nq_status nq_vocab_distill(const void* H, int64_t ldh, const void* W, int64_t ldw, int32_t dtype,
                           int64_t T, int64_t V, int64_t d, const int32_t* ids, int64_t ldi,
                           const float* logq, int64_t ldq, int64_t K, float scale, int32_t tail,
                           float* loss, float* lse, float* rest, float* hit, float* logits,
                           void* work, void* stream) {
  nq_status st = check_head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  if (st != NQ_OK || T == 0) return st;
  if ((st = check_listed(ids, ldi, logq, ldq, K)) != NQ_OK) return st;
  if (!loss || !lse || !rest || !hit) return bad("loss, lse, rest and hit are required");
  if (misaligned(loss, 4) || misaligned(lse, 4) || misaligned(rest, 4) || misaligned(hit, 4))
    return bad("an output is not aligned to its type");
  if (misaligned(logits, 16)) return bad("logits must be 16-byte aligned");
  Distill a{};
  a.v = head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  a.ids = ids; a.logq = logq; a.K = K; a.ldi = ldi; a.ldq = ldq; a.tail = tail != 0;
  a.loss = loss; a.lse = lse; a.rest = rest; a.hit = hit; a.z = logits;
  NQ_HIPCHK(launch_vocab_distill(a, (hipStream_t)stream));
  return NQ_OK;
}

nq_status nq_vocab_distill_backward(const void* H, int64_t ldh, const void* W, int64_t ldw,
                                    int32_t dtype, int64_t T, int64_t V, int64_t d,
                                    const int32_t* ids, int64_t ldi, const float* logq, int64_t ldq,
                                    int64_t K, float scale, int32_t tail, const float* lse,
                                    const float* rest, const float* hit, const float* logits,
                                    const float* dloss, void* dH, int64_t lddh, void* dW,
                                    int64_t lddw, void* work, void* stream) {
  if (T == 0 && dW && V >= 1 && d >= 1)
    return bad("T == 0: there is no gradient (dW is all zero)");
  nq_status st = check_head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  if (st != NQ_OK || T == 0) return st;
  if ((st = check_listed(ids, ldi, logq, ldq, K)) != NQ_OK) return st;
  if (!lse || !rest || !hit || !dloss) return bad("lse, rest, hit and dloss are required");
  if (!dH && !dW) return bad("dH or dW is required");
  if ((dH && lddh < d) || (dW && lddw < d)) return bad("lddh < d or lddw < d");
  if (misaligned(dH, dtype_bytes(dtype)) || misaligned(dW, dtype_bytes(dtype)))
    return bad("dH or dW is not aligned to its type");
  if (misaligned(lse, 4) || misaligned(rest, 4) || misaligned(hit, 4) || misaligned(dloss, 4))
    return bad("lse, rest, hit or dloss is not aligned to its type");
  if (misaligned(logits, 16)) return bad("logits must be 16-byte aligned");
  Distill a{};
  a.v = head(H, ldh, W, ldw, dtype, T, V, d, scale, work);
  a.v.dloss = dloss; a.v.dH = dH; a.v.lddh = lddh; a.v.dW = dW; a.v.lddw = lddw;
  a.ids = ids; a.logq = logq; a.K = K; a.ldi = ldi; a.ldq = ldq; a.tail = tail != 0;
  a.lse = (float*)lse; a.rest = (float*)rest; a.hit = (float*)hit; a.z = (float*)logits;
  NQ_HIPCHK(launch_vocab_distill_backward(a, (hipStream_t)stream));
  return NQ_OK;
}

}  // extern "C"
