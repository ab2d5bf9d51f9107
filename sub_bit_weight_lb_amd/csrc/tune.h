// Internal declarations of the kernels that tune a packed model: 8-bit
// activation checkpoints (act8.hip), the gradient of a packed layer
// (binback.hip) and the loss over a large vocabulary (vocab.hip).
#pragma once

#include "common.h"

namespace nq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// (the device's own min and max take two 64-bit integers of different
// spellings to double)
__device__ __forceinline__ int64_t lmin(int64_t a, int64_t b) { return a < b ? a : b; }
__device__ __forceinline__ int64_t lmax(int64_t a, int64_t b) { return a > b ? a : b; }

// A uniform value in a scalar register, for operands of inline assembly: read
// from a vector register that the compiler cannot see through (it drops a
// v_readfirstlane of what it knows to be uniform, and may then hand the assembly
// a vector register).
__device__ __forceinline__ int scalar(int x) {
  asm("" : "+v"(x));
  return __builtin_amdgcn_readfirstlane(x);
}

// One element of type D as the caller stores it, and its conversions; from()
// rounds to nearest even.
template <int D> struct Elem;
template <> struct Elem<kF32> {
  typedef float type;
  static __device__ __forceinline__ float to(float x) { return x; }
  static __device__ __forceinline__ float from(float x) { return x; }
};
template <> struct Elem<kBF16> {
  typedef uint16_t type;
  static __device__ __forceinline__ float to(uint16_t x) {
    return __uint_as_float((uint32_t)x << 16);
  }
  static __device__ __forceinline__ uint16_t from(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
  }
};
template <> struct Elem<kF16> {
  typedef _Float16 type;
  static __device__ __forceinline__ float to(_Float16 x) { return (float)x; }
  static __device__ __forceinline__ _Float16 from(float x) { return (_Float16)x; }
};

// Columns that share one exponent of an 8-bit checkpoint.
constexpr int kActGroup = 32;

// An 8-bit checkpoint of rows x cols activations on the device: codes (row
// stride ldc bytes) and, per row, ceil(cols / 32) biased exponents (row
// stride lde): value = code * 2^(exponent - 127), NaN where it is 255.
struct Act8 {
  const int8_t* codes;
  int64_t ldc;
  const uint8_t* exps;
  int64_t lde;
};
// 2^(e - 127) for a stored exponent (1 .. 254), NaN for 255. (0, which no
// quantiser writes, gives 0.)
__device__ __forceinline__ float act8_step(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e << 23);
}

hipError_t launch_act8_quantize(const void* X, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                                int8_t* codes, int64_t ldc, uint8_t* exps, int64_t lde,
                                hipStream_t s);
hipError_t launch_act8_dequantize(const Act8& q, int64_t rows, int64_t cols, void* X, int dtype,
                                  int64_t ldx, hipStream_t s);
hipError_t launch_act8_steps(const uint8_t* exps, int64_t lde, int64_t rows, int64_t groups,
                             float* steps, int64_t lds, hipStream_t s);

// ---------------------------------------------------------------- packed layer's gradient (binback.hip)
// Y = X^ W^T for W = diag(s1) S_U S_V^T diag(s2) and the checkpoint X^ of
// T x n inputs; dY = dL/dY (T x m). Writes dX (T x n, dY's type, nullable),
// ds1 (m), ds2 (n).
struct BinBack {
  const uint32_t *u, *ut, *v, *vt;   // signs: m x r, r x m, n x r, r x n
  int64_t ldu, ldut, ldv, ldvt;      // their row strides in words
  int64_t m, n, r, T;
  const float *s1, *s2;
  Act8 x;
  const void* dY;
  int dtype;                         // of dY and dX
  int64_t lddy;
  void* dX;
  int64_t lddx;
  float *ds1, *ds2;
  void* work;                        // binback_work_bytes, 16-byte aligned
};
int64_t binback_work_bytes(int64_t m, int64_t n, int64_t r, int64_t T);
hipError_t launch_binback(const BinBack& a, hipStream_t s);

// ---------------------------------------------------------------- loss over a vocabulary (vocab.hip)
struct Vocab {
  const void *H, *W;                 // T x d and V x d, of type dtype
  int dtype;
  int64_t ldh, ldw, T, V, d;
  const int32_t* labels;             // T; negative: ignored
  float scale;                       // logits = scale H W^T
  float *loss, *lse;                 // T each; lse is read by the gradient
  const float* dloss;                // T (gradient)
  void *dH, *dW;                     // T x d, V x d (gradient; either nullable)
  int64_t lddh, lddw;
  void* work;                        // vocab_work_bytes, 16-byte aligned
  // a gradient whose G is exp(z - lse) share dloss scale, but val dloss scale at the
  // `listed` words of each token (0: none; a negative one: no entry); |G| <= wr dloss scale, wr: T,
  // overwritten
  const float* share;
  float* wr;
  const int32_t* ids;
  int64_t listed, ldi;
  const float* val;                  // T x listed
  const float* z;                    // nullable: the logits, ldz apart
  int64_t ldz;
};
int64_t vocab_work_bytes(int64_t T, int64_t V, int64_t d, int dtype, bool grad);
hipError_t launch_vocab_loss(const Vocab& a, hipStream_t s);
hipError_t launch_vocab_loss_backward(const Vocab& a, hipStream_t s);

// ---------------------------------------------------------------- single logits (vocab_top.hip)
struct Logprobs {
  Vocab v;                           // H, W, sizes, scale, work
  const int32_t* tokens;             // T x given, ldt apart; negative: none
  int64_t given, ldt, k;
  float *logprobs, *entropy, *lse;   // T x given, T, T
  int32_t* top_ids;                  // T x k
  float* top_logprobs;
};
struct Distill {
  Vocab v;                           // H, W, sizes, scale, dloss, dH, dW, work
  const int32_t* ids;                // T x K, ldi apart; negative: no entry
  const float* logq;                 // T x K, ldq apart
  int64_t K, ldi, ldq;
  int tail;
  float *loss, *lse, *rest, *hit;    // T, T, T, T x K; but for loss read by the gradient
  float* z;                          // T x (V to 128), nullable: logits that are kept for it
};
// few tokens' gradient: z, G (T rows of FewPlan's ldz), part: FewPlan's; labels: T, scratch
struct Few {
  Distill a;
  const float* z;
  float *G, *part;
  int32_t* labels;
};
hipError_t launch_few_gradient(const Few& a, hipStream_t s);
int64_t logprobs_work_bytes(int64_t T, int64_t V, int64_t d, int dtype, int64_t given, int64_t k);
int64_t distill_work_bytes(int64_t T, int64_t V, int64_t d, int dtype, int64_t K, bool grad);
hipError_t launch_vocab_logprobs(const Logprobs& a, hipStream_t s);
hipError_t launch_vocab_distill(const Distill& a, hipStream_t s);
hipError_t launch_vocab_distill_backward(const Distill& a, hipStream_t s);

}  // namespace nq
