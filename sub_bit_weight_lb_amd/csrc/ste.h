// Launches of the STE refinement's kernels (ste.hip), for ste.cpp.
#pragma once

#include "tune.h"

namespace nq {

// The batch's inputs as float32 rows; an 8-bit checkpoint of them is an Act8.
struct SteFloat {
  const float* X;
  int64_t ldx;
};

hipError_t launch_ste_signs(const float* F, int64_t rows, int64_t r, int64_t rp, int64_t rows_pad,
                            float* S, float* St, hipStream_t s);
template <class Src>
hipError_t launch_ste_stage(const Src& X, const int32_t* idx, int64_t T, int64_t n,
                            const float* s2, int64_t np_, int64_t tp, float* A, float* At,
                            hipStream_t s);
hipError_t launch_ste_loss(const float* Q, const float* Y, int64_t ldy, const int32_t* idx,
                           int64_t T, int64_t m, const float* s1, int64_t mp, int64_t tp,
                           float* dQ, float* dQt, float* ds1p, double* lossp, float* ds1,
                           double* loss, hipStream_t s);
template <class Src>
hipError_t launch_ste_ds2(const float* dA, const Src& X, const int32_t* idx, int64_t T, int64_t n,
                          int64_t np_, int64_t tp, float* ds2p, float* ds2, hipStream_t s);
hipError_t launch_ste_adam(float* p, const float* g, float* m, float* v, int64_t rows,
                           int64_t cols, int64_t ld, float lr, float b1, float b2, float c1,
                           float c2, float eps, hipStream_t s);

}  // namespace nq
