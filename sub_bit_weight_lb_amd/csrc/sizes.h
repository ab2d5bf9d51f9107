// Element types and sizes that host code without HIP shares with the kernels.
#pragma once

#include <stdint.h>

namespace nq {

inline int64_t round_up(int64_t x, int64_t q) { return (x + q - 1) / q * q; }

// Element types of caller tensors (nq_dtype in include/nq.h).
enum DType : int { kF32 = 0, kBF16 = 1, kF16 = 2 };
inline int64_t dtype_bytes(int t) { return t == kF32 ? 4 : 2; }

}  // namespace nq
