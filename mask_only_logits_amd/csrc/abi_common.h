// What the C ABI's source files share: size and alignment checks, chunk sizes, and the debug
// check of the index lists.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/mosaic.h"

namespace mosaic {
namespace abi {

constexpr int64_t kMaxPos = 0x7fffffffLL;   // positions and rows are int32

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

// ceil(a / b) for a >= 0, b > 0, without the overflow of (a + b - 1) / b near INT64_MAX.
inline int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

inline int64_t esize_of(mosaic_dtype_t t) { return t == MOSAIC_F32 ? 4 : (t == MOSAIC_BF16 ? 2 : 0); }

// M * V * esize without int64 overflow; -1 on overflow.
inline int64_t checked_bytes(int64_t rows, int64_t V, int64_t esize)
{
    if (rows < 0 || V < 0 || esize <= 0)
        return -1;
    if (rows != 0 && V > INT64_MAX / rows)
        return -1;
    const int64_t n = rows * V;
    if (n != 0 && esize > INT64_MAX / n)
        return -1;
    return n * esize;
}

// MOSAIC_CHECK_IDX=1: checks on the device that every idx[i] (i < M) lies in [0, L), and waits
// for the answer (defined in mosaic_abi.cpp).
mosaic_status_t check_idx_if_asked(const int32_t *idx, int64_t M, int64_t L, hipStream_t stream);

}  // namespace abi
}  // namespace mosaic
