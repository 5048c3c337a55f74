// Device helpers of the row kernels (norm, quantization, distillation): wave and workgroup
// reductions, 16-byte element loads and stores, and row counts read from device memory.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mosaic {
namespace rows {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct AddOp {
    __device__ __forceinline__ static float id() { return 0.0f; }
    __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// Maximum that ignores NaN (a NaN shows up in the sums taken beside it).
struct MaxOp {
    __device__ __forceinline__ static float id() { return -__builtin_inff(); }
    __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
// Maximum of non-negative values by their bits: a NaN counts above infinity and stays.
struct MaxBitsOp {
    __device__ __forceinline__ static float id() { return 0.0f; }
    __device__ __forceinline__ float operator()(float a, float b) const
    {
        const uint32_t x = __builtin_bit_cast(uint32_t, a), y = __builtin_bit_cast(uint32_t, b);
        return __builtin_bit_cast(float, x > y ? x : y);
    }
};

template <typename Op>
__device__ __forceinline__ float wave_reduce(float v, Op op)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1)
        v = op(v, __shfl_xor(v, o, 64));
    return v;
}

// Reduction over a workgroup of NW waves, the result in every thread.  `red` holds NW floats
// and is free again for the next call (both barriers are inside).  The waves' values are
// combined in wave order, so the result does not depend on timing.
template <int NW, typename Op>
__device__ __forceinline__ float block_reduce(float v, Op op, float *red)
{
    v = wave_reduce(v, op);
    if constexpr (NW == 1)
        return v;
    if ((threadIdx.x & 63) == 0)
        red[threadIdx.x >> 6] = v;
    __syncthreads();
    float r = red[0];
#pragma unroll
    for (int w = 1; w < NW; ++w)
        r = op(r, red[w]);
    __syncthreads();
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }

// two floats to a pair of bf16 (round to nearest even)
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __bf16 a = static_cast<__bf16>(lo), b = static_cast<__bf16>(hi);
    return (uint32_t)__builtin_bit_cast(uint16_t, a) | ((uint32_t)__builtin_bit_cast(uint16_t, b) << 16);
}

// VEC elements from element offset off: VEC == 8 with 16-byte loads (off a multiple of 8,
// base 16-byte aligned), VEC == 1 with one element's load.
template <bool BF16, int VEC>
__device__ __forceinline__ void load(const void *p, int64_t off, float (&x)[VEC])
{
    if constexpr (VEC == 8) {
        if constexpr (BF16) {
            const u32x4_t w = *(const u32x4_t *)((const uint16_t *)p + off);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = bf16_lo(w[i]);
                x[2 * i + 1] = bf16_hi(w[i]);
            }
        } else {
            const f32x4_t a = *(const f32x4_t *)((const float *)p + off);
            const f32x4_t b = *(const f32x4_t *)((const float *)p + off + 4);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[i] = a[i];
                x[4 + i] = b[i];
            }
        }
    } else {
        static_assert(VEC == 1, "one element or eight");
        if constexpr (BF16)
            x[0] = bf16_lo(((const uint16_t *)p)[off]);
        else
            x[0] = ((const float *)p)[off];
    }
}

// The same for a store; bf16 values are rounded to nearest even here.
template <bool BF16, int VEC>
__device__ __forceinline__ void store(void *p, int64_t off, const float (&x)[VEC])
{
    if constexpr (VEC == 8) {
        if constexpr (BF16) {
            *(u32x4_t *)((uint16_t *)p + off) = u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                        pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
        } else {
            *(f32x4_t *)((float *)p + off) = f32x4_t{x[0], x[1], x[2], x[3]};
            *(f32x4_t *)((float *)p + off + 4) = f32x4_t{x[4], x[5], x[6], x[7]};
        }
    } else {
        if constexpr (BF16)
            ((__bf16 *)p)[off] = static_cast<__bf16>(x[0]);
        else
            ((float *)p)[off] = x[0];
    }
}

// rows, or min(max(*count, 0), rows) where a device-side count is given.
__device__ __forceinline__ int64_t row_count(const int32_t *count, int64_t rows)
{
    if (!count)
        return rows;
    const int64_t n = *count;
    return n < 0 ? 0 : (n < rows ? n : rows);
}

}  // namespace rows
}  // namespace mosaic
