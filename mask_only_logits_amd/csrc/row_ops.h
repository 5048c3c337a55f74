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

// Rows may start at any element, so the vector types are aligned to one: gfx950 takes the
// same 16-byte loads and stores at any address, at full rate where it is aligned.
typedef u32x4_t u32x4_any __attribute__((aligned(2)));

template <bool NT>
__device__ __forceinline__ u32x4_t get16(const u32x4_any *p)
{
    if constexpr (NT)
        return __builtin_nontemporal_load(p);
    else
        return *p;
}

template <bool NT>
__device__ __forceinline__ void put16(u32x4_any *p, const u32x4_t &w)
{
    if constexpr (NT)
        __builtin_nontemporal_store(w, p);
    else
        *p = w;
}

// Eight elements as they are stored: 16 bytes (bf16) or 32 (fp32).
template <bool BF16>
struct Raw8 {
    u32x4_t w[BF16 ? 1 : 2];

    // NT: with the streaming cache policy, for data that is read once
    template <bool NT = false>
    __device__ __forceinline__ void load(const void *p, int64_t off)
    {
        if constexpr (BF16) {
            w[0] = get16<NT>((const u32x4_any *)((const uint16_t *)p + off));
        } else {
            w[0] = get16<NT>((const u32x4_any *)((const float *)p + off));
            w[1] = get16<NT>((const u32x4_any *)((const float *)p + off + 4));
        }
    }
    __device__ __forceinline__ void get(float (&x)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16) {
                x[2 * i] = bf16_lo(w[0][i]);
                x[2 * i + 1] = bf16_hi(w[0][i]);
            } else {
                // (copies: a bit cast of a vector's element itself takes its first one)
                const uint32_t lo = w[0][i], hi = w[1][i];
                x[i] = __builtin_bit_cast(float, lo);
                x[4 + i] = __builtin_bit_cast(float, hi);
            }
        }
    }
    __device__ __forceinline__ void fill(float v)
    {
        const uint32_t b = __builtin_bit_cast(uint32_t, v), f = BF16 ? (b & 0xffff0000u) | (b >> 16) : b;
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            w[i] = u32x4_t{f, f, f, f};
    }
    // Keeps the compiler from carrying the unpacked floats of an earlier use past this point:
    // rows held in registers are held as they are stored.
    __device__ __forceinline__ void opaque()
    {
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i)
            asm volatile("" : "+v"(w[i]));
    }
    // the first n < 8 elements (n >= 1), the rest left as they are
    __device__ __forceinline__ void load_part(const void *p, int64_t off, int n)
    {
#pragma unroll
        for (int i = 0; i < 7; ++i) {
            if (i >= n)
                continue;
            if constexpr (BF16) {
                const uint32_t e = ((const uint16_t *)p)[off + i];
                w[0][i >> 1] = i & 1 ? (w[0][i >> 1] & 0xffffu) | (e << 16) : (w[0][i >> 1] & 0xffff0000u) | e;
            } else {
                w[i >> 2][i & 3] = ((const uint32_t *)p)[off + i];
            }
        }
    }
};

__device__ __forceinline__ float load1(const void *p, int64_t off, bool bf16)
{
    return bf16 ? bf16_lo(((const uint16_t *)p)[off]) : ((const float *)p)[off];
}

template <bool BF16>
__device__ __forceinline__ void store1(void *p, int64_t off, float x)
{
    if constexpr (BF16)
        ((__bf16 *)p)[off] = static_cast<__bf16>(x);
    else
        ((float *)p)[off] = x;
}

// Eight results; bf16 values are rounded to nearest even here.  NT: streaming cache policy.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void store8(void *p, int64_t off, const float (&x)[8])
{
    if constexpr (BF16) {
        put16<NT>((u32x4_any *)((uint16_t *)p + off), u32x4_t{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])});
    } else {
        u32x4_t w[2];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i >> 2][i & 3] = __builtin_bit_cast(uint32_t, x[i]);
        put16<NT>((u32x4_any *)((float *)p + off), w[0]);
        put16<NT>((u32x4_any *)((float *)p + off + 4), w[1]);
    }
}

// The first n of eight results.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void store_upto(void *p, int64_t off, const float (&x)[8], int n)
{
    if (n >= 8)
        return store8<BF16, NT>(p, off, x);
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < n)
            store1<BF16>(p, off + i, x[i]);
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
