// Device helpers of the row kernels (norm, quantization, distillation): wave and workgroup
// reductions, 16-byte loads and stores of elements, and row counts read from device memory.
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

// Elements of a chunk: what one 16-byte access holds.
template <bool BF16>
constexpr int kChunk = BF16 ? 8 : 4;

// A chunk as it is stored.
template <bool BF16>
struct Raw {
    static constexpr int N = kChunk<BF16>;
    u32x4_t w;

    // NT: with the streaming cache policy, for data that is read once
    template <bool NT = false>
    __device__ __forceinline__ void load(const void *p, int64_t off)
    {
        w = get16<NT>((const u32x4_any *)((const char *)p + off * (BF16 ? 2 : 4)));
    }
    __device__ __forceinline__ void get(float (&x)[N]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = w[i];   // (a copy: a bit cast of a vector's element takes its first one)
            if constexpr (BF16) {
                x[2 * i] = bf16_lo(e);
                x[2 * i + 1] = bf16_hi(e);
            } else {
                x[i] = __builtin_bit_cast(float, e);
            }
        }
    }
    __device__ __forceinline__ void fill(float v)
    {
        const uint32_t b = __builtin_bit_cast(uint32_t, v), f = BF16 ? (b & 0xffff0000u) | (b >> 16) : b;
        w = u32x4_t{f, f, f, f};
    }
    // Keeps the compiler from carrying the unpacked floats of an earlier use past this point:
    // rows held in registers are held as they are stored.
    __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(w)); }
    // the first n < N elements (n >= 1), the rest left as they are
    __device__ __forceinline__ void load_part(const void *p, int64_t off, int n)
    {
#pragma unroll
        for (int i = 0; i < N - 1; ++i) {
            if (i >= n)
                continue;
            if constexpr (BF16) {
                const uint32_t e = ((const uint16_t *)p)[off + i];
                w[i >> 1] = i & 1 ? (w[i >> 1] & 0xffffu) | (e << 16) : (w[i >> 1] & 0xffff0000u) | e;
            } else {
                w[i] = ((const uint32_t *)p)[off + i];
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

// A chunk of results; bf16 values are rounded to nearest even here.  NT: streaming cache policy.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void store(void *p, int64_t off, const float (&x)[kChunk<BF16>])
{
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (BF16)
            w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
        else
            w[i] = __builtin_bit_cast(uint32_t, x[i]);
    }
    put16<NT>((u32x4_any *)((char *)p + off * (BF16 ? 2 : 4)), w);
}

// The first n results of a chunk.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void store_upto(void *p, int64_t off, const float (&x)[kChunk<BF16>], int n)
{
    if (n >= kChunk<BF16>)
        return store<BF16, NT>(p, off, x);
#pragma unroll
    for (int i = 0; i < kChunk<BF16> - 1; ++i)
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
