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
    // v, rounded, in the place of the elements from the n-th on
    __device__ __forceinline__ void fill_from(int n, float v)
    {
        const uint32_t e = BF16 ? pack_bf16(v, v) : __builtin_bit_cast(uint32_t, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (BF16)
                w[i] = 2 * i >= n ? e : 2 * i + 1 >= n ? (w[i] & 0xffffu) | (e & 0xffff0000u) : w[i];
            else
                w[i] = i >= n ? e : w[i];
        }
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

// A thread's CH chunks of a row of d elements, chunk c from element c * STEP + t0 on, zeros
// behind the row's end.  The whole chunks' loads go first, without a branch between them.
template <bool BF16, int CH, int STEP, bool STREAM>
__device__ __forceinline__ void load_row(const void *p, int64_t off, int t0, int d, Raw<BF16> (&r)[CH])
{
    constexpr int N = kChunk<BF16>;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        r[c].fill(0.0f);
        if (c * STEP + t0 + N <= d)
            r[c].template load<STREAM>(p, off + c * STEP + t0);
    }
    if (d % N) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = c * STEP + t0;
            if (k < d && k + N > d)
                r[c].load_part(p, off + k, d - k);
        }
    }
}

// The gain's elements beside a chunk of N of the row's, as stored: 8, 16 or 32 bytes.
template <bool BF16, int N>
struct Gain {
    static constexpr int WORDS = N * (BF16 ? 2 : 4) / 4, V = WORDS < 4 ? WORDS : 4;
    typedef uint32_t vec_t __attribute__((ext_vector_type(V)));
    typedef vec_t vec_any __attribute__((aligned(2)));
    vec_t w[WORDS / V];

    __device__ __forceinline__ void load(const void *p, int k, int d)
    {
#pragma unroll
        for (int i = 0; i < WORDS / V; ++i) {
            w[i] = (vec_t)(0u);
            if (k + N <= d)
                w[i] = ((const vec_any *)((const char *)p + (int64_t)k * (BF16 ? 2 : 4)))[i];
        }
    }
    // the chunk that the row's end cuts: its first n elements
    __device__ __forceinline__ void load_part(const void *p, int k, int n)
    {
#pragma unroll
        for (int i = 0; i < N - 1; ++i) {
            if (i >= n)
                continue;
            if constexpr (BF16)
                w[i / 2 / V][i / 2 % V] |= (uint32_t)((const uint16_t *)p)[k + i] << (16 * (i % 2));
            else
                w[i / V][i % V] = ((const uint32_t *)p)[k + i];
        }
    }
    // keeps the elements packed up to here (as Raw::opaque does)
    __device__ __forceinline__ void opaque()
    {
#pragma unroll
        for (int i = 0; i < WORDS / V; ++i)
            asm volatile("" : "+v"(w[i]));
    }
    __device__ __forceinline__ float get(int i) const
    {
        const uint32_t e = BF16 ? w[i / 2 / V][i / 2 % V] : w[i / V % (WORDS / V)][i % V];
        if constexpr (BF16)
            return i % 2 ? bf16_hi(e) : bf16_lo(e);
        else
            return __builtin_bit_cast(float, e);
    }
};

// Reduction over the LPR threads of a row: lanes of a wave, or a workgroup's waves.
template <int LPR, typename Op>
__device__ __forceinline__ float row_reduce(float v, Op op, float *red)
{
    if constexpr (LPR > 64)
        return block_reduce<LPR / 64>(v, op, red);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1)
        v = op(v, __shfl_xor(v, o, 64));
    return v;
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
