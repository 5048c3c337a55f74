// Residual addition with root-mean-square norm, and 8-bit row codes.
//
// For a row of d elements, with x the layer's output and r the residual stream:
//   s = x + r,   y_k = s_k * g_k / sqrt(mean_k(s_k^2) + eps),
//   amax = max_k |y_k|,  scale = amax / top,  q_k = RNE(y_k * (top / amax)),
// top = 448 for E4M3 codes and 127 for INT8 codes; a row of zeros has zero codes and
// scale 0.  Sums, the norm and the scale are fp32; s, y and q are each rounded once, from
// the unrounded fp32 value of the one before (rounding s to bf16 first would move y by up
// to half a bf16 step, 2^-9 of its value, for nothing: s is in registers).  The INT8
// quantization of plain rows is the same kernel without the norm.
//
// Rows are gathered through a list of row ids where one is given: the LM head needs the
// final norm of the masked rows only.
//
// One pass: a row's elements stay in registers from the loads to the last store, so each
// input is read once and each output written once, and HBM is what bounds the kernel.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch_ops.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

// |x| as MaxBitsOp takes it
__device__ __forceinline__ float abs_bits(float x)
{
    return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0x7fffffffu);
}

// Codes of N = 4 or 8 values already multiplied by top / amax (|y| <= top up to fp32 rounding).
// INT8: adding 1.5 * 2^23 leaves the nearest even integer in the sum's low bits.  E4M3:
// v_cvt_pk_fp8_f32 rounds to nearest even, and 448 (1 + 2^-23) is still 448.
template <int N>
__device__ __forceinline__ void make_codes(const float (&y)[N], bool int8, uint32_t (&w)[N / 4])
{
#pragma clang fp contract(off)   // y * inv rounds before the addition
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        if (int8) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                b[e] = __builtin_bit_cast(uint32_t, y[4 * i + e] + 12582912.0f);
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
            const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u);
            w[i] = lo | (hi << 16);
        } else {
            const int p = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
            w[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], p, true);
        }
    }
}

// The first n of N codes, at any byte.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *q, const uint32_t (&w)[N / 4], int n)
{
    if (n >= N) {
        __builtin_memcpy(q, w, N);
        return;
    }
#pragma unroll
    for (int i = 0; i < N - 1; ++i)
        if (i < n)
            q[i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
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

// Power of two that keeps top / amax inside fp32 for the smallest rows (1 for all others).
__device__ __forceinline__ float code_lift(float amax) { return amax < 0x1p-100f ? 0x1p100f : 1.0f; }

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

// LPR threads per row, a thread holding CH chunks of 16 bytes (d <= LPR CH kChunk): lanes of a
// wave, which then has 64 / LPR rows, or whole waves.
// NORM off: y = x (plain quantization).  STREAM: streaming cache policy.
// Bound: HBM.  32768 x 4096 bf16 with residual, sum, out and codes moves 1.21 GB in 185 us, 6.5
// TB/s (a large copy runs at 4.75); 1229 gathered rows to codes alone take 8.5 us, where the
// chain of row id, row, two reductions and store counts.
template <bool BF16, bool GAIN_BF16, bool NORM, int LPR, int CH, bool STREAM>
__global__ __launch_bounds__(LPR <= 64 ? 256 : LPR) void rows_norm_kernel(const RowsNorm a)
{
    constexpr int RPB = LPR <= 64 ? 256 / LPR : 1;   // rows per workgroup
    constexpr int N = kChunk<BF16>, STEP = LPR * N;
    __shared__ float red[LPR <= 64 ? 1 : LPR / 64];
    const int t = threadIdx.x % LPR;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < n; row += (int64_t)gridDim.x * RPB) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;   // a row id outside gives a row of NaN
        float v[CH][N];
        Raw<BF16> x[CH], r[CH];
        Gain<GAIN_BF16, N> gain[CH];   // taken with the row, not after its reduction
        if (inside) {
            load_row<BF16, CH, STEP, STREAM>(a.X, src * a.ldx, t * N, a.d, x);
            if (NORM && a.R)
                load_row<BF16, CH, STEP, STREAM>(a.R, src * a.ldr, t * N, a.d, r);
        }
        if (NORM) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                gain[c].load(a.gain, c * STEP + t * N, a.d);
            if (a.d % N) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int k = c * STEP + t * N;
                    if (k < a.d && k + N > a.d)
                        gain[c].load_part(a.gain, k, a.d - k);
                }
            }
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (!inside)
                x[c].fill(__builtin_nanf(""));
            x[c].get(v[c]);
            if (NORM && a.R && inside) {
                float y[N];
                r[c].get(y);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[c][i] += y[i];
            }
        }
        if constexpr (NORM) {
            if (a.sum) {
#pragma unroll
                for (int c = 0; c < CH; ++c) {
                    const int k = c * STEP + t * N;
                    if (k < a.d)
                        store_upto<BF16, STREAM>(a.sum, row * a.ldsum + k, v[c], a.d - k);
                }
            }
            float ss = 0.0f;
#pragma unroll
            for (int c = 0; c < CH; ++c)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    ss += v[c][i] * v[c][i];
            ss = row_reduce<LPR>(ss, AddOp{}, red);
            float rstd = 1.0f / sqrtf(ss / (float)a.d + a.eps);
            if (rstd == 0.0f) {
                // the squares of finite values, or eps beside them, passed fp32's range: take all
                // of it 2^-160 smaller, eps too (2^128 and d < 2^31 terms then stay inside)
                constexpr float down = 0x1p-80f;
                float s2 = 0.0f;
#pragma unroll
                for (int c = 0; c < CH; ++c)
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        s2 += (v[c][i] * down) * (v[c][i] * down);
                s2 = row_reduce<LPR>(s2, AddOp{}, red);
                rstd = 1.0f / sqrtf(s2 / (float)a.d + a.eps_low) * down;
            }
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = c * STEP + t * N;
                gain[c].opaque();
                if (k < a.d) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        v[c][i] = v[c][i] * rstd * gain[c].get(i);
                    if (a.out)
                        store_upto<BF16, STREAM>(a.out, row * a.d + k, v[c], a.d - k);
                }
            }
            if (!a.q)
                continue;
        }
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i)
                amax = MaxBitsOp{}(amax, abs_bits(v[c][i]));
        amax = row_reduce<LPR>(amax, MaxBitsOp{}, red);
        const float top = a.code_int8 ? 127.0f : 448.0f;
        // a row with a NaN or an infinity has zero codes and that scale, so that what is
        // computed from it is not finite either
        const bool fine = amax > 0.0f && amax < __builtin_inff();
        const float up = code_lift(amax), inv = fine ? top / (amax * up) : 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = c * STEP + t * N;
            if (k < a.d) {
                float y[N];
#pragma unroll
                for (int i = 0; i < N; ++i)
                    y[i] = fine ? v[c][i] * up * inv : 0.0f;
                uint32_t w[N / 4];
                make_codes(y, a.code_int8, w);
                store_codes<N>(a.q + row * a.d + k, w, a.d - k);
            }
        }
        if (t == 0)
            a.scale[row] = amax / top;
    }
}

// Rows too long for the registers: the row is read again for each of the three passes (sum
// of squares, maximum, results), from L2 after the first.  `sum` is written in the last pass,
// each element by the thread that has read it for the last time, so that it may be X or R.
// A thread adds up to 2^20 squares: in 64 bits, since in fp32 equal squares, whose additions all
// round the same way, would take the row off by 114 half steps at d = 2^20, by 551 at 2^24.
template <bool BF16, bool NORM>
__global__ __launch_bounds__(1024) void rows_norm_long_kernel(const RowsNorm a)
{
    __shared__ float red[16];
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;
        auto element = [&](int k) {
            if (!inside)
                return __builtin_nanf("");
            const float x = load1(a.X, src * a.ldx + k, BF16);
            return NORM && a.R ? x + load1(a.R, src * a.ldr + k, BF16) : x;
        };
        float rstd = 1.0f;
        if constexpr (NORM) {
            double sum = 0.0;
            for (int k = threadIdx.x; k < a.d; k += 1024) {
                const float x = element(k);
                sum += (double)(x * x);
            }
            const float ss = block_reduce<16>((float)sum, AddOp{}, red);
            rstd = 1.0f / sqrtf(ss / (float)a.d + a.eps);
            if (rstd == 0.0f) {   // as in rows_norm_kernel
                constexpr float down = 0x1p-80f;
                sum = 0.0;
                for (int k = threadIdx.x; k < a.d; k += 1024) {
                    const float x = element(k) * down;
                    sum += (double)(x * x);
                }
                const float s2 = block_reduce<16>((float)sum, AddOp{}, red);
                rstd = 1.0f / sqrtf(s2 / (float)a.d + a.eps_low) * down;
            }
        }
        auto normed = [&](float x, int k) { return NORM ? x * rstd * load1(a.gain, k, a.gain_bf16) : x; };
        float amax = 0.0f;
        if (a.q) {
            for (int k = threadIdx.x; k < a.d; k += 1024)
                amax = MaxBitsOp{}(amax, abs_bits(normed(element(k), k)));
            amax = block_reduce<16>(amax, MaxBitsOp{}, red);
        }
        const float top = a.code_int8 ? 127.0f : 448.0f;
        const bool fine = amax > 0.0f && amax < __builtin_inff();
        const float up = code_lift(amax), inv = fine ? top / (amax * up) : 0.0f;
        for (int k = threadIdx.x; k < a.d; k += 1024) {
            const float x = element(k), y = normed(x, k);
            if (NORM && a.sum)
                store1<BF16>(a.sum, row * a.ldsum + k, x);
            if (NORM && a.out)
                store1<BF16>(a.out, row * a.d + k, y);
            if (a.q) {
                const float z[4] = {fine ? y * up * inv : 0.0f};
                uint32_t w[1];
                make_codes(z, a.code_int8, w);
                a.q[row * a.d + k] = (uint8_t)w[0];
            }
        }
        if (a.q && threadIdx.x == 0)
            a.scale[row] = amax / top;
    }
}

// Workgroups of a launch: one for each row (or 4 to 32), and no more than 2^20, over which the
// kernels walk: a launch holds at most 2^32 - 1 threads.
unsigned grid_of(int64_t rows, int per_block)
{
    return (unsigned)std::min<int64_t>((rows + per_block - 1) / per_block, 1 << 20);
}

// Rows that pass the 256 MB Infinity Cache by far are read and written with the streaming cache
// policy: bf16, d = 4096, residual, sum, out and codes, 32768 rows (1.2 GB): 187 against 211 us,
// 16384 rows: 93 against 106 us; 8192 rows (0.3 GB) run alike, and what reads their results
// next finds them in the cache.
bool is_large(const RowsNorm &a, int64_t esize)
{
    const int64_t streams = 1 + (a.R != nullptr) + (a.sum != nullptr) + (a.out != nullptr);
    return streams * a.rows * a.d * esize >= (int64_t)512 << 20;
}

// CH: chunks of eight elements per thread
template <bool BF16, bool NORM, int LPR, int CH>
void run(const RowsNorm &a, hipStream_t stream)
{
    constexpr int C = CH * 8 / kChunk<BF16>;
    const dim3 grid(grid_of(a.rows, LPR <= 64 ? 256 / LPR : 1)), block(LPR <= 64 ? 256 : LPR);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    if (NORM && is_large(a, BF16 ? 2 : 4))
        a.gain_bf16 ? go(rows_norm_kernel<BF16, true, NORM, LPR, C, NORM>)
                    : go(rows_norm_kernel<BF16, false, NORM, LPR, C, NORM>);
    else
        a.gain_bf16 || !NORM ? go(rows_norm_kernel<BF16, true, NORM, LPR, C, false>)
                             : go(rows_norm_kernel<BF16, !NORM, NORM, LPR, C, false>);
}

// Threads per row and chunks per thread, by the row's length: enough threads for the row to
// finish soon, few enough that several rows share a wave or a CU and one's reductions lie under
// the others' reads (bf16, residual, sum, out and codes: 16384 x 8192: 182 us with 512 threads,
// 285 us with 1024; 32768 x 4096: 187 us with 256, 238 us with 512; 131072 x 127: 54 us with 16,
// 148 us with 64; 131072 x 64: 14 us with 8, 63 us with 64).  Three chunks where two would leave
// many threads without one (bf16: 131072 x 260: 79 us with 16 threads, 139 us with 64; 131072 x
// 700: 173 us with 32, 198 us with 64; 32768 x 1100: 85 us with 64, 98 us with 128; 32768 x 2500:
// 152 us with 128, 175 us with 256; 32768 x 4097: 265 us with 256, 286 us with 512; but 32768 x
// 3000: 153 us with 128, 146 us with 256); in fp32, whose chunks of eight are two loads, only the
// last of these gains (381 against 407 us).
template <bool BF16, bool NORM>
void pick(const RowsNorm &a, hipStream_t stream)
{
    if (a.d <= 64)
        return run<BF16, NORM, 8, 1>(a, stream);
    if (a.d <= 128)
        return run<BF16, NORM, 16, 1>(a, stream);
    if constexpr (BF16) {
        if (a.d <= 192)
            return run<BF16, NORM, 8, 3>(a, stream);
        if (a.d > 256 && a.d <= 384)
            return run<BF16, NORM, 16, 3>(a, stream);
        if (a.d > 512 && a.d <= 768)
            return run<BF16, NORM, 32, 3>(a, stream);
        if (a.d > 1024 && a.d <= 1536)
            return run<BF16, NORM, 64, 3>(a, stream);
        if (a.d > 2048 && a.d <= 2560)
            return run<BF16, NORM, 128, 3>(a, stream);
    }
    if (a.d <= 256)
        return run<BF16, NORM, 32, 1>(a, stream);
    if (a.d <= 512)
        return run<BF16, NORM, 64, 1>(a, stream);
    if (a.d <= 1024)
        return run<BF16, NORM, 64, 2>(a, stream);
    if (a.d <= 2048)
        return run<BF16, NORM, 128, 2>(a, stream);
    if (a.d <= 4096)
        return run<BF16, NORM, 256, 2>(a, stream);
    if (a.d <= 6144)
        return run<BF16, NORM, 256, 3>(a, stream);
    if (a.d <= 8192)
        return run<BF16, NORM, 512, 2>(a, stream);
    if (a.d <= 16384)
        return run<BF16, NORM, 512, 4>(a, stream);
    hipLaunchKernelGGL((rows_norm_long_kernel<BF16, NORM>), dim3(grid_of(a.rows, 1)), dim3(1024), 0, stream, a);
}

}  // namespace

hipError_t launch_rows_norm(const RowsNorm &a, bool in_bf16, bool norm, hipStream_t stream)
{
    if (in_bf16)
        norm ? pick<true, true>(a, stream) : pick<true, false>(a, stream);
    else
        norm ? pick<false, true>(a, stream) : pick<false, false>(a, stream);
    return hipGetLastError();
}

}  // namespace mosaic
