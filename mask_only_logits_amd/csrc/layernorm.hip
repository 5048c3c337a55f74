// Layer norm with residual addition, and its backward pass.
//
// For a row of d elements, with x a layer's output and r the residual stream:
//   s = x + r,  mu = mean_k(s_k),  var = mean_k((s_k - mu)^2),  rho = 1 / sqrt(var + eps),
//   xh_k = (s_k - mu) rho,  y_k = xh_k g_k + b_k.
// With a_k = dy_k g_k, the gradients are
//   dx_k = rho (a_k - mean(a) - xh_k mean(a xh)) + dsum_k,
//   dg_k = sum over rows of dy_k xh_k,  db_k = sum over rows of dy_k,
// where dsum is the gradient that reaches s by the residual stream.
//
// The statistics are taken in 64 bits: squares of any fp32 values stay finite, and a mean far
// from zero costs the differences nothing.  One pass does with the sums of (s - s_0) and its
// square: the variance is at least (s_0 - mu)^2 / d, so the difference of the two moments
// loses at most a factor d of 2^53.  s is rounded once, where it is stored; y is computed from
// the unrounded one.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch_head.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

// Sums of two values over a workgroup of NW waves, in every thread, always in the same order.
// `red` holds 2 NW values and is free again for the next call.
template <int NW, typename T>
__device__ __forceinline__ void block_sum2(T &a, T &b, T *red)
{
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) {
        a += __shfl_xor(a, o, 64);
        b += __shfl_xor(b, o, 64);
    }
    if constexpr (NW == 1)
        return;
    if ((threadIdx.x & 63) == 0) {
        red[threadIdx.x >> 6] = a;
        red[NW + (threadIdx.x >> 6)] = b;
    }
    __syncthreads();
    a = red[0];
    b = red[NW];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
        a += red[w];
        b += red[NW + w];
    }
    __syncthreads();
}

// Mean and 1 / sqrt(var + eps) from the sums of s - s0 and of its square.
__device__ __forceinline__ void moments(double s0, double sum, double sum2, int d, double eps, double &mean, double &rstd)
{
    const double m = sum / d, var = sum2 / d - m * m;
    mean = s0 + m;
    rstd = 1.0 / sqrt((var < 0.0 ? 0.0 : var) + eps);   // (a NaN stays)
}

// Gain (or bias) of a thread's CH chunks of N elements, chunk c from element c * STEP + t0 on;
// `none` where there is no such array.
template <bool BF16, int CH, int N, int STEP>
__device__ __forceinline__ void load_weights(const void *p, float none, int t0, int d, Gain<BF16, N> (&g)[CH])
{
    if (!p) {
        const uint32_t b = __builtin_bit_cast(uint32_t, none);
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (auto &w : g[c].w)
                w = (typename Gain<BF16, N>::vec_t)(BF16 ? (b & 0xffff0000u) | (b >> 16) : b);
        return;
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
        g[c].load(p, c * STEP + t0, d);
    if (d % N) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = c * STEP + t0;
            if (k < d && k + N > d)
                g[c].load_part(p, k, d - k);
        }
    }
}

// Sums of two values over the LPR threads of a row.
template <int LPR, typename T>
__device__ __forceinline__ void row_sum2(T &a, T &b, T *red)
{
    if constexpr (LPR > 64)
        return block_sum2<LPR / 64>(a, b, red);
#pragma unroll
    for (int o = LPR / 2; o >= 1; o >>= 1) {
        a += __shfl_xor(a, o, 64);
        b += __shfl_xor(b, o, 64);
    }
}

// LPR threads per row, a thread holding CH chunks of 16 bytes (d <= LPR CH kChunk): lanes of a
// wave, which then has 64 / LPR rows, or whole waves.  STREAM: streaming cache policy.
template <bool BF16, bool GAIN_BF16, int LPR, int CH, bool STREAM>
__global__ __launch_bounds__(LPR <= 64 ? 256 : LPR) void layernorm_kernel(const LayerNorm a)
{
    constexpr int RPB = LPR <= 64 ? 256 / LPR : 1;   // rows per workgroup
    constexpr int N = kChunk<BF16>, STEP = LPR * N;
    __shared__ double red[LPR <= 64 ? 1 : LPR / 32];
    const int t = threadIdx.x % LPR;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR; row < n; row += (int64_t)gridDim.x * RPB) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;   // a row id outside gives a row of NaN
        float v[CH][N], s0 = __builtin_nanf("");
        Raw<BF16> x[CH], r[CH];
        Gain<GAIN_BF16, N> gain[CH], bias[CH];   // taken with the row, not after its reduction
        if (inside) {
            load_row<BF16, CH, STEP, STREAM>(a.X, src * a.ldx, t * N, a.d, x);
            s0 = load1(a.X, src * a.ldx, BF16);
            if (a.R) {
                load_row<BF16, CH, STEP, STREAM>(a.R, src * a.ldr, t * N, a.d, r);
                s0 += load1(a.R, src * a.ldr, BF16);
            }
        }
        load_weights<GAIN_BF16, CH, N, STEP>(a.gain, 1.0f, t * N, a.d, gain);
        load_weights<GAIN_BF16, CH, N, STEP>(a.bias, 0.0f, t * N, a.d, bias);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            if (!inside)
                x[c].fill(__builtin_nanf(""));
            x[c].get(v[c]);
            if (a.R && inside) {
                float y[N];
                r[c].get(y);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[c][i] += y[i];
            }
        }
        double sum = 0.0, sum2 = 0.0, mean, rstd;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int left = a.d - c * STEP - t * N;
            if (left < N) {   // what lies behind the row's end counts nothing
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[c][i] = i < left ? v[c][i] : s0;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const double u = (double)v[c][i] - (double)s0;
                sum += u;
                sum2 = __builtin_fma(u, u, sum2);
            }
        }
        row_sum2<LPR>(sum, sum2, red);
        if (a.sum) {   // (after the sums: with several waves to a row s_0 has then been read by all of them)
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = c * STEP + t * N;
                if (k < a.d)
                    store_upto<BF16, STREAM>(a.sum, row * a.ldsum + k, v[c], a.d - k);
            }
        }
        moments(s0, sum, sum2, a.d, a.eps, mean, rstd);
        if (a.stats && t == 0) {
            a.stats[2 * row] = mean;
            a.stats[2 * row + 1] = rstd;
        }
        if (a.out) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = c * STEP + t * N;
                gain[c].opaque();
                bias[c].opaque();
#pragma unroll
                for (int i = 0; i < N; ++i)
                    asm volatile("" : "+v"(v[c][i]));   // (or its fp64 form is kept over the reduction)
                if (k < a.d) {
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        v[c][i] = __builtin_fmaf((float)(((double)v[c][i] - mean) * rstd), gain[c].get(i), bias[c].get(i));
                    store_upto<BF16, STREAM>(a.out, row * a.d + k, v[c], a.d - k);
                }
            }
        }
    }
}

// Rows too long for the registers: read once for the sums and again for the results.
template <bool BF16>
__global__ __launch_bounds__(1024) void layernorm_long_kernel(const LayerNorm a)
{
    __shared__ double red[32];
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;   // a row id outside gives a row of NaN
        auto element = [&](int k) {
            if (!inside)
                return __builtin_nanf("");
            const float x = load1(a.X, src * a.ldx + k, BF16);
            return a.R ? x + load1(a.R, src * a.ldr + k, BF16) : x;
        };
        const double s0 = element(0);
        double sum = 0.0, sum2 = 0.0, mean, rstd;
        for (int k = threadIdx.x; k < a.d; k += 1024) {
            const double u = (double)element(k) - s0;
            sum += u;
            sum2 += u * u;
        }
        block_sum2<16>(sum, sum2, red);
        moments(s0, sum, sum2, a.d, a.eps, mean, rstd);
        // each element of `sum` is written by the thread that has read it for the last time (and
        // element 0, which all threads read, after the barriers above), so that it may be X or R
        for (int k = threadIdx.x; k < a.d; k += 1024) {
            const float x = element(k);
            if (a.sum)
                store1<BF16>(a.sum, row * a.ldsum + k, x);
            if (a.out) {
                const float xh = (float)(((double)x - mean) * rstd);
                const float g = a.gain ? load1(a.gain, k, a.gain_bf16) : 1.0f;
                store1<BF16>(a.out, row * a.d + k, __builtin_fmaf(xh, g, a.bias ? load1(a.bias, k, a.gain_bf16) : 0.0f));
            }
        }
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * row] = mean;
            a.stats[2 * row + 1] = rstd;
        }
    }
}

// Partial sums of the weight gradients: [parts][2][width], width = d rounded up to 64 (for
// 16-byte accesses), in fp32 where a part has kRun rows at most, else in fp64.
constexpr int kRun = 128;
__host__ __device__ inline int64_t partial_width(int64_t d) { return (d + 63) / 64 * 64; }

// LPR threads per row and CH chunks a thread, as above; a workgroup of NT threads walks over its
// rows, NT / LPR at a time, and the threads keep the sums of the weight gradients of their
// columns in registers.  NEXT: the next row's loads are issued before this row is computed.
// `parts` = gridDim.x * NT / LPR with weight gradients, each row group a part; 0: none.
template <bool BF16, bool GAIN_BF16, int LPR, int CH, int NT, bool NEXT, bool STREAM>
__global__ __launch_bounds__(NT) void layernorm_grad_kernel(const LayerNormGrad a, int parts, bool in_runs)
{
    constexpr int RPB = NT / LPR, NW = LPR <= 64 ? 1 : LPR / 64;
    static_assert(LPR <= 64 || RPB == 1, "a row's waves meet at workgroup barriers");
    constexpr int N = kChunk<BF16>, STEP = LPR * N;
    __shared__ float red[2][2 * NW];
    const int t = threadIdx.x % LPR;
    const int64_t n = row_count(a.count, a.rows);
    Gain<GAIN_BF16, N> gain[CH];
    load_weights<GAIN_BF16, CH, N, STEP>(a.gain, 1.0f, t * N, a.d, gain);
    float dg[CH][N] = {}, db[CH][N] = {};
    struct Loaded {
        Raw<BF16> s[CH], dy[CH], ds[CH];
        double mean, rstd;
    };
    auto fetch = [&](int64_t row, Loaded &x) __attribute__((always_inline)) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        x.mean = a.stats[2 * row];
        x.rstd = a.stats[2 * row + 1];
        load_row<BF16, CH, STEP, STREAM>(a.dY, row * a.lddy, t * N, a.d, x.dy);
        if (src >= 0 && src < a.nsrc) {
            load_row<BF16, CH, STEP, STREAM>(a.S, src * a.lds, t * N, a.d, x.s);
        } else {   // a row id outside gives a row of NaN
#pragma unroll
            for (int c = 0; c < CH; ++c)
                x.s[c].fill(__builtin_nanf(""));
        }
        if (a.dsum)
            load_row<BF16, CH, STEP, STREAM>(a.dsum, row * a.lddsum, t * N, a.d, x.ds);
    };
    const double over_d = 1.0 / a.d;
    Loaded x, next;
    const int64_t first = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR, step = (int64_t)gridDim.x * RPB;
    if (first < n)
        fetch(first, x);
    int run = 0, odd = 0;
    bool flushed = false;
    const int64_t width = partial_width(a.d);
    const int64_t part = (int64_t)blockIdx.x * RPB + threadIdx.x / LPR;
    // the sums so far, to fp64 partials of this row group's own
    auto flush = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int k = c * STEP + t * N;
            if (k < width) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    double *g = (double *)a.partials + part * 2 * width + k + i, *b = g + width;
                    *g = (flushed ? *g : 0.0) + (double)dg[c][i];
                    *b = (flushed ? *b : 0.0) + (double)db[c][i];
                    dg[c][i] = db[c][i] = 0.0f;
                }
            }
        }
        flushed = true;
    };
    // every thread of a row's waves takes the same number of turns (LPR > 64: the workgroup is the row)
    for (int64_t row = first; row < n; row += step) {
        if (NEXT && row + step < n)
            fetch(row + step, next);
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float xh[N], dy[N];   // dy is 0 behind the row's end, where s is 0 too
            gain[c].opaque();
            x.s[c].get(xh);
            x.dy[c].get(dy);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                xh[i] = (float)(((double)xh[i] - x.mean) * x.rstd);
                dg[c][i] = __builtin_fmaf(dy[i], xh[i], dg[c][i]);
                db[c][i] += dy[i];
                dy[i] *= gain[c].get(i);
                c1 += dy[i];
                c2 = __builtin_fmaf(dy[i], xh[i], c2);
            }
        }
        if constexpr (LPR > 64) {
#pragma unroll
            for (int o = 32; o >= 1; o >>= 1) {
                c1 += __shfl_xor(c1, o, 64);
                c2 += __shfl_xor(c2, o, 64);
            }
            // (one barrier a row: the other half of `red` is written next, and this one again only
            // when every wave has passed that row's barrier)
            if ((threadIdx.x & 63) == 0) {
                red[odd][threadIdx.x >> 6] = c1;
                red[odd][NW + (threadIdx.x >> 6)] = c2;
            }
            __syncthreads();
            c1 = red[odd][0];
            c2 = red[odd][NW];
#pragma unroll
            for (int w = 1; w < NW; ++w) {
                c1 += red[odd][w];
                c2 += red[odd][NW + w];
            }
            odd ^= 1;
        } else {
            row_sum2<LPR>(c1, c2, (float *)nullptr);
        }
        const float m1 = (float)(c1 * over_d), m2 = (float)(c2 * over_d);
        if (a.dX) {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = c * STEP + t * N;
                // the terms are made again: kept, they would take the registers of another row
                x.s[c].opaque();
                x.dy[c].opaque();
                gain[c].opaque();
                if (k < a.d) {
                    float xh[N], dy[N], y[N] = {};
                    x.s[c].get(xh);
                    x.dy[c].get(dy);
                    if (a.dsum)
                        x.ds[c].get(y);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        xh[i] = (float)(((double)xh[i] - x.mean) * x.rstd);
                        y[i] += (float)(x.rstd * (double)(dy[i] * gain[c].get(i) - m1 - xh[i] * m2));
                    }
                    store_upto<BF16, STREAM>(a.dX, row * a.lddx + k, y, a.d - k);
                }
            }
        }
        if (in_runs && ++run == kRun) {
            flush();
            run = 0;
        }
        if (NEXT)
            x = next;
        else if (row + step < n)
            fetch(row + step, x);
    }
    if (parts == 0)
        return;
    if (in_runs)
        return flush();
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int k = c * STEP + t * N;
        if (k < width) {
            float *g = (float *)a.partials + part * 2 * width + k;
            store<false>(g, 0, *(float(*)[4])&dg[c][0]);
            store<false>(g + width, 0, *(float(*)[4])&db[c][0]);
            if constexpr (N == 8) {
                store<false>(g + 4, 0, *(float(*)[4])&dg[c][4]);
                store<false>(g + width + 4, 0, *(float(*)[4])&db[c][4]);
            }
        }
    }
}

// The gradient of rows too long for the registers: read twice.
template <bool BF16>
__global__ __launch_bounds__(1024) void layernorm_grad_long_kernel(const LayerNormGrad a)
{
    __shared__ double red[32];
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;
        const double mean = a.stats[2 * row], rstd = a.stats[2 * row + 1];
        auto terms = [&](int k, float &x, float &xh) {
            const float s = inside ? load1(a.S, src * a.lds + k, BF16) : __builtin_nanf("");
            xh = (float)(((double)s - mean) * rstd);
            x = load1(a.dY, row * a.lddy + k, BF16) * (a.gain ? load1(a.gain, k, a.gain_bf16) : 1.0f);
        };
        double c1 = 0.0, c2 = 0.0;
        for (int k = threadIdx.x; k < a.d; k += 1024) {
            float x, xh;
            terms(k, x, xh);
            c1 += x;
            c2 += (double)x * xh;
        }
        block_sum2<16>(c1, c2, red);
        const float m1 = (float)(c1 / a.d), m2 = (float)(c2 / a.d);
        for (int k = threadIdx.x; k < a.d; k += 1024) {
            float x, xh;
            terms(k, x, xh);
            float g = (float)(rstd * (double)(x - m1 - xh * m2));
            if (a.dsum)
                g += load1(a.dsum, row * a.lddsum + k, BF16);
            store1<BF16>(a.dX, row * a.lddx + k, g);
        }
    }
}

constexpr int kColumns = 256;   // columns of a workgroup of the two kernels below

// Sums of the weight gradients' terms over the rows r of part blockIdx.y of gridDim.y, a column to a
// thread, into partials[part][2][d].
template <bool BF16>
__global__ __launch_bounds__(kColumns) void layernorm_columns_kernel(const LayerNormGrad a, double *__restrict__ partials)
{
    const int k = blockIdx.x * kColumns + threadIdx.x;
    if (k >= a.d)
        return;
    const int64_t n = row_count(a.count, a.rows);
    double dg = 0.0, db = 0.0;
    for (int64_t row = blockIdx.y; row < n; row += gridDim.y) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;
        const float s = inside ? load1(a.S, src * a.lds + k, BF16) : __builtin_nanf("");
        const float xh = (float)(((double)s - a.stats[2 * row]) * a.stats[2 * row + 1]);
        const double dy = load1(a.dY, row * a.lddy + k, BF16);
        dg += dy * xh;
        db += dy;
    }
    const int64_t width = partial_width(a.d);
    partials[(int64_t)blockIdx.y * 2 * width + k] = dg;
    partials[((int64_t)blockIdx.y * 2 + 1) * width + k] = db;
}

// The weight gradients from `parts` partial sums [parts][2][width]: a workgroup takes 64 columns of
// [2][width], 16 threads side by side with four each, and the parts go round its 64 groups of
// these.  The groups' sums are added in a fixed order.
template <typename T>
__global__ __launch_bounds__(1024) void layernorm_join_kernel(const T *__restrict__ partials, int parts, int32_t d,
                                                              float *__restrict__ dgain, float *__restrict__ dbias)
{
    __shared__ double sums[64][65];
    const int64_t width = partial_width(d), stride = 2 * width;
    const int q = threadIdx.x & 15, group = threadIdx.x >> 4;
    const T *p = partials + (int64_t)blockIdx.x * 64 + q * 4;
    double s[4] = {};
#pragma unroll 8
    for (int i = group; i < parts; i += 64) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            s[e] += (double)p[i * stride + e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
        sums[group][q * 4 + e] = s[e];
    __syncthreads();
    // 16 threads a column, four groups each
    const int column = threadIdx.x >> 4;
    double x = 0.0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        x += sums[q * 4 + e][column];
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1)
        x += __shfl_xor(x, o, 64);
    const int64_t at = (int64_t)blockIdx.x * 64 + column;
    float *to = at < width ? dgain : dbias;
    const int64_t k = at < width ? at : at - width;
    if (q == 0 && to && k < d)
        to[k] = (float)x;
}

// Workgroups of a launch: one for each row (or 4 to 32), and no more than 2^20, over which the
// kernels walk: a launch holds at most 2^32 - 1 threads.
unsigned grid_of(int64_t rows, int per_block)
{
    return (unsigned)std::min<int64_t>((rows + per_block - 1) / per_block, 1 << 20);
}

// Rows that pass the 256 MB Infinity Cache by far are read and written with the streaming cache
// policy, which leaves the cache to what is used next.
bool is_large(int64_t streams, int64_t rows, int64_t d, int64_t esize)
{
    return streams * rows * d * esize >= (int64_t)512 << 20;
}

// CH: chunks of eight elements per thread
template <bool BF16, int LPR, int CH>
void run(const LayerNorm &a, hipStream_t stream)
{
    constexpr int C = CH * 8 / kChunk<BF16>;
    const dim3 grid(grid_of(a.rows, LPR <= 64 ? 256 / LPR : 1)), block(LPR <= 64 ? 256 : LPR);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, a); };
    if (is_large(1 + (a.R != nullptr) + (a.sum != nullptr) + (a.out != nullptr), a.rows, a.d, BF16 ? 2 : 4))
        a.gain_bf16 ? go(layernorm_kernel<BF16, true, LPR, C, true>) : go(layernorm_kernel<BF16, false, LPR, C, true>);
    else
        a.gain_bf16 ? go(layernorm_kernel<BF16, true, LPR, C, false>) : go(layernorm_kernel<BF16, false, LPR, C, false>);
}

// Threads per row and chunks per thread, by the row's length: enough threads for the row to
// finish soon, few enough that several rows share a wave or a CU and one's reductions lie under
// the others' reads.
template <bool BF16>
void pick(const LayerNorm &a, hipStream_t stream)
{
    if (a.d <= 64)
        return run<BF16, 8, 1>(a, stream);
    if (a.d <= 128)
        return run<BF16, 16, 1>(a, stream);
    if (a.d <= 256)
        return run<BF16, 32, 1>(a, stream);
    if (a.d <= 512)
        return run<BF16, 64, 1>(a, stream);
    if (a.d <= 1024)
        return run<BF16, 64, 2>(a, stream);
    if (a.d <= 2048)
        return run<BF16, 128, 2>(a, stream);
    if (a.d <= 4096)
        return run<BF16, 256, 2>(a, stream);
    if (a.d <= 6144)
        return run<BF16, 256, 3>(a, stream);
    if (a.d <= 8192)
        return run<BF16, 512, 2>(a, stream);
    if (a.d <= 16384)
        return run<BF16, 512, 4>(a, stream);
    hipLaunchKernelGGL((layernorm_long_kernel<BF16>), dim3(grid_of(a.rows, 1)), dim3(1024), 0, stream, a);
}

// The forms of the gradient by the row's length: threads per row, chunks of eight elements a
// thread, threads of a workgroup, and workgroups that the chip is given.
struct GradForm {
    int lpr, nt, groups;
};
constexpr int64_t kGradWidest = 16384;   // longer rows are read twice
GradForm grad_form(int64_t d)
{
    if (d <= 64)
        return {8, 256, 1024};
    if (d <= 128)
        return {16, 256, 1024};
    if (d <= 256)
        return {32, 256, 1024};
    if (d <= 1024)
        return {64, 256, 768};
    if (d <= 2048)
        return {128, 128, 1024};
    if (d <= 4096)
        return {256, 256, 512};
    return {512, 512, 256};
}

// Parts of the rows for the weight gradients: the row groups of the gradient kernel, or (rows
// too long for it) enough workgroups of columns for the chip.
int64_t parts_of(int64_t rows, int64_t d)
{
    if (d > kGradWidest) {
        const int64_t wide = (d + kColumns - 1) / kColumns;
        return std::max<int64_t>(1, std::min<int64_t>({rows, 512, 4096 / wide}));
    }
    const GradForm f = grad_form(d);
    const int rpb = f.nt / f.lpr;
    return std::min<int64_t>((rows + rpb - 1) / rpb, f.groups) * rpb;
}
// whether a part has so many rows that its sums are taken in runs, into fp64 partials
bool in_runs(int64_t rows, int64_t d) { return d > kGradWidest || rows > kRun * parts_of(rows, d); }

template <bool BF16, int LPR, int CH, int NT>
void run_grad(const LayerNormGrad &a, hipStream_t stream)
{
    constexpr int C = CH * 8 / kChunk<BF16>;
    constexpr bool NEXT = CH < 4;   // (32 elements a thread leave no registers for another row)
    const bool weights = a.dgain || a.dbias;
    const int parts = (int)parts_of(a.rows, a.d);
    const dim3 grid((unsigned)(parts / (NT / LPR)));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, stream, a, weights ? parts : 0, weights && in_runs(a.rows, a.d));
    };
    if (is_large(2 + (a.dsum != nullptr) + (a.dX != nullptr), a.rows, a.d, BF16 ? 2 : 4))
        a.gain_bf16 ? go(layernorm_grad_kernel<BF16, true, LPR, C, NT, NEXT, true>)
                    : go(layernorm_grad_kernel<BF16, false, LPR, C, NT, NEXT, true>);
    else
        a.gain_bf16 ? go(layernorm_grad_kernel<BF16, true, LPR, C, NT, NEXT, false>)
                    : go(layernorm_grad_kernel<BF16, false, LPR, C, NT, NEXT, false>);
}

template <bool BF16>
hipError_t pick_grad(const LayerNormGrad &a, hipStream_t stream)
{
    const bool weights = a.dgain || a.dbias;
    if (a.rows > 0 && a.d <= kGradWidest) {
        if (a.d <= 64)
            run_grad<BF16, 8, 1, 256>(a, stream);
        else if (a.d <= 128)
            run_grad<BF16, 16, 1, 256>(a, stream);
        else if (a.d <= 256)
            run_grad<BF16, 32, 1, 256>(a, stream);
        else if (a.d <= 512)
            run_grad<BF16, 64, 1, 256>(a, stream);
        else if (a.d <= 1024)
            run_grad<BF16, 64, 2, 256>(a, stream);
        else if (a.d <= 2048)
            run_grad<BF16, 128, 2, 128>(a, stream);
        else if (a.d <= 4096)
            run_grad<BF16, 256, 2, 256>(a, stream);
        else if (a.d <= 8192)
            run_grad<BF16, 512, 2, 512>(a, stream);
        else
            run_grad<BF16, 512, 4, 512>(a, stream);
    }
    const int parts = a.rows > 0 ? (int)parts_of(a.rows, a.d) : 0;
    if (weights && a.rows > 0 && a.d > kGradWidest)
        hipLaunchKernelGGL((layernorm_columns_kernel<BF16>), dim3((unsigned)((a.d + kColumns - 1) / kColumns), (unsigned)parts),
                           dim3(kColumns), 0, stream, a, (double *)a.partials);
    if (a.dX && a.rows > 0 && a.d > kGradWidest)   // after it: dX may be dY itself
        hipLaunchKernelGGL((layernorm_grad_long_kernel<BF16>), dim3(grid_of(a.rows, 1)), dim3(1024), 0, stream, a);
    if (weights) {
        const dim3 grid((unsigned)(partial_width(a.d) / 32));
        if (parts > 0 && in_runs(a.rows, a.d))
            hipLaunchKernelGGL((layernorm_join_kernel<double>), grid, dim3(1024), 0, stream, (const double *)a.partials,
                               parts, a.d, a.dgain, a.dbias);
        else
            hipLaunchKernelGGL((layernorm_join_kernel<float>), grid, dim3(1024), 0, stream, (const float *)a.partials,
                               parts, a.d, a.dgain, a.dbias);
    }
    return hipGetLastError();
}

}  // namespace

int64_t layernorm_grad_workspace_bytes(int64_t rows, int64_t d)
{
    return rows == 0 || d == 0 ? 0 : parts_of(rows, d) * 2 * partial_width(d) * (in_runs(rows, d) ? 8 : 4);
}

hipError_t launch_layernorm(const LayerNorm &a, bool in_bf16, hipStream_t stream)
{
    in_bf16 ? pick<true>(a, stream) : pick<false>(a, stream);
    return hipGetLastError();
}

hipError_t launch_layernorm_grad(const LayerNormGrad &a, bool in_bf16, hipStream_t stream)
{
    return in_bf16 ? pick_grad<true>(a, stream) : pick_grad<false>(a, stream);
}

}  // namespace mosaic
