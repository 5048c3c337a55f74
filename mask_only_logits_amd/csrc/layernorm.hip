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

// A row's statistics for fp32 arithmetic: xh = (fma(s, h, -mu_hi) - mu_lo) * r.  Each of the two
// differences rounds relative to itself, so a mean far from zero costs xh nothing.  h is 1, or 2^-60
// for rows whose differences could pass fp32's range or whose rho lies below its normal numbers: with
// rho >= 2^-60 no element is further than 2^60 sqrt(d) from the mean, and no r passes 2^63.
struct RowStats {
    float h, mu_hi, mu_lo, r;

    __device__ __forceinline__ RowStats(double mean, double rstd)
    {
        const bool wide = rstd < 0x1p-60;
        h = wide ? 0x1p-60f : 1.0f;
        const double m = wide ? mean * 0x1p-60 : mean;
        mu_hi = (float)m;
        mu_lo = (float)(m - (double)mu_hi);
        r = (float)(wide ? rstd * 0x1p60 : rstd);
    }
    __device__ __forceinline__ float xh(float s) const { return (__builtin_fmaf(s, h, -mu_hi) - mu_lo) * r; }
    // rho t (r first: below 1 where h is not, so that neither product leaves fp32's range before the result does)
    __device__ __forceinline__ float times_rho(float t) const { return t * r * h; }
};

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

// Row of a thread within its workgroup's row groups; the same for a wave's lanes where it is, so
// that the row's addresses are a uniform pointer and a lane's offset.
template <int LPR>
__device__ __forceinline__ int row_group()
{
    if constexpr (LPR > 64)
        return 0;
    const int g = threadIdx.x / LPR;
    return LPR == 64 ? __builtin_amdgcn_readfirstlane(g) : g;
}

// Where a row of elements starts.
template <bool BF16>
__device__ __forceinline__ const void *row_at(const void *p, int64_t row, int64_t ld)
{
    return (const char *)p + row * ld * (BF16 ? 2 : 4);
}
template <bool BF16>
__device__ __forceinline__ void *row_at(void *p, int64_t row, int64_t ld)
{
    return (char *)p + row * ld * (BF16 ? 2 : 4);
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
// Bound: HBM.  32768 x 4096 bf16 with residual and sum moves 1.07 GB in 180 us, 5.95 TB/s (a
// large copy runs at 5.2); the same with the rows' differences in fp64 184 us.
template <bool BF16, bool GAIN_BF16, int LPR, int CH, bool STREAM>
__global__ __launch_bounds__(LPR <= 64 ? 256 : LPR) void layernorm_kernel(const LayerNorm a)
{
    constexpr int RPB = LPR <= 64 ? 256 / LPR : 1;   // rows per workgroup
    constexpr int N = kChunk<BF16>, STEP = LPR * N;
    __shared__ double red[LPR <= 64 ? 1 : LPR / 32];
    const int t = threadIdx.x % LPR;
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = (int64_t)blockIdx.x * RPB + row_group<LPR>(); row < n; row += (int64_t)gridDim.x * RPB) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;   // a row id outside gives a row of NaN
        float v[CH][N], s0 = __builtin_nanf("");
        Raw<BF16> x[CH], r[CH];
        Gain<GAIN_BF16, N> gain[CH], bias[CH];   // taken with the row, not after its reduction
        if (inside) {
            load_row<BF16, CH, STEP, STREAM>(row_at<BF16>(a.X, src, a.ldx), 0, t * N, a.d, x);
            s0 = load1(a.X, src * a.ldx, BF16);
            if (a.R) {
                load_row<BF16, CH, STEP, STREAM>(row_at<BF16>(a.R, src, a.ldr), 0, t * N, a.d, r);
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
                    store_upto<BF16, STREAM>(row_at<BF16>(a.sum, row, a.ldsum), k, v[c], a.d - k);
            }
        }
        moments(s0, sum, sum2, a.d, a.eps, mean, rstd);
        if (a.stats && t == 0) {
            a.stats[2 * row] = mean;
            a.stats[2 * row + 1] = rstd;
        }
        if (a.out) {
            const RowStats st(mean, rstd);
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
                        v[c][i] = __builtin_fmaf(st.xh(v[c][i]), gain[c].get(i), bias[c].get(i));
                    store_upto<BF16, STREAM>(row_at<BF16>(a.out, row, a.d), k, v[c], a.d - k);
                }
            }
        }
    }
}

// Chunks of N elements of a row of d, chunk by chunk over NT threads: f(k, n) for elements k .. k + n - 1,
// n < N at the row's end.
template <int N, int NT, typename F>
__device__ __forceinline__ void over_row(int d, F f)
{
    for (int k = threadIdx.x * N; k < d; k += NT * N)
        f(k, min(N, d - k));
}

// Elements k .. k + n - 1 of a row, zeros behind them.
template <bool BF16>
__device__ __forceinline__ void load_some(const void *row, int k, int n, float (&x)[kChunk<BF16>])
{
    Raw<BF16> r;
    if (n == kChunk<BF16>) {
        r.load(row, k);
    } else {
        r.fill(0.0f);
        r.load_part(row, k, n);
    }
    r.get(x);
}

// The weights beside them, `none` where there is no array.
template <int N>
__device__ __forceinline__ void load_weight_some(const void *p, bool bf16, float none, int k, int n, float (&x)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = p && i < n ? load1(p, k + i, bf16) : none;
}

// Rows too long for the registers: read once for the sums and again for the results.
template <bool BF16>
__global__ __launch_bounds__(1024) void layernorm_long_kernel(const LayerNorm a)
{
    constexpr int N = kChunk<BF16>;
    __shared__ double red[32];
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;   // a row id outside gives a row of NaN
        const void *x = row_at<BF16>(a.X, inside ? src : 0, a.ldx);
        const void *r = a.R ? row_at<BF16>(a.R, inside ? src : 0, a.ldr) : nullptr;
        auto elements = [&](int k, int cnt, float (&v)[N]) __attribute__((always_inline)) {
            load_some<BF16>(x, k, cnt, v);
            if (r) {
                float y[N];
                load_some<BF16>(r, k, cnt, y);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[i] += y[i];
            }
        };
        const float first = load1(x, 0, BF16) + (r ? load1(r, 0, BF16) : 0.0f);
        const double s0 = inside ? first : __builtin_nanf("");
        double sum = 0.0, sum2 = 0.0, mean, rstd;
        over_row<N, 1024>(a.d, [&](int k, int cnt) {
            float v[N];
            elements(k, cnt, v);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const double u = i < cnt ? (double)v[i] - s0 : 0.0;
                sum += u;
                sum2 = __builtin_fma(u, u, sum2);
            }
        });
        block_sum2<16>(sum, sum2, red);
        moments(s0, sum, sum2, a.d, a.eps, mean, rstd);
        const RowStats st(mean, rstd);
        // each element of `sum` is written by the thread that has read it for the last time (and
        // element 0, which all threads read, after the barriers above), so that it may be X or R
        over_row<N, 1024>(a.d, [&](int k, int cnt) {
            float v[N], g[N], b[N];
            elements(k, cnt, v);
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] = inside ? v[i] : __builtin_nanf("");
            if (a.sum)
                store_upto<BF16>(row_at<BF16>(a.sum, row, a.ldsum), k, v, cnt);
            if (a.out) {
                load_weight_some(a.gain, a.gain_bf16, 1.0f, k, cnt, g);
                load_weight_some(a.bias, a.gain_bf16, 0.0f, k, cnt, b);
#pragma unroll
                for (int i = 0; i < N; ++i)
                    v[i] = __builtin_fmaf(st.xh(v[i]), g[i], b[i]);
                store_upto<BF16>(row_at<BF16>(a.out, row, a.d), k, v, cnt);
            }
        });
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * row] = mean;
            a.stats[2 * row + 1] = rstd;
        }
    }
}

// Partial sums of the weight gradients: [parts][2][width], width = d rounded up to 64 (for
// 16-byte accesses).  Where a row group (the threads of a row) has kRun rows at most, its sums are
// fp32, those of a workgroup's groups (32 at most) are joined in fp32, and a part is a workgroup; else
// a part is a row group, in fp64, to which it adds its fp32 sums of every kRun rows.
constexpr int kRun = 128;
__host__ __device__ inline int64_t partial_width(int64_t d) { return (d + 63) / 64 * 64; }

// LPR threads per row and CH chunks a thread, as above; a workgroup of NT threads walks over its
// rows, NT / LPR at a time, and the threads keep the sums of the weight gradients of their
// columns in registers, so that no row is read a second time for them.  NEXT: the next row's
// loads are issued before this row is computed.
// Bound: HBM.  32768 x 4096 bf16 with dsum and both weight gradients, join included: 195 us for 1.07
// GB, 5.5 TB/s.  216 us with the differences in fp64 (eleven conversions and fp64 operations an
// element), and before that 211 us with the terms kept in registers over the reduction (177
// registers, two waves to a SIMD, instead of 139 and three).
// Each workgroup leaves a part of the weight gradients; in_runs: each of its row groups does.
template <bool BF16, bool GAIN_BF16, int LPR, int CH, int NT, bool NEXT, bool STREAM>
__global__ __launch_bounds__(NT) void layernorm_grad_kernel(const LayerNormGrad a, bool weights, bool in_runs)
{
    constexpr int RPB = NT / LPR, NW = LPR <= 64 ? 1 : LPR / 64;
    static_assert(LPR <= 64 || RPB == 1, "a row's waves meet at workgroup barriers");
    constexpr int N = kChunk<BF16>, STEP = LPR * N;
    __shared__ float red[2][2 * NW];
    __shared__ __attribute__((aligned(16))) float joined[RPB > 1 ? NT / 64 * 64 * CH * 4 : 4];
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
        load_row<BF16, CH, STEP, STREAM>(row_at<BF16>(a.dY, row, a.lddy), 0, t * N, a.d, x.dy);
        if (src >= 0 && src < a.nsrc) {
            load_row<BF16, CH, STEP, STREAM>(row_at<BF16>(a.S, src, a.lds), 0, t * N, a.d, x.s);
        } else {   // a row id outside gives a row of NaN
#pragma unroll
            for (int c = 0; c < CH; ++c)
                x.s[c].fill(__builtin_nanf(""));
        }
        if (a.dsum)
            load_row<BF16, CH, STEP, STREAM>(row_at<BF16>(a.dsum, row, a.lddsum), 0, t * N, a.d, x.ds);
    };
    const double over_d = 1.0 / a.d;
    const bool ragged = a.d < LPR * CH * N;   // some threads have nothing in a place
    Loaded x, next;
    const int64_t first = (int64_t)blockIdx.x * RPB + row_group<LPR>(), step = (int64_t)gridDim.x * RPB;
    if (first < n)
        fetch(first, x);
    int run = 0, odd = 0;
    bool flushed = false;
    const int64_t width = partial_width(a.d);
    const int64_t part = first;
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
                    __builtin_amdgcn_sched_barrier(0);   // (or the registers for all of them are taken)
                }
            }
        }
        flushed = true;
    };
    // every thread of a row's waves takes the same number of turns (LPR > 64: the workgroup is the row)
    for (int64_t row = first; row < n; row += step) {
        if (NEXT && row + step < n)
            fetch(row + step, next);
        const RowStats st(x.mean, x.rstd);
        // Behind the row's end dy and s are 0.  Where mu rho passes fp32's range so would xh, and 0 times it
        // is no number: there s takes mu, which is what such a row's elements are, all but equal in fp32.
        // (Leaving the row's end out of the sums takes up to 36 registers.)
        if (ragged && __builtin_expect(fabsf(st.xh(0.0f)) == __builtin_inff(), 0)) {
#pragma unroll
            for (int c = 0; c < CH; ++c)
                x.s[c].fill_from(a.d - c * STEP - t * N, (float)x.mean);
        }
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float xh[N], dy[N];   // dy is 0 behind the row's end, where s is 0 too
            gain[c].opaque();
            x.s[c].get(xh);
            x.dy[c].get(dy);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                xh[i] = st.xh(xh[i]);
                dg[c][i] = __builtin_fmaf(dy[i], xh[i], dg[c][i]);
                db[c][i] += dy[i];
                asm volatile("" : "+v"(dg[c][i]), "+v"(db[c][i]));   // (or done later, with the terms kept)
                dy[i] *= gain[c].get(i);
                c1 += dy[i];
                c2 = __builtin_fmaf(dy[i], xh[i], c2);
            }
            __builtin_amdgcn_sched_barrier(0);   // one chunk unpacked at a time
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
                    for (int i = 0; i < N; ++i)
                        y[i] += st.times_rho(dy[i] * gain[c].get(i) - m1 - st.xh(xh[i]) * m2);
                    store_upto<BF16, STREAM>(row_at<BF16>(a.dX, row, a.lddx), k, y, a.d - k);
                }
                __builtin_amdgcn_sched_barrier(0);
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
    if (!weights)
        return;
    if (in_runs)
        return flush();
    // the row groups of a wave, then its waves, in a fixed order
    if constexpr (LPR < 64) {
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
                for (int o = LPR; o < 64; o <<= 1) {
                    dg[c][i] += __shfl_xor(dg[c][i], o, 64);
                    db[c][i] += __shfl_xor(db[c][i], o, 64);
                }
    }
    auto put = [&](float (&x)[CH][N], float *to) __attribute__((always_inline)) {
        if constexpr (RPB > 1) {
            // four elements of each chunk a time, [wave][chunk][thread of the row]
            constexpr int WAVES = NT / 64, SIDE = LPR < 64 ? LPR : 64;
#pragma unroll
            for (int h = 0; h < N; h += 4) {
                __syncthreads();
                if ((threadIdx.x & 63) < SIDE)
#pragma unroll
                    for (int c = 0; c < CH; ++c)
                        *(f32x4_t *)&joined[(((threadIdx.x >> 6) * CH + c) * SIDE + t) * 4] =
                            f32x4_t{x[c][h], x[c][h + 1], x[c][h + 2], x[c][h + 3]};
                __syncthreads();
                for (int j = threadIdx.x; j < CH * SIDE; j += NT) {
                    f32x4_t s = *(const f32x4_t *)&joined[j * 4];
#pragma unroll
                    for (int w = 1; w < WAVES; ++w)
                        s += *(const f32x4_t *)&joined[(w * CH * SIDE + j) * 4];
                    const int k = j / SIDE * STEP + j % SIDE * N + h;
                    if (k < width)
                        *(f32x4_t *)(to + k) = s;
                }
            }
        } else {
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int k = c * STEP + t * N;
                if (k < width) {
#pragma unroll
                    for (int h = 0; h < N; h += 4)
                        *(f32x4_t *)(to + k + h) = f32x4_t{x[c][h], x[c][h + 1], x[c][h + 2], x[c][h + 3]};
                }
            }
        }
    };
    float *to = (float *)a.partials + (int64_t)blockIdx.x * 2 * width;
    put(dg, to);
    put(db, to + width);
}

// The gradient of rows too long for the registers: read twice.
template <bool BF16>
__global__ __launch_bounds__(1024) void layernorm_grad_long_kernel(const LayerNormGrad a)
{
    constexpr int N = kChunk<BF16>;
    __shared__ double red[32];
    const int64_t n = row_count(a.count, a.rows);
    for (int64_t row = blockIdx.x; row < n; row += gridDim.x) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;
        const void *s = row_at<BF16>(a.S, inside ? src : 0, a.lds), *dy = row_at<BF16>(a.dY, row, a.lddy);
        const RowStats st(a.stats[2 * row], inside ? a.stats[2 * row + 1] : (double)__builtin_nanf(""));
        // dy g and xh, both 0 behind the row's end
        auto terms = [&](int k, int cnt, float (&x)[N], float (&xh)[N]) __attribute__((always_inline)) {
            float g[N];
            load_some<BF16>(s, k, cnt, xh);
            load_some<BF16>(dy, k, cnt, x);
            load_weight_some(a.gain, a.gain_bf16, 1.0f, k, cnt, g);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                xh[i] = i < cnt ? st.xh(xh[i]) : 0.0f;
                x[i] *= g[i];
            }
        };
        double c1 = 0.0, c2 = 0.0;
        over_row<N, 1024>(a.d, [&](int k, int cnt) {
            float x[N], xh[N];
            terms(k, cnt, x, xh);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                c1 += (double)x[i];
                c2 = __builtin_fma((double)x[i], (double)xh[i], c2);
            }
        });
        block_sum2<16>(c1, c2, red);
        const float m1 = (float)(c1 / a.d), m2 = (float)(c2 / a.d);
        over_row<N, 1024>(a.d, [&](int k, int cnt) {
            float x[N], xh[N], y[N] = {};
            terms(k, cnt, x, xh);
            if (a.dsum)
                load_some<BF16>(row_at<BF16>(a.dsum, row, a.lddsum), k, cnt, y);
#pragma unroll
            for (int i = 0; i < N; ++i)
                y[i] += st.times_rho(x[i] - m1 - xh[i] * m2);
            store_upto<BF16>(row_at<BF16>(a.dX, row, a.lddx), k, y, cnt);
        });
    }
}

// Sums of the weight gradients' terms over the rows of part blockIdx.y of gridDim.y, a chunk of
// columns to a thread, into partials[part][2][width].
constexpr int kColumnThreads = 256;
template <bool BF16>
__global__ __launch_bounds__(kColumnThreads) void layernorm_columns_kernel(const LayerNormGrad a,
                                                                           double *__restrict__ partials)
{
    constexpr int N = kChunk<BF16>;
    const int k = (blockIdx.x * kColumnThreads + threadIdx.x) * N, cnt = min(N, a.d - k);
    if (cnt <= 0)
        return;
    const int64_t n = row_count(a.count, a.rows);
    double dg[N] = {}, db[N] = {};
#pragma unroll 2
    for (int64_t row = blockIdx.y; row < n; row += gridDim.y) {
        const int64_t src = a.row_idx ? (int64_t)a.row_idx[row] : row;
        const bool inside = src >= 0 && src < a.nsrc;
        const RowStats st(a.stats[2 * row], inside ? a.stats[2 * row + 1] : (double)__builtin_nanf(""));
        float s[N], dy[N];
        load_some<BF16>(row_at<BF16>(a.S, inside ? src : 0, a.lds), k, cnt, s);
        load_some<BF16>(row_at<BF16>(a.dY, row, a.lddy), k, cnt, dy);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            dg[i] = __builtin_fma((double)dy[i], (double)st.xh(s[i]), dg[i]);
            db[i] += (double)dy[i];
        }
    }
    const int64_t width = partial_width(a.d);
    double *to = partials + (int64_t)blockIdx.y * 2 * width + k;
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < cnt) {
            to[i] = dg[i];
            to[width + i] = db[i];
        }
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
// the others' reads.  Three chunks where two would leave many threads without one (bf16: 131072 x
// 700: 181 against 236 us, 32768 x 2560: 112 against 158 us; the gradient of these 250 against
// 259 and 132 against 179 us).
template <bool BF16>
void pick(const LayerNorm &a, hipStream_t stream)
{
    if (a.d <= 64)
        return run<BF16, 8, 1>(a, stream);
    if (a.d <= 128)
        return run<BF16, 16, 1>(a, stream);
    if constexpr (BF16) {
        if (a.d <= 192)
            return run<BF16, 8, 3>(a, stream);
        if (a.d > 256 && a.d <= 384)
            return run<BF16, 16, 3>(a, stream);
        if (a.d > 512 && a.d <= 768)
            return run<BF16, 32, 3>(a, stream);
        if (a.d > 1024 && a.d <= 1536)
            return run<BF16, 64, 3>(a, stream);
        if (a.d > 2048 && a.d <= 2560)
            return run<BF16, 128, 3>(a, stream);
    }
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
    if (a.d <= 12288)
        return run<BF16, 512, 3>(a, stream);
    if (a.d <= 16384)
        return run<BF16, 512, 4>(a, stream);
    hipLaunchKernelGGL((layernorm_long_kernel<BF16>), dim3(grid_of(a.rows, 1)), dim3(1024), 0, stream, a);
}

// The forms of the gradient by the row's length: threads per row, threads of a workgroup, and
// workgroups that the chip is given, two to four on a CU: more leave more partial sums to write and
// join (bf16: 32768 x 4096: 195 us with 512 or 768 workgroups, 16384 x 6144: 151 against 173 us, 16384 x
// 8192: 214 us with 256, 266 with 384; 131072 x 1024: 185 us with 512, 193 with 768).
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
    if (d <= 384)
        return {16, 256, 768};
    if (d <= 512)
        return {64, 256, 512};
    if (d <= 768)
        return {32, 256, 768};
    if (d <= 1536)
        return {64, 256, 512};
    if (d <= 2560)
        return {128, 128, 1024};
    if (d <= 6144)
        return {256, 256, 512};
    return {512, 512, 256};
}

// Workgroups of the gradient kernel, and the rows that one takes at a time.
int64_t groups_of(int64_t rows, int64_t d, int *per_group)
{
    const GradForm f = grad_form(d);
    *per_group = f.nt / f.lpr;
    return std::min<int64_t>((rows + *per_group - 1) / *per_group, f.groups);
}
// Whether a row group has so many rows that its sums are taken in runs, into fp64 partials.
bool in_runs(int64_t rows, int64_t d)
{
    int per_group;
    return d > kGradWidest || rows > kRun * groups_of(rows, d, &per_group) * per_group;
}
// Parts of the rows for the weight gradients; for rows too long for the gradient kernel enough
// workgroups of columns for the chip.
int64_t parts_of(int64_t rows, int64_t d)
{
    if (d > kGradWidest)
        return std::max<int64_t>(1, std::min<int64_t>({rows / 4, 512, (8 << 20) / d}));
    int per_group;
    const int64_t groups = groups_of(rows, d, &per_group);
    return groups * (in_runs(rows, d) ? per_group : 1);
}

template <bool BF16, int LPR, int CH, int NT>
void run_grad(const LayerNormGrad &a, hipStream_t stream)
{
    constexpr int C = CH * 8 / kChunk<BF16>;
    constexpr bool NEXT = CH < (BF16 ? 4 : 3);   // (more elements a thread leave no registers for another row)
    const bool weights = a.dgain || a.dbias;
    int per_group;
    const dim3 grid((unsigned)groups_of(a.rows, a.d, &per_group));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, stream, a, weights, weights && in_runs(a.rows, a.d));
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
        else if (a.d <= 384)
            run_grad<BF16, 16, 3, 256>(a, stream);
        else if (a.d <= 512)
            run_grad<BF16, 64, 1, 256>(a, stream);
        else if (a.d <= 768)
            run_grad<BF16, 32, 3, 256>(a, stream);
        else if (a.d <= 1024)
            run_grad<BF16, 64, 2, 256>(a, stream);
        else if (a.d <= 1536)
            run_grad<BF16, 64, 3, 256>(a, stream);
        else if (a.d <= 2048)
            run_grad<BF16, 128, 2, 128>(a, stream);
        else if (a.d <= 2560)
            run_grad<BF16, 128, 3, 128>(a, stream);
        else if (a.d <= 4096)
            run_grad<BF16, 256, 2, 256>(a, stream);
        else if (a.d <= 6144)
            run_grad<BF16, 256, 3, 256>(a, stream);
        else if (a.d <= 8192)
            run_grad<BF16, 512, 2, 512>(a, stream);
        else if (a.d <= 12288)
            run_grad<BF16, 512, 3, 512>(a, stream);
        else
            run_grad<BF16, 512, 4, 512>(a, stream);
    }
    const int parts = a.rows > 0 ? (int)parts_of(a.rows, a.d) : 0;
    if (weights && a.rows > 0 && a.d > kGradWidest)
        hipLaunchKernelGGL((layernorm_columns_kernel<BF16>),
                           dim3((unsigned)((a.d + kColumnThreads * kChunk<BF16> - 1) / (kColumnThreads * kChunk<BF16>)),
                                (unsigned)parts),
                           dim3(kColumnThreads), 0, stream, a, (double *)a.partials);
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
