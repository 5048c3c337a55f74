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

// Rows of any length: read once for the sums and again for the results.
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

// The gradient of rows of any length: read twice.
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
    partials[(int64_t)blockIdx.y * 2 * a.d + k] = dg;
    partials[((int64_t)blockIdx.y * 2 + 1) * a.d + k] = db;
}

// The weight gradients from `parts` partial sums [parts][2][d].
template <typename T>
__global__ __launch_bounds__(kColumns) void layernorm_join_kernel(const T *__restrict__ partials, int parts, int32_t d,
                                                                  float *__restrict__ dgain, float *__restrict__ dbias)
{
    const int k = blockIdx.x * kColumns + threadIdx.x;
    if (k >= d)
        return;
    double dg = 0.0, db = 0.0;
    for (int p = 0; p < parts; ++p) {
        dg += (double)partials[(int64_t)p * 2 * d + k];
        db += (double)partials[((int64_t)p * 2 + 1) * d + k];
    }
    if (dgain)
        dgain[k] = (float)dg;
    if (dbias)
        dbias[k] = (float)db;
}

unsigned grid_of(int64_t rows) { return (unsigned)std::min<int64_t>(rows, 1 << 20); }

// Parts of the rows for the weight gradients: enough workgroups of columns for the chip.
int column_parts(int64_t rows, int64_t d)
{
    const int64_t wide = (d + kColumns - 1) / kColumns;
    return (int)std::max<int64_t>(1, std::min<int64_t>({rows, 512, 4096 / wide}));
}

template <bool BF16>
hipError_t run_grad(const LayerNormGrad &a, hipStream_t stream)
{
    if (a.dgain || a.dbias) {
        const int parts = a.rows > 0 ? column_parts(a.rows, a.d) : 0;
        const unsigned wide = (unsigned)((a.d + (int64_t)kColumns - 1) / kColumns);
        double *p = (double *)a.partials;
        if (parts > 0)
            hipLaunchKernelGGL((layernorm_columns_kernel<BF16>), dim3(wide, (unsigned)parts), dim3(kColumns), 0, stream, a,
                               p);
        hipLaunchKernelGGL((layernorm_join_kernel<double>), dim3(wide), dim3(kColumns), 0, stream, (const double *)p,
                           parts, a.d, a.dgain, a.dbias);
    }
    // last: dX may be dY itself
    if (a.dX && a.rows > 0)
        hipLaunchKernelGGL((layernorm_grad_long_kernel<BF16>), dim3(grid_of(a.rows)), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

}  // namespace

int64_t layernorm_grad_workspace_bytes(int64_t rows, int64_t d)
{
    return rows == 0 || d == 0 ? 0 : (int64_t)column_parts(rows, d) * 2 * d * 8;
}

hipError_t launch_layernorm(const LayerNorm &a, bool in_bf16, hipStream_t stream)
{
    if (in_bf16)
        hipLaunchKernelGGL((layernorm_long_kernel<true>), dim3(grid_of(a.rows)), dim3(1024), 0, stream, a);
    else
        hipLaunchKernelGGL((layernorm_long_kernel<false>), dim3(grid_of(a.rows)), dim3(1024), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_layernorm_grad(const LayerNormGrad &a, bool in_bf16, hipStream_t stream)
{
    return in_bf16 ? run_grad<true>(a, stream) : run_grad<false>(a, stream);
}

}  // namespace mosaic
