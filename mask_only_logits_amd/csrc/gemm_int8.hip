// INT8 LM head: products of 8-bit integer codes with a scale per row (token) and per
// vocabulary entry (channel),
//   out[i, v] = (sum_k Hq[i, k] Wq[v, k]) * hs[i] * ws[v].
// The sums are exact in int32 (d <= 131071, codes of magnitude 128 at most), so every form
// below gives the same bits, whatever its order: the sum is converted to fp32 (one rounding
// above 2^24), multiplied by hs[i], then by ws[v], and rounded to bf16 where that is the
// output's type.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"
#include "row_ops.h"

namespace mosaic {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Four consecutive vocabulary entries v .. v + 3 of one row; vec: the address is a multiple of
// the four values' size.
template <bool OUT_BF16>
__device__ __forceinline__ void store4(void *out, int64_t off, const float (&x)[4], int v, int V, bool vec)
{
    if (vec && v + 3 < V) {
        if constexpr (OUT_BF16)
            *(u32x2_t *)((uint16_t *)out + off) = u32x2_t{rows::pack_bf16(x[0], x[1]), rows::pack_bf16(x[2], x[3])};
        else
            *(f32x4_t *)((float *)out + off) = f32x4_t{x[0], x[1], x[2], x[3]};
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (v + e < V) {
            if constexpr (OUT_BF16)
                ((__bf16 *)out)[off + e] = static_cast<__bf16>(x[e]);
            else
                ((float *)out)[off + e] = x[e];
        }
    }
}

// Any shape and alignment.  64 x 64 outputs per workgroup of four waves, 32 x 32 each; K in
// steps of 64 codes, staged through registers into LDS (rows of 64 + 16 bytes, so that the
// 16-byte fragment reads spread over the banks); codes past d, V or the rows are zeros.
template <bool OUT_BF16, bool ALIGNED>
__global__ __launch_bounds__(256) void gemm_int8_any_kernel(const int8_t *__restrict__ Hq,
                                                            const float *__restrict__ hs,
                                                            const int32_t *__restrict__ count, int32_t max_rows,
                                                            const int8_t *__restrict__ Wq,
                                                            const float *__restrict__ ws, int32_t V, int32_t d,
                                                            void *__restrict__ out, int64_t ldo)
{
    constexpr int BK = 64, PITCH = BK + 16;
    __shared__ __attribute__((aligned(16))) char smem[2 * 128 * PITCH];
    const int rows = (int)rows::row_count(count, max_rows);
    const int nvt = (V + 63) / 64;
    const int v0 = (int)(blockIdx.x % nvt) * 64, m0 = (int)(blockIdx.x / nvt) * 64;
    if (m0 >= rows)
        return;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // thread t stages 16 codes of W row t / 4 and of H row t / 4
    const int sr = tid >> 2, sk = (tid & 3) * 16;
    const bool w_ok = v0 + sr < V, h_ok = m0 + sr < rows;
    const int8_t *wp = Wq + (int64_t)(w_ok ? v0 + sr : 0) * d;
    const int8_t *hp = Hq + (int64_t)(h_ok ? m0 + sr : 0) * d;
    auto fetch = [&](const int8_t *p, bool ok, int k) {
        i32x4_t r = {0, 0, 0, 0};
        if (!ok || k >= d)
            return r;
        if constexpr (ALIGNED)   // d % 16 == 0 and 16-byte aligned rows: whole or nothing
            return *(const i32x4_t *)(p + k);
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (k + b < d)
                r[b >> 2] |= (int)((uint32_t)(uint8_t)p[k + b] << (8 * (b & 3)));
        return r;
    };
    auto put = [&](int stage, const i32x4_t &w, const i32x4_t &h) {
        char *s = smem + stage * 128 * PITCH + sr * PITCH + sk;
        *(i32x4_t *)s = w;
        *(i32x4_t *)(s + 64 * PITCH) = h;
    };
    const int wv = (wave & 1) * 32, wm = (wave >> 1) * 32;
    const int fr = lane & 15, kg = lane >> 4;
    i32x4_t acc[2][2];
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int b = 0; b < 2; ++b)
            acc[a][b] = i32x4_t{0, 0, 0, 0};
    const int nk = (d + BK - 1) / BK;
    i32x4_t w = fetch(wp, w_ok, sk), h = fetch(hp, h_ok, sk);
    put(0, w, h);
    __syncthreads();
    for (int kt = 0; kt < nk; ++kt) {
        const char *s = smem + (kt & 1) * 128 * PITCH;
        if (kt + 1 < nk) {
            w = fetch(wp, w_ok, (kt + 1) * BK + sk);
            h = fetch(hp, h_ok, (kt + 1) * BK + sk);
        }
        i32x4_t af[2], bf[2];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            af[a] = *(const i32x4_t *)(s + (wv + a * 16 + fr) * PITCH + kg * 16);
            bf[a] = *(const i32x4_t *)(s + (64 + wm + a * 16 + fr) * PITCH + kg * 16);
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
                acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[a], bf[b], acc[a][b], 0, 0, 0);
        if (kt + 1 < nk)
            put((kt + 1) & 1, w, h);   // last read two steps ago, a barrier in between
        __syncthreads();
    }
    // lane (fr, kg) holds entries 4 kg .. 4 kg + 3 of a 16-entry block for row fr of a 16-row block
    const bool vec = OUT_BF16 ? ((uintptr_t)out & 7) == 0 && (ldo & 3) == 0
                              : ((uintptr_t)out & 15) == 0 && (ldo & 3) == 0;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int row = m0 + wm + b * 16 + fr;
        if (row >= rows)
            continue;
        const float hsc = hs[row];
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const int v = v0 + wv + a * 16 + kg * 4;
            if (v >= V)
                continue;
            float x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = (float)acc[a][b][e] * hsc * ws[min(v + e, V - 1)];
            store4<OUT_BF16>(out, (int64_t)row * ldo + v, x, v, V, vec);
        }
    }
}

}  // namespace

hipError_t launch_gemm_int8(const int8_t *Hq, const float *hs, const int32_t *count, int64_t rows, const int8_t *Wq,
                            const float *ws, int64_t V, int64_t d, void *out, bool out_bf16, int64_t ldo,
                            hipStream_t stream)
{
    const bool aligned = d % 16 == 0 && ((uintptr_t)Hq & 15) == 0 && ((uintptr_t)Wq & 15) == 0;
    const dim3 grid((unsigned)(((V + 63) / 64) * ((rows + 63) / 64)));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, Hq, hs, count, (int32_t)rows, Wq, ws, (int32_t)V,
                           (int32_t)d, out, ldo);
    };
    if (out_bf16)
        aligned ? go(gemm_int8_any_kernel<true, true>) : go(gemm_int8_any_kernel<true, false>);
    else
        aligned ? go(gemm_int8_any_kernel<false, true>) : go(gemm_int8_any_kernel<false, false>);
    return hipGetLastError();
}

}  // namespace mosaic
