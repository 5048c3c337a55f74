// MXFP4 (OCP microscaling, 4-bit floating point): row codes, and the LM head on them.
//
// A row of d elements is cut into blocks of 32 (the last one filled up with zeros).  With amax
// the largest magnitude of a block,
//   e = clamp(floor(log2(amax)) - 2, -127, 127),  scale byte = e + 127 (E8M0),
//   code_k = the E2M1 value nearest to x_k 2^-e (ties to the even code, at most 6),
// so a code's value is 0, 0.5, 1, 1.5, 2, 3, 4 or 6 with a sign, and amax 2^-e lies in [4, 8): what
// is above 6 there is taken to 6, the rule of the format's specification.  x 2^-e is
// exact.  A block of zeros has scale byte 0; a block holding a NaN or an infinity has scale byte
// 255 (NaN) and codes 0.  Two codes make a byte, the even element in its low half.
//
// The product is out[i, v] = sum_b 2^(eh + ew) sum_{k in b} h_k w_k.  v_mfma_scale_f32_16x16x128
// multiplies four blocks a time: of each eight in turn, lanes (r, g) of the first instruction hold
// the 16 bytes of row r's block 2 g and their scale byte, those of the second block 2 g + 1.
// Products of codes are exact and sums are fp32; every form below adds the blocks in this order
// and so gives the same bits.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "launch.h"
#include "launch_head.h"
#include "row_ops.h"

namespace mosaic {
namespace {

using namespace rows;

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// Eight consecutive elements of a row a thread, four threads a block.  Bound: HBM.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(const void *__restrict__ X, int64_t nsrc, int32_t d,
                                                             int32_t blocks, const int32_t *__restrict__ row_idx,
                                                             int64_t rows, uint8_t *__restrict__ q,
                                                             uint8_t *__restrict__ scale, void *__restrict__ values)
{
    constexpr int ES = BF16 ? 2 : 4;
    const int64_t total = rows * blocks * 4;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / (blocks * 4);
        const int c = (int)(i - row * (blocks * 4)), k = c * 8;
        const int64_t src = row_idx ? (int64_t)row_idx[row] : row;
        const bool inside = src >= 0 && src < nsrc;   // a row id outside gives a row of NaN
        float x[8];
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            x[e] = k + e < d ? (inside ? load1(X, src * d + k + e, BF16) : __builtin_nanf("")) : 0.0f;
            top = max(top, __builtin_bit_cast(uint32_t, x[e]) & 0x7fffffffu);
        }
        // the four threads of a block are neighbours, and in the loop together
        top = max(top, (uint32_t)__shfl_xor((int)top, 1, 64));
        top = max(top, (uint32_t)__shfl_xor((int)top, 2, 64));
        const int field = (int)(top >> 23);
        const bool fine = field != 255;
        const int byte = fine ? max(field - 2, 0) : 255;
        const float down = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
        const float up = byte ? __builtin_bit_cast(float, (uint32_t)byte << 23) : 0x1p-127f;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = fine ? fabsf(x[e]) * down : 0.0f;
            // the number of midpoints that y has passed; a tie goes to the even code
            const uint32_t code = (uint32_t)(y > 0.25f) + (y >= 0.75f) + (y > 1.25f) + (y >= 1.75f) + (y > 2.5f) +
                                  (y >= 3.5f) + (y > 5.0f);
            const uint32_t sign = fine ? __builtin_bit_cast(uint32_t, x[e]) >> 31 : 0u;
            w |= (code | sign << 3) << (4 * e);
            const float v = code < 2 ? 0.5f * code : (code & 1 ? 1.5f : 1.0f) * (float)(1 << ((code >> 1) - 1));
            x[e] = fine ? (sign ? -v : v) * up : __builtin_nanf("");
        }
        if (q)
            *(uint32_t *)(q + (row * blocks + (c >> 2)) * 16 + (c & 3) * 4) = w;
        if (scale && (c & 3) == 0)
            scale[row * blocks + (c >> 2)] = (uint8_t)byte;
        if (values)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (k + e < d)
                    store1<BF16>((char *)values + row * d * ES, k + e, x[e]);
    }
}

__device__ __forceinline__ f32x4_t mfma_fp4(const i32x4_t &a, const i32x4_t &b, const f32x4_t &c, int sa, int sb)
{
    const i32x8_t x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
    const i32x8_t y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sa, 0, sb);
}

// Any sizes: a wave for 16 x 16 outputs, its operands straight from memory.
template <bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_mxfp4_any_kernel(const uint8_t *__restrict__ Hq,
                                                             const uint8_t *__restrict__ hs,
                                                             const int32_t *__restrict__ count, int32_t max_rows,
                                                             const uint8_t *__restrict__ Wq,
                                                             const uint8_t *__restrict__ ws, int32_t V, int32_t blocks,
                                                             void *__restrict__ out)
{
    const int rows = (int)row_count(count, max_rows);
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int64_t row_tiles = (rows + 15) / 16, tiles = row_tiles * ((V + 15) / 16);
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < tiles; t += (int64_t)gridDim.x * 4) {
        const int v0 = (int)(t / row_tiles) * 16, m0 = (int)(t % row_tiles) * 16;
        const int64_t wrow = (int64_t)min(v0 + r, V - 1) * blocks, hrow = (int64_t)min(m0 + r, rows - 1) * blocks;
        f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int kt = 0; kt < blocks; kt += 8) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int b = kt + 2 * g + s;
                i32x4_t w = {0, 0, 0, 0}, h = w;
                int sw = 0, sh = 0;
                if (b < blocks) {
                    w = *(const i32x4_t *)(Wq + (wrow + b) * 16);
                    h = *(const i32x4_t *)(Hq + (hrow + b) * 16);
                    sw = ws[wrow + b];
                    sh = hs[hrow + b];
                }
                acc = mfma_fp4(w, h, acc, sw, sh);
            }
        }
        // lane (r, g) holds entries 4 g .. 4 g + 3 of the tile for its row r
        const int row = m0 + r;
        if (row >= rows)
            continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (v0 + 4 * g + e < V)
                store1<OUT_BF16>(out, (int64_t)row * V + v0 + 4 * g + e, acc[e]);
    }
}

}  // namespace

hipError_t launch_quantize_rows_mxfp4(const void *X, bool in_bf16, int64_t nsrc, int64_t d, const int32_t *row_idx,
                                      int64_t rows, uint8_t *q, uint8_t *scale, void *values, hipStream_t stream)
{
    const int64_t blocks = mxfp4_blocks(d);
    const dim3 grid((unsigned)std::min<int64_t>((rows * blocks * 4 + 255) / 256, 1 << 20));
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, X, nsrc, (int32_t)d, (int32_t)blocks, row_idx, rows, q,
                           scale, values);
    };
    in_bf16 ? go(quantize_mxfp4_kernel<true>) : go(quantize_mxfp4_kernel<false>);
    return hipGetLastError();
}

hipError_t launch_gemm_mxfp4(const uint8_t *Hq, const uint8_t *hs, const int32_t *count, int64_t rows,
                             const uint8_t *Wq, const uint8_t *ws, int64_t V, int64_t blocks, void *out, bool out_bf16,
                             hipStream_t stream)
{
    const int64_t row_tiles = (rows + 15) / 16, tiles = row_tiles * ((V + 15) / 16);
    auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)std::min<int64_t>((tiles + 3) / 4, 1 << 20)), dim3(256), 0, stream, Hq,
                           hs, count, (int32_t)rows, Wq, ws, (int32_t)V, (int32_t)blocks, out);
    };
    out_bf16 ? go(gemm_mxfp4_any_kernel<true>) : go(gemm_mxfp4_any_kernel<false>);
    return hipGetLastError();
}

}  // namespace mosaic
