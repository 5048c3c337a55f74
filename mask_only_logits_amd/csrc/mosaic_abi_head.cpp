// C ABI of the layer norm, the MXFP4 head and the token log-probabilities (declared in
// include/mosaic.h).  Argument validation and the row-chunk driver; all of it on the host,
// before any HIP call, so a rejected call touches neither the device nor an output.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mosaic.h"
#include "abi_common.h"
#include "launch_head.h"
#include "launch_ops.h"

namespace {

using namespace mosaic::abi;

bool aligned_to(const void *p, int64_t bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// [rows, cols] with row stride ld: the bytes up to its last element stay inside int64.
bool strided_ok(int64_t rows, int64_t cols, int64_t ld, int64_t esize)
{
    return ld >= cols && checked_bytes(rows, ld, esize) >= 0;
}

mosaic_status_t status_of(hipError_t e) { return e == hipSuccess ? MOSAIC_OK : MOSAIC_ERR_DEVICE; }

// 64 x 64 tiles of outputs that one launch takes
bool tiles_fit(int64_t M, int64_t V) { return ceil_div(M, 64) <= ((1 << 24) - 1) / ceil_div(V, 64); }

}  // namespace

extern "C" {

mosaic_status_t mosaic_add_layernorm(const void *X, int64_t ldx, const void *R, int64_t ldr, int64_t nsrc, int64_t d,
                                     mosaic_dtype_t in_dtype, const void *gain, const void *bias,
                                     mosaic_dtype_t gain_dtype, float eps, const int32_t *row_idx,
                                     const int32_t *count, int64_t rows, void *sum, int64_t ldsum, void *out,
                                     double *stats, void *stream)
{
    const int64_t es = esize_of(in_dtype), gs = esize_of(gain_dtype);
    if (nsrc < 0 || d < 0 || rows < 0 || es == 0 || gs == 0 || !(eps >= 0x1p-126f) || !isfinite(eps))
        return MOSAIC_ERR_INVALID_ARG;
    if (rows == 0)
        return MOSAIC_OK;
    if (!X || d == 0 || nsrc == 0 || (!sum && !out && !stats) || (!row_idx && rows > nsrc))
        return MOSAIC_ERR_INVALID_ARG;
    if (!strided_ok(nsrc, d, ldx, es) || (R && !strided_ok(nsrc, d, ldr, es)) ||
        (sum && !strided_ok(rows, d, ldsum, es)) || checked_bytes(rows, d, es) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(X, es) || !aligned_to(R, es) || !aligned_to(sum, es) || !aligned_to(out, es) ||
        !aligned_to(gain, gs) || !aligned_to(bias, gs) || !aligned_to(row_idx, 4) || !aligned_to(count, 4) ||
        !aligned_to(stats, 8))
        return MOSAIC_ERR_INVALID_ARG;
    // in place: each element of the stream is read and written by the same thread, which
    // holds only when result row i is source row i
    if (sum && ((sum == X && (row_idx || ldsum != ldx)) || (sum == R && (row_idx || ldsum != ldr))))
        return MOSAIC_ERR_INVALID_ARG;
    if (out && (out == X || out == R || out == sum))
        return MOSAIC_ERR_INVALID_ARG;
    if (nsrc > kMaxPos || d > mosaic::kNormMaxWidth || rows > kMaxPos)
        return MOSAIC_ERR_UNSUPPORTED;
    mosaic::LayerNorm a;
    a.X = X;
    a.ldx = ldx;
    a.R = R;
    a.ldr = ldr;
    a.nsrc = nsrc;
    a.d = (int32_t)d;
    a.gain = gain;
    a.bias = bias;
    a.gain_bf16 = gain_dtype == MOSAIC_BF16;
    a.eps = (double)eps;
    a.row_idx = row_idx;
    a.count = count;
    a.rows = rows;
    a.sum = sum;
    a.ldsum = ldsum;
    a.out = out;
    a.stats = stats;
    return status_of(mosaic::launch_layernorm(a, in_dtype == MOSAIC_BF16, (hipStream_t)stream));
}

int64_t mosaic_layernorm_grad_workspace_bytes(int64_t rows, int64_t d)
{
    return rows < 0 || d < 0 || rows > kMaxPos || d > mosaic::kNormMaxWidth
               ? -1
               : mosaic::layernorm_grad_workspace_bytes(rows, d);
}

mosaic_status_t mosaic_layernorm_grad(const void *dY, int64_t lddy, const void *S, int64_t lds, int64_t nsrc, int64_t d,
                                      mosaic_dtype_t in_dtype, const double *stats, const void *gain,
                                      mosaic_dtype_t gain_dtype, const int32_t *row_idx, const int32_t *count,
                                      int64_t rows, const void *dsum, int64_t lddsum, void *dX, int64_t lddx,
                                      float *dgain, float *dbias, void *workspace, int64_t workspace_bytes,
                                      void *stream)
{
    const int64_t es = esize_of(in_dtype), gs = esize_of(gain_dtype);
    if (nsrc < 0 || d < 0 || rows < 0 || es == 0 || gs == 0)
        return MOSAIC_ERR_INVALID_ARG;
    const bool weights = dgain || dbias;
    if (d == 0 || (!dX && !weights) || !aligned_to(dgain, 4) || !aligned_to(dbias, 4) ||
        (dgain && dgain == dbias))
        return MOSAIC_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!dY || !S || !stats || nsrc == 0 || (!row_idx && rows > nsrc))
            return MOSAIC_ERR_INVALID_ARG;
        if (!strided_ok(rows, d, lddy, es) || !strided_ok(nsrc, d, lds, es) ||
            (dsum && !strided_ok(rows, d, lddsum, es)) || (dX && !strided_ok(rows, d, lddx, es)))
            return MOSAIC_ERR_INVALID_ARG;
        if (!aligned_to(dY, es) || !aligned_to(S, es) || !aligned_to(stats, 8) || !aligned_to(gain, gs) ||
            !aligned_to(row_idx, 4) || !aligned_to(count, 4) || !aligned_to(dsum, es) || !aligned_to(dX, es))
            return MOSAIC_ERR_INVALID_ARG;
        // in place: element by element, so the strides have to agree; S is read by other rows
        // too where a list names its rows
        if (dX && ((dX == dY && lddx != lddy) || (dX == dsum && lddx != lddsum) ||
                   (dX == S && (row_idx || lddx != lds))))
            return MOSAIC_ERR_INVALID_ARG;
    }
    if (nsrc > kMaxPos || d > mosaic::kNormMaxWidth || rows > kMaxPos)
        return MOSAIC_ERR_UNSUPPORTED;
    const int64_t need = mosaic::layernorm_grad_workspace_bytes(rows, d);
    if (weights && (!aligned16(workspace) || workspace_bytes < need || (need > 0 && !workspace)))
        return MOSAIC_ERR_INVALID_ARG;
    if (rows == 0 && !weights)
        return MOSAIC_OK;
    mosaic::LayerNormGrad a;
    a.dY = dY;
    a.lddy = lddy;
    a.S = S;
    a.lds = lds;
    a.nsrc = nsrc;
    a.d = (int32_t)d;
    a.stats = stats;
    a.gain = gain;
    a.gain_bf16 = gain_dtype == MOSAIC_BF16;
    a.row_idx = row_idx;
    a.count = count;
    a.rows = rows;
    a.dsum = dsum;
    a.lddsum = lddsum;
    a.dX = dX;
    a.lddx = lddx;
    a.dgain = dgain;
    a.dbias = dbias;
    a.partials = workspace;
    return status_of(mosaic::launch_layernorm_grad(a, in_dtype == MOSAIC_BF16, (hipStream_t)stream));
}

mosaic_status_t mosaic_quantize_rows_mxfp4(const void *X, int64_t nsrc, int64_t d, mosaic_dtype_t in_dtype,
                                           const int32_t *row_idx, int64_t rows, uint8_t *q, uint8_t *scale,
                                           void *values, void *stream)
{
    const int64_t es = esize_of(in_dtype);
    if (nsrc < 0 || d < 0 || rows < 0 || es == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (rows == 0 || d == 0)
        return MOSAIC_OK;
    if (!X || (!q && !values) || (q == nullptr) != (scale == nullptr) || nsrc == 0 || (!row_idx && rows > nsrc))
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(X, es) || !aligned16(q) || !aligned_to(values, es) || !aligned_to(row_idx, 4))
        return MOSAIC_ERR_INVALID_ARG;
    if (values == X && row_idx)   // in place: each element is read and written by the same thread
        return MOSAIC_ERR_INVALID_ARG;
    if (checked_bytes(nsrc, d, es) < 0 || checked_bytes(rows, d, es) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (nsrc > kMaxPos || d > mosaic::kNormMaxWidth || rows > kMaxPos)
        return MOSAIC_ERR_UNSUPPORTED;
    return status_of(mosaic::launch_quantize_rows_mxfp4(X, in_dtype == MOSAIC_BF16, nsrc, d, row_idx, rows, q, scale,
                                                        values, (hipStream_t)stream));
}

mosaic_status_t mosaic_quantized_logits_mxfp4(const uint8_t *Hq, const uint8_t *h_scale, int64_t M, const int32_t *count,
                                              const uint8_t *Wq, const uint8_t *w_scale, int64_t V, int64_t d, void *out,
                                              mosaic_dtype_t out_dtype, void *stream)
{
    const int64_t es = esize_of(out_dtype);
    if (M < 0 || V < 0 || d < 0 || es == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (M == 0 || V == 0)
        return MOSAIC_OK;
    if (!Hq || !h_scale || !Wq || !w_scale || !out || d == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned16(Hq) || !aligned16(Wq) || !aligned16(out) || !aligned_to(count, 4))
        return MOSAIC_ERR_INVALID_ARG;
    const int64_t blocks = mosaic::mxfp4_blocks(d);
    if (checked_bytes(M, V, es) < 0 || checked_bytes(M, blocks, 16) < 0 || checked_bytes(V, blocks, 16) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (M > kMaxPos || V > kMaxPos || !tiles_fit(M, V) || blocks > mosaic::kMxfp4MaxBlocks)
        return MOSAIC_ERR_UNSUPPORTED;
    return status_of(mosaic::launch_gemm_mxfp4(Hq, h_scale, count, M, Wq, w_scale, V, blocks, out,
                                               out_dtype == MOSAIC_BF16, (hipStream_t)stream));
}

int64_t mosaic_logits_mxfp4_workspace_bytes(int64_t M, int64_t chunk_rows, int64_t d)
{
    if (M < 0 || d < 0)
        return -1;
    const int64_t C = chunk_rows <= 0 || chunk_rows >= M ? M : chunk_rows;
    return checked_bytes(C, mosaic::mxfp4_blocks(d), 17);   // codes, then scale bytes
}

mosaic_status_t mosaic_masked_logits_mxfp4(const void *H, int64_t L, int64_t d, mosaic_dtype_t in_dtype,
                                           const int32_t *idx, int64_t M, const uint8_t *Wq, const uint8_t *w_scale,
                                           int64_t V, void *out, int64_t chunk_rows, mosaic_dtype_t out_dtype,
                                           void *workspace, int64_t workspace_bytes, void *stream)
{
    const int64_t in_es = esize_of(in_dtype), es = esize_of(out_dtype);
    if (M < 0 || V < 0 || L < 0 || d < 0 || in_es == 0 || es == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (M == 0 || V == 0)
        return MOSAIC_OK;
    if (!H || !idx || !Wq || !w_scale || !out || !workspace || L == 0 || d == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(H, in_es) || !aligned16(Wq) || !aligned16(out) || !aligned16(workspace) || !aligned_to(idx, 4))
        return MOSAIC_ERR_INVALID_ARG;
    const int64_t blocks = mosaic::mxfp4_blocks(d);
    if (checked_bytes(M, V, es) < 0 || checked_bytes(L, d, in_es) < 0 || checked_bytes(V, blocks, 16) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    const int64_t K = mosaic_num_chunks(M, chunk_rows);
    const int64_t C = K == 1 ? M : chunk_rows;
    const int64_t need = mosaic_logits_mxfp4_workspace_bytes(M, chunk_rows, d);
    if (need < 0 || workspace_bytes < need)
        return MOSAIC_ERR_INVALID_ARG;
    // (M: the list may hold more rows than a chunk, but the debug check counts it in one)
    if (L > kMaxPos || V > kMaxPos || C > kMaxPos || blocks > mosaic::kMxfp4MaxBlocks || !tiles_fit(C, V))
        return MOSAIC_ERR_UNSUPPORTED;
    const mosaic_status_t ck = check_idx_if_asked(idx, M, L, (hipStream_t)stream);
    if (ck != MOSAIC_OK)
        return ck;
    uint8_t *hq = (uint8_t *)workspace, *hs = hq + C * blocks * 16;
    for (int64_t k = 0; k < K; ++k) {
        const int64_t r0 = k * C, n = r0 + C < M ? C : M - r0;
        // out starts at a multiple of 16 bytes in the first chunk only; the kernels take any
        if (mosaic::launch_quantize_rows_mxfp4(H, in_dtype == MOSAIC_BF16, L, d, idx + r0, n, hq, hs, nullptr,
                                               (hipStream_t)stream) != hipSuccess ||
            mosaic::launch_gemm_mxfp4(hq, hs, nullptr, n, Wq, w_scale, V, blocks, (char *)out + r0 * V * es,
                                      out_dtype == MOSAIC_BF16, (hipStream_t)stream) != hipSuccess)
            return MOSAIC_ERR_DEVICE;
    }
    return MOSAIC_OK;
}

int64_t mosaic_token_logprobs_workspace_bytes(int64_t M, int64_t V, int64_t top_n)
{
    return M < 0 || V < 0 || top_n < 0 || top_n > mosaic::kTopMax || M > kMaxPos || V > mosaic::kTokenLogprobsMaxV
               ? -1
               : mosaic::token_logprobs_workspace_bytes(M, V, top_n);
}

// What both entry points check of the arguments they share, and `a` filled from them.
// MOSAIC_OK with a.rows == 0: nothing to do.
static mosaic_status_t logprob_args(const void *logits, int64_t ldz, int64_t M, int64_t V, mosaic_dtype_t dtype,
                                    const int32_t *tokens, float temperature, const int32_t *count,
                                    mosaic::TokenLogprobs &a)
{
    const int64_t es = esize_of(dtype);
    if (M < 0 || V < 0 || es == 0 || !(temperature >= 0x1p-20f && temperature <= 0x1p20f))
        return MOSAIC_ERR_INVALID_ARG;
    if (M == 0)
        return MOSAIC_OK;
    if (!logits || V == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(tokens, 4) || !aligned_to(count, 4) || !strided_ok(M, V, ldz, es))
        return MOSAIC_ERR_INVALID_ARG;
    if (M > kMaxPos || V > mosaic::kTokenLogprobsMaxV)
        return MOSAIC_ERR_UNSUPPORTED;
    a.Z = logits;
    a.ldz = ldz;
    a.rows = M;
    a.count = count;
    a.V = (int32_t)V;
    a.temperature = temperature;
    a.tokens = tokens;
    return MOSAIC_OK;
}

mosaic_status_t mosaic_token_logprobs(const void *logits, int64_t ldz, int64_t M, int64_t V, mosaic_dtype_t dtype,
                                      const int32_t *tokens, float temperature, const int32_t *count, float *logprob,
                                      float *entropy, int64_t top_n, int32_t *top_ids, float *top_logprobs,
                                      float *stats, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (top_n < 0)
        return MOSAIC_ERR_INVALID_ARG;
    mosaic::TokenLogprobs a;
    const mosaic_status_t s = logprob_args(logits, ldz, M, V, dtype, tokens, temperature, count, a);
    if (s != MOSAIC_OK || a.rows == 0)
        return s;
    if (!stats || (tokens == nullptr) != (logprob == nullptr) || (top_n > 0 && (!top_ids || !top_logprobs)) ||
        !aligned_to(logprob, 4) || !aligned_to(entropy, 4) || !aligned_to(stats, 8) || !aligned_to(top_ids, 4) ||
        !aligned_to(top_logprobs, 4))
        return MOSAIC_ERR_INVALID_ARG;
    if (top_n > mosaic::kTopMax)
        return MOSAIC_ERR_UNSUPPORTED;
    const int64_t need = mosaic::token_logprobs_workspace_bytes(M, V, top_n);
    if (!aligned16(workspace) || workspace_bytes < need || (need > 0 && !workspace))
        return MOSAIC_ERR_INVALID_ARG;
    a.logprob = logprob;
    a.entropy = entropy;
    a.top_n = (int32_t)top_n;
    a.top_ids = top_ids;
    a.top_logprobs = top_logprobs;
    a.stats = stats;
    a.workspace = workspace;
    return status_of(mosaic::launch_token_logprobs(a, dtype == MOSAIC_BF16, (hipStream_t)stream));
}

mosaic_status_t mosaic_token_logprobs_grad(const void *logits, int64_t ldz, int64_t M, int64_t V, mosaic_dtype_t dtype,
                                           const int32_t *tokens, float temperature, const int32_t *count,
                                           const float *stats, const float *entropy, const float *grad_logprob,
                                           const float *grad_entropy, void *grad, int64_t ldg, void *stream)
{
    mosaic::TokenLogprobs a;
    const mosaic_status_t s = logprob_args(logits, ldz, M, V, dtype, tokens, temperature, count, a);
    if (s != MOSAIC_OK || a.rows == 0)
        return s;
    if (!stats || !grad || (!grad_logprob && !grad_entropy) || (tokens == nullptr) != (grad_logprob == nullptr) ||
        (grad_entropy && !entropy))
        return MOSAIC_ERR_INVALID_ARG;
    const int64_t es = esize_of(dtype);
    if (!aligned_to(stats, 8) || !aligned_to(entropy, 4) || !aligned_to(grad_logprob, 4) ||
        !aligned_to(grad_entropy, 4) || !aligned_to(grad, es) || !strided_ok(M, V, ldg, es) ||
        (grad == logits && ldg != ldz))
        return MOSAIC_ERR_INVALID_ARG;
    a.stats = const_cast<float *>(stats);
    a.entropy = const_cast<float *>(entropy);
    a.grad_logprob = grad_logprob;
    a.grad_entropy = grad_entropy;
    a.grad = grad;
    a.ldg = ldg;
    return status_of(mosaic::launch_token_logprobs_grad(a, dtype == MOSAIC_BF16, (hipStream_t)stream));
}

}  // extern "C"
