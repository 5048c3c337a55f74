// C ABI of the operators around the LM head (declared in include/mosaic.h): residual
// addition with root-mean-square norm, the INT8 head and the distillation loss.  Argument
// validation and the row-chunk driver; all of it on the host, before any HIP call, so a
// rejected call touches neither the device nor an output.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/mosaic.h"
#include "abi_common.h"
#include "launch.h"
#include "launch_ops.h"

namespace {

using namespace mosaic::abi;

bool aligned_to(const void *p, int64_t bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

bool known(mosaic_code_t c) { return c == MOSAIC_E4M3 || c == MOSAIC_INT8; }

// [rows, cols] with row stride ld: the bytes up to its last element stay inside int64.
bool strided_ok(int64_t rows, int64_t cols, int64_t ld, int64_t esize)
{
    return ld >= cols && checked_bytes(rows, ld, esize) >= 0;
}

mosaic_status_t status_of(hipError_t e) { return e == hipSuccess ? MOSAIC_OK : MOSAIC_ERR_DEVICE; }

// A launch of 256 threads for each 64 x 64 tile of outputs stays inside the grid's limit.
bool int8_grid_fits(int64_t M, int64_t V) { return ceil_div(M, 64) <= ((1 << 24) - 1) / ceil_div(V, 64); }

}  // namespace

extern "C" {

mosaic_status_t mosaic_add_rmsnorm(const void *X, int64_t ldx, const void *R, int64_t ldr, int64_t nsrc, int64_t d,
                                   mosaic_dtype_t in_dtype, const void *gain, mosaic_dtype_t gain_dtype, float eps,
                                   const int32_t *row_idx, const int32_t *count, int64_t rows, void *sum,
                                   int64_t ldsum, void *out, mosaic_code_t code, void *q, float *scale,
                                   void *stream)
{
    const int64_t es = esize_of(in_dtype), gs = esize_of(gain_dtype);
    if (nsrc < 0 || d < 0 || rows < 0 || es == 0 || gs == 0 || !(eps >= 0x1p-126f) || !isfinite(eps) ||
        (q && !known(code)))
        return MOSAIC_ERR_INVALID_ARG;
    if (rows == 0)
        return MOSAIC_OK;
    if (!X || !gain || d == 0 || nsrc == 0 || (!sum && !out && !q) || (q && !scale) || (!row_idx && rows > nsrc))
        return MOSAIC_ERR_INVALID_ARG;
    if (!strided_ok(nsrc, d, ldx, es) || (R && !strided_ok(nsrc, d, ldr, es)) ||
        (sum && !strided_ok(rows, d, ldsum, es)) || checked_bytes(rows, d, es) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(X, es) || !aligned_to(R, es) || !aligned_to(sum, es) || !aligned_to(out, es) ||
        !aligned_to(gain, gs) || !aligned_to(row_idx, 4) || !aligned_to(count, 4) || !aligned_to(scale, 4))
        return MOSAIC_ERR_INVALID_ARG;
    // in place: each element of the stream is read and written by the same thread, which
    // holds only when result row i is source row i
    if (sum && ((sum == X && (row_idx || ldsum != ldx)) || (sum == R && (row_idx || ldsum != ldr))))
        return MOSAIC_ERR_INVALID_ARG;
    if (out && (out == X || out == R || out == sum))
        return MOSAIC_ERR_INVALID_ARG;
    if (nsrc > kMaxPos || d > mosaic::kNormMaxWidth || rows > kMaxPos)
        return MOSAIC_ERR_UNSUPPORTED;
    mosaic::RowsNorm a;
    a.X = X;
    a.ldx = ldx;
    a.R = R;
    a.ldr = ldr;
    a.nsrc = nsrc;
    a.d = (int32_t)d;
    a.gain = gain;
    a.gain_bf16 = gain_dtype == MOSAIC_BF16;
    a.eps = eps;
    a.eps_low = eps * 0x1p-80f * 0x1p-80f;   // (2^-160 itself is no fp32 number)
    a.row_idx = row_idx;
    a.count = count;
    a.rows = rows;
    a.sum = sum;
    a.ldsum = ldsum;
    a.out = out;
    a.code_int8 = code == MOSAIC_INT8;
    a.q = (uint8_t *)q;
    a.scale = scale;
    return status_of(mosaic::launch_rows_norm(a, in_dtype == MOSAIC_BF16, true, (hipStream_t)stream));
}

// Rows X[row_idx[r]] (or X[r]) to INT8 codes and scales; the arguments have been checked.
static hipError_t quantize_int8(const void *X, int64_t nsrc, int64_t d, mosaic_dtype_t in_dtype,
                                const int32_t *row_idx, int64_t rows, int8_t *q, float *scale, hipStream_t stream)
{
    mosaic::RowsNorm a;
    a.X = X;
    a.ldx = d;
    a.nsrc = nsrc;
    a.d = (int32_t)d;
    a.row_idx = row_idx;
    a.rows = rows;
    a.code_int8 = true;
    a.q = (uint8_t *)q;
    a.scale = scale;
    return mosaic::launch_rows_norm(a, in_dtype == MOSAIC_BF16, false, stream);
}

mosaic_status_t mosaic_quantize_rows_int8(const void *X, int64_t nsrc, int64_t d, mosaic_dtype_t in_dtype,
                                          const int32_t *row_idx, int64_t rows, int8_t *q, float *scale,
                                          void *stream)
{
    const int64_t es = esize_of(in_dtype);
    if (nsrc < 0 || d < 0 || rows < 0 || es == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (rows == 0 || d == 0)
        return MOSAIC_OK;
    if (!X || !q || !scale || nsrc == 0 || (!row_idx && rows > nsrc))
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(X, es) || !aligned_to(scale, 4) || !aligned_to(row_idx, 4))
        return MOSAIC_ERR_INVALID_ARG;
    if (checked_bytes(nsrc, d, es) < 0 || checked_bytes(rows, d, 1) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (nsrc > kMaxPos || d > mosaic::kNormMaxWidth || rows > kMaxPos)
        return MOSAIC_ERR_UNSUPPORTED;
    return status_of(quantize_int8(X, nsrc, d, in_dtype, row_idx, rows, q, scale, (hipStream_t)stream));
}

mosaic_status_t mosaic_quantized_logits(mosaic_code_t code, const void *Hq, const float *h_scale, int64_t M,
                                        const int32_t *count, const void *Wq, const float *w_scale, int64_t V,
                                        int64_t d, void *out, mosaic_dtype_t out_dtype, void *stream)
{
    const int64_t es = esize_of(out_dtype);
    if (M < 0 || V < 0 || d < 0 || es == 0 || !known(code))
        return MOSAIC_ERR_INVALID_ARG;
    if (M == 0 || V == 0)
        return MOSAIC_OK;
    const bool e4m3 = code == MOSAIC_E4M3;
    if (e4m3 && (out_dtype != MOSAIC_BF16 || d % 128 != 0 || d > (1 << 22) || count))
        return MOSAIC_ERR_UNSUPPORTED;
    if (!Hq || !h_scale || !Wq || !w_scale || !out || d == 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned_to(h_scale, 4) || !aligned_to(w_scale, e4m3 ? 16 : 4) || !aligned_to(count, 4) ||
        (e4m3 && (!aligned16(Hq) || !aligned16(Wq))))
        return MOSAIC_ERR_INVALID_ARG;
    if (checked_bytes(M, V, es) < 0 || checked_bytes(M, d, 1) < 0 || checked_bytes(V, d, 1) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (M > kMaxPos || V > kMaxPos || d > kMaxPos || !int8_grid_fits(M, V) || (!e4m3 && d > mosaic::kInt8MaxDepth))
        return MOSAIC_ERR_UNSUPPORTED;
    if (!e4m3)
        return status_of(mosaic::launch_gemm_int8((const int8_t *)Hq, h_scale, count, M, (const int8_t *)Wq, w_scale,
                                                  V, d, out, out_dtype == MOSAIC_BF16, V, (hipStream_t)stream));
    const uint8_t *hq = (const uint8_t *)Hq, *wq = (const uint8_t *)Wq;
    return status_of(M <= 64 ? mosaic::launch_gemm_fp8_lowm(hq, h_scale, M, wq, w_scale, V, d, out, V,
                                                            (hipStream_t)stream)
                             : mosaic::launch_gemm_fp8(hq, h_scale, M, wq, w_scale, V, d, out, V, 0, 0,
                                                       (hipStream_t)stream));
}

int64_t mosaic_logits_int8_workspace_bytes(int64_t M, int64_t chunk_rows, int64_t d)
{
    return mosaic_logits_fp8_workspace_bytes(M, chunk_rows, d);   // one byte a code, four a scale, as there
}

mosaic_status_t mosaic_masked_logits_int8(const void *H, int64_t L, int64_t d, mosaic_dtype_t in_dtype,
                                          const int32_t *idx, int64_t M, const int8_t *Wq, const float *w_scale,
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
    if (!aligned_to(H, in_es) || !aligned16(out) || !aligned16(workspace) || !aligned_to(idx, 4) ||
        !aligned_to(w_scale, 4))
        return MOSAIC_ERR_INVALID_ARG;
    if (checked_bytes(M, V, es) < 0 || checked_bytes(L, d, in_es) < 0 || checked_bytes(V, d, 1) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    const int64_t K = mosaic_num_chunks(M, chunk_rows);
    const int64_t C = K == 1 ? M : chunk_rows;
    const int64_t need = mosaic_logits_int8_workspace_bytes(M, chunk_rows, d);
    if (need < 0 || workspace_bytes < need)
        return MOSAIC_ERR_INVALID_ARG;
    if (L > kMaxPos || V > kMaxPos || C > kMaxPos || d > mosaic::kInt8MaxDepth || !int8_grid_fits(C, V))
        return MOSAIC_ERR_UNSUPPORTED;
    const mosaic_status_t ck = check_idx_if_asked(idx, M, L, (hipStream_t)stream);
    if (ck != MOSAIC_OK)
        return ck;
    // workspace: the chunk's codes [C, d], then its row scales [C]
    int8_t *hq = (int8_t *)workspace;
    float *hs = (float *)((char *)workspace + ceil_div(C * d, 16) * 16);
    for (int64_t k = 0; k < K; ++k) {
        const int64_t r0 = k * C, n = r0 + C < M ? C : M - r0;
        if (quantize_int8(H, L, d, in_dtype, idx + r0, n, hq, hs, (hipStream_t)stream) != hipSuccess ||
            mosaic::launch_gemm_int8(hq, hs, nullptr, n, Wq, w_scale, V, d, (char *)out + r0 * V * es,
                                     out_dtype == MOSAIC_BF16, V, (hipStream_t)stream) != hipSuccess)
            return MOSAIC_ERR_DEVICE;
    }
    return MOSAIC_OK;
}

int64_t mosaic_distill_topk_workspace_bytes(int64_t M, int64_t V, int64_t K)
{
    return M < 0 || V < 0 || K < 0 || K > mosaic::kDistillMaxK ? -1 : mosaic::distill_workspace_bytes(M, V, K);
}

// What both distillation entry points check of the arguments they share, and `a` filled from
// them.  MOSAIC_OK with a.rows == 0: nothing to do.
static mosaic_status_t distill_args(const void *logits, int64_t ldz, int64_t M, int64_t V, mosaic_dtype_t dtype,
                                    const void *top, mosaic_dtype_t top_dtype, const int32_t *ids, int64_t K,
                                    float temperature, const int32_t *count, const float *grad_loss, void *grad,
                                    int64_t ldg, mosaic::Distill &a)
{
    const int64_t es = esize_of(dtype), ts = esize_of(top_dtype);
    if (M < 0 || V < 0 || K < 0 || es == 0 || ts == 0 || !(temperature >= 0x1p-20f && temperature <= 0x1p20f))
        return MOSAIC_ERR_INVALID_ARG;
    if (M == 0)
        return MOSAIC_OK;
    if (!logits || V == 0 || (K > 0 && (!top || !ids)))
        return MOSAIC_ERR_INVALID_ARG;
    if (!aligned_to(logits, es) || !aligned_to(grad, es) || !aligned_to(top, ts) || !aligned_to(ids, 4) ||
        !aligned_to(count, 4) || !aligned_to(grad_loss, 4))
        return MOSAIC_ERR_INVALID_ARG;
    if (!strided_ok(M, V, ldz, es) || (grad && !strided_ok(M, V, ldg, es)) || checked_bytes(M, K, 4) < 0)
        return MOSAIC_ERR_INVALID_ARG;
    if (grad == logits && ldg != ldz)
        return MOSAIC_ERR_INVALID_ARG;
    if (M > kMaxPos || V > mosaic::kDistillMaxV || K > mosaic::kDistillMaxK)
        return MOSAIC_ERR_UNSUPPORTED;
    a.Z = logits;
    a.ldz = ldz;
    a.rows = M;
    a.count = count;
    a.V = (int32_t)V;
    a.top = top;
    a.top_bf16 = top_dtype == MOSAIC_BF16;
    a.ids = ids;
    a.K = (int32_t)K;
    a.temperature = temperature;
    a.grad_loss = grad_loss;
    a.grad = grad;
    a.ldg = ldg;
    return MOSAIC_OK;
}

mosaic_status_t mosaic_distill_topk(const void *logits, int64_t ldz, int64_t M, int64_t V, mosaic_dtype_t dtype,
                                    const void *teacher_logits, mosaic_dtype_t teacher_dtype,
                                    const int32_t *teacher_ids, int64_t K, float temperature, const int32_t *count,
                                    float *loss, float *stats, const float *grad_loss, void *grad, int64_t ldg,
                                    void *workspace, int64_t workspace_bytes, void *stream)
{
    mosaic::Distill a;
    const mosaic_status_t s = distill_args(logits, ldz, M, V, dtype, teacher_logits, teacher_dtype, teacher_ids, K,
                                           temperature, count, grad_loss, grad, ldg, a);
    if (s != MOSAIC_OK || a.rows == 0)
        return s;
    const int64_t need = mosaic::distill_workspace_bytes(M, V, K);
    if (!loss || !stats || !aligned_to(loss, 4) || !aligned_to(stats, 8) || !aligned16(workspace) ||
        workspace_bytes < need || (need > 0 && !workspace))
        return MOSAIC_ERR_INVALID_ARG;
    a.loss = loss;
    a.stats = stats;
    a.partials = (float *)workspace;
    return status_of(mosaic::launch_distill(a, dtype == MOSAIC_BF16, (hipStream_t)stream));
}

mosaic_status_t mosaic_distill_topk_grad(const void *logits, int64_t ldz, int64_t M, int64_t V,
                                         mosaic_dtype_t dtype, const void *teacher_logits,
                                         mosaic_dtype_t teacher_dtype, const int32_t *teacher_ids, int64_t K,
                                         float temperature, const int32_t *count, const float *stats,
                                         const float *grad_loss, void *grad, int64_t ldg, void *stream)
{
    mosaic::Distill a;
    const mosaic_status_t s = distill_args(logits, ldz, M, V, dtype, teacher_logits, teacher_dtype, teacher_ids, K,
                                           temperature, count, grad_loss, grad, ldg, a);
    if (s != MOSAIC_OK || a.rows == 0)
        return s;
    if (!grad || !stats || !aligned_to(stats, 8))
        return MOSAIC_ERR_INVALID_ARG;
    a.stats = const_cast<float *>(stats);
    return status_of(mosaic::launch_distill_grad(a, dtype == MOSAIC_BF16, (hipStream_t)stream));
}

}  // extern "C"
