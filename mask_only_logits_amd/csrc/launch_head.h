// Launchers of the layer norm, the MXFP4 head and the token log-probabilities.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mosaic {

// Layer norm with residual addition (layernorm.hip).
struct LayerNorm {
    const void *X = nullptr;            // [nsrc, d], row stride ldx elements
    int64_t ldx = 0;
    const void *R = nullptr;            // residual, as X, or null
    int64_t ldr = 0;
    int64_t nsrc = 0;
    int32_t d = 0;
    const void *gain = nullptr;         // [d] or null (1)
    const void *bias = nullptr;         // [d] or null (0)
    bool gain_bf16 = false;             // type of both
    double eps = 0.0;
    const int32_t *row_idx = nullptr;   // row r of the results is source row row_idx[r] (null: r)
    const int32_t *count = nullptr;     // device-side row count (null: rows)
    int64_t rows = 0;
    void *sum = nullptr;                // [rows, d], row stride ldsum, or null
    int64_t ldsum = 0;
    void *out = nullptr;                // [rows, d] or null
    double *stats = nullptr;            // [rows, 2]: mean, 1 / sqrt(variance + eps); or null
};
// 1 <= d <= kNormMaxWidth (launch_ops.h), rows >= 1
hipError_t launch_layernorm(const LayerNorm &a, bool in_bf16, hipStream_t stream);

struct LayerNormGrad {
    const void *dY = nullptr;           // [rows, d], row stride lddy elements
    int64_t lddy = 0;
    const void *S = nullptr;            // [nsrc, d] the rows that were normed, row stride lds
    int64_t lds = 0;
    int64_t nsrc = 0;
    int32_t d = 0;
    const double *stats = nullptr;      // [rows, 2]
    const void *gain = nullptr;         // [d] or null (1)
    bool gain_bf16 = false;
    const int32_t *row_idx = nullptr;   // S's row of each result (null: r)
    const int32_t *count = nullptr;     // device-side row count (null: rows)
    int64_t rows = 0;
    const void *dsum = nullptr;         // [rows, d] gradient that joins dX, row stride lddsum, or null
    int64_t lddsum = 0;
    void *dX = nullptr;                 // [rows, d], row stride lddx, or null
    int64_t lddx = 0;
    float *dgain = nullptr;             // [d] or null
    float *dbias = nullptr;             // [d] or null
    void *partials = nullptr;           // workspace
};
int64_t layernorm_grad_workspace_bytes(int64_t rows, int64_t d);
// rows >= 0: no rows give weight gradients of zero
hipError_t launch_layernorm_grad(const LayerNormGrad &a, bool in_bf16, hipStream_t stream);

// MXFP4 codes (gemm_mxfp4.hip): a row of d elements is ceil(d / 32) blocks of 16 bytes and as
// many scale bytes.
inline int64_t mxfp4_blocks(int64_t d) { return d / 32 + (d % 32 != 0); }
hipError_t launch_quantize_rows_mxfp4(const void *X, bool in_bf16, int64_t nsrc, int64_t d, const int32_t *row_idx,
                                      int64_t rows, uint8_t *q, uint8_t *scale, void *values, hipStream_t stream);
// out[i, v] for i < min(max(*count, 0), rows) (count null: rows), v < V, row stride V; codes
// 16-byte aligned; 1 <= blocks <= kMxfp4MaxBlocks.
constexpr int64_t kMxfp4MaxBlocks = 1 << 20;
hipError_t launch_gemm_mxfp4(const uint8_t *Hq, const uint8_t *hs, const int32_t *count, int64_t rows,
                             const uint8_t *Wq, const uint8_t *ws, int64_t V, int64_t blocks, void *out, bool out_bf16,
                             hipStream_t stream);

// Log-probabilities of given tokens, entropy and top alternatives (token_logprobs.hip).
struct TokenLogprobs {
    const void *Z = nullptr;            // logits [rows, V], row stride ldz elements
    int64_t ldz = 0;
    int64_t rows = 0;
    const int32_t *count = nullptr;     // device-side row count (null: rows)
    int32_t V = 0;
    float temperature = 1.0f;
    const int32_t *tokens = nullptr;    // [rows] or null
    float *logprob = nullptr;           // [rows] where tokens is given
    float *entropy = nullptr;           // [rows] or null
    int32_t top_n = 0;
    int32_t *top_ids = nullptr;         // [rows, top_n]
    float *top_logprobs = nullptr;      // [rows, top_n]
    float *stats = nullptr;             // [rows, 2]: row maximum, log of the sum of exp((z - max) / T)
    void *workspace = nullptr;
    // gradient
    const float *grad_logprob = nullptr;   // [rows] or null
    const float *grad_entropy = nullptr;   // [rows] or null
    void *grad = nullptr;                  // [rows, V], row stride ldg, Z's type
    int64_t ldg = 0;
};
constexpr int kTopMax = 64;
constexpr int64_t kTokenLogprobsMaxV = (int64_t)1 << 30;
int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t V, int64_t top_n);
hipError_t launch_token_logprobs(const TokenLogprobs &a, bool z_bf16, hipStream_t stream);
hipError_t launch_token_logprobs_grad(const TokenLogprobs &a, bool z_bf16, hipStream_t stream);

}  // namespace mosaic
