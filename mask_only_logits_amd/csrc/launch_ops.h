// Launchers of the operators around the LM head: norm, INT8 product, distillation loss.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mosaic {

// Residual addition with root-mean-square norm, and 8-bit row codes (rmsnorm.hip).
struct RowsNorm {
    const void *X = nullptr;            // [nsrc, d], row stride ldx elements
    int64_t ldx = 0;
    const void *R = nullptr;            // residual, as X, or null
    int64_t ldr = 0;
    int64_t nsrc = 0;
    int32_t d = 0;
    const void *gain = nullptr;         // [d]
    bool gain_bf16 = false;
    float eps = 0.0f, eps_low = 0.0f;   // and eps 2^-160
    const int32_t *row_idx = nullptr;   // row r of the results is source row row_idx[r] (null: r)
    const int32_t *count = nullptr;     // device-side row count (null: rows)
    int64_t rows = 0;
    void *sum = nullptr;                // [rows, d], row stride ldsum, or null
    int64_t ldsum = 0;
    void *out = nullptr;                // [rows, d] or null
    bool code_int8 = false;             // codes: INT8, else E4M3
    uint8_t *q = nullptr;               // [rows, d] or null
    float *scale = nullptr;             // [rows] where q is given
};
// 1 <= d <= kNormMaxWidth, rows >= 1; norm off: q and scale of X's rows themselves.
constexpr int64_t kNormMaxWidth = (int64_t)1 << 30;
hipError_t launch_rows_norm(const RowsNorm &a, bool in_bf16, bool norm, hipStream_t stream);

// INT8 product (gemm_int8.hip): out[i, v] = (sum_k Hq[i, k] Wq[v, k]) * hs[i] * ws[v] for
// i < min(max(*count, 0), rows) (count null: rows), v < V; out is bf16 or fp32 with row
// stride ldo.  1 <= d <= kInt8MaxDepth.
constexpr int64_t kInt8MaxDepth = 131071;   // d products of at most 2^14 stay inside int32
hipError_t launch_gemm_int8(const int8_t *Hq, const float *hs, const int32_t *count, int64_t rows, const int8_t *Wq,
                            const float *ws, int64_t V, int64_t d, void *out, bool out_bf16, int64_t ldo,
                            hipStream_t stream);

// Distillation from a teacher's top logits (distill.hip).
struct Distill {
    const void *Z = nullptr;            // student logits [rows, V], row stride ldz elements
    int64_t ldz = 0;
    int64_t rows = 0;
    const int32_t *count = nullptr;     // device-side row count (null: rows)
    int32_t V = 0;
    const void *top = nullptr;          // teacher logits [rows, K]
    bool top_bf16 = false;
    const int32_t *ids = nullptr;       // their vocabulary entries [rows, K]
    int32_t K = 0;
    float temperature = 1.0f;
    const float *grad_loss = nullptr;   // [rows] or null (1)
    float *loss = nullptr;              // [rows]
    float *stats = nullptr;             // [rows, 2]: row maximum, log of the sum of exp((z - max) / T)
    void *grad = nullptr;               // [rows, V], row stride ldg, Z's type; null: no gradient
    int64_t ldg = 0;
    float *partials = nullptr;          // workspace of the split form
};
constexpr int kDistillMaxK = 1024;
constexpr int64_t kDistillMaxV = (int64_t)1 << 30;
// Workspace bytes of launch_distill (0: none needed).
int64_t distill_workspace_bytes(int64_t rows, int64_t V, int64_t K);
// loss and stats, and grad where it is given.
hipError_t launch_distill(const Distill &a, bool z_bf16, hipStream_t stream);
// grad from the stats.
hipError_t launch_distill_grad(const Distill &a, bool z_bf16, hipStream_t stream);

}  // namespace mosaic
