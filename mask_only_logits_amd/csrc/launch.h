// Internal launchers of the HIP kernels (not part of the public C ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mosaic {

// flag[0] = 1 if some idx[i] (i < M) is outside [0, L), else 0 (clears flag first).
hipError_t launch_idx_range_check(const int32_t *idx, int64_t M, int64_t L, int32_t *flag, hipStream_t stream);

hipError_t launch_mask_compact(const int32_t *tokens, int64_t L, int32_t mask_id, int32_t *idx,
                               int32_t *count, hipStream_t stream);
hipError_t launch_mask_compact_flags(const uint8_t *flags, int64_t L, int32_t *idx, int32_t *count,
                                     hipStream_t stream);
hipError_t launch_mask_compact_batched(const int32_t *tokens, int64_t L, const int32_t *seq_offsets,
                                       int32_t nseq, int32_t mask_id, int32_t *idx,
                                       int32_t *idx_offsets, hipStream_t stream);

// Kernel variants of the logits GEMM.  The numbers are stable identifiers (reported by
// mosaic_logits_variant and accepted by MOSAIC_TUNE); gaps are retired experiment forms.
enum LogitsVariant : int {
    kVariantF32 = 0,               // fp32 inputs: LDS-tiled FMA kernel
    kVariantBf16Simple = 2,        // bf16 inputs, any d % 8 == 0: LDS-tiled FMA kernel
    kVariantBf16PersistK32 = 11,   // bf16, d % 32 == 0: persistent 256 x 256, 4 waves, BK 32, 4 stages
    kVariantBf16W8K64S2 = 12,      // bf16, d % 64 == 0: 256 x 256, 8 waves, BK 64 (the bf16 -> fp32 default)
    kVariantBf16DeferS4I8 = 16,    // bf16 -> bf16, d % 64 == 0: persistent 8-wave, 32 x 32 x 16 MFMA,
                                   // half the stores deferred over 4 K steps (comparison form)
    kVariantBf16M16S1 = 19,        // bf16 -> bf16, d % 64 == 0: persistent 8-wave, 16 x 16 x 32 MFMA,
                                   // every wave requests K tiles
    kVariantBf16LowMShared = 20,   // bf16, d % 64 == 0, M <= 64: W streaming with a workgroup-shared H tile
    kVariantBf16M16Dma4 = 21,      // bf16 -> bf16, d % 64 == 0: as 19, K tiles requested by one wave per
                                   // SIMD
    kVariantBf16M16Dma4W3 = 22,    // as 21 with a third W stage (the bf16-output default)
};

// Default number of row tiles that share the W slabs of one XCD (tile order).
constexpr int kDefaultGroupM = 8;



// Whether a chunk of `rows` rows over V vocabulary rows fits the variant's launch grid.
bool gather_gemm_grid_fits(int variant, int64_t rows, int64_t V);

// One chunk: out[i, v] for i < rows, v < V, out row stride ldo elements.
hipError_t launch_gather_gemm(int variant, const void *H, const int32_t *idx, int64_t rows,
                              const void *W, int64_t V, int64_t d, void *out, int64_t ldo,
                              bool out_bf16, int group_m, hipStream_t stream);

// One launch whose row count is read by the kernel from device memory: rows =
// clamp(*rows_dev, 0, max_rows) (bf16 -> bf16, d % 64 == 0; the default persistent form,
// its grid sized for max_rows).
hipError_t launch_gather_gemm_device_rows(const void *H, const int32_t *idx, const int32_t *rows_dev,
                                          int64_t max_rows, const void *W, int64_t V, int64_t d, void *out,
                                          int64_t ldo, int group_m, hipStream_t stream);

// One chunk of the per-row consumer (bf16 in, d % 64 == 0): the persistent kernel
// reduces every (row, 256-entry vocabulary tile) to a partial in pmax / parg / psum
// ([ceil(V/256)][rows] each) and, when `out` is not null, also stores the bf16 logits;
// a finish kernel combines the partials into row_max / row_argmax / row_lse.  With rows_dev,
// both kernels take clamp(*rows_dev, 0, rows) rows from device memory (rows is then the
// capacity: the grids and the partials' row stride).  m16 selects
// the 16 x 16 x 32 MFMA form of the kernel (else 32 x 32 x 16); the two give the same
// logits, maxima and argmax, and exp sums added in different orders.
hipError_t launch_logits_argmax_lse(const void *H, const int32_t *idx, int64_t rows, const void *W, int64_t V,
                                    int64_t d, void *out, int64_t ldo, float *pmax, int32_t *parg, float *psum,
                                    float *row_max, int32_t *row_argmax, float *row_lse, int group_m,
                                    bool m16, hipStream_t stream, const int32_t *rows_dev = nullptr);

// FP8 LM head.  Quantize `rows` rows of X ([*, d], bf16 or fp32, d % 8 == 0; row r is
// source row row_idx[r], or r when row_idx is null) to E4M3 codes q ([rows, d]) and
// fp32 row scales.
hipError_t launch_quantize_rows_e4m3(const void *X, bool in_bf16, int64_t d, const int32_t *row_idx, int64_t rows,
                                     uint8_t *q, float *scale, hipStream_t stream);

// out[i, v] (bf16) = (sum_k Hq[i, k] Wq[v, k]) * hs[i] * ws[v] for i < rows, v < V;
// d % 128 == 0; nwaves 4 or 8: the comparison forms with every wave requesting K tiles,
// anything else: the default (eight waves, four requesting, three W stages).  All three
// give the same bits.
hipError_t launch_gemm_fp8(const uint8_t *Hq, const float *hs, int64_t rows, const uint8_t *Wq, const float *ws,
                           int64_t V, int64_t d, void *out, int64_t ldo, int group_m, int nwaves, hipStream_t stream);

// The same logits for rows <= 64 (d % 128 == 0): a W-streaming kernel, bit-identical to
// launch_gemm_fp8.
hipError_t launch_gemm_fp8_lowm(const uint8_t *Hq, const float *hs, int64_t rows, const uint8_t *Wq, const float *ws,
                                int64_t V, int64_t d, void *out, int64_t ldo, hipStream_t stream);

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
    float eps = 0.0f;
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
