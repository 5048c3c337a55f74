// Host sanitizer run of the norm, INT8 head and distillation entry points (test
// infrastructure): their validation with every size at the edges of int64 in turn, and the
// empty problems.  A call that gets past validation reaches a stand-in launcher and reports
// MOSAIC_ERR_DEVICE; no GPU is needed.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mosaic.h"

static int failures = 0;
#define EXPECT(cond)                                                                \
    do {                                                                            \
        if (!(cond)) {                                                              \
            fprintf(stderr, "ops driver: %s failed at line %d\n", #cond, __LINE__); \
            ++failures;                                                             \
        }                                                                           \
    } while (0)

int main()
{
    char *A = (char *)(uintptr_t)(1 << 20), *B = A + (1 << 20), *C = B + (1 << 20);   // never dereferenced
    const int32_t *idx = (const int32_t *)A;
    float *f = (float *)A;
    const int64_t big = INT64_MAX;
    const int64_t edge[] = {INT64_MIN, -1, 0, 1, 63, 64, (int64_t)1 << 30, ((int64_t)1 << 31) - 1, (int64_t)1 << 31,
                            (int64_t)1 << 62, big};
    auto known = [](mosaic_status_t s) { return s >= MOSAIC_OK && s <= MOSAIC_ERR_DEVICE; };
    for (int64_t x : edge)
        for (int64_t y : edge) {
            EXPECT(known(mosaic_add_rmsnorm(A, x, B, y, 100, 64, MOSAIC_BF16, A, MOSAIC_F32, 1e-6f, idx, idx, 10, C, y,
                                            nullptr, MOSAIC_INT8, A, f, nullptr)));
            EXPECT(known(mosaic_add_rmsnorm(A, x, nullptr, 0, y, x, MOSAIC_F32, A, MOSAIC_BF16, 1e-6f, nullptr, nullptr,
                                            y, nullptr, 0, C, MOSAIC_E4M3, nullptr, nullptr, nullptr)));
            EXPECT(known(mosaic_quantize_rows_int8(A, x, y, MOSAIC_BF16, idx, x, (int8_t *)B, f, nullptr)));
            for (mosaic_code_t c : {MOSAIC_E4M3, MOSAIC_INT8})
                EXPECT(known(mosaic_quantized_logits(c, A, f, x, nullptr, A, f, y, 128, C, MOSAIC_BF16, nullptr)));
            EXPECT(known(mosaic_quantized_logits(MOSAIC_INT8, A, f, x, idx, A, f, 70, y, C, MOSAIC_F32, nullptr)));
            EXPECT(mosaic_logits_int8_workspace_bytes(x, y, 64) >= -1);
            EXPECT(mosaic_logits_int8_workspace_bytes(x, 0, y) >= -1);
            EXPECT(known(mosaic_masked_logits_int8(A, 100, x, MOSAIC_BF16, nullptr, y, (const int8_t *)A, f, 50, C, 0,
                                                   MOSAIC_BF16, B, big, nullptr)));
            EXPECT(known(mosaic_distill_topk(A, x, y, 64, MOSAIC_BF16, B, MOSAIC_F32, idx, 4, 1.0f, idx, f, f, f, C, x,
                                             B, big, nullptr)));
            EXPECT(known(mosaic_distill_topk(A, x, 10, x, MOSAIC_F32, B, MOSAIC_BF16, idx, y, 1.0f, nullptr, f, f,
                                             nullptr, nullptr, 0, B, big, nullptr)));
            EXPECT(known(mosaic_distill_topk_grad(A, x, y, x, MOSAIC_F32, B, MOSAIC_F32, idx, y, 1.0f, nullptr, f,
                                                  nullptr, C, x, nullptr)));
            EXPECT(mosaic_distill_topk_workspace_bytes(x, y, 4) >= -1);
        }
    // past validation: the stand-ins
    EXPECT(mosaic_add_rmsnorm(A, 64, A, 64, 100, 64, MOSAIC_BF16, A, MOSAIC_BF16, 1e-6f, nullptr, nullptr, 100, A, 64,
                              C, MOSAIC_INT8, B, f, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_quantize_rows_int8(A, 100, 65, MOSAIC_F32, idx, 10, (int8_t *)B, f, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_quantized_logits(MOSAIC_INT8, A, f, 10, idx, A, f, 50, 33, C, MOSAIC_F32, nullptr) ==
           MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_quantized_logits(MOSAIC_E4M3, A, f, 100, nullptr, A, f, 50, 128, C, MOSAIC_BF16, nullptr) ==
           MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_masked_logits_int8(A, 100, 64, MOSAIC_BF16, idx, 10, (const int8_t *)A, f, 50, C, 3, MOSAIC_BF16, B,
                                     mosaic_logits_int8_workspace_bytes(10, 3, 64), nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_distill_topk(A, 64, 10, 64, MOSAIC_BF16, B, MOSAIC_F32, idx, 4, 1.0f, nullptr, f, f, nullptr, A, 64,
                               B, big, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_distill_topk_grad(A, 64, 10, 64, MOSAIC_BF16, B, MOSAIC_F32, idx, 4, 1.0f, nullptr, f, nullptr, A, 64,
                                    nullptr) == MOSAIC_ERR_DEVICE);
    // refusals of numbers that compare with nothing
    EXPECT(mosaic_add_rmsnorm(A, 64, nullptr, 0, 100, 64, MOSAIC_BF16, A, MOSAIC_BF16, NAN, idx, nullptr, 10, nullptr, 0,
                              C, MOSAIC_INT8, nullptr, nullptr, nullptr) == MOSAIC_ERR_INVALID_ARG);
    EXPECT(mosaic_distill_topk(A, 64, 10, 64, MOSAIC_BF16, B, MOSAIC_F32, idx, 4, NAN, nullptr, f, f, nullptr, nullptr, 0,
                               B, big, nullptr) == MOSAIC_ERR_INVALID_ARG);
    if (failures == 0)
        printf("ops sanitizer driver ok\n");
    return failures != 0;
}
