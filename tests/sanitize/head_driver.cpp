// Host sanitizer run of the layer norm, MXFP4 head and token log-probability entry points (test
// infrastructure): their validation with every size at the edges of int64 in turn, and the empty
// problems.  A call that gets past validation reaches a stand-in launcher and reports
// MOSAIC_ERR_DEVICE; no GPU is needed.
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mosaic.h"

static int failures = 0;
#define EXPECT(cond)                                                                 \
    do {                                                                             \
        if (!(cond)) {                                                               \
            fprintf(stderr, "head driver: %s failed at line %d\n", #cond, __LINE__); \
            ++failures;                                                              \
        }                                                                            \
    } while (0)

int main()
{
    char *A = (char *)(uintptr_t)(1 << 20), *B = A + (1 << 20), *C = B + (1 << 20);   // never dereferenced
    const int32_t *idx = (const int32_t *)A;
    float *f = (float *)A, *g = (float *)B;
    double *st = (double *)A;
    uint8_t *u = (uint8_t *)A;
    const int64_t big = INT64_MAX;
    const int64_t edge[] = {INT64_MIN, -1, 0, 1, 31, 32, 64, (int64_t)1 << 25, (int64_t)1 << 30, ((int64_t)1 << 31) - 1,
                            (int64_t)1 << 31, (int64_t)1 << 62, big};
    auto known = [](mosaic_status_t s) { return s >= MOSAIC_OK && s <= MOSAIC_ERR_DEVICE; };
    for (int64_t x : edge)
        for (int64_t y : edge) {
            EXPECT(known(mosaic_add_layernorm(A, x, B, y, 100, 64, MOSAIC_BF16, A, A, MOSAIC_F32, 1e-5f, idx, idx, 10, C, y,
                                              nullptr, st, nullptr)));
            EXPECT(known(mosaic_add_layernorm(A, x, nullptr, 0, y, x, MOSAIC_F32, nullptr, A, MOSAIC_BF16, 1e-5f, nullptr,
                                              nullptr, y, nullptr, 0, C, nullptr, nullptr)));
            EXPECT(known(mosaic_layernorm_grad(A, x, B, y, 100, 64, MOSAIC_BF16, st, A, MOSAIC_F32, idx, idx, 10, A, x, C, y,
                                               f, g, B, big, nullptr)));
            EXPECT(known(mosaic_layernorm_grad(A, y, B, y, x, y, MOSAIC_F32, st, nullptr, MOSAIC_F32, nullptr, nullptr, x,
                                               nullptr, 0, C, y, f, nullptr, B, big, nullptr)));
            EXPECT(mosaic_layernorm_grad_workspace_bytes(x, y) >= -1);
            EXPECT(known(mosaic_quantize_rows_mxfp4(A, x, y, MOSAIC_BF16, idx, x, u, u, B, nullptr)));
            EXPECT(known(mosaic_quantized_logits_mxfp4(u, u, x, idx, u, u, y, 128, C, MOSAIC_BF16, nullptr)));
            EXPECT(known(mosaic_quantized_logits_mxfp4(u, u, x, nullptr, u, u, 70, y, C, MOSAIC_F32, nullptr)));
            EXPECT(mosaic_logits_mxfp4_workspace_bytes(x, y, 64) >= -1);
            EXPECT(mosaic_logits_mxfp4_workspace_bytes(x, 0, y) >= -1);
            EXPECT(known(mosaic_masked_logits_mxfp4(A, 100, x, MOSAIC_BF16, nullptr, y, u, u, 50, C, 0, MOSAIC_BF16, B, big,
                                                    nullptr)));
            EXPECT(known(mosaic_masked_logits_mxfp4(A, y, 64, MOSAIC_F32, idx, 7, u, u, x, C, 2, MOSAIC_F32, B, big,
                                                    nullptr)));
            EXPECT(known(mosaic_token_logprobs(A, x, y, 64, MOSAIC_BF16, idx, 1.0f, idx, f, f, 4, (int32_t *)A, f, f, B, big,
                                               nullptr)));
            EXPECT(known(mosaic_token_logprobs(A, x, 10, x, MOSAIC_F32, nullptr, 1.0f, nullptr, nullptr, nullptr, y,
                                               (int32_t *)A, f, f, B, big, nullptr)));
            EXPECT(known(mosaic_token_logprobs_grad(A, x, y, x, MOSAIC_F32, idx, 1.0f, nullptr, f, f, f, f, C, x, nullptr)));
            EXPECT(mosaic_token_logprobs_workspace_bytes(x, y, 4) >= -1 && mosaic_token_logprobs_workspace_bytes(4, x, y) >= -1);
        }
    // past validation: the stand-ins
    EXPECT(mosaic_add_layernorm(A, 64, A, 64, 100, 64, MOSAIC_BF16, A, A, MOSAIC_BF16, 1e-5f, nullptr, nullptr, 100, A, 64,
                                C, st, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_layernorm_grad(A, 64, B, 64, 100, 64, MOSAIC_BF16, st, A, MOSAIC_BF16, nullptr, nullptr, 100, C, 64, C, 64,
                                 f, g, B, big, nullptr) == MOSAIC_ERR_DEVICE);
    // no rows: the weight gradients are written all the same
    EXPECT(mosaic_layernorm_grad(nullptr, 64, nullptr, 64, 0, 64, MOSAIC_BF16, nullptr, A, MOSAIC_BF16, nullptr, nullptr, 0,
                                 nullptr, 0, nullptr, 0, f, g, nullptr, 0, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_quantize_rows_mxfp4(A, 100, 65, MOSAIC_F32, nullptr, 10, u, u, A, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_quantized_logits_mxfp4(u, u + 1, 10, idx, u, u + 3, 50, 33, C, MOSAIC_F32, nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_masked_logits_mxfp4(A, 100, 64, MOSAIC_BF16, idx, 10, u, u, 50, C, 3, MOSAIC_BF16, B,
                                      mosaic_logits_mxfp4_workspace_bytes(10, 3, 64), nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_token_logprobs(A, 64, 10, 64, MOSAIC_BF16, idx, 1.0f, nullptr, f, f, 64, (int32_t *)A, f, f, B, big,
                                 nullptr) == MOSAIC_ERR_DEVICE);
    EXPECT(mosaic_token_logprobs_grad(A, 64, 10, 64, MOSAIC_BF16, nullptr, 1.0f, nullptr, f, f, nullptr, f, A, 64,
                                      nullptr) == MOSAIC_ERR_DEVICE);
    // refusals of numbers that compare with nothing
    EXPECT(mosaic_add_layernorm(A, 64, nullptr, 0, 100, 64, MOSAIC_BF16, A, A, MOSAIC_BF16, NAN, idx, nullptr, 10, nullptr, 0,
                                C, nullptr, nullptr) == MOSAIC_ERR_INVALID_ARG);
    EXPECT(mosaic_token_logprobs(A, 64, 10, 64, MOSAIC_BF16, idx, NAN, nullptr, f, f, 0, nullptr, nullptr, f, B, big,
                                 nullptr) == MOSAIC_ERR_INVALID_ARG);
    if (failures == 0)
        printf("head sanitizer driver ok\n");
    return failures != 0;
}
