// Stand-ins for the launchers behind the layer norm, MXFP4 head and token log-probability entry
// points, for the host sanitizer build of the C ABI (test infrastructure): they enqueue nothing
// and report a launch failure.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../mask_only_logits_amd/csrc/launch_head.h"

namespace mosaic {

hipError_t launch_layernorm(const LayerNorm &, bool, hipStream_t) { return hipErrorInvalidValue; }
int64_t layernorm_grad_workspace_bytes(int64_t rows, int64_t d) { return rows == 0 ? 0 : 16 * d; }
hipError_t launch_layernorm_grad(const LayerNormGrad &, bool, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_quantize_rows_mxfp4(const void *, bool, int64_t, int64_t, const int32_t *, int64_t, uint8_t *, uint8_t *,
                                      void *, hipStream_t)
{
    return hipErrorInvalidValue;
}
hipError_t launch_gemm_mxfp4(const uint8_t *, const uint8_t *, const int32_t *, int64_t, const uint8_t *, const uint8_t *,
                             int64_t, int64_t, void *, bool, hipStream_t)
{
    return hipErrorInvalidValue;
}
int64_t token_logprobs_workspace_bytes(int64_t rows, int64_t, int64_t n) { return rows <= 128 ? 8 * rows * (3 + n) : 0; }
hipError_t launch_token_logprobs(const TokenLogprobs &, bool, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_token_logprobs_grad(const TokenLogprobs &, bool, hipStream_t) { return hipErrorInvalidValue; }

}  // namespace mosaic
