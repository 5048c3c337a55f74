// Stand-ins for the launchers behind the norm, INT8 head and distillation entry points, for the
// host sanitizer build of the C ABI (test infrastructure): they enqueue nothing and report a
// launch failure.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../mask_only_logits_amd/csrc/launch_ops.h"

namespace mosaic {

hipError_t launch_rows_norm(const RowsNorm &, bool, bool, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_gemm_int8(const int8_t *, const float *, const int32_t *, int64_t, const int8_t *, const float *,
                            int64_t, int64_t, void *, bool, int64_t, hipStream_t)
{
    return hipErrorInvalidValue;
}
int64_t distill_workspace_bytes(int64_t rows, int64_t, int64_t K) { return rows <= 1024 ? 4 * rows * (2 + K) : 0; }
hipError_t launch_distill(const Distill &, bool, hipStream_t) { return hipErrorInvalidValue; }
hipError_t launch_distill_grad(const Distill &, bool, hipStream_t) { return hipErrorInvalidValue; }

}  // namespace mosaic
