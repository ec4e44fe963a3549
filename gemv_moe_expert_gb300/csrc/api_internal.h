// api_internal.h -- what the entry points in several translation units share
// (defined in api.cu): the per-thread error string, the fault-injection hook
// that every kernel is asked through, and the launch accounting.
#pragma once

#include <cuda_runtime.h>

#include "../../include/gbmm.h"

namespace gbmm {

// sets gbmm_last_error() and returns `status`
int record_error(int status, const char *message);
// false (and the error string set) when a test made kernel `name` unavailable
bool resolve_kernel(const char *name);
// status of a launch that returned `e`; counts it, and synchronises under GBMM_DEBUG_SYNC=1
gbmm_status finish_launch(cudaError_t e, const char *name, cudaStream_t s);

}  // namespace gbmm
