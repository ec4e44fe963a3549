// api_internal.h -- what the entry points in several translation units share
// (defined in api.cu): the per-thread error string, the fault-injection hook
// that every kernel is asked through, and the launch accounting.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/gbmm.h"

namespace gbmm {

// sets gbmm_last_error() and returns `status`
int record_error(int status, const char *message);
// false (and the error string set) when a test made kernel `name` unavailable
bool resolve_kernel(const char *name);
// status of a launch that returned `e`; counts it, and synchronises under GBMM_DEBUG_SYNC=1
gbmm_status finish_launch(cudaError_t e, const char *name, cudaStream_t s);

// Tensor map of a 16-bit matrix [outer][inner], rows ld elements apart, boxes of box_outer x 64, 128-byte
// swizzle.  False where TMA cannot read it (16-byte aligned base and rows).
bool encode_matrix16(CUtensorMap *map, int dt, const void *base, int64_t inner, int64_t outer, int64_t ld,
                     uint32_t box_outer);

// Tensor map of a matrix of bytes [outer][inner], boxes of box_outer x 128, 128-byte swizzle.
bool encode_matrix8(CUtensorMap *map, const void *base, int64_t inner, int64_t outer, int64_t ld, uint32_t box_outer);
// Tensor map for storing 32 x 32 pieces of a matrix [rows][cols] of type dt: rows of 64 bytes with 64-byte
// swizzle (16-bit types), of 128 bytes with 128-byte swizzle (f32).  False where TMA cannot write it.
bool encode_store32(CUtensorMap *map, int dt, const void *base, int64_t cols, int64_t rows, int64_t ld);

}  // namespace gbmm
