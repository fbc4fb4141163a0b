// Host-side parts of gemm_api.hip that the library's other translation units use.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>

namespace gemm {

// Records e as the thread's last HIP error; returns GEMM_ERR_HIP.
int host_fail(hipError_t e);

// Compute units to plan for in a query that launches nothing.
int host_planning_cus();

// The current device, which must be gfx950, and its compute units. Returns a status.
int host_check_device(int *dev, int *cus);

// Whether the byte ranges [p, p + pb) and [q, q + qb) meet.
bool host_overlaps(const void *p, size_t pb, const void *q, size_t qb);

// Runs body(context, workspace) with a buffer of the library's pool (a null
// workspace if none could be had); GEMM_ERR_CAPTURING on a stream that captures
// a graph.
int host_with_library_workspace(int dev, size_t need, hipStream_t stream,
                                int (*body)(void *context, void *workspace), void *context);

}  // namespace gemm
