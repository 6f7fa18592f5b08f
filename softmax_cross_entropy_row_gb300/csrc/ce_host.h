// What the host layers of the library share (defined in ce_api.cu).
// Internal to the library.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ce {

// Records a CUDA error's text for ce_last_cuda_error; returns CE_ERR_CUDA.
int host_cuda_fail(cudaError_t e);

// The current device and its number of SMs.
int host_device(int *dev, int *sms);

// CE_OK for memory of the current device (or managed memory): what a tensor
// copy may be pointed at.
int host_check_device_pointer(const void *p, int dev);

bool host_overlap(const void *a, size_t na, const void *b, size_t nb);

// The device error counters of `stream` on `dev` (ce_get_device_errors),
// created if the stream has none yet, also while it is being captured.
int host_error_counters(int dev, cudaStream_t stream, int **err);

// cudaMalloc that is allowed while a stream is being captured (the memory is
// not part of the capture), zeroed over its first `zero` bytes.
cudaError_t host_malloc_zeroed(void **p, size_t bytes, size_t zero);

// Frees the workspaces of the projection's operators (ce_head_api.cu); part of
// ce_release_workspaces.
int release_head_workspaces();

}  // namespace ce
