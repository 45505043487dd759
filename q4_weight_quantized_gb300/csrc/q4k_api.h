// What the C-ABI layer's translation units share: the device gate, the record of
// a failed CUDA call and the pointer checks.
#pragma once

#include "q4k.h"
#include "q4k_internal.h"

namespace q4k {

// Q4K_OK if a compute capability 10.3 device is current (its properties in *di).
q4k_status check_device(DeviceInfo *di);

// The setting of q4k_set_batch_invariant.
bool batch_invariant();

// The limit of the waits that q4k_set_gemv_wait_limit_ns can shorten.
unsigned long long wait_limit_ns();

// Records e for q4k_last_cuda_error and returns Q4K_ERR_CUDA.
q4k_status cuda_fail(cudaError_t e);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace q4k
