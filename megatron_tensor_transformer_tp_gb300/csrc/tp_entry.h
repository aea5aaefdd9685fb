// What an entry point outside tp_api.cu needs of it (not part of the ABI).
#pragma once

#include <cuda_runtime.h>

#include "tp.h"

namespace tp {

// SM count and error word of the current device, after its one-time set-up.
tp_status entry_device(int* num_sms, unsigned** err);
// Runs work(arg), which enqueues kernels on s, as the profiled work `name`.
cudaError_t entry_timed(const char* name, cudaStream_t s, cudaError_t (*work)(void*), void* arg);

}  // namespace tp
