// api.h -- what the files of the C ABI share: error reporting and checks of arguments.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/fp8gb.h"
#include "kernels.h"

namespace fp8gb {

// Record the message of a failed call on this thread and return its status.
fp8_status_t fail(fp8_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fp8_status_t cuda_fail(cudaError_t e, const char* where);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

QuantState to_qs(const fp8_tensor_state_t* st);
fp8_status_t check_state(const fp8_tensor_state_t* st, fp8_scaling_t mode, const char* who);

}  // namespace fp8gb
