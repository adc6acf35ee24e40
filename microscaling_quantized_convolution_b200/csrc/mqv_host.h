// Host helpers shared by the library's source files (internal): the
// per-thread error message, argument checks and the device error word.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mqv.h"

namespace mqv {

constexpr int kMaxDevices = 64;

// Sets the calling thread's message and returns st; ok() clears it.
mqv_status fail(mqv_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mqv_status ok();
mqv_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device's error word, which bounded waits set on timeout.
mqv_status device_error_word(uint32_t** out);

}  // namespace mqv
