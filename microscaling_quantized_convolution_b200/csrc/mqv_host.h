// Host helpers shared by the library's source files (internal): the
// per-thread error message, argument checks and the device error word.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "mqv.h"
#include "mqv_ptx.cuh"

namespace mqv {

constexpr int kMaxDevices = 64;

// Sets the calling thread's message and returns st; ok() clears it.
mqv_status fail(mqv_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
mqv_status ok();
mqv_status cuda_fail(cudaError_t e, const char* what);

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// The current device's error word, which bounded waits set on timeout.
mqv_status device_error_word(uint32_t** out);

// The constants of a division by d (see FastDiv).
inline FastDiv make_fastdiv(int64_t d) {
  FastDiv f;
  uint32_t s = 0;
  while ((int64_t(1) << s) < d) ++s;
  const unsigned __int128 num = (static_cast<unsigned __int128>(1) << (32 + s)) + (d - 1);
  f.m = static_cast<uint32_t>(static_cast<uint64_t>(num / static_cast<unsigned __int128>(d)) - (uint64_t(1) << 32));
  f.s = s;
  return f;
}

}  // namespace mqv
