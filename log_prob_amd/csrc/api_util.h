// Error reporting and argument checks shared by the C ABI's source files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "flce.h"

namespace flce {

// Record the calling thread's last error and return its status; ok() clears it.
flce_status_t fail(flce_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
flce_status_t ok();

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes every call accepts (the limits stated in flce.h).
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxHidden = int64_t(1) << 20;

}  // namespace flce
