// host.hpp -- checks and errors shared by the C ABI's host files (defined in lora_host.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lora {

// Sets the calling thread's error message and returns `code`.
int fail(int code, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
void clear_err();
int launch_status(hipError_t e, const char *what);
// LORA_OK on a gfx950, an error anywhere else.
int check_device(const char *what);
// Records the caller's profile event i, if set (lora_set_profile_events).
void prof_record(int i, hipStream_t st);
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
constexpr uint32_t kMaxRows = 16384;  // of any call's batch

}  // namespace lora
