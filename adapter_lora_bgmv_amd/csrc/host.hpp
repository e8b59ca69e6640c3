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
// LORA_OK for a known dtype.
int check_type(const char *what, int32_t dtype);
// Rows of `width` elements: 16-byte accesses at every multiple of 16 bytes.
int check_rows(const char *what, int32_t dtype, const char *name, const void *p, uint32_t stride, uint64_t width, uint32_t n);
// A call of one main kernel, between the caller's profile events.
template <typename F>
int timed(const char *what, hipStream_t st, F launch) {
  prof_record(0, st);
  prof_record(1, st);
  const int e = launch_status(launch(), what);
  prof_record(2, st);
  prof_record(3, st);
  return e;
}
inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
constexpr uint32_t kMaxRows = 16384;  // of any call's batch

}  // namespace lora
