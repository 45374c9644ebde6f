// Host-side helpers that the C ABI's sources share (defined in api.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ma {

// Records the calling thread's error message and returns `code`.
int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int hip_fail(hipError_t e, const char* what);

// A launch bracketed by the two events of ma_profile_begin's pool.
struct ProfScope {
  int slot = -1;
  hipStream_t s;
  ProfScope(int kind, hipStream_t st);
  ~ProfScope();
  ProfScope(const ProfScope&) = delete;
  ProfScope& operator=(const ProfScope&) = delete;
};

// A roctx range over the host side of an entry point.
struct EntryMark {
  explicit EntryMark(const char* what);
  ~EntryMark();
  EntryMark(const EntryMark&) = delete;
  EntryMark& operator=(const EntryMark&) = delete;
};

// MA_OK if `stream` belongs to the current device, else MA_ERR_INVALID_ARG.
int check_stream_device(void* stream, const char* what);

}  // namespace ma
