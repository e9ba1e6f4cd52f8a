// handle.hpp -- the handle behind lin_gemm_t and what the C entry points
// share: error texts and the growth of handle-owned buffers.
#pragma once

#include <hip/hip_runtime.h>

#include <string>
#include <vector>

#include "../../include/lin_gemm.h"
#include "dispatch.hpp"

struct lin_gemm_ctx {
  std::vector<lg::TableEntry> table;
  bool forced = false;
  lg::Variant force;
  std::string last_error;
  void* ws = nullptr;         // split-K workspace
  size_t ws_bytes = 0;
  int* counters = nullptr;    // per-16-row-group arrival counters (kept at zero between calls)
  size_t counters_n = 0;
  void* dq = nullptr;         // staging of lin_gemm_run_dynamic: codes, then scales
  size_t dq_bytes = 0;
  // Buffers replaced by bigger ones.  They stay allocated until the handle
  // is destroyed: a graph captured before the growth still holds their
  // addresses and may be replayed.
  std::vector<void*> retired;
};

namespace lg {

inline int fail(lin_gemm_t h, int status, const std::string& msg) {
  if (h) h->last_error = msg;
  return status;
}

// An error that a call reports is taken off the runtime's record, where the
// launch check of the next call would find it.
inline int hip_fail(lin_gemm_t h, hipError_t e, const char* what) {
  (void)hipGetLastError();
  return fail(h, LIN_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

// Device memory, or null (with no error on the record).
inline void* device_alloc(size_t bytes) {
  void* p = nullptr;
  if (hipMalloc(&p, bytes) == hipSuccess) return p;
  (void)hipGetLastError();
  return nullptr;
}

// Sizes of handle-owned buffers grow in powers of two (at least 1 MiB), so
// the retired ones add up to less than the live one.
inline size_t grow_size(size_t need) {
  size_t b = (size_t)1 << 20;
  while (b < need) b <<= 1;
  return b;
}

inline bool misaligned(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

}  // namespace lg
