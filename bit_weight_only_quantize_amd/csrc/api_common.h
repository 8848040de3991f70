// What the C ABI's translation units share (api.cpp, api_kv.cpp).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/awq355.h"

namespace awq {

// Records the calling thread's message and returns `st`.
awq_status fail(awq_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears it.
awq_status ok();
awq_status hip_status(hipError_t e, const char *where);

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// Bytes [p, p + n) and [q, q + m) share none.
inline bool apart(const void *p, size_t n, const void *q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n == 0 || m == 0 || a + n <= b || b + m <= a;
}
inline hipStream_t as_stream(awq_stream_t s) { return reinterpret_cast<hipStream_t>(s); }

constexpr size_t kAlign = 256;      // of workspaces and their regions
inline size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

}  // namespace awq
