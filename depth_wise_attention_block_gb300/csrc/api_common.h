// What the C entry points share (api.cu, body_api.cu): the per-thread error
// message, and checks of argument values.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "attnres.h"

namespace attnres {

// Set this host thread's error message and return `code`.
int fail(int code, const char* fmt, ...);
// Clear it; returns ATTNRES_OK.
int ok();
// ATTNRES_ECUDA with CUDA's message.
int cuda_fail(cudaError_t e, const char* what);

inline bool valid_dtype(int dt) { return dt == ATTNRES_F32 || dt == ATTNRES_BF16; }
inline int64_t dtype_bytes(int dt) { return dt == ATTNRES_BF16 ? 2 : 4; }
inline int64_t align256(int64_t x) { return (x + 255) & ~int64_t(255); }

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
inline bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return na > 0 && nb > 0 && pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

}  // namespace attnres
