// Argument-check helpers shared by the C entry points (host side).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/dora.h"

namespace dora {

constexpr size_t kAlign = 256;

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool valid_dtype(int dt) { return dt == DORA_BF16 || dt == DORA_F32 || dt == DORA_F16; }
inline int64_t esize(int dt) { return dt == DORA_F32 ? 4 : 2; }
inline int64_t epc(int dt) { return dt == DORA_F32 ? 4 : 8; }

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte ranges [a, a+na) and [b, b+nb) intersect (empty ranges never do).
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (a == nullptr || b == nullptr || na <= 0 || nb <= 0) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
  return pa < pb + (uintptr_t)nb && pb < pa + (uintptr_t)na;
}

// Upper bound that keeps every index and grid dimension in range.
constexpr int64_t kMaxDim = (int64_t)1 << 31;

inline dora_status hip_status(hipError_t e) { return e == hipSuccess ? DORA_OK : DORA_ERR_HIP; }

}  // namespace dora
