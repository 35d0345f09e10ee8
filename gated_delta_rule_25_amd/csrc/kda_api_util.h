// kda_api_util.h — argument checks shared by the C ABI files.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstddef>
#include <cstdint>

#include "kda.h"

namespace kda {
namespace api {

constexpr int kD = 128;

struct Range {
  uintptr_t lo = 0, hi = 0;  // [lo, hi); empty when lo == hi
};

inline Range range_of(const void* p, size_t bytes) {
  Range r;
  if (p && bytes) {
    r.lo = reinterpret_cast<uintptr_t>(p);
    r.hi = r.lo + bytes;
  }
  return r;
}

inline bool overlap(const Range& a, const Range& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}

inline int cu_count_for_current_device() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64) {
    int v = cache[dev].load(std::memory_order_relaxed);
    if (v > 0) return v;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) n = 256;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

inline size_t elem_size(kda_dtype dt) { return dt == KDA_DTYPE_BF16 ? 2 : 4; }

inline bool dtype_ok(kda_dtype dt) { return dt == KDA_DTYPE_F32 || dt == KDA_DTYPE_BF16; }

// q, k, v, log_alpha, gate, o and the states move as 16-byte vectors; the
// rest (beta, cu_seqlens, conv and norm weights, workspace) are read as scalars.
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace api

// Whether KDA_DEBUG_CHECKS asks for the precondition checks (read at every
// call), and the failed checks of the calling thread's last checked call
// (kda_last_precondition_flags).
bool debug_checks();
void set_check_flags(uint32_t flags);

}  // namespace kda
