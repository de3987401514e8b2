// Host helpers shared by the API's source files.
#ifndef KDA_API_UTIL_H_
#define KDA_API_UTIL_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

struct Range {
  uintptr_t lo;
  uintptr_t hi;  // exclusive
};

inline Range make_range(const void* p, int64_t bytes) {
  Range r;
  r.lo = reinterpret_cast<uintptr_t>(p);
  r.hi = r.lo + (bytes > 0 ? static_cast<uintptr_t>(bytes) : 0);
  return r;
}

inline bool overlaps(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;  // empty ranges never overlap
  return a.lo < b.hi && b.lo < a.hi;
}

// Compute units of the current device (256 on MI355X when the query fails, e.g.
// without a GPU).
inline int device_cus() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
      cus <= 0)
    return 256;
  return cus;
}

}  // namespace kda

#endif  // KDA_API_UTIL_H_
