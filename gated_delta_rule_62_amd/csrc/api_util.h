// Host helpers shared by the API's source files.
#ifndef KDA_API_UTIL_H_
#define KDA_API_UTIL_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <limits>

#include "../../include/kda.h"

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

constexpr int64_t kMaxBytes = (int64_t)1 << 62;  // of one tensor: the range arithmetic cannot wrap

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// A row stride in elements: whole 16-byte units, at least the row itself.
inline bool row_ok(int64_t row, int64_t heads, int64_t D) {
  return row >= heads * D && row % 8 == 0;
}

// Bytes from the first element of `rows` bf16 rows to the last, or -1 beyond kMaxBytes.
inline int64_t span_bytes(int64_t rows, int64_t row, int64_t heads, int64_t D) {
  if (rows <= 0) return 0;
  if (row > kMaxBytes / 2 / rows) return -1;
  return ((rows - 1) * row + heads * D) * 2;
}

inline bool any_overlap(Range out, const Range* ins, int n) {
  for (int i = 0; i < n; ++i)
    if (overlaps(out, ins[i])) return true;
  return false;
}

// The sizes of a packed or batched call; num_seqs sequences.
inline int batch_ok(const int64_t* cu, int64_t N, int64_t B, int64_t T) {
  if (B < 1 || T < 0) return KDA_ERR_BAD_SHAPE;
  if (T == 0 && !cu) return KDA_ERR_BAD_SHAPE;
  if (T > ((int64_t)1 << 40) / B) return KDA_ERR_BAD_SHAPE;
  if (cu ? (B != 1 || N < 1) : N != B) return KDA_ERR_BAD_VARLEN;
  return KDA_OK;
}

// The factor of the scores in base 2.
inline float attn_c(float scale) { return static_cast<float>(scale * 1.4426950408889634); }

// The same for the kernels, never zero: minus infinity times it stands for a masked score.  The
// smallest float in place of zero moves a finite score by 2^-21 at most, six roundings of its
// exponential.
inline float attn_factor(float scale) {
  return std::fmax(attn_c(scale), std::numeric_limits<float>::denorm_min());
}

inline int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

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
