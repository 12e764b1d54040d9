// kda_check.h -- host-side argument checks shared by the C ABI sources.
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstdint>

#include "kda.h"

namespace kda {

// KDA_OK, or KDA_ERR_HIP with the error kept for kda_last_hip_error().
int hip_status(hipError_t e);

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = (uintptr_t)p;
  return Range{lo, lo + (uintptr_t)(bytes > 0 ? bytes : 0)};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.hi > a.lo && b.hi > b.lo; }

// Rows of `row` bytes, `stride` bytes apart (stride >= row).
struct RowSet {
  uintptr_t p;
  int64_t rows, stride, row;
};

inline RowSet row_set(const void* p, int64_t rows, int64_t stride, int64_t row, int64_t es) {
  return RowSet{(uintptr_t)p, p ? rows : 0, stride * es, row * es};
}

inline Range range_of(const RowSet& r) {
  return range_of((const void*)r.p, r.rows > 0 ? (r.rows - 1) * r.stride + r.row : 0);
}

// Whether two row sets share a byte; for different strides, whether their
// extents do.  Rows of one stride that lie side by side (two slices of a wider
// buffer) are apart.
inline bool overlap(const RowSet& a, const RowSet& b) {
  if (!overlap(range_of(a), range_of(b))) return false;
  if (a.stride != b.stride) return true;
  const int64_t s = a.stride;
  const int64_t d = (int64_t)((a.p >= b.p ? a.p - b.p : b.p - a.p) % (uintptr_t)s);
  const int64_t to_a = a.p >= b.p ? d : (s - d) % s;  // a's rows start this far into b's
  return !(to_a >= b.row && to_a + a.row <= s);
}

inline bool supported_d(int d) { return d == 32 || d == 64 || d == 128; }

// State dtype: 0 or fp32, or bf16 with bf16 inputs.  Sets *bf16_state.
inline int check_state_dtype(int32_t state_dtype, int32_t dtype, bool* bf16_state) {
  if (state_dtype == 0 || state_dtype == KDA_DTYPE_F32) {
    *bf16_state = false;
    return KDA_OK;
  }
  if (state_dtype != KDA_DTYPE_BF16) return KDA_ERR_DTYPE;
  if (dtype != KDA_DTYPE_BF16) return KDA_ERR_UNSUPPORTED;
  *bf16_state = true;
  return KDA_OK;
}

}  // namespace kda
