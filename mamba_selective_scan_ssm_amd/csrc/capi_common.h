// Host-side checks shared by the files of the C ABI.
#pragma once

#include "../../include/ssm_scan.h"

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

namespace ssm {
namespace capi {

constexpr int64_t kMaxGridYZ = 65535;

inline bool valid_dtype(ssm_dtype dt) { return dt == SSM_F32 || dt == SSM_BF16; }
inline int64_t esize(ssm_dtype dt) { return dt == SSM_BF16 ? 2 : 4; }

struct Range {
  const void *p;
  int64_t bytes;
};

inline bool overlap(Range a, Range b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

template <size_t K>
inline bool overlaps_any(Range out, const Range (&ins)[K]) {
  for (size_t i = 0; i < K; ++i)
    if (overlap(out, ins[i])) return true;
  return false;
}

// Whether two of the outputs share memory.
inline bool any_pair(const Range *r, size_t n) {
  for (size_t i = 0; i < n; ++i)
    for (size_t j = i + 1; j < n; ++j)
      if (overlap(r[i], r[j])) return true;
  return false;
}

inline bool dopts_ok(const ssm_delta_opts *o) {
  if (!o) return true;
  for (int i = 0; i < 3; ++i)
    if (o->reserved[i] != 0) return false;
  return o->softplus == 0 || o->softplus == 1;
}
inline const float *dbias_of(const ssm_delta_opts *o) { return o ? o->bias : nullptr; }
inline bool dsoft_of(const ssm_delta_opts *o) { return o && o->softplus == 1; }

inline ssm_status hip_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

// The product of non-negative sizes; false where it passes 2^58 (no array of
// that many elements exists, and byte counts formed from it stay in range).
inline bool product(std::initializer_list<int64_t> sizes, int64_t *out) {
  int64_t n = 1;
  for (int64_t s : sizes)
    if (__builtin_mul_overflow(n, s, &n) || n > (int64_t(1) << 58)) return false;
  *out = n;
  return true;
}

}  // namespace capi
}  // namespace ssm
