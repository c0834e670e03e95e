// host_checks.h -- argument checks that the C ABI's files share.  Nothing is thrown: a check returns a
// status and describes it for moe_last_error().
#pragma once
#include <cuda_runtime.h>
#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "moe_internal.h"

namespace moe {

inline moe_status fail(moe_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
inline moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return set_last_error(st, buf);
}

inline moe_status cuda_status(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  return fail(MOE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Ptr {
  const void* p;
  const char* name;
  size_t align;
  bool may_be_null;
};
template <size_t N>
moe_status check(const Ptr (&ptrs)[N]) {
  for (const Ptr& q : ptrs) {
    if (!q.p && !q.may_be_null) return fail(MOE_ERR_INVALID_ARG, "%s is null", q.name);
    if (!aligned(q.p, q.align)) return fail(MOE_ERR_INVALID_ARG, "%s is not %zu-byte aligned", q.name, q.align);
  }
  return MOE_OK;
}

// Whether [a, a + na) and [b, b + nb) share a byte.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return na && nb && x < y + nb && y < x + na;
}

inline bool is_dtype(int32_t t) { return t == MOE_F32 || t == MOE_BF16; }
inline size_t esize(int32_t t) { return t == MOE_BF16 ? 2 : 4; }

}  // namespace moe
