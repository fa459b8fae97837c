// api_checks.hpp -- argument checks shared by the C-ABI files of the block
// operators (block_api.cpp, mixer_api.cpp).  Each returns SSM_OK or stores the
// message and returns the status.
#pragma once

#include <stdint.h>

#include "../../include/ssm_block.h"
#include "api_error.hpp"

namespace ssm {

constexpr int64_t kMaxElems = (int64_t)1 << 40;  // of one tensor
constexpr int64_t kMaxStep = (int64_t)1 << 23;   // elements from one step to the next

inline bool product_ok(int64_t a, int64_t b, int64_t *out) {
  if (b > kMaxElems / a) return false;
  *out = a * b;
  return true;
}

inline int check_dtype(int io_dtype) {
  if (io_dtype != SSM_F32 && io_dtype != SSM_BF16)
    return api_fail(SSM_ERR_UNSUPPORTED, "io_dtype=%d is neither SSM_F32 (0) nor SSM_BF16 (1)", io_dtype);
  return SSM_OK;
}

// A stride of a view, or its step's (which stays below kMaxStep).
inline int check_stride(const char *name, int64_t s, int io_dtype) {
  const int64_t es = io_dtype == SSM_F32 ? 4 : 2;
  if (s < 0 || s > kMaxElems) return api_fail(SSM_ERR_BAD_SHAPE, "%s has stride %lld", name, (long long)s);
  if (s * es % 16 != 0) return api_fail(SSM_ERR_ALIGNMENT, "%s has stride %lld, not a multiple of 16 bytes", name, (long long)s);
  return SSM_OK;
}

inline int check_view_ptr(const char *name, const void *view, const void *ptr) {
  if (view == nullptr || ptr == nullptr) return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", name);
  if (((uintptr_t)ptr & 15u) != 0) return api_fail(SSM_ERR_ALIGNMENT, "%s is not 16-byte aligned", name);
  return SSM_OK;
}

struct Ptr {
  const char *name;
  const void *p;
  bool required;
  unsigned align;
};

inline int check_ptrs(const Ptr *ps, int n) {
  for (int i = 0; i < n; ++i) {
    if (ps[i].required && ps[i].p == nullptr) return api_fail(SSM_ERR_NULL_ARG, "%s is NULL", ps[i].name);
    if (((uintptr_t)ps[i].p & (ps[i].align - 1)) != 0)
      return api_fail(SSM_ERR_ALIGNMENT, "%s is not %u-byte aligned", ps[i].name, ps[i].align);
  }
  return SSM_OK;
}

inline int check_workspace(const void *workspace, int64_t got, int64_t need) {
  if (need == 0) return SSM_OK;
  if (workspace == nullptr || got < need)
    return api_fail(SSM_ERR_WORKSPACE, "needs %lld workspace bytes, got %lld", (long long)need, workspace ? (long long)got : 0LL);
  if (((uintptr_t)workspace & 15u) != 0) return api_fail(SSM_ERR_ALIGNMENT, "workspace is not 16-byte aligned");
  return SSM_OK;
}

}  // namespace ssm

#define SSM_TRY(call)              \
  do {                             \
    const int st_ = (call);        \
    if (st_ != SSM_OK) return st_; \
  } while (0)
#define SSM_TRY_PTRS(ps) SSM_TRY(ssm::check_ptrs(ps, (int)(sizeof(ps) / sizeof(ps[0]))))
