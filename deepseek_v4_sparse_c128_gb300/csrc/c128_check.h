// Descriptor checks shared by the entry points (host only, nothing here touches CUDA).
#pragma once
#include <stdint.h>

#include "c128compress.h"

namespace c128 {
namespace check {

inline int check_desc(const c128_tensor_t* t, int dtype, int ndim) {
  if (t == nullptr) return C128_ERR_NULL_PTR;
  if (t->dtype != dtype) return C128_ERR_DTYPE;
  if (t->ndim != ndim) return C128_ERR_SHAPE;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] < 0) return C128_ERR_SHAPE;
  return C128_OK;
}
inline int64_t numel(const c128_tensor_t* t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}
inline int check_data(const c128_tensor_t* t) {
  if (numel(t) > 0 && t->data == nullptr) return C128_ERR_NULL_PTR;
  return C128_OK;
}
inline int check_vector(const c128_tensor_t* t, int dtype, int64_t n) {
  int rc = check_desc(t, dtype, 1);
  if (rc) return rc;
  if (t->shape[0] != n) return C128_ERR_SHAPE;
  if (n > 1 && t->stride[0] != 1) return C128_ERR_STRIDE;
  return check_data(t);
}
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

}  // namespace check
}  // namespace c128

#define C128_TRY(expr)         \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_ != C128_OK) return rc_; \
  } while (0)
