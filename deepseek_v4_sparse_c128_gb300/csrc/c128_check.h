// Descriptor checks shared by the entry points (host only, nothing here touches CUDA).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "c128_internal.h"
#include "c128_serving.h"
#include "c128compress.h"

#define C128_TRY(expr)         \
  do {                         \
    const int rc_ = (expr);    \
    if (rc_ != C128_OK) return rc_; \
  } while (0)

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

constexpr int64_t kMaxCount = 0x7fffffffLL;

// Element size of a descriptor's type.
inline uintptr_t item_bytes(const c128_tensor_t* t) {
  switch (t->dtype) {
    case C128_I64: return 8;
    case C128_I32: case C128_F32: return 4;
    case C128_BF16: return 2;
    default: return 1;
  }
}

// A vector of n elements of one type, aligned to its elements.
inline int check_array(const c128_tensor_t* t, int dtype, int64_t n) {
  C128_TRY(check_vector(t, dtype, n));
  return aligned(t->data, item_bytes(t)) ? C128_OK : C128_ERR_ALIGN;
}

// A block table [requests, columns] whose rows may be padded; its row stride in *stride.
inline int check_table(const c128_tensor_t* t, int64_t requests, int64_t* stride) {
  C128_TRY(check_desc(t, C128_I32, 2));
  if (t->shape[0] != requests || t->shape[1] > kMaxCount) return C128_ERR_SHAPE;
  *stride = t->shape[1];
  if (numel(t) == 0) return C128_OK;
  if (t->shape[1] > 1 && t->stride[1] != 1) return C128_ERR_STRIDE;
  if (t->shape[0] > 1 && t->stride[0] < t->shape[1]) return C128_ERR_STRIDE;
  C128_TRY(check_data(t));
  if (!aligned(t->data, 4)) return C128_ERR_ALIGN;
  *stride = t->shape[0] > 1 ? t->stride[0] : t->shape[1];
  return C128_OK;
}

// A statistic [.., R, H] fp32 with positive strides of any order.
inline int check_lse(const c128_tensor_t* t, int ndim) {
  C128_TRY(check_desc(t, C128_F32, ndim));
  if (numel(t) == 0) return C128_OK;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] < 1) return C128_ERR_STRIDE;
  C128_TRY(check_data(t));
  return aligned(t->data, 4) ? C128_OK : C128_ERR_ALIGN;
}

// Rows of 512 values [.., R, H, 512], bf16 or (where `f32` is not NULL) fp32, each row starting on a
// 16-byte boundary.
inline int check_rows(const c128_tensor_t* t, int ndim, int32_t* f32) {
  if (t == nullptr) return C128_ERR_NULL_PTR;
  const bool is_f32 = t->dtype == C128_F32;
  C128_TRY(check_desc(t, f32 != nullptr && is_f32 ? C128_F32 : C128_BF16, ndim));
  if (f32 != nullptr) *f32 = is_f32 ? 1 : 0;
  if (t->shape[ndim - 1] != kHead) return C128_ERR_UNSUPPORTED;
  if (numel(t) == 0) return C128_OK;  // its strides say nothing
  if (t->stride[ndim - 1] != 1) return C128_ERR_STRIDE;
  for (int i = 0; i + 1 < ndim; ++i) {
    if (t->shape[i] > 1 && t->stride[i] < kHead) return C128_ERR_STRIDE;
    if (t->shape[i] > 1 && (t->stride[i] * item_bytes(t)) % 16 != 0) return C128_ERR_ALIGN;
  }
  C128_TRY(check_data(t));
  return aligned(t->data, 16) ? C128_OK : C128_ERR_ALIGN;
}
// The results [R, H, width] (width 1: [R, H]) are stored by many CTAs at once, so no two rows may share an element: the
// rows of one of the two dimensions have to lie between two neighbours of the other.
inline int check_apart(const c128_tensor_t* t, int64_t width) {
  int64_t inner = t->shape[1], at = t->stride[1], outer = t->stride[0];
  if (t->shape[0] <= 1 || t->shape[1] <= 1) return C128_OK;
  if (at > outer) at = t->stride[0], outer = t->stride[1], inner = t->shape[0];
  return (outer - width) / at >= inner - 1 ? C128_OK : C128_ERR_STRIDE;
}
// The cache as the compressor takes it: slots of 584 bytes or more, a block a flat byte range.
inline int check_cache(const c128_tensor_t* t, int64_t block_size) {
  C128_TRY(check_desc(t, C128_U8, 3));
  if (block_size < 1 || block_size > kMaxCount || t->shape[1] != block_size) return C128_ERR_ARG;
  if (t->shape[0] > kMaxCount) return C128_ERR_ARG;
  if (t->shape[2] < kSlotBytes) return C128_ERR_SHAPE;
  if (t->stride[2] != 1 || t->stride[1] != t->shape[2]) return C128_ERR_STRIDE;
  if (t->shape[0] > 1 && t->stride[0] < t->shape[1] * t->shape[2]) return C128_ERR_STRIDE;
  if ((t->shape[0] > 1 && t->stride[0] % 8 != 0) || !aligned(t->data, 16)) return C128_ERR_ALIGN;
  return check_data(t);
}
// Stride of dimension i, 0 where it has a single index (whatever the descriptor says there).
inline int64_t step(const c128_tensor_t* t, int i) { return t->shape[i] > 1 ? t->stride[i] : 0; }

inline int done(cudaError_t e) { return e == cudaSuccess ? C128_OK : C128_ERR_CUDA; }

inline bool partly_overlap(const void* a, const void* b, int64_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != y && (x < y ? y - x : x - y) < static_cast<uintptr_t>(bytes);
}

// What the two attentions over a paged cache have in common, into *p: queries [R, H, 512], cache, scale, sink,
// results and scratch.
inline int check_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size, float scale,
                           const c128_tensor_t* sink, const c128_tensor_t* out, const c128_tensor_t* lse,
                           const c128_tensor_t* workspace, DecodeParams* p) {
  C128_TRY(check_rows(q, 3, nullptr));
  const int64_t R = q->shape[0], H = q->shape[1];
  if (R > kMaxCount) return C128_ERR_ARG;
  if (H > kMaxDecodeHeads) return C128_ERR_UNSUPPORTED;
  C128_TRY(check_rows(out, 3, &p->out_f32));
  if (out->shape[0] != R || out->shape[1] != H) return C128_ERR_SHAPE;
  if (R > 0 && H > 0) C128_TRY(check_apart(out, kHead));
  C128_TRY(check_cache(k_cache, kv_block_size));
  if (!std::isfinite(scale * 1.44269504f)) return C128_ERR_ARG;  // times log2(e), the kernel's factor
  if (sink != nullptr) C128_TRY(check_array(sink, C128_F32, H));
  if (lse != nullptr) {
    C128_TRY(check_lse(lse, 2));
    if (lse->shape[0] != R || lse->shape[1] != H) return C128_ERR_SHAPE;
    if (R > 0 && H > 0) C128_TRY(check_apart(lse, 1));
  }
  C128_TRY(check_desc(workspace, C128_U8, 1));
  C128_TRY(check_array(workspace, C128_U8, workspace->shape[0]));
  if (!aligned(workspace->data, 256)) return C128_ERR_ALIGN;
  p->q = static_cast<const uint16_t*>(q->data);
  p->q_stride_r = step(q, 0);
  p->q_stride_h = step(q, 1);
  p->kc = static_cast<const uint8_t*>(k_cache->data);
  p->nkb = k_cache->shape[0];
  p->kv_bs = kv_block_size;
  p->kv_div = Divisor(kv_block_size);
  p->kc_stride0 = step(k_cache, 0);
  p->requests = R;
  p->heads = static_cast<int32_t>(H);
  p->scale = scale;
  p->sink = sink != nullptr ? static_cast<const float*>(sink->data) : nullptr;
  p->out = out->data;
  p->out_stride_r = step(out, 0);
  p->out_stride_h = step(out, 1);
  p->lse = lse != nullptr ? static_cast<float*>(lse->data) : nullptr;
  p->lse_stride_r = lse != nullptr ? step(lse, 0) : 0;
  p->lse_stride_h = lse != nullptr ? step(lse, 1) : 0;
  p->workspace = static_cast<uint8_t*>(workspace->data);
  return C128_OK;
}

}  // namespace check
}  // namespace c128
