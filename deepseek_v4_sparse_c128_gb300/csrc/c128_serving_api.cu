// C entry points of the operators around the compressor: argument checks (host only, before
// anything is launched) and the launches. Declarations and their contract are in
// include/c128compress.h.
#include <cuda_runtime.h>

#include <cmath>

#include "c128_check.h"
#include "c128_serving.h"
#include "c128compress.h"

namespace {

using namespace c128::check;

constexpr int64_t kMaxCount = 0x7fffffffLL;

// Element size of a descriptor's type.
uintptr_t item_bytes(const c128_tensor_t* t) {
  switch (t->dtype) {
    case C128_I64: return 8;
    case C128_I32: case C128_F32: return 4;
    case C128_BF16: return 2;
    default: return 1;
  }
}

// A vector of n elements of one type, aligned to its elements.
int check_array(const c128_tensor_t* t, int dtype, int64_t n) {
  C128_TRY(check_vector(t, dtype, n));
  return aligned(t->data, item_bytes(t)) ? C128_OK : C128_ERR_ALIGN;
}

// A block table [requests, columns] whose rows may be padded; its row stride in *stride.
int check_table(const c128_tensor_t* t, int64_t requests, int64_t* stride) {
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
int check_lse(const c128_tensor_t* t, int ndim) {
  C128_TRY(check_desc(t, C128_F32, ndim));
  if (numel(t) == 0) return C128_OK;
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] > 1 && t->stride[i] < 1) return C128_ERR_STRIDE;
  C128_TRY(check_data(t));
  return aligned(t->data, 4) ? C128_OK : C128_ERR_ALIGN;
}

// Rows of 512 values [.., R, H, 512], bf16 or (where `f32` is not NULL) fp32, each row starting on a
// 16-byte boundary.
int check_rows(const c128_tensor_t* t, int ndim, int32_t* f32) {
  if (t == nullptr) return C128_ERR_NULL_PTR;
  const bool is_f32 = t->dtype == C128_F32;
  C128_TRY(check_desc(t, f32 != nullptr && is_f32 ? C128_F32 : C128_BF16, ndim));
  if (f32 != nullptr) *f32 = is_f32 ? 1 : 0;
  if (t->shape[ndim - 1] != c128::kHead) return C128_ERR_UNSUPPORTED;
  if (numel(t) == 0) return C128_OK;  // its strides say nothing
  if (t->stride[ndim - 1] != 1) return C128_ERR_STRIDE;
  for (int i = 0; i + 1 < ndim; ++i) {
    if (t->shape[i] > 1 && t->stride[i] < c128::kHead) return C128_ERR_STRIDE;
    if (t->shape[i] > 1 && (t->stride[i] * item_bytes(t)) % 16 != 0) return C128_ERR_ALIGN;
  }
  C128_TRY(check_data(t));
  return aligned(t->data, 16) ? C128_OK : C128_ERR_ALIGN;
}
// The results [R, H, width] (width 1: [R, H]) are stored by many CTAs at once, so no two rows may share an element: the
// rows of one of the two dimensions have to lie between two neighbours of the other.
int check_apart(const c128_tensor_t* t, int64_t width) {
  int64_t inner = t->shape[1], at = t->stride[1], outer = t->stride[0];
  if (t->shape[0] <= 1 || t->shape[1] <= 1) return C128_OK;
  if (at > outer) at = t->stride[0], outer = t->stride[1], inner = t->shape[0];
  return (outer - width) / at >= inner - 1 ? C128_OK : C128_ERR_STRIDE;
}
// Stride of dimension i, 0 where it has a single index (whatever the descriptor says there).
int64_t step(const c128_tensor_t* t, int i) { return t->shape[i] > 1 ? t->stride[i] : 0; }

int done(cudaError_t e) { return e == cudaSuccess ? C128_OK : C128_ERR_CUDA; }

bool partly_overlap(const void* a, const void* b, int64_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x != y && (x < y ? y - x : x - y) < static_cast<uintptr_t>(bytes);
}

// c128_decode_attention; `stall`: the test of its waits.
int decode(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
           const c128_tensor_t* block_table, const c128_tensor_t* kv_lens, float scale,
           const c128_tensor_t* sink, const c128_tensor_t* out, const c128_tensor_t* lse,
           const c128_tensor_t* workspace, c128_stream_t stream, bool stall) {
  c128::DecodeParams p{};
  C128_TRY(check_rows(q, 3, nullptr));
  const int64_t R = q->shape[0], H = q->shape[1];
  if (R > kMaxCount) return C128_ERR_ARG;
  if (H > c128::kMaxDecodeHeads) return C128_ERR_UNSUPPORTED;
  C128_TRY(check_rows(out, 3, &p.out_f32));
  if (out->shape[0] != R || out->shape[1] != H) return C128_ERR_SHAPE;
  if (R > 0 && H > 0) C128_TRY(check_apart(out, c128::kHead));
  // the cache as the compressor takes it (slots of 584 bytes or more, a block a flat byte range)
  C128_TRY(check_desc(k_cache, C128_U8, 3));
  if (kv_block_size < 1 || kv_block_size > kMaxCount || k_cache->shape[1] != kv_block_size) return C128_ERR_ARG;
  if (k_cache->shape[0] > kMaxCount) return C128_ERR_ARG;
  if (k_cache->shape[2] < c128::kSlotBytes) return C128_ERR_SHAPE;
  if (k_cache->stride[2] != 1 || k_cache->stride[1] != k_cache->shape[2]) return C128_ERR_STRIDE;
  if (k_cache->shape[0] > 1 && k_cache->stride[0] < k_cache->shape[1] * k_cache->shape[2]) return C128_ERR_STRIDE;
  if ((k_cache->shape[0] > 1 && k_cache->stride[0] % 8 != 0) || !aligned(k_cache->data, 16)) return C128_ERR_ALIGN;
  C128_TRY(check_data(k_cache));
  C128_TRY(check_table(block_table, R, &p.table_stride));
  C128_TRY(check_array(kv_lens, C128_I32, R));
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
  if (R == 0 || H == 0) return C128_OK;
  // what the table can hold, in tiles of 64 entries: the kernel counts those, and the requests, in 32 bits
  const int64_t most = block_table->shape[1] > kMaxCount / kv_block_size ? kMaxCount : block_table->shape[1] * kv_block_size;
  if (R * (most / 64 + 2) > kMaxCount) return C128_ERR_ARG;
  p.most = static_cast<int32_t>(most);
  p.q = static_cast<const uint16_t*>(q->data);
  p.q_stride_r = step(q, 0);
  p.q_stride_h = step(q, 1);
  p.kc = static_cast<const uint8_t*>(k_cache->data);
  p.nkb = k_cache->shape[0];
  p.kv_bs = kv_block_size;
  p.kv_div = c128::Divisor(kv_block_size);
  p.kc_stride0 = step(k_cache, 0);
  p.table = static_cast<const int32_t*>(block_table->data);
  p.requests = R;
  p.kv_lens = static_cast<const int32_t*>(kv_lens->data);
  p.heads = static_cast<int32_t>(H);
  p.scale = scale;
  p.sink = sink != nullptr ? static_cast<const float*>(sink->data) : nullptr;
  p.out = out->data;
  p.out_stride_r = step(out, 0);
  p.out_stride_h = step(out, 1);
  p.lse = lse != nullptr ? static_cast<float*>(lse->data) : nullptr;
  p.lse_stride_r = lse != nullptr ? step(lse, 0) : 0;
  p.lse_stride_h = lse != nullptr ? step(lse, 1) : 0;
  p.workspace = static_cast<uint8_t*>(workspace->data);
  p.stall = stall ? 1 : 0;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  C128_TRY(c128::stream_errors(s, &p.err, &sms));
  if (workspace->shape[0] < c128::decode_workspace_bytes(p.heads, sms)) return C128_ERR_ARG;
  return done(c128::launch_decode(p, sms, s));
}

}  // namespace

extern "C" {

int c128_extend_block_tables(const c128_tensor_t* seq_lens, const c128_tensor_t* held, const c128_tensor_t* block_table,
                             const c128_tensor_t* free_blocks, const c128_tensor_t* taken, int32_t compress_ratio,
                             int64_t block_size, const c128_tensor_t* held_out, const c128_tensor_t* taken_out,
                             c128_stream_t stream) {
  C128_TRY(check_desc(seq_lens, C128_I32, 1));
  const int64_t R = seq_lens->shape[0];
  if (R > kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_array(seq_lens, C128_I32, R));
  C128_TRY(check_array(held, C128_I32, R));
  C128_TRY(check_array(held_out, C128_I32, R));
  c128::ExtendParams p{};
  C128_TRY(check_table(block_table, R, &p.stride));
  C128_TRY(check_desc(free_blocks, C128_I32, 1));
  if (free_blocks->shape[0] >= kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_array(free_blocks, C128_I32, free_blocks->shape[0]));
  C128_TRY(check_array(taken, C128_I64, 1));
  C128_TRY(check_array(taken_out, C128_I64, 1));
  if (compress_ratio < 1 || block_size < 1 || block_size > kMaxCount) return C128_ERR_ARG;
  if (partly_overlap(held->data, held_out->data, 4 * R)) return C128_ERR_ARG;
  p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  p.held = static_cast<const int32_t*>(held->data);
  p.held_out = static_cast<int32_t*>(held_out->data);
  p.table = static_cast<int32_t*>(block_table->data);
  p.requests = R;
  p.columns = block_table->shape[1];
  p.free_blocks = static_cast<const int32_t*>(free_blocks->data);
  p.num_free = free_blocks->shape[0];
  p.taken = static_cast<const int64_t*>(taken->data);
  p.taken_out = static_cast<int64_t*>(taken_out->data);
  p.ratio = c128::Divisor(compress_ratio);
  p.block = c128::Divisor(block_size);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  C128_TRY(c128::stream_errors(s, &p.err, &sms));
  return done(c128::launch_extend(p, sms, s));
}

int c128_build_slot_maps(const c128_tensor_t* seq_lens, const c128_tensor_t* query_lens, const c128_tensor_t* state_table,
                         int64_t state_block, const c128_tensor_t* kv_table, int64_t kv_block_size, int32_t compress_ratio,
                         const c128_tensor_t* query_start, const c128_tensor_t* token_to_req_indices,
                         const c128_tensor_t* positions, const c128_tensor_t* slot_mapping,
                         const c128_tensor_t* kv_slot_mapping, const c128_tensor_t* kv_lens, c128_stream_t stream) {
  C128_TRY(check_desc(seq_lens, C128_I32, 1));
  const int64_t R = seq_lens->shape[0];
  if (R >= kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_array(seq_lens, C128_I32, R));
  C128_TRY(check_array(query_lens, C128_I32, R));
  C128_TRY(check_array(kv_lens, C128_I32, R));
  C128_TRY(check_array(query_start, C128_I32, R + 1));
  C128_TRY(check_desc(positions, C128_I64, 1));
  const int64_t T = positions->shape[0];
  if (T >= kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_array(positions, C128_I64, T));
  C128_TRY(check_array(token_to_req_indices, C128_I32, T));
  C128_TRY(check_array(slot_mapping, C128_I64, T));
  C128_TRY(check_array(kv_slot_mapping, C128_I64, T));
  c128::SlotMapParams p{};
  C128_TRY(check_table(state_table, R, &p.state_stride));
  C128_TRY(check_table(kv_table, R, &p.kv_stride));
  if (compress_ratio < 1 || state_block < 1 || state_block > kMaxCount || kv_block_size < 1 || kv_block_size > kMaxCount)
    return C128_ERR_ARG;
  p.seq_lens = static_cast<const int32_t*>(seq_lens->data);
  p.query_lens = static_cast<const int32_t*>(query_lens->data);
  p.requests = R;
  p.state_table = static_cast<const int32_t*>(state_table->data);
  p.state_cols = state_table->shape[1];
  p.state_block = c128::Divisor(state_block);
  p.kv_table = static_cast<const int32_t*>(kv_table->data);
  p.kv_cols = kv_table->shape[1];
  p.kv_block = c128::Divisor(kv_block_size);
  p.ratio = c128::Divisor(compress_ratio);
  p.query_start = static_cast<int32_t*>(query_start->data);
  p.token_to_req = static_cast<int32_t*>(token_to_req_indices->data);
  p.positions = static_cast<int64_t*>(positions->data);
  p.slots = static_cast<int64_t*>(slot_mapping->data);
  p.kv_slots = static_cast<int64_t*>(kv_slot_mapping->data);
  p.kv_lens = static_cast<int32_t*>(kv_lens->data);
  p.tokens = T;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  C128_TRY(c128::stream_errors(s, &p.err, &sms));
  return done(c128::launch_slot_maps(p, s));
}

int c128_decode_attention_workspace(int64_t num_heads, int64_t* bytes) {
  if (bytes == nullptr) return C128_ERR_NULL_PTR;
  if (num_heads < 1 || num_heads > c128::kMaxDecodeHeads) return C128_ERR_UNSUPPORTED;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return C128_ERR_CUDA;
  *bytes = c128::decode_workspace_bytes(static_cast<int>(num_heads), sms);
  return C128_OK;
}

int c128_decode_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                          const c128_tensor_t* block_table, const c128_tensor_t* kv_lens, float scale,
                          const c128_tensor_t* sink, const c128_tensor_t* out, const c128_tensor_t* lse,
                          const c128_tensor_t* workspace, c128_stream_t stream) {
  return decode(q, k_cache, kv_block_size, block_table, kv_lens, scale, sink, out, lse, workspace, stream, false);
}

int c128_debug_stall_decode_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                                      const c128_tensor_t* block_table, const c128_tensor_t* kv_lens, float scale,
                                      const c128_tensor_t* sink, const c128_tensor_t* out, const c128_tensor_t* lse,
                                      const c128_tensor_t* workspace, c128_stream_t stream) {
  return decode(q, k_cache, kv_block_size, block_table, kv_lens, scale, sink, out, lse, workspace, stream, true);
}

int c128_merge_attention(const c128_tensor_t* part_out, const c128_tensor_t* part_lse, const c128_tensor_t* out,
                         const c128_tensor_t* lse, c128_stream_t stream) {
  c128::MergeParams p{};
  C128_TRY(check_rows(part_out, 4, &p.part_f32));
  const int64_t P = part_out->shape[0], R = part_out->shape[1], H = part_out->shape[2];
  if (P < 1 || P > kMaxCount || R > kMaxCount || H > kMaxCount) return C128_ERR_ARG;
  if (R * H > kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_lse(part_lse, 3));
  if (part_lse->shape[0] != P || part_lse->shape[1] != R || part_lse->shape[2] != H) return C128_ERR_SHAPE;
  C128_TRY(check_rows(out, 3, &p.out_f32));
  if (out->shape[0] != R || out->shape[1] != H) return C128_ERR_SHAPE;
  if (R > 0 && H > 0) C128_TRY(check_apart(out, c128::kHead));
  if (lse != nullptr) {
    C128_TRY(check_lse(lse, 2));
    if (lse->shape[0] != R || lse->shape[1] != H) return C128_ERR_SHAPE;
    if (R > 0 && H > 0) C128_TRY(check_apart(lse, 1));
  }
  if (R == 0 || H == 0) return C128_OK;
  p.part = part_out->data;
  p.part_stride_p = step(part_out, 0);
  p.part_stride_r = step(part_out, 1);
  p.part_stride_h = step(part_out, 2);
  p.part_lse = static_cast<const float*>(part_lse->data);
  p.lse_in_p = step(part_lse, 0);
  p.lse_in_r = step(part_lse, 1);
  p.lse_in_h = step(part_lse, 2);
  p.parts = P;
  p.requests = R;
  p.heads = H;
  p.out = out->data;
  p.out_stride_r = step(out, 0);
  p.out_stride_h = step(out, 1);
  p.lse = lse != nullptr ? static_cast<float*>(lse->data) : nullptr;
  p.lse_stride_r = lse != nullptr ? step(lse, 0) : 0;
  p.lse_stride_h = lse != nullptr ? step(lse, 1) : 0;
  return done(c128::launch_merge(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
