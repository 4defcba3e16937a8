// C entry points of the operators around the attention of recent tokens: argument checks (host only,
// before anything is launched) and the launches. Declarations and their contract are in
// include/c128compress.h.
#include <cuda_runtime.h>

#include <cmath>

#include "c128_check.h"
#include "c128_step.h"
#include "c128compress.h"

namespace {

using namespace c128::check;

// A table of rotations [MP, R] with R even; its row stride in *stride.
int check_cos_sin(const c128_tensor_t* t, int64_t* stride) {
  C128_TRY(check_desc(t, C128_F32, 2));
  const int64_t R = t->shape[1];
  if (R < 2 || R % 2 != 0 || R > c128::kMaxTurned) return C128_ERR_UNSUPPORTED;
  *stride = R;
  if (t->shape[0] == 0) return C128_OK;
  if (t->stride[1] != 1 || (t->shape[0] > 1 && t->stride[0] < R)) return C128_ERR_STRIDE;
  C128_TRY(check_data(t));
  if (!aligned(t->data, 4)) return C128_ERR_ALIGN;
  *stride = step(t, 0);
  return C128_OK;
}

// Values [T, H, D] of one of two types.
int check_heads(const c128_tensor_t* t, int32_t* f32) {
  if (t == nullptr) return C128_ERR_NULL_PTR;
  *f32 = t->dtype == C128_F32 ? 1 : 0;
  C128_TRY(check_desc(t, *f32 ? C128_F32 : C128_BF16, 3));
  if (numel(t) == 0) return C128_OK;
  if (t->stride[2] != 1) return C128_ERR_STRIDE;
  for (int i = 0; i < 2; ++i)
    if (t->shape[i] > 1 && t->stride[i] < t->shape[2]) return C128_ERR_STRIDE;
  C128_TRY(check_data(t));
  return aligned(t->data, item_bytes(t)) ? C128_OK : C128_ERR_ALIGN;
}

// A norm's weight, which may be missing.
int check_weight(const c128_tensor_t* t) {
  if (t == nullptr) return C128_OK;
  C128_TRY(check_array(t, C128_F32, c128::kHead));
  return aligned(t->data, 16) ? C128_OK : C128_ERR_ALIGN;
}

bool positive(double x) { return x > 0 && std::isfinite(x); }

// Turns per position that a step may have. (In 53 bits, 33 or more of them behind the point; past 2^53 nothing would be left.)
constexpr double kMostTurns = 0x1p20;

// The steps of c128_rope_t in turns per position, as fractions of 2^64.
int rope_steps(const c128_rope_t* rope, int turned, uint64_t* step) {
  if (rope == nullptr) return C128_ERR_NULL_PTR;
  const int scaling = rope->scaling;
  if (scaling != C128_ROPE_PLAIN && scaling != C128_ROPE_LINEAR && scaling != C128_ROPE_YARN) return C128_ERR_UNSUPPORTED;
  if (!(rope->theta > 1) || !std::isfinite(rope->theta) || rope->reserved != 0) return C128_ERR_ARG;
  if (!std::isfinite(rope->magnitude) || !std::isfinite(static_cast<float>(rope->magnitude))) return C128_ERR_ARG;
  if (scaling != C128_ROPE_PLAIN && !positive(rope->factor)) return C128_ERR_ARG;
  const double kTurn = 6.283185307179586476925286766559;
  double low = 0, high = 0;
  if (scaling == C128_ROPE_YARN) {
    if (!positive(rope->original_positions) || !positive(rope->beta_fast) || !positive(rope->beta_slow)) return C128_ERR_ARG;
    auto pair = [&](double turns) {
      return turned * std::log(rope->original_positions / (kTurn * turns)) / (2 * std::log(rope->theta));
    };
    low = std::fmax(std::floor(pair(rope->beta_fast)), 0);
    high = std::fmin(std::ceil(pair(rope->beta_slow)), turned - 1);
  }
  for (int i = 0; i < turned / 2; ++i) {
    double f = std::pow(rope->theta, -2.0 * i / turned);
    if (scaling == C128_ROPE_LINEAR) f /= rope->factor;
    if (scaling == C128_ROPE_YARN) {
      const double g = std::fmin(std::fmax((i - low) / std::fmax(high - low, 0.001), 0), 1);
      f = f * (1 - g) + f / rope->factor * g;
    }
    const double turns = f / kTurn;
    if (!(turns <= kMostTurns)) return C128_ERR_ARG;  // NaN too: of an infinite step times a ramp of 0
    const double part = turns - std::floor(turns);
    const double scaled = std::nearbyint(part * 0x1p64);
    step[i] = scaled >= 0x1p64 ? 0 : static_cast<uint64_t>(scaled);
  }
  return C128_OK;
}

// c128_window_attention; `stall`: the test of its waits.
int window_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                     const c128_tensor_t* block_table, const c128_tensor_t* token_to_req_indices,
                     const c128_tensor_t* positions, const c128_tensor_t* slot_mapping, int64_t window,
                     int64_t first, float scale, const c128_tensor_t* sink, const c128_tensor_t* out,
                     const c128_tensor_t* lse, const c128_tensor_t* workspace, c128_stream_t stream, bool stall) {
  c128::DecodeParams p{};
  C128_TRY(check_attention(q, k_cache, kv_block_size, scale, sink, out, lse, workspace, &p));
  const int64_t T = q->shape[0];
  C128_TRY(check_desc(block_table, C128_I32, 2));
  p.table_rows = block_table->shape[0];
  if (p.table_rows > kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_table(block_table, p.table_rows, &p.table_stride));
  C128_TRY(check_array(token_to_req_indices, C128_I32, T));
  C128_TRY(check_array(positions, C128_I64, T));
  C128_TRY(check_array(slot_mapping, C128_I64, T));
  if (window < 1 || window > kMaxCount || first < 0 || first > kMaxCount) return C128_ERR_ARG;
  if (T == 0 || q->shape[1] == 0) return C128_OK;
  // what the table can hold, and what a token can see of it, in tiles of 64 entries: counted in 32 bits
  const int64_t most = block_table->shape[1] > kMaxCount / kv_block_size ? kMaxCount : block_table->shape[1] * kv_block_size;
  const int64_t seen = most < window + first ? most : window + first;
  if (T * (seen / 64 + 2) > kMaxCount) return C128_ERR_ARG;
  p.most = static_cast<int32_t>(most);
  p.table = static_cast<const int32_t*>(block_table->data);
  p.token_req = static_cast<const int32_t*>(token_to_req_indices->data);
  p.positions = static_cast<const int64_t*>(positions->data);
  p.slots = static_cast<const int64_t*>(slot_mapping->data);
  p.window = window;
  p.first = static_cast<int32_t>(first);
  p.stall = stall ? 1 : 0;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  C128_TRY(c128::stream_errors(s, &p.err, &sms));
  if (c128::window_fits(window, first)) return done(c128::launch_window(p, sms, s));
  if (workspace->shape[0] < c128::decode_workspace_bytes(p.heads, sms)) return C128_ERR_ARG;
  return done(c128::launch_decode(p, workspace->shape[0], sms, s));
}

}  // namespace

extern "C" {

int c128_build_cos_sin(const c128_rope_t* rope, int64_t first_position, const c128_tensor_t* cos_sin_cache,
                       c128_stream_t stream) {
  c128::CosSinParams p{};
  C128_TRY(check_cos_sin(cos_sin_cache, &p.stride));
  const int64_t rows = cos_sin_cache->shape[0], turned = cos_sin_cache->shape[1];
  C128_TRY(rope_steps(rope, static_cast<int>(turned), p.step));
  constexpr int64_t kMostPositions = 1ll << 32;
  if (first_position < 0 || first_position > kMostPositions || rows > kMostPositions - first_position) return C128_ERR_ARG;
  if (rows == 0) return C128_OK;
  p.table = static_cast<float*>(cos_sin_cache->data);
  p.rows = rows;
  p.first = static_cast<uint64_t>(first_position);
  p.half = static_cast<int32_t>(turned / 2);
  p.magnitude = static_cast<float>(rope->magnitude);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return C128_ERR_CUDA;
  return done(c128::launch_cos_sin(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int c128_rotate(const c128_tensor_t* x, const c128_tensor_t* positions, const c128_tensor_t* cos_sin_cache,
                int64_t first_column, int32_t layout, int32_t inverse, const c128_tensor_t* out, c128_stream_t stream) {
  c128::RotateParams p{};
  C128_TRY(check_heads(x, &p.f32));
  const int64_t T = x->shape[0], H = x->shape[1], D = x->shape[2];
  if (T > kMaxCount || H > kMaxCount || D > kMaxCount || H * D > kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_array(positions, C128_I64, T));
  C128_TRY(check_cos_sin(cos_sin_cache, &p.cs_stride));
  const int64_t turned = cos_sin_cache->shape[1];
  if (layout != C128_ROPE_PAIRS && layout != C128_ROPE_HALVES) return C128_ERR_UNSUPPORTED;
  if (inverse != 0 && inverse != 1) return C128_ERR_ARG;
  if (first_column < 0 || first_column > D || turned > D - first_column) return C128_ERR_ARG;
  int32_t out_f32 = 0;
  C128_TRY(check_heads(out, &out_f32));
  if (out_f32 != p.f32) return C128_ERR_DTYPE;
  if (out->shape[0] != T || out->shape[1] != H || out->shape[2] != D) return C128_ERR_SHAPE;
  if (T == 0 || H == 0) return C128_OK;
  C128_TRY(check_apart(out, D));
  p.x = x->data;
  p.x_stride_t = step(x, 0);
  p.x_stride_h = step(x, 1);
  p.out = out->data;
  p.out_stride_t = step(out, 0);
  p.out_stride_h = step(out, 1);
  p.in_place = x->data == out->data ? 1 : 0;
  if (p.in_place && (p.x_stride_t != p.out_stride_t || p.x_stride_h != p.out_stride_h)) return C128_ERR_STRIDE;
  p.tokens = T;
  p.heads = static_cast<int32_t>(H);
  p.width = static_cast<int32_t>(D);
  p.first = static_cast<int32_t>(first_column);
  p.half = static_cast<int32_t>(turned / 2);
  p.halves = layout == C128_ROPE_HALVES ? 1 : 0;
  p.sign = inverse ? -1.f : 1.f;
  p.positions = static_cast<const int64_t*>(positions->data);
  p.cos_sin = static_cast<const float*>(cos_sin_cache->data);
  p.rows = cos_sin_cache->shape[0];
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  C128_TRY(c128::stream_errors(s, &p.err, &sms));
  return done(c128::launch_rotate(p, s));
}

int c128_norm_rope_store(const c128_tensor_t* positions, const c128_tensor_t* slot_mapping, float eps,
                         const c128_tensor_t* cos_sin_cache, const c128_tensor_t* q, const c128_tensor_t* q_w,
                         const c128_tensor_t* q_out, const c128_tensor_t* k, const c128_tensor_t* k_w,
                         const c128_tensor_t* k_cache, int64_t kv_block_size, c128_stream_t stream) {
  c128::NormParams p{};
  C128_TRY(check_desc(positions, C128_I64, 1));
  const int64_t T = positions->shape[0];
  if (T > kMaxCount) return C128_ERR_ARG;
  C128_TRY(check_array(positions, C128_I64, T));
  C128_TRY(check_array(slot_mapping, C128_I64, T));
  C128_TRY(check_cos_sin(cos_sin_cache, &p.cs_stride));
  if (cos_sin_cache->shape[1] != c128::kRope) return C128_ERR_UNSUPPORTED;
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_cache == nullptr) || (q == nullptr && k == nullptr))
    return C128_ERR_NULL_PTR;
  if (q == nullptr && q_w != nullptr) return C128_ERR_NULL_PTR;
  if (k == nullptr && k_w != nullptr) return C128_ERR_NULL_PTR;
  C128_TRY(check_weight(q_w));
  C128_TRY(check_weight(k_w));
  int64_t H = 0;
  if (q != nullptr) {
    C128_TRY(check_rows(q, 3, &p.q_f32));
    C128_TRY(check_rows(q_out, 3, &p.out_f32));
    H = q->shape[1];
    if (q->shape[0] != T || q_out->shape[0] != T || q_out->shape[1] != H) return C128_ERR_SHAPE;
    if (H > kMaxCount) return C128_ERR_ARG;
    if (T > 0 && H > 0) C128_TRY(check_apart(q_out, c128::kHead));
    if (q->data != nullptr && q->data == q_out->data &&
        (p.q_f32 != p.out_f32 || step(q, 0) != step(q_out, 0) || step(q, 1) != step(q_out, 1)))
      return p.q_f32 != p.out_f32 ? C128_ERR_DTYPE : C128_ERR_STRIDE;
    p.q = q->data;
    p.q_stride_t = step(q, 0);
    p.q_stride_h = step(q, 1);
    p.q_w = q_w != nullptr ? static_cast<const float*>(q_w->data) : nullptr;
    p.q_out = q_out->data;
    p.out_stride_t = step(q_out, 0);
    p.out_stride_h = step(q_out, 1);
    p.heads = static_cast<int32_t>(H);
  }
  if (k != nullptr) {
    C128_TRY(check_rows(k, 2, &p.k_f32));
    if (k->shape[0] != T) return C128_ERR_SHAPE;
    C128_TRY(check_cache(k_cache, kv_block_size));
    p.k = k->data;
    p.k_stride = step(k, 0);
    p.k_w = k_w != nullptr ? static_cast<const float*>(k_w->data) : nullptr;
    p.kc = static_cast<uint8_t*>(k_cache->data);
    p.nkb = k_cache->shape[0];
    p.kv_bs = kv_block_size;
    p.kc_stride0 = step(k_cache, 0);
    p.kv_div = c128::Divisor(kv_block_size);
  }
  if (T * ((H + 3) / 4 + 1) > kMaxCount) return C128_ERR_ARG;
  if (T == 0 || (k == nullptr && H == 0)) return C128_OK;
  p.positions = static_cast<const int64_t*>(positions->data);
  p.slots = static_cast<const int64_t*>(slot_mapping->data);
  p.tokens = T;
  p.eps = eps;
  p.cos_sin = static_cast<const float*>(cos_sin_cache->data);
  p.rows = cos_sin_cache->shape[0];
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  int sms = 0;
  C128_TRY(c128::stream_errors(s, &p.err, &sms));
  return done(c128::launch_norm(p, sms, s));
}

int c128_window_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                          const c128_tensor_t* block_table, const c128_tensor_t* token_to_req_indices,
                          const c128_tensor_t* positions, const c128_tensor_t* slot_mapping, int64_t window,
                          int64_t first, float scale, const c128_tensor_t* sink, const c128_tensor_t* out,
                          const c128_tensor_t* lse, const c128_tensor_t* workspace, c128_stream_t stream) {
  return window_attention(q, k_cache, kv_block_size, block_table, token_to_req_indices, positions, slot_mapping, window, first,
                          scale, sink, out, lse, workspace, stream, false);
}

int c128_window_attention_workspace(int64_t num_heads, int64_t window, int64_t first, int64_t* bytes) {
  if (bytes == nullptr) return C128_ERR_NULL_PTR;
  if (num_heads < 1 || num_heads > c128::kMaxDecodeHeads) return C128_ERR_UNSUPPORTED;
  if (window < 1 || window > kMaxCount || first < 0 || first > kMaxCount) return C128_ERR_ARG;
  *bytes = 0;
  if (c128::window_fits(window, first)) return C128_OK;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return C128_ERR_CUDA;
  *bytes = c128::runs_workspace_bytes(static_cast<int>(num_heads), sms);
  return C128_OK;
}

int c128_debug_stall_window_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                                      const c128_tensor_t* block_table, const c128_tensor_t* token_to_req_indices,
                                      const c128_tensor_t* positions, const c128_tensor_t* slot_mapping, int64_t window,
                                      int64_t first, float scale, const c128_tensor_t* sink, const c128_tensor_t* out,
                                      const c128_tensor_t* lse, const c128_tensor_t* workspace, c128_stream_t stream) {
  return window_attention(q, k_cache, kv_block_size, block_table, token_to_req_indices, positions, slot_mapping, window, first,
                          scale, sink, out, lse, workspace, stream, true);
}

}  // extern "C"
