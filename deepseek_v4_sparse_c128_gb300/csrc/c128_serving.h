// Parameters and launchers of the operators around the compressor (c128_serving_api.cu checks the
// arguments; c128_tables.cu, c128_attention.cu and c128_merge.cu hold the kernels).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "c128_internal.h"

namespace c128 {

constexpr int kMaxDecodeHeads = 1024;

struct Divisor {
  uint32_t value;
  int32_t shift;  // log2(value), -1 if that is none
  Divisor() = default;
  explicit Divisor(int64_t v) : value(static_cast<uint32_t>(v)), shift(-1) {
    for (int i = 0; i < 32; ++i)
      if (value == 1u << i) shift = i;
  }
};
// x / d, with a shift where d is a power of two (shift >= 0): block sizes and ratios mostly are.
__device__ __forceinline__ uint32_t divide(uint32_t x, const Divisor d) { return d.shift >= 0 ? x >> d.shift : x / d.value; }

struct ExtendParams {
  const int32_t* seq_lens;
  const int32_t* held;
  int32_t* held_out;
  int32_t* table;
  int64_t requests, columns, stride;
  const int32_t* free_blocks;
  int64_t num_free;
  const int64_t* taken;
  int64_t* taken_out;
  Divisor ratio, block;
  unsigned int* err;
};
cudaError_t launch_extend(const ExtendParams& p, int sm_count, cudaStream_t stream);

struct SlotMapParams {
  const int32_t* seq_lens;
  const int32_t* query_lens;
  int64_t requests;
  const int32_t* state_table;
  int64_t state_cols, state_stride;
  Divisor state_block;
  const int32_t* kv_table;
  int64_t kv_cols, kv_stride;
  Divisor kv_block, ratio;
  int32_t* query_start;
  int32_t* token_to_req;
  int64_t* positions;
  int64_t* slots;
  int64_t* kv_slots;
  int32_t* kv_lens;
  int64_t tokens;
  unsigned int* err;
};
cudaError_t launch_slot_maps(const SlotMapParams& p, cudaStream_t stream);

struct DecodeParams {
  const uint16_t* q;             // bf16
  int64_t q_stride_r, q_stride_h;
  const uint8_t* kc;
  int64_t nkb, kv_bs, kc_stride0;
  Divisor kv_div;                // kv_bs
  const int32_t* table;
  int64_t requests, table_stride;
  int32_t most;                  // entries that a row of the table holds, at most 2^31 - 1
  const int32_t* kv_lens;        // NULL: c128_window_attention, and `requests` are tokens
  const int32_t* token_req;      // its arrays: the row of each token's request in the table,
  const int64_t* positions;      // its position (the entry that is its own),
  const int64_t* slots;          // and its cache slot (< 0: skipped)
  int64_t table_rows, window;    // a token sees the last `window` entries and the `first` ones
  int32_t first;
  int32_t heads;
  float scale;
  const float* sink;             // nullable
  void* out;
  int64_t out_stride_r, out_stride_h;
  int32_t out_f32;
  float* lse;                    // nullable
  int64_t lse_stride_r, lse_stride_h;
  uint8_t* workspace;
  int32_t stall;                 // test only: CTA 0 never learns of its tiles, and its waits run out
  unsigned int* err;
};
cudaError_t launch_decode(const DecodeParams& p, int64_t workspace_bytes, int sm_count, cudaStream_t stream);
cudaError_t prepare_decode();  // function attributes, once per device
int64_t decode_workspace_bytes(int heads, int sm_count);
int64_t runs_workspace_bytes(int heads, int sm_count);  // where tokens that follow one another may be taken together

struct MergeParams {
  const void* part;
  int64_t part_stride_p, part_stride_r, part_stride_h;
  int32_t part_f32;
  const float* part_lse;
  int64_t lse_in_p, lse_in_r, lse_in_h;
  int64_t parts, requests, heads;
  void* out;
  int64_t out_stride_r, out_stride_h;
  int32_t out_f32;
  float* lse;                    // nullable
  int64_t lse_stride_r, lse_stride_h;
};
cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream);

}  // namespace c128
