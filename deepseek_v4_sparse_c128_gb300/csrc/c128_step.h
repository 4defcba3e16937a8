// Parameters and launchers of the operators around the attention of recent tokens (c128_step_api.cu checks
// the arguments; c128_rotary.cu, c128_norm.cu and c128_window.cu hold the kernels).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "c128_internal.h"
#include "c128_serving.h"

namespace c128 {

constexpr int kMaxTurned = 512;  // columns that a table of rotations may have

struct CosSinParams {
  float* table;
  int64_t stride, rows;
  uint64_t first;
  int32_t half;                      // angles per position
  float magnitude;
  uint64_t step[kMaxTurned / 2];     // of each pair, in 2^-64 turns
};
cudaError_t launch_cos_sin(const CosSinParams& p, int sm_count, cudaStream_t stream);

struct RotateParams {
  const void* x;
  int64_t x_stride_t, x_stride_h;    // elements
  void* out;
  int64_t out_stride_t, out_stride_h;
  int64_t tokens;
  int32_t heads, width, first, half; // half: pairs
  int32_t f32, halves, in_place;
  float sign;                        // of the sines
  const int64_t* positions;
  const float* cos_sin;
  int64_t rows, cs_stride;
  unsigned int* err;
};
cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream);

struct NormParams {
  const int64_t* positions;
  const int64_t* slots;
  int64_t tokens;
  float eps;
  const float* cos_sin;
  int64_t rows, cs_stride;
  const void* q;                     // nullable
  int64_t q_stride_t, q_stride_h;
  int32_t q_f32, heads;
  const float* q_w;                  // nullable
  void* q_out;
  int64_t out_stride_t, out_stride_h;
  int32_t out_f32;
  const void* k;                     // nullable
  int64_t k_stride;
  int32_t k_f32;
  const float* k_w;                  // nullable
  uint8_t* kc;
  int64_t nkb, kv_bs, kc_stride0;
  Divisor kv_div;
  unsigned int* err;
};
cudaError_t launch_norm(const NormParams& p, int sm_count, cudaStream_t stream);

// c128_window_attention's parameters are DecodeParams (kv_lens NULL). Windows that fit into shared memory have a kernel of
// their own, which takes no workspace.
bool window_fits(int64_t window, int64_t first);
cudaError_t prepare_window();  // function attributes, once per device
cudaError_t launch_window(const DecodeParams& p, int sm_count, cudaStream_t stream);

}  // namespace c128
