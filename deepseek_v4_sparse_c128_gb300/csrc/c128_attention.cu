// c128_decode_attention: attention of one new token per request over its entries of the paged FP8
// cache. First form: one CTA per request and 8 heads, a warp per head, the entries decoded to fp32
// in shared memory 16 at a time, one online-softmax step per entry.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "c128_device.cuh"
#include "c128_serving.h"

namespace c128 {
namespace {

constexpr int kDecThreads = 256;
constexpr int kDecHeads = kDecThreads / 32;
constexpr int kDecTile = 16;

__device__ __forceinline__ float e4m3_value(uint32_t b) {
  const uint32_t mag = b & 0x7fu;
  float v = mag == 0x7fu ? NAN : __uint_as_float(mag << 20) * 0x1p120f;
  return b & 0x80u ? -v : v;
}

__global__ void __launch_bounds__(kDecThreads) decode_simple_kernel(const DecodeParams p) {
  __shared__ float s_k[kDecTile][kHead];
  __shared__ int s_ok[kDecTile];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r = blockIdx.x;
  const int h = static_cast<int>(blockIdx.y) * kDecHeads + warp;
  unsigned int err = 0;
  int64_t n = p.kv_lens[r];
  if (n < 0) {
    err |= C128_DEV_BAD_LENGTH;
    n = 0;
  }
  if (n > p.columns * p.kv_bs) {
    err |= C128_DEV_BAD_BT_COL;
    n = p.columns * p.kv_bs;
  }
  float q[16], acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t b = h < p.heads ? p.q[r * p.q_stride_r + h * p.q_stride_h + lane + 32 * i] : 0u;
    q[i] = __uint_as_float(b << 16);
    acc[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int64_t j0 = 0; j0 < n; j0 += kDecTile) {
    __syncthreads();
    for (int e = threadIdx.x; e < kDecTile * kHead; e += kDecThreads) {
      const int jj = e / kHead, c = e % kHead;
      const int64_t j = j0 + jj;
      float v = 0.f;
      int ok = 0;
      if (j < n) {
        const int id = p.table[r * p.table_stride + j / p.kv_bs];
        if (id < 0 || id >= p.nkb) {
          err |= C128_DEV_BAD_BLOCK;
        } else {
          ok = 1;
          const uint8_t* blk = p.kc + id * p.kc_stride0;
          const int64_t off = j % p.kv_bs;
          const uint8_t* rec = blk + off * kTokenStride;
          if (c < kNope) {
            const int sb = blk[p.kv_bs * kTokenStride + off * kScaleDim + c / kQuantBlock];
            v = ldexpf(e4m3_value(rec[c]), sb - 127);
          } else {
            v = __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(rec + kNope + 2 * (c - kNope))) << 16);
          }
        }
      }
      s_k[jj][c] = v;
      if (c == 0) s_ok[jj] = ok;
    }
    __syncthreads();
    for (int jj = 0; jj < kDecTile; ++jj) {
      if (!s_ok[jj]) continue;
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) s = fmaf(q[i], s_k[jj][lane + 32 * i], s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= p.scale;
      const float m2 = fmaxf(m, s), f = m2 == -INFINITY ? 1.f : expf(m - m2), w = expf(s - (m2 == -INFINITY ? 0.f : m2));
      m = m2;
      l = l * f + w;
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] = acc[i] * f + w * s_k[jj][lane + 32 * i];
    }
  }
  if (err) atomicOr(p.err, err);
  if (h >= p.heads) return;
  if (p.sink != nullptr) {
    const float s = p.sink[h], m2 = fmaxf(m, s), f = m2 == -INFINITY ? 1.f : expf(m - m2);
    l = l * f + expf(s - (m2 == -INFINITY ? 0.f : m2));
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] *= f;
    m = m2;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t at = r * p.out_stride_r + h * p.out_stride_h + lane + 32 * i;
    if (p.out_f32) static_cast<float*>(p.out)[at] = acc[i] * inv;
    else static_cast<uint16_t*>(p.out)[at] = static_cast<uint16_t>(pack_bf16x2(acc[i] * inv, 0.f));
  }
  if (p.lse != nullptr && lane == 0) p.lse[r * p.lse_stride_r + h * p.lse_stride_h] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

int64_t decode_workspace_bytes(int heads, int sm_count) { return 256; }

cudaError_t launch_decode(const DecodeParams& p, int sm_count, cudaStream_t stream) {
  decode_simple_kernel<<<dim3(static_cast<unsigned>(p.requests), (p.heads + kDecHeads - 1) / kDecHeads), kDecThreads, 0,
                         stream>>>(p);
  return cudaGetLastError();
}

}  // namespace c128
