// c128_merge_attention: partial attentions joined by their log-sum-exp. With top = max_p lse_p and
// w_p = exp(lse_p - top): out = sum_p w_p o_p / sum_p w_p, lse = top + log(sum_p w_p).
//
// A pass over memory and nothing else: 1 KB per part and row read, 1 KB written. One warp per row of
// 512 values, 16 per lane in two 16-byte pieces (bf16), so that each load of a warp covers 512
// consecutive bytes and the loads of four parts are in flight before the first is used.
//
// Measured in a graph: 256 requests x 128 heads, 4 bf16 parts (168 MB) 25.6 us, 6.56 TB/s, 0.97 of the measured copy; one
// request, 64 heads, 2 parts 1.8 us, which is a launch. (Weights first and values behind them 34.2 us;
// CTAs of 256 threads, whose rows end together, 28.2, of 512 38.9, of 32 33.4; streaming loads 26.7.)
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "c128_serving.h"

namespace c128 {
namespace {

constexpr int kMergeThreads = 64;

// 16 bytes past L1, and never ahead of the wait for the kernels before this one, which may be writing them. (__ldcg does
// not say that it keeps that order.)
__device__ __forceinline__ uint4 ld16(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}

// Values [c, c + 8) of a row.
template <bool F32>
struct Piece;
template <>
struct Piece<true> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* row, int c) {
    a = ld16(static_cast<const float*>(row) + c);
    b = ld16(static_cast<const float*>(row) + c + 4);
  }
  __device__ __forceinline__ void add(float w, float (&acc)[8]) const {
    const uint32_t v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, __uint_as_float(v[i]), acc[i]);
  }
};
template <>
struct Piece<false> {
  uint4 a;
  __device__ __forceinline__ void load(const void* row, int c) {
    a = ld16(static_cast<const uint16_t*>(row) + c);
  }
  __device__ __forceinline__ void add(float w, float (&acc)[8]) const {
    const uint32_t v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[2 * i] = fmaf(w, __uint_as_float(v[i] << 16), acc[2 * i]);
      acc[2 * i + 1] = fmaf(w, __uint_as_float(v[i] & 0xffff0000u), acc[2 * i + 1]);
    }
  }
};
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

template <bool PART_F32, bool OUT_F32>
__global__ void __launch_bounds__(kMergeThreads) merge_kernel(const MergeParams p) {
  const int lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.launch_dependents;" :::);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kMergeThreads / 32) + (threadIdx.x >> 5);
  if (row >= p.requests * p.heads) return;
  const int64_t r = row / p.heads, h = row % p.heads;
  constexpr int kPartBytes = PART_F32 ? 4 : 2;
  const float* lse_in = p.part_lse + r * p.lse_in_r + h * p.lse_in_h;
  const char* part = static_cast<const char*>(p.part) + (r * p.part_stride_r + h * p.part_stride_h) * kPartBytes;

  constexpr int kFlight = 4;
  Piece<PART_F32> v[kFlight][2];
  auto load = [&](int64_t i0) {
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (i0 + k < p.parts) {
        const char* src = part + (i0 + k) * p.part_stride_p * kPartBytes;
        v[k][0].load(src, 8 * lane);
        v[k][1].load(src, 256 + 8 * lane);
      }
    }
  };
  load(0);  // on its way while the weights are made, a part's by each lane
  float top = -INFINITY;
  bool nan = false;
  for (int64_t i = lane; i < p.parts; i += 32) {
    const float l = lse_in[i * p.lse_in_p];
    top = fmaxf(top, l);
    nan |= l != l;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (__any_sync(0xffffffffu, nan)) top = NAN;
  const float shift = top == -INFINITY ? 0.f : top;
  float acc[2][8] = {};
  float sum = 0.f, own = 0.f;
  for (int64_t i0 = 0; i0 < p.parts; i0 += kFlight) {
    if (i0 % 32 == 0) own = i0 + lane < p.parts ? expf(lse_in[(i0 + lane) * p.lse_in_p] - shift) : 0.f;
    if (i0 > 0) load(i0);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const float w = __shfl_sync(0xffffffffu, own, static_cast<int>(i0 % 32) + k);
      if (w != 0.f) {  // a part without weight may hold anything (and one behind the last has none)
        sum += w;
        v[k][0].add(w, acc[0]);
        v[k][1].add(w, acc[1]);
      }
    }
  }
  __syncwarp();  // out and lse may be one of the parts: every lane has read them by here
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    float* a = acc[g];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] *= inv;
    const int64_t at = r * p.out_stride_r + h * p.out_stride_h + 256 * g + 8 * lane;
    if (OUT_F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.out) + at);
      o[0] = make_float4(a[0], a[1], a[2], a[3]);
      o[1] = make_float4(a[4], a[5], a[6], a[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + at) =
          make_uint4(pack2(a[0], a[1]), pack2(a[2], a[3]), pack2(a[4], a[5]), pack2(a[6], a[7]));
    }
  }
  if (p.lse != nullptr && lane == 0) p.lse[r * p.lse_stride_r + h * p.lse_stride_h] = sum == 0.f ? -INFINITY : top + logf(sum);
}

}  // namespace

cudaError_t launch_merge(const MergeParams& p, cudaStream_t stream) {
  constexpr int kRows = kMergeThreads / 32;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>((p.requests * p.heads + kRows - 1) / kRows));
  lc.blockDim = dim3(kMergeThreads);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  if (p.part_f32) return p.out_f32 ? cudaLaunchKernelEx(&lc, merge_kernel<true, true>, p) : cudaLaunchKernelEx(&lc, merge_kernel<true, false>, p);
  return p.out_f32 ? cudaLaunchKernelEx(&lc, merge_kernel<false, true>, p) : cudaLaunchKernelEx(&lc, merge_kernel<false, false>, p);
}

}  // namespace c128
