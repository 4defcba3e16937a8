// c128_norm_rope_store: queries and keys normalised and turned by their position, keys into the paged cache.
//
//   n = x * rrms * w,  rrms = 1 / sqrt(mean(x^2) + eps);  the last 64 columns: (e, o) -> (e c - o s, o c + e s)
//
// One pass: a warp takes a row of 512 values, 16 per lane in two pieces of 8 (columns 8l .. and 256 + 8l ..),
// keeps it in registers between the sum and the result, and has ROWS heads of one token on their way at
// once, for which it reads the token's position and angles once. Lanes 24 .. 31 hold the turned columns in
// their second piece, four pairs each. A key's groups of 64 columns are eight lanes of a piece.
//
// A query is 1 KB read and 1 KB written (bf16) for some 180 instructions of a warp, so DRAM bounds it: 7,777 tokens of 64
// heads and a key 163 us, 6.33 TB/s, 0.94 of the measured copy; 200 tokens of 128 heads and a key 11.9 us, 4.4 TB/s (the
// launch and one chain position - angles - result stand before and behind 8 us of bytes); one token of 64 heads 3.6 us, a
// launch and that chain. With 4 heads to a warp instead of 8 the 7,777 tokens took 178 us: too few loads on their way.
#include <cuda_runtime.h>

#include <cstdint>

#include "c128_step.h"
#include "c128_warp_epilogue.cuh"

namespace c128 {
namespace {

constexpr int kNormThreads = 64;

// Not ahead of the wait: see grid_dependency_wait.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
template <bool F32>
struct Row {  // a lane's 16 values, as they are in memory
  uint4 v[F32 ? 4 : 2];
  __device__ __forceinline__ void load(const void* row, int lane) {
    if constexpr (F32) {
      const float* p = static_cast<const float*>(row) + 8 * lane;
      v[0] = load16(p), v[1] = load16(p + 4), v[2] = load16(p + 256), v[3] = load16(p + 260);
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(row) + 8 * lane;
      v[0] = load16(p), v[1] = load16(p + 256);
    }
  }
  __device__ __forceinline__ void values(float (&x)[16]) const {
#pragma unroll
    for (int i = 0; i < (F32 ? 4 : 2); ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (F32) x[4 * i + k] = __uint_as_float(w[k]);
        else x[8 * i + 2 * k] = __uint_as_float(w[k] << 16), x[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    }
  }
};
__device__ __forceinline__ void load_weight(const float* w, int lane, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = w == nullptr ? make_float4(1.f, 1.f, 1.f, 1.f)
                                  : *reinterpret_cast<const float4*>(w + 8 * lane + 4 * (i & 1) + 256 * (i >> 1));
    x[4 * i] = f.x, x[4 * i + 1] = f.y, x[4 * i + 2] = f.z, x[4 * i + 3] = f.w;
  }
}
// The angles of the four pairs x[8 ..] of lanes 24 .. 31 (of the other lanes: any).
struct Angles {
  float c[4], s[4];
  __device__ __forceinline__ Angles(float cos_of_lane, float sin_of_lane, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int pair = (4 * (lane - 24) + i) & 31;
      c[i] = __shfl_sync(0xffffffffu, cos_of_lane, pair), s[i] = __shfl_sync(0xffffffffu, sin_of_lane, pair);
    }
  }
  __device__ __forceinline__ void turn(float (&x)[16], int lane) const {
    if (lane < 24) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = x[8 + 2 * i], o = x[9 + 2 * i];
      x[8 + 2 * i] = __fsub_rn(__fmul_rn(e, c[i]), __fmul_rn(o, s[i]));
      x[9 + 2 * i] = __fadd_rn(__fmul_rn(o, c[i]), __fmul_rn(e, s[i]));
    }
  }
};

// A token's angles, of pair `lane`; false where it is skipped (and said why, by the warp with `report`).
__device__ __forceinline__ bool token_angles(const NormParams& p, int64_t t, bool report, int lane, float& c, float& s) {
  const int64_t slot = p.slots[t], pos = p.positions[t];
  if (slot < 0 || pos < 0) return false;
  unsigned int err = 0;
  if (pos >= p.rows) err |= C128_DEV_BAD_COS_ROW;
  if (p.k != nullptr && slot >= p.nkb * p.kv_bs) err |= C128_DEV_BAD_KV_SLOT;
  if (err) {
    if (report && lane == 0) atomicOr(p.err, err);
    return false;
  }
  const float* row = p.cos_sin + pos * p.cs_stride;
  c = __ldcg(row + lane), s = __ldcg(row + 32 + lane);
  return true;
}

// ---------------------------------------------------------------------------------------- queries
template <bool F32, bool OUT_F32, int ROWS>
__device__ __forceinline__ void queries(const NormParams& p, int64_t t, int head0, bool report, int lane) {
  Row<F32> row[ROWS];
  const char* src = static_cast<const char*>(p.q) + (t * p.q_stride_t + head0 * p.q_stride_h) * (F32 ? 4 : 2);
#pragma unroll
  for (int r = 0; r < ROWS; ++r)
    if (head0 + r < p.heads) row[r].load(src + r * p.q_stride_h * (F32 ? 4 : 2), lane);
  float c, s;
  if (!token_angles(p, t, report, lane, c, s)) return;
  const Angles angles(c, s, lane);
  float w[16];
  if (p.q_w != nullptr) load_weight(p.q_w, lane, w);
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (head0 + r >= p.heads) break;
    float x[16];
    row[r].values(x);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum = fmaf(x[i], x[i], sum);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float rrms = __frsqrt_rn(fmaf(sum, 1.f / kHead, p.eps));
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x[i] * rrms;
    if (p.q_w != nullptr) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * w[i];
    }
    angles.turn(x, lane);
    const int64_t at = t * p.out_stride_t + (head0 + r) * p.out_stride_h + 8 * lane;
    if constexpr (OUT_F32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.q_out) + at);
      dst[0] = make_float4(x[0], x[1], x[2], x[3]), dst[1] = make_float4(x[4], x[5], x[6], x[7]);
      dst[64] = make_float4(x[8], x[9], x[10], x[11]), dst[65] = make_float4(x[12], x[13], x[14], x[15]);
    } else {
      uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + at);
      dst[0] = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
      dst[32] = make_uint4(pack_bf16x2(x[8], x[9]), pack_bf16x2(x[10], x[11]), pack_bf16x2(x[12], x[13]), pack_bf16x2(x[14], x[15]));
    }
  }
}

// ------------------------------------------------------------------------------------------- keys
// 2^e of a group of 64 columns (the lane's 8 and those of the seven lanes beside it), as the compressor has
// it: e = ceil(log2(RN(absmax * RN(1/448)))), absmax of the values rounded to bf16.
__device__ __forceinline__ int group_exponent(const uint32_t (&b)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, max(b[i] << 16 & 0x7fffffffu, b[i] & 0x7fff0000u));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  const float most = fmaxf(__uint_as_float(top), __uint_as_float(kAbsmaxFloorBits));
  const uint32_t raw = __float_as_uint(__fmul_rn(most, __uint_as_float(kInv448Bits)));
  return static_cast<int>(raw >> 23) - 127 + ((raw & 0x7fffffu) ? 1 : 0);
}
__device__ __forceinline__ uint2 group_codes(const uint32_t (&b)[4], int e) {
  const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  uint32_t two[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = __fmul_rn(__uint_as_float(b[i] << 16), inv), y = __fmul_rn(__uint_as_float(b[i] & 0xffff0000u), inv);
    two[i] = pack_e4m3x2(x, y);  // saturates, and keeps NaN
  }
  return make_uint2(two[0] | two[1] << 16, two[2] | two[3] << 16);
}

template <bool F32>
__device__ __forceinline__ void key(const NormParams& p, int64_t t, int lane, float* scratch) {
  Row<F32> row;
  row.load(static_cast<const char*>(p.k) + t * p.k_stride * (F32 ? 4 : 2), lane);
  float c, s;
  if (!token_angles(p, t, true, lane, c, s)) return;
  float x[16], w[16];
  row.values(x);
  load_weight(p.k_w, lane, w);
  // RN(exact(sum x^2) / 512), as the compressor has it: squares as 128-bit integers, aligned to the largest
  uint32_t most = 0, special = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
    most = max(most, biased_exp(u));
    special |= special_bits(u);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  special = __reduce_or_sync(0xffffffffu, special);
  unsigned long long lo = 0, hi = 0;
  bool wide = false;  // values too far apart for that
  if (special == 0) {
#pragma unroll
    for (int i = 0; i < 16; ++i) add_square(__float_as_uint(x[i]) & 0x7fffffffu, most, lo, hi, wide);
  }
  warp_sum128(lo, hi);
  wide = __any_sync(0xffffffffu, wide);
  if (wide) {
#pragma unroll
    for (int i = 0; i < 16; ++i) scratch[8 * lane + (i & 7) + 256 * (i >> 3)] = x[i];
    __syncwarp();
  }
  float rrms = 0.f;
  if (lane == 0) {
    const float var = special & 2u ? __int_as_float(0x7fc00000) : special & 1u ? INFINITY
                      : wide ? mean_square_exact_slow(scratch, kHead, 9)
                             : round_u128_to_f32(lo, hi, 2 * static_cast<int>(most) - 373, false);
    rrms = __frsqrt_rn(__fadd_rn(var, p.eps));
  }
  __syncwarp();
  rrms = __shfl_sync(0xffffffffu, rrms, 0);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = p.k_w != nullptr ? __fmul_rn(__fmul_rn(x[i], rrms), w[i]) : __fmul_rn(x[i], rrms);
  Angles(c, s, lane).turn(x, lane);
  uint32_t a[4], b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) a[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]), b[i] = pack_bf16x2(x[8 + 2 * i], x[9 + 2 * i]);
  const int ea = group_exponent(a), eb = group_exponent(b);  // (the last of eb's is of turned columns, and not used)
  const int64_t slot = p.slots[t], block = p.kv_div.shift >= 0 ? slot >> p.kv_div.shift : slot / p.kv_bs, at = slot - block * p.kv_bs;
  uint8_t* blk = p.kc + block * p.kc_stride0;
  uint8_t* rec = blk + at * kTokenStride;
  *reinterpret_cast<uint2*>(rec + 8 * lane) = group_codes(a, ea);
  if (lane < 24) {
    *reinterpret_cast<uint2*>(rec + 256 + 8 * lane) = group_codes(b, eb);
  } else {
    uint2* dst = reinterpret_cast<uint2*>(rec + kNope + 16 * (lane - 24));  // (records start on 8 bytes)
    dst[0] = make_uint2(b[0], b[1]), dst[1] = make_uint2(b[2], b[3]);
  }
  const uint32_t ba = min(max(ea + 127, 0), 255), bb = lane < 24 ? min(max(eb + 127, 0), 255) : 0;
  uint32_t low = 0, high = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    low |= __shfl_sync(0xffffffffu, ba, 8 * i) << (8 * i);
    high |= __shfl_sync(0xffffffffu, bb, 8 * i) << (8 * i);
  }
  if (lane == 0) *reinterpret_cast<uint2*>(blk + p.kv_bs * kTokenStride + at * kScaleDim) = make_uint2(low, high);
}

template <bool F32, bool OUT_F32, int ROWS>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(const NormParams p, const uint32_t pieces, const int64_t key_warps) {
  __shared__ float scratch[kNormThreads / 32][kHead];
  launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kNormThreads / 32) + (threadIdx.x >> 5);
  grid_dependency_wait();
  if (warp < key_warps) {  // the keys first: one takes longer than a query
    if (warp >= p.tokens) return;
    if (p.k_f32) key<true>(p, warp, lane, scratch[threadIdx.x >> 5]);
    else key<false>(p, warp, lane, scratch[threadIdx.x >> 5]);
    return;
  }
  if (p.q == nullptr) return;
  const uint32_t item = static_cast<uint32_t>(warp - key_warps);
  const uint32_t t = item / pieces, piece = item - t * pieces;
  if (t >= p.tokens) return;
  queries<F32, OUT_F32, ROWS>(p, t, piece * ROWS, p.k == nullptr && piece == 0, lane);
}

template <int ROWS>
const void* norm_kernel_for(bool f32, bool out_f32) {
  if (f32) return out_f32 ? reinterpret_cast<const void*>(norm_kernel<true, true, ROWS>) : reinterpret_cast<const void*>(norm_kernel<true, false, ROWS>);
  return out_f32 ? reinterpret_cast<const void*>(norm_kernel<false, true, ROWS>) : reinterpret_cast<const void*>(norm_kernel<false, false, ROWS>);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, int sm_count, cudaStream_t stream) {
  if (p.tokens == 0) return cudaSuccess;
  constexpr int kWarps = kNormThreads / 32;
  const int64_t rows = p.q != nullptr ? p.tokens * p.heads : 0;
  // Heads of a token to a warp: 1 while every row has a warp to itself (one token of 64 heads, 64 warps); 8 where there are rows for several waves of CTAs (64
  // heads: 4,096 tokens 94.4 us with 4, 88.9 with 8; 1,024 tokens 25.2 and 25.0; 512 tokens 13.7 and 14.5)
  const int per = rows <= 32ll * sm_count ? 1 : rows < 400ll * sm_count ? 4 : 8;
  uint32_t pieces = static_cast<uint32_t>(p.q != nullptr ? (p.heads + per - 1) / per : 0);
  int64_t key_warps = p.k != nullptr ? p.tokens : 0;
  const int64_t ctas = (key_warps + p.tokens * pieces + kWarps - 1) / kWarps;
  if (ctas == 0) return cudaSuccess;
  if (pieces == 0) pieces = 1;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(ctas));
  lc.blockDim = dim3(kNormThreads);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  void* args[] = {const_cast<NormParams*>(&p), &pieces, &key_warps};
  const void* kernel = per == 1 ? norm_kernel_for<1>(p.q_f32, p.out_f32) : per == 4 ? norm_kernel_for<4>(p.q_f32, p.out_f32) : norm_kernel_for<8>(p.q_f32, p.out_f32);
  return cudaLaunchKernelExC(&lc, kernel, args);
}

}  // namespace c128
