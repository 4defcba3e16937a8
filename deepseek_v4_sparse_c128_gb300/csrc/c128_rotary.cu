// c128_build_cos_sin and c128_rotate: positions as rotations.
#include <cuda_runtime.h>

#include <cstdint>

#include "c128_device.cuh"
#include "c128_step.h"

namespace c128 {
namespace {

// ------------------------------------------------------------------------------------------ table
// cos and sin of position * step. A step is kept in 2^-64 turns, so the low 64 bits of the product are the
// angle with its whole turns gone, exactly. The nearest quarter turn is taken off it (the two highest bits,
// rounded), and what is left, under an eighth of a turn either way, becomes a float: sines near zero keep their
// relative precision. With |x| <= pi / 4 the Taylor series of both, to x^10 and x^11, are 2^-33 of a value off; their
// steps in z = x^2 are the same, so a packed multiply-add takes both.
// Stores bound it where the table is long: a million positions of 32 pairs, 268 MB, 38.9 us, 6.9 TB/s (with the library's
// cosine and sine of each angle, one pair to a thread, 67 us: instructions bound that). 16,384 positions 3.3 us: a launch.
constexpr int kTableThreads = 256;

__device__ __forceinline__ void cos_sin_of(uint64_t turn, float magnitude, float& c, float& s) {
  const uint32_t high = static_cast<uint32_t>(turn >> 32), quarter = (high + (1u << 29)) >> 30;
  const float rest = fmaf(static_cast<float>(static_cast<int32_t>(high - (quarter << 30))), 0x1p32f, static_cast<float>(static_cast<uint32_t>(turn)));
  const float x = rest * (6.283185307179586f * 0x1p-64f), z = x * x, xm = x * magnitude;
  const float2 zz = make_float2(z, z);
  float2 p = make_float2(-1.f / 3628800.f, -1.f / 39916800.f);
  p = __ffma2_rn(p, zz, make_float2(1.f / 40320.f, 1.f / 362880.f));
  p = __ffma2_rn(p, zz, make_float2(-1.f / 720.f, -1.f / 5040.f));
  p = __ffma2_rn(p, zz, make_float2(1.f / 24.f, 1.f / 120.f));
  p = __ffma2_rn(p, zz, make_float2(-1.f / 2.f, -1.f / 6.f));
  p = __fmul2_rn(p, zz);
  const float a = fmaf(p.x, magnitude, magnitude), b = fmaf(p.y, xm, xm);
  const bool swap = quarter & 1;
  c = __uint_as_float(__float_as_uint(swap ? b : a) ^ ((quarter + 1) & 2) << 30);
  s = __uint_as_float(__float_as_uint(swap ? a : b) ^ (quarter & 2) << 30);
}

// A thread keeps its N pairs and goes from row to row, the angles by addition. No kernel behind this one starts early: the
// compressor's read tables as read-only data, which nobody may write while they are resident.
template <int N>
__global__ void __launch_bounds__(kTableThreads) cos_sin_kernel(const __grid_constant__ CosSinParams p) {
  __shared__ uint64_t steps[kMaxTurned / 2];  // (parameters are slow to read by an index of the thread's own)
  for (int i = threadIdx.x; i < p.half; i += kTableThreads) steps[i] = p.step[i];
  __syncthreads();
  const unsigned threads = p.half / N, at_once = kTableThreads / threads, below = threadIdx.x / threads;
  const unsigned pair = (threadIdx.x - below * threads) * N;
  if (below >= at_once) return;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * at_once;
  int64_t row = static_cast<int64_t>(blockIdx.x) * at_once + below;
  uint64_t turn[N], add[N];
#pragma unroll
  for (int k = 0; k < N; ++k) turn[k] = (p.first + row) * steps[pair + k], add[k] = stride * steps[pair + k];
  float* dst = p.table + row * p.stride + pair;
  const int64_t next = stride * p.stride;
  grid_dependency_wait();  // the table may still be read by kernels before this one
  for (; row < p.rows; row += stride, dst += next) {
    float c[N], s[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      cos_sin_of(turn[k], p.magnitude, c[k], s[k]);
      turn[k] += add[k];
    }
    if constexpr (N == 4) {
      *reinterpret_cast<float4*>(dst) = make_float4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<float4*>(dst + p.half) = make_float4(s[0], s[1], s[2], s[3]);
    } else {
      dst[0] = c[0], dst[p.half] = s[0];
    }
  }
}

// --------------------------------------------------------------------------------------- rotation
// A pass over memory, bound by it: 4,096 tokens x 64 heads x 512 columns 79.6 us, 6.75 TB/s, as the measured copy; 4,099 x 40
// x 128 in fp32 28.4 us, 5.9 TB/s; 64 x 64 x 512, a decode step, 3.5 us, about a launch. Work is dealt out in units: a vector of 16 bytes (of halves: one of either half) to
// turn, or one to copy; a CTA takes kUnits of them, of one token or of several whole ones. Without the
// alignment for vectors a unit is a pair, or a value to copy. Two units to a thread of 128: one took the three cases 3.8, 133.6
// and 35.2 us, four 4.6, 81.7 and 32.8, eight 5.9, 112.9 and 49.5.
constexpr int kRotateThreads = 128, kFlight = 2, kUnits = kRotateThreads * kFlight;

template <typename T>
struct Vec {  // 16 bytes of T
  static constexpr int kN = 16 / sizeof(T);
};
// Behind the wait, and never ahead of it: see grid_dependency_wait.
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  asm volatile("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
  return v;
}
template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) f[i] = __uint_as_float(w[i]);
    else f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* f) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const uint16_t* p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }
__device__ __forceinline__ void turn(float& u, float& v, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s)), b = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
  u = a, v = b;
}

// x / d as a product, where that is exact: x < 2^32 / d.
struct Quotient {
  uint32_t value, inverse;  // inverse 0: a division
  Quotient() = default;
  Quotient(int64_t d, int64_t most) : value(static_cast<uint32_t>(d)), inverse(0) {
    // (2^32 / d rounded up is less than 1 too large, so the product is off by less than x / 2^32 < 1 / d)
    if (d > 1 && d * most < 1ll << 32) inverse = static_cast<uint32_t>(((1ull << 32) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t of(uint32_t x) const { return inverse ? __umulhi(x, inverse) : x / value; }
};
struct RotateShape {
  Quotient units, token_units;  // of a row; of a token
  int32_t turned;              // units of a row to turn, the rest are copied
  uint32_t tokens_per_cta;     // with 1 of them, `pieces` CTAs to a token
  uint32_t pieces;
};

// T: float or uint16_t (the bits of a bf16)
template <typename T, bool HALVES, bool VECTOR>
__global__ void __launch_bounds__(kRotateThreads) rotate_kernel(const RotateParams p, const RotateShape shape) {
  launch_dependents();
  const uint32_t group = blockIdx.x / shape.pieces, piece = blockIdx.x - group * shape.pieces;
  const int64_t token0 = static_cast<int64_t>(group) * shape.tokens_per_cta;
  const uint32_t tokens = static_cast<uint32_t>(p.tokens - token0 < shape.tokens_per_cta ? p.tokens - token0 : shape.tokens_per_cta);
  const uint32_t begin = piece * kUnits, end = min(tokens * shape.token_units.value, begin + kUnits);
  grid_dependency_wait();
  constexpr int N = VECTOR ? Vec<T>::kN : 1;
  constexpr int kTwo = HALVES && VECTOR ? 2 : 1;  // vectors of a unit to turn
  const T* src[kFlight];
  T* dst[kFlight];
  int64_t pos[kFlight];
  int pairs[kFlight];  // the first to turn; -1: to copy
  bool first[kFlight];
  uint4 v[kFlight][kTwo];
  const int apart = HALVES ? p.half : 1;  // columns between the two of a pair
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    const uint32_t at = begin + k * kRotateThreads + threadIdx.x;
    src[k] = nullptr;
    if (at >= end) continue;
    const uint32_t t = shape.tokens_per_cta == 1 ? 0 : shape.token_units.of(at), in_token = at - t * shape.token_units.value;
    const uint32_t h = shape.units.of(in_token), unit = in_token - h * shape.units.value;
    const int64_t token = token0 + t;
    pos[k] = p.positions[token];
    const bool turned = unit < static_cast<uint32_t>(shape.turned);
    int column, pair = 0;
    if (turned) {
      pair = HALVES ? unit * N : VECTOR ? unit * (N / 2) : unit;
      column = p.first + (HALVES ? pair : 2 * pair);
    } else {
      column = (unit - shape.turned) * N;
      if (column >= p.first) column += 2 * p.half;
    }
    src[k] = static_cast<const T*>(p.x) + token * p.x_stride_t + h * p.x_stride_h + column;
    dst[k] = static_cast<T*>(p.out) + token * p.out_stride_t + h * p.out_stride_h + column;
    pairs[k] = turned ? pair : -1;
    first[k] = in_token == 0;
    if constexpr (VECTOR) {
      v[k][0] = load16(src[k]);
      if constexpr (HALVES)
        if (turned) v[k][1] = load16(src[k] + apart);
    }
  }
#pragma unroll
  for (int k = 0; k < kFlight; ++k) {
    if (src[k] == nullptr || pos[k] < 0) continue;  // (a skipped token's values have been read, and are not used)
    if (pos[k] >= p.rows) {
      if (first[k]) atomicOr(p.err, static_cast<unsigned int>(C128_DEV_BAD_COS_ROW));
      continue;
    }
    const float* c = pairs[k] < 0 ? nullptr : p.cos_sin + pos[k] * p.cs_stride + pairs[k];
    if constexpr (!VECTOR) {
      float a = value(src[k]);
      if (c != nullptr) {
        float b = value(src[k] + apart);
        turn(a, b, __ldcg(c), p.sign * __ldcg(c + p.half));
        put(dst[k] + apart, b);
      }
      put(dst[k], a);
    } else if (c == nullptr) {
      *reinterpret_cast<uint4*>(dst[k]) = v[k][0];
    } else if constexpr (HALVES) {
      float a[N], b[N];
      unpack<T>(v[k][0], a);
      unpack<T>(v[k][1], b);
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const float4 cc = __ldcg(reinterpret_cast<const float4*>(c + i)), ss = __ldcg(reinterpret_cast<const float4*>(c + p.half + i));
        turn(a[i], b[i], cc.x, p.sign * ss.x), turn(a[i + 1], b[i + 1], cc.y, p.sign * ss.y);
        turn(a[i + 2], b[i + 2], cc.z, p.sign * ss.z), turn(a[i + 3], b[i + 3], cc.w, p.sign * ss.w);
      }
      *reinterpret_cast<uint4*>(dst[k]) = pack<T>(a);
      *reinterpret_cast<uint4*>(dst[k] + apart) = pack<T>(b);
    } else {
      float a[N];
      unpack<T>(v[k][0], a);
#pragma unroll
      for (int i = 0; i < N / 2; i += 2) {
        const float2 cc = __ldcg(reinterpret_cast<const float2*>(c + i)), ss = __ldcg(reinterpret_cast<const float2*>(c + p.half + i));
        turn(a[2 * i], a[2 * i + 1], cc.x, p.sign * ss.x), turn(a[2 * i + 2], a[2 * i + 3], cc.y, p.sign * ss.y);
      }
      *reinterpret_cast<uint4*>(dst[k]) = pack<T>(a);
    }
  }
}

template <typename T>
const void* rotate_kernel_for(bool halves, bool vector) {
  if (halves) return vector ? reinterpret_cast<const void*>(rotate_kernel<T, true, true>) : reinterpret_cast<const void*>(rotate_kernel<T, true, false>);
  return vector ? reinterpret_cast<const void*>(rotate_kernel<T, false, true>) : reinterpret_cast<const void*>(rotate_kernel<T, false, false>);
}

cudaError_t launch_pdl(const void* kernel, int64_t ctas, int threads, void** args, cudaStream_t stream) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(ctas));
  lc.blockDim = dim3(threads);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelExC(&lc, kernel, args);
}

}  // namespace

cudaError_t launch_cos_sin(const CosSinParams& p, int sm_count, cudaStream_t stream) {
  if (p.rows == 0) return cudaSuccess;
  // four pairs to a thread, and stores of 16 bytes, where rows and their halves allow it
  const bool four = p.half % 4 == 0 && p.stride % 4 == 0 && reinterpret_cast<uintptr_t>(p.table) % 16 == 0;
  const int64_t at_once = kTableThreads / (p.half / (four ? 4 : 1)), need = (p.rows + at_once - 1) / at_once, most = 8ll * sm_count;
  void* args[] = {const_cast<CosSinParams*>(&p)};
  return launch_pdl(four ? reinterpret_cast<const void*>(cos_sin_kernel<4>) : reinterpret_cast<const void*>(cos_sin_kernel<1>),
                    need < most ? need : most, kTableThreads, args, stream);
}

cudaError_t launch_rotate(const RotateParams& p, cudaStream_t stream) {
  if (p.tokens == 0 || p.heads == 0) return cudaSuccess;
  const int item = p.f32 ? 4 : 2, n = 16 / item;
  auto whole = [&](int64_t v) { return v % n == 0; };
  auto on16 = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  // The table's loads are of four values (halves) or two; a vector's first pair is a multiple of that.
  const int table = p.halves ? 4 : 2;
  const bool vector = on16(p.x) && on16(p.out) && whole(p.x_stride_t) && whole(p.x_stride_h) && whole(p.out_stride_t) &&
                      whole(p.out_stride_h) && whole(p.first) && whole(p.width) && whole(p.halves ? p.half : 2 * p.half) &&
                      p.half % table == 0 && p.cs_stride % table == 0 && on16(p.cos_sin);
  RotateShape shape;
  const int copied = p.in_place ? 0 : p.width - 2 * p.half;
  shape.turned = !vector ? p.half : p.halves ? p.half / n : 2 * p.half / n;
  const int64_t units = shape.turned + (vector ? copied / n : copied), token_units = units * p.heads;
  shape.tokens_per_cta = token_units >= kUnits ? 1 : static_cast<uint32_t>(kUnits / token_units);
  shape.units = Quotient(units, token_units);
  shape.token_units = Quotient(token_units, token_units * shape.tokens_per_cta);
  shape.pieces = static_cast<uint32_t>((token_units * shape.tokens_per_cta + kUnits - 1) / kUnits);
  const int64_t ctas = (p.tokens + shape.tokens_per_cta - 1) / shape.tokens_per_cta * shape.pieces;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  void* args[] = {const_cast<RotateParams*>(&p), &shape};
  return launch_pdl(p.f32 ? rotate_kernel_for<float>(p.halves, vector) : rotate_kernel_for<uint16_t>(p.halves, vector), ctas,
                    kRotateThreads, args, stream);
}

}  // namespace c128
