// Block tables and per-token arrays from request lengths: c128_extend_block_tables and
// c128_build_slot_maps. Both are prefix sums over the requests followed by one pass over the blocks
// (or tokens) that finds each one's request in the sums.
//
// Decode steps make a few kilobytes of either, so what counts there is the number of dependent trips
// to memory: one launch, in which every CTA sums the requests for itself (2048 per round, a few KB
// that all CTAs read from L2) instead of a scan kernel and a second one behind it, then looks its
// own blocks or tokens up in shared memory. Nothing is accumulated across CTAs: no atomics but the
// error bits, and no scratch.
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "c128_serving.h"

namespace c128 {
namespace {

constexpr int kChunk = 2048;  // requests per round of the prefix sum

// Exclusive prefix sum of one value per thread over the CTA, and the total. `warp_sums` holds one
// value per warp and may be used again after the next __syncthreads.
template <int THREADS>
__device__ __forceinline__ int64_t block_exclusive_sum(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    const int64_t s = warp_sums[w];
    if (w < warp) before += s;
    all += s;
  }
  *total = all;
  return before + incl - v;
}

// The last index in [0, n) whose start is <= x (starts ascend, starts[0] <= x).
__device__ __forceinline__ int last_at_or_before(const int* starts, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (starts[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// N values v[r .. r + N - 1] of a vector of n, zero behind its end; 16-byte loads where they fit.
template <int N>
__device__ __forceinline__ void load_run(const int32_t* v, int64_t r, int64_t n, int (&out)[N]) {
  if (r + N <= n && (reinterpret_cast<uintptr_t>(v) & 15) == 0) {
#pragma unroll
    for (int k = 0; k < N; k += 4) {
      const int4 x = *reinterpret_cast<const int4*>(v + r + k);
      out[k] = x.x, out[k + 1] = x.y, out[k + 2] = x.z, out[k + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = r + k < n ? v[r + k] : 0;
  }
}

// ------------------------------------------------------------------------------- block tables
constexpr int kExtendThreads = 512;
constexpr int kPerThread = kChunk / kExtendThreads;  // requests of a round, blocks of a tile
constexpr int kExtendTile = kExtendThreads * kPerThread;

// Every CTA sums all requests; the given blocks are dealt out in tiles of kExtendTile. With
// `write_counts` the CTAs also write held_out (a round each) and CTA 0 taken_out, which must then not
// be `held` and `taken` themselves unless the grid is one CTA.
__global__ void __launch_bounds__(kExtendThreads) extend_kernel(const ExtendParams p, bool write_table, bool write_counts) {
  __shared__ int s_start[kChunk];  // first block of each request of the round, counted from the round's first
  __shared__ int s_held[kChunk];
  __shared__ int64_t s_warp[kExtendThreads / 32];
  __shared__ unsigned long long s_fail;

  const int64_t taken = *p.taken;
  unsigned int err = 0;
  const bool bad_taken = taken < 0 || taken > p.num_free;
  if (bad_taken) err |= C128_DEV_BAD_LENGTH;
  const int64_t avail = bad_taken ? 0 : p.num_free - taken;
  int64_t base = 0;  // blocks needed by the requests of earlier rounds
  int64_t given = 0;
  bool failed = false;
  const uint32_t ratio = static_cast<uint32_t>(p.ratio), block = static_cast<uint32_t>(p.block);
  const int64_t rounds = (p.requests + kChunk - 1) / kChunk;

  for (int64_t c = 0; c < rounds; ++c) {
    if (threadIdx.x == 0) s_fail = ULLONG_MAX;
    const int64_t r = c * kChunk + threadIdx.x * kPerThread;
    int len[kPerThread], held[kPerThread], need[kPerThread];
    load_run(p.seq_lens, r, p.requests, len);
    load_run(p.held, r, p.requests, held);
    int64_t sum = 0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      if (len[k] < 0) err |= C128_DEV_BAD_LENGTH;
      const uint32_t entries = static_cast<uint32_t>(max(len[k], 0)) / ratio;
      const uint32_t needed = entries / block + (entries % block != 0);  // <= 2^31 - 1
      need[k] = 0;
      if (held[k] < 0) {
        err |= C128_DEV_BAD_LENGTH;
      } else if (needed > static_cast<uint32_t>(held[k])) {
        if (needed > p.columns) err |= C128_DEV_BAD_BT_COL;
        else need[k] = static_cast<int>(needed) - held[k];
      }
      sum += need[k];
    }
    int64_t total;
    int64_t off = base + block_exclusive_sum<kExtendThreads>(sum, s_warp, &total);  // a barrier, also for s_fail
    int64_t first = off;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      if (need[k] > 0 && first + need[k] > avail) {
        err |= C128_DEV_NO_FREE_BLOCK;
        atomicMin(&s_fail, static_cast<unsigned long long>(first));
        break;
      }
      first += need[k];
    }
    __syncthreads();
    // blocks are given up to the first request that the list cannot serve; none after it
    const int64_t end = s_fail == ULLONG_MAX ? base + total : min(static_cast<int64_t>(s_fail), base + total);
    const int64_t round_given = failed ? 0 : end - base;  // <= num_free < 2^31
    int out[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
      const int i = threadIdx.x * kPerThread + k;
      s_start[i] = static_cast<int>(min(off - base, round_given));
      s_held[i] = held[k];
      out[k] = held[k] + (off - base + need[k] <= round_given ? need[k] : 0);
      off += need[k];
    }
    if (write_counts && c % gridDim.x == blockIdx.x) {
#pragma unroll
      for (int k = 0; k < kPerThread; ++k)
        if (r + k < p.requests) p.held_out[r + k] = out[k];
    }
    __syncthreads();
    if (write_table) {
      const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), p.requests - c * kChunk));
      const int32_t* from = p.free_blocks + taken + base;
      for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * kExtendTile; i0 < round_given;
           i0 += static_cast<int64_t>(gridDim.x) * kExtendTile) {
#pragma unroll
        for (int k = 0; k < kPerThread; ++k) {
          const int64_t i = i0 + k * kExtendThreads + threadIdx.x;
          if (i < round_given) {
            const int id = from[i];
            const int q = last_at_or_before(s_start, n, static_cast<int>(i));
            p.table[(c * kChunk + q) * p.stride + s_held[q] + (static_cast<int>(i) - s_start[q])] = id;
          }
        }
      }
    }
    failed = failed || s_fail != ULLONG_MAX;
    given += round_given;
    base += total;
    __syncthreads();  // s_start, s_held, s_warp and s_fail are written again
  }
  if (write_counts && blockIdx.x == 0 && threadIdx.x == 0) *p.taken_out = taken + given;
  if (write_counts && blockIdx.x == 0 && err) atomicOr(p.err, err);
}

// ----------------------------------------------------------------------------------- slot maps
constexpr int kMapThreads = 256;
constexpr int kMapRequests = kChunk / kMapThreads;  // requests per thread and round
constexpr int kMapTokens = 4;                       // consecutive tokens per thread
constexpr int kMapTile = kMapThreads * kMapTokens;

// Slot of `index` in row r of a block table, -1 with an error bit if the table has none.
__device__ __forceinline__ int64_t slot_of(const int32_t* table, int64_t stride, int64_t cols, uint32_t block, int r,
                                           uint32_t index, unsigned int* err) {
  const uint32_t col = index / block;
  if (col >= cols) {
    *err |= C128_DEV_BAD_BT_COL;
    return -1;
  }
  const int id = table[r * stride + col];
  if (id < 0) {
    *err |= C128_DEV_BAD_BLOCK;
    return -1;
  }
  return static_cast<int64_t>(id) * block + index % block;
}

template <class T, int N>
__device__ __forceinline__ void store_run(T* v, int64_t t, int64_t n, const T (&x)[N]) {
  constexpr int kPer16 = 16 / sizeof(T);
  if (t + N <= n && (reinterpret_cast<uintptr_t>(v) & 15) == 0) {
#pragma unroll
    for (int k = 0; k < N; k += kPer16) *reinterpret_cast<int4*>(v + t + k) = *reinterpret_cast<const int4*>(&x[k]);
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k)
      if (t + k < n) v[t + k] = x[k];
  }
}

// CTA b makes the arrays of tokens [b * kMapTile, (b + 1) * kMapTile) and the per-request outputs of
// rounds b, b + grid, ...; it sums requests until it has passed both.
__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(const SlotMapParams p) {
  __shared__ int s_start[kChunk];  // first token of each request of the round
  __shared__ int s_pos[kChunk];    // and its position
  __shared__ int64_t s_warp[kMapThreads / 32];

  const int64_t tile = static_cast<int64_t>(blockIdx.x) * kMapTile;
  const int64_t tile_end = min(tile + kMapTile, p.tokens);
  const int64_t t0 = tile + threadIdx.x * kMapTokens;
  unsigned int err = 0;
  alignas(16) int32_t req[kMapTokens];
  alignas(16) int64_t pos[kMapTokens], slot[kMapTokens], kv_slot[kMapTokens];
#pragma unroll
  for (int k = 0; k < kMapTokens; ++k) req[k] = 0, pos[k] = 0, slot[k] = kv_slot[k] = -1;

  const uint32_t ratio = static_cast<uint32_t>(p.ratio);
  const int64_t rounds = max(static_cast<int64_t>(1), (p.requests + kChunk - 1) / kChunk);
  int64_t base = 0;
  int64_t duty = blockIdx.x;  // the next round whose per-request outputs are this CTA's
  for (int64_t c = 0; c < rounds && (base < tile_end || duty < rounds); ++c) {
    const int64_t r = c * kChunk + threadIdx.x * kMapRequests;
    int len[kMapRequests], query[kMapRequests];
    load_run(p.seq_lens, r, p.requests, len);
    load_run(p.query_lens, r, p.requests, query);
    int64_t sum = 0;
    unsigned int bad = 0;
#pragma unroll
    for (int k = 0; k < kMapRequests; ++k) {
      if (len[k] < 0 || query[k] < 0) bad = C128_DEV_BAD_LENGTH;
      len[k] = max(len[k], 0);
      query[k] = max(query[k], 0);
      if (query[k] > len[k]) bad = C128_DEV_BAD_LENGTH;
      sum += query[k];
    }
    int64_t total;
    int64_t start = base + block_exclusive_sum<kMapThreads>(sum, s_warp, &total);
#pragma unroll
    for (int k = 0; k < kMapRequests; ++k) {
      const int i = threadIdx.x * kMapRequests + k;
      const int clipped = static_cast<int>(min(start, static_cast<int64_t>(INT_MAX)));
      s_start[i] = clipped;
      s_pos[i] = len[k] - query[k];
      if (c == duty && r + k < p.requests) {
        p.query_start[r + k] = clipped;
        p.kv_lens[r + k] = static_cast<int32_t>(static_cast<uint32_t>(len[k]) / ratio);
      }
      start += query[k];
    }
    if (c == duty) {
      err |= bad;
      if (c == rounds - 1 && threadIdx.x == 0) {
        p.query_start[p.requests] = static_cast<int>(min(base + total, static_cast<int64_t>(INT_MAX)));
        if (base + total > p.tokens) err |= C128_DEV_BAD_LENGTH;
      }
      duty += gridDim.x;
    }
    __syncthreads();
    const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), p.requests - c * kChunk));
    int q = -1;
#pragma unroll
    for (int k = 0; k < kMapTokens; ++k) {
      const int64_t t = t0 + k;
      if (t < base || t >= base + total || t >= tile_end) continue;
      if (q < 0 || (q + 1 < n && s_start[q + 1] <= t)) q = last_at_or_before(s_start, n, static_cast<int>(t));
      const int rq = static_cast<int>(c * kChunk) + q;
      const int64_t at = static_cast<int64_t>(s_pos[q]) + (t - s_start[q]);
      req[k] = rq;
      pos[k] = at;
      if (at < 0) continue;
      const uint32_t u = static_cast<uint32_t>(at);
      slot[k] = slot_of(p.state_table, p.state_stride, p.state_cols, static_cast<uint32_t>(p.state_block), rq, u, &err);
      if ((u + 1) % ratio == 0)
        kv_slot[k] = slot_of(p.kv_table, p.kv_stride, p.kv_cols, static_cast<uint32_t>(p.kv_block), rq, u / ratio, &err);
    }
    base += total;
    __syncthreads();  // s_start, s_pos and s_warp are written again
  }
  store_run(p.token_to_req, t0, tile_end, req);
  store_run(p.positions, t0, tile_end, pos);
  store_run(p.slots, t0, tile_end, slot);
  store_run(p.kv_slots, t0, tile_end, kv_slot);
  if (err) atomicOr(p.err, err);
}

}  // namespace

// One launch where held_out and taken_out are other memory than held and taken. In place, a CTA
// could read a count that another has already raised, so the counts are written by a launch of their
// own behind the one that fills the tables.
cudaError_t launch_extend(const ExtendParams& p, int sm_count, cudaStream_t stream) {
  const bool in_place = p.held_out == p.held || p.taken_out == p.taken;
  const int64_t most = p.columns > 0 && p.requests > p.num_free / p.columns ? p.num_free : p.requests * p.columns;
  const int64_t tiles = (most + kExtendTile - 1) / kExtendTile;
  const int grid = static_cast<int>(tiles < 1 ? 1 : tiles < sm_count ? tiles : sm_count);
  if (!in_place || grid == 1) {
    extend_kernel<<<grid, kExtendThreads, 0, stream>>>(p, true, true);
    return cudaGetLastError();
  }
  extend_kernel<<<grid, kExtendThreads, 0, stream>>>(p, true, false);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  extend_kernel<<<1, kExtendThreads, 0, stream>>>(p, false, true);
  return cudaGetLastError();
}

cudaError_t launch_slot_maps(const SlotMapParams& p, cudaStream_t stream) {
  const int64_t tiles = (p.tokens + kMapTile - 1) / kMapTile;
  slot_map_kernel<<<static_cast<unsigned>(tiles < 1 ? 1 : tiles), kMapThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace c128
