// Block tables and per-token arrays from request lengths: c128_extend_block_tables and
// c128_build_slot_maps. Both are prefix sums over the requests followed by one pass over the blocks
// (or tokens) that finds each one's request in the sums.
//
// Decode steps make a few kilobytes of either, so what counts there is the number of dependent trips
// to memory: one launch, in which every CTA sums the requests for itself (512 or 1024 in a round, a few KB
// that all CTAs read from L2) instead of a scan kernel and a second one behind it, then looks its
// own blocks or tokens up in shared memory. Nothing is accumulated across CTAs, and there is no scratch. The
// only atomics are the error bits and, within a CTA, the minimum that finds the first request that the list cannot
// serve: the order of neither matters.
//
// Measured, device time per call in a graph: tables of 256 requests that each grow by one token 2.0 us (in place, with
// two launches, 4.0), of 16 requests that get all blocks of up to a million tokens (1.1 M blocks, 9 MB) 3.8 us; maps of
// 256 rows 2.3 us, of 32 thousand tokens 2.6, of 215 thousand (6 MB) 4.0. A launch that does nothing takes about 2 us
// this way, and what is left is the chain of loads, sum, search and loads. (Sums in 64 bits, divisions
// and several tokens to a thread took 7 to 8 us for the maps.)
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "c128_serving.h"

namespace c128 {
namespace {

// Sums stop at INT_MAX (blocks and tokens are fewer, so a sum that large is an error anyhow): 32-bit
// words, and the order of additions does not matter.
__device__ __forceinline__ uint32_t add_clipped(uint32_t a, uint32_t b) { return min(a + b, static_cast<uint32_t>(INT_MAX)); }

// Exclusive prefix sum of one value per thread over the CTA, and the total. `warp_sums` holds one
// value per warp and may be used again after the next __syncthreads.
template <int THREADS>
__device__ __forceinline__ uint32_t block_exclusive_sum(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl = add_clipped(incl, u);
  }
  const uint32_t before = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t w = lane < THREADS / 32 ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < THREADS / 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w = add_clipped(w, u);
  }
  *total = __shfl_sync(0xffffffffu, w, THREADS / 32 - 1);
  const uint32_t warps_before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return add_clipped(warp > 0 ? warps_before : 0, lane > 0 ? before : 0);
}

__device__ __forceinline__ void wait_for_inputs() {
  asm volatile("griddepcontrol.launch_dependents;" :::);
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

// N values v[r .. r + N - 1] of a vector of n, zero behind its end; in 16-byte loads where those fit.
template <int N>
__device__ __forceinline__ void load_run(const int32_t* v, int64_t r, int64_t n, int (&out)[N]) {
  if (N % 4 == 0 && r + N <= n && (reinterpret_cast<uintptr_t>(v) & 15) == 0) {
#pragma unroll
    for (int k = 0; k + 3 < N; k += 4) {
      const int4 x = *reinterpret_cast<const int4*>(v + r + k);
      out[k] = x.x, out[k + 1] = x.y, out[k + 2] = x.z, out[k + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) out[k] = r + k < n ? v[r + k] : 0;
  }
}

// ------------------------------------------------------------------------------- block tables
// One CTA to an SM, and a request to a thread: with 512 threads, two CTAs to an SM and four requests 1.1 M blocks took
// 6.3 us, not 4.0, and a step of 256 requests 2.2, not 2.1.
constexpr int kExtendThreads = 1024;
constexpr int kExtendChunk = kExtendThreads;         // requests of a round
constexpr int kTileBlocks = 8;                       // blocks of a tile per thread, their loads in flight together
constexpr int kExtendTile = kExtendThreads * kTileBlocks;

// Every CTA sums all requests; the given blocks are dealt out in tiles of kExtendTile. With
// `write_counts` the CTAs also write held_out (a round each) and CTA 0 taken_out, which must then not
// be `held` and `taken` themselves unless the grid is one CTA.
__global__ void __launch_bounds__(kExtendThreads) extend_kernel(const ExtendParams p, bool write_table, bool write_counts) {
  __shared__ int s_start[kExtendChunk];  // first block of each request of the round, counted from the round's first
  __shared__ int s_held[kExtendChunk];
  __shared__ uint32_t s_warp[kExtendThreads / 32];
  __shared__ uint32_t s_fail;

  wait_for_inputs();
  const int64_t taken = *p.taken;
  unsigned int err = 0;
  const bool bad_taken = taken < 0 || taken > p.num_free;
  if (bad_taken) err |= C128_DEV_BAD_LENGTH;
  const uint32_t avail = bad_taken ? 0 : static_cast<uint32_t>(p.num_free - taken);
  uint32_t base = 0;   // blocks needed by the requests of earlier rounds
  uint32_t given = 0;
  const int64_t rounds = (p.requests + kExtendChunk - 1) / kExtendChunk;

  for (int64_t c = 0; c < rounds; ++c) {
    if (threadIdx.x == 0) s_fail = UINT_MAX;
    const int64_t r = c * kExtendChunk + threadIdx.x;
    const int len = r < p.requests ? p.seq_lens[r] : 0, held = r < p.requests ? p.held[r] : 0;
    if (len < 0) err |= C128_DEV_BAD_LENGTH;
    const uint32_t entries = divide(static_cast<uint32_t>(max(len, 0)), p.ratio);
    const uint32_t full = divide(entries, p.block), needed = full + (full * p.block.value != entries);  // <= INT_MAX
    uint32_t need = 0;
    if (held < 0) {
      err |= C128_DEV_BAD_LENGTH;
    } else if (needed > static_cast<uint32_t>(held)) {
      if (needed > p.columns) err |= C128_DEV_BAD_BT_COL;
      else need = needed - static_cast<uint32_t>(held);
    }
    uint32_t total;
    // (a barrier, also for s_fail)
    const uint32_t off = add_clipped(base, block_exclusive_sum<kExtendThreads>(need, s_warp, &total));
    if (need > 0 && add_clipped(off, need) > avail) {  // avail < INT_MAX
      err |= C128_DEV_NO_FREE_BLOCK;
      atomicMin(&s_fail, off);
    }
    __syncthreads();
    // Blocks are given up to the first request that the list cannot serve, and none after it: the sum
    // only grows, so later rounds find nothing left either.
    const uint32_t end = min(s_fail, add_clipped(base, total));
    const uint32_t round_given = base <= avail ? end - base : 0;
    s_start[threadIdx.x] = static_cast<int>(min(off - base, round_given));
    s_held[threadIdx.x] = held;
    if (write_counts && c % gridDim.x == blockIdx.x && r < p.requests)
      p.held_out[r] = held + (need <= round_given && off - base <= round_given - need ? static_cast<int>(need) : 0);
    __syncthreads();
    if (write_table) {
      const int n = static_cast<int>(min(static_cast<int64_t>(kExtendChunk), p.requests - c * kExtendChunk));
      const int32_t* from = p.free_blocks + taken + base;
      for (uint32_t i0 = blockIdx.x * kExtendTile; i0 < round_given; i0 += gridDim.x * kExtendTile) {
        int id[kTileBlocks];
#pragma unroll
        for (int k = 0; k < kTileBlocks; ++k) {
          const uint32_t i = i0 + k * kExtendThreads + threadIdx.x;
          id[k] = i < round_given ? from[i] : 0;
        }
        int q = -1;
#pragma unroll
        for (int k = 0; k < kTileBlocks; ++k) {
          const uint32_t i = i0 + k * kExtendThreads + threadIdx.x;
          if (i >= round_given) break;
          if (q < 0 || (q + 1 < n && static_cast<uint32_t>(s_start[q + 1]) <= i)) q = last_at_or_before(s_start, n, static_cast<int>(i));
          p.table[(c * kExtendChunk + q) * p.stride + s_held[q] + (static_cast<int>(i) - s_start[q])] = id[k];
        }
      }
    }
    given += round_given;
    base = add_clipped(base, total);
    __syncthreads();  // s_start, s_held, s_warp and s_fail are written again
  }
  if (write_counts && blockIdx.x == 0 && threadIdx.x == 0) *p.taken_out = taken + given;
  if (write_counts && blockIdx.x == 0 && err) atomicOr(p.err, err);
}

// ----------------------------------------------------------------------------------- slot maps
// CTA b makes the arrays of tokens [b * THREADS, (b + 1) * THREADS) and the per-request outputs
// of rounds b, b + grid, ...; it sums requests until it has passed both. A token per thread, not
// several: a decode step has a few hundred, and what counts is the chain of dependent steps of one.
template <int THREADS, int PER>  // requests per thread and round
__global__ void __launch_bounds__(THREADS) slot_map_kernel(const SlotMapParams p) {
  constexpr int kChunk = PER * THREADS;
  __shared__ int s_start[kChunk];  // first token of each request of the round
  __shared__ int s_pos[kChunk];    // and its position
  __shared__ uint32_t s_warp[THREADS / 32];

  wait_for_inputs();
  const uint32_t t = blockIdx.x * THREADS + threadIdx.x;
  const uint32_t tile_end = static_cast<uint32_t>(min(static_cast<int64_t>(blockIdx.x + 1) * THREADS, p.tokens));
  unsigned int err = 0;
  int req = 0, pos = 0;
  int64_t slot = -1, kv_slot = -1;

  const int64_t rounds = max(static_cast<int64_t>(1), (p.requests + kChunk - 1) / kChunk);
  uint32_t base = 0;
  int64_t duty = blockIdx.x;  // the next round whose per-request outputs are this CTA's
  for (int64_t c = 0; c < rounds && (base < tile_end || duty < rounds); ++c) {
    const int64_t r = c * kChunk + threadIdx.x * PER;
    int len[PER], query[PER];
    load_run(p.seq_lens, r, p.requests, len);
    load_run(p.query_lens, r, p.requests, query);
    uint32_t sum = 0;
    unsigned int bad = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (len[k] < 0 || query[k] < 0) bad = C128_DEV_BAD_LENGTH;
      len[k] = max(len[k], 0);
      query[k] = max(query[k], 0);
      if (query[k] > len[k]) bad = C128_DEV_BAD_LENGTH;
      sum = add_clipped(sum, static_cast<uint32_t>(query[k]));
    }
    uint32_t total;
    uint32_t start = add_clipped(base, block_exclusive_sum<THREADS>(sum, s_warp, &total));
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const int i = threadIdx.x * PER + k;
      s_start[i] = static_cast<int>(start);
      s_pos[i] = len[k] - query[k];
      if (c == duty && r + k < p.requests) {
        p.query_start[r + k] = static_cast<int>(start);
        p.kv_lens[r + k] = static_cast<int32_t>(divide(static_cast<uint32_t>(len[k]), p.ratio));
      }
      start = add_clipped(start, static_cast<uint32_t>(query[k]));
    }
    const uint32_t end = add_clipped(base, total);
    if (c == duty) {
      err |= bad;
      if (c == rounds - 1 && threadIdx.x == 0) {
        p.query_start[p.requests] = static_cast<int>(end);
        if (end > p.tokens) err |= C128_DEV_BAD_LENGTH;
      }
      duty += gridDim.x;
    }
    __syncthreads();
    if (t >= base && t < end && t < tile_end) {
      const int n = static_cast<int>(min(static_cast<int64_t>(kChunk), p.requests - c * kChunk));
      const int q = last_at_or_before(s_start, n, static_cast<int>(t));
      req = static_cast<int>(c * kChunk) + q;
      pos = s_pos[q] + (static_cast<int>(t) - s_start[q]);
      if (pos >= 0) {
        // both tables are read before either is looked at
        const uint32_t u = static_cast<uint32_t>(pos), entry = divide(u, p.ratio);
        const bool ends = u + 1 == (entry + 1) * p.ratio.value;
        const uint32_t col = divide(u, p.state_block), kv_col = divide(entry, p.kv_block);
        const bool in = col < p.state_cols, kv_in = ends && kv_col < p.kv_cols;
        const int id = in ? p.state_table[req * p.state_stride + col] : 0;
        const int kv_id = kv_in ? p.kv_table[req * p.kv_stride + kv_col] : 0;
        if (!in || (ends && !kv_in)) err |= C128_DEV_BAD_BT_COL;
        if (id < 0 || kv_id < 0) err |= C128_DEV_BAD_BLOCK;
        if (in && id >= 0) slot = static_cast<int64_t>(id) * p.state_block.value + (u - col * p.state_block.value);
        if (kv_in && kv_id >= 0) kv_slot = static_cast<int64_t>(kv_id) * p.kv_block.value + (entry - kv_col * p.kv_block.value);
      }
    }
    base = end;
    __syncthreads();  // s_start, s_pos and s_warp are written again
  }
  if (t < tile_end) {
    p.token_to_req[t] = req;
    p.positions[t] = pos;
    p.slots[t] = slot;
    p.kv_slots[t] = kv_slot;
  }
  if (err) atomicOr(p.err, err);
}

}  // namespace

namespace {
// Launched so that its start overlaps the end of the kernel before it (it waits for that one's writes).
template <class P, class... A>
cudaError_t launch_early(void (*kernel)(P, A...), unsigned grid, unsigned threads, cudaStream_t stream, const P& p, A... args) {
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(threads);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, kernel, p, args...);
}
}  // namespace

// One launch where held_out and taken_out are other memory than held and taken. In place, a CTA
// could read a count that another has already raised, so the counts are written by a launch of their
// own behind the one that fills the tables.
cudaError_t launch_extend(const ExtendParams& p, int sm_count, cudaStream_t stream) {
  const bool in_place = p.held_out == p.held || p.taken_out == p.taken;
  const int64_t most = p.columns > 0 && p.requests > p.num_free / p.columns ? p.num_free : p.requests * p.columns;
  const int64_t tiles = (most + kExtendTile - 1) / kExtendTile;
  const unsigned grid = static_cast<unsigned>(tiles < 1 ? 1 : tiles < sm_count ? tiles : sm_count);
  if (!in_place || grid == 1) return launch_early(extend_kernel, grid, kExtendThreads, stream, p, true, true);
  const cudaError_t e = launch_early(extend_kernel, grid, kExtendThreads, stream, p, true, false);
  return e != cudaSuccess ? e : launch_early(extend_kernel, 1u, kExtendThreads, stream, p, false, true);
}

// A request to a thread while one round takes them all; else four, and the rounds are fewer: 200 requests 2.4 us and
// 2.5, 333 with 32 thousand tokens 2.6 and 3.2; 2048 4.5 and 3.4, 1000 with 100 thousand tokens 5.2 and 4.4.
cudaError_t launch_slot_maps(const SlotMapParams& p, cudaStream_t stream) {
  const bool one_round = p.requests <= 512;
  const int threads = one_round ? 512 : 256;  // a token each
  const int64_t tiles = (p.tokens + threads - 1) / threads;
  const unsigned grid = static_cast<unsigned>(tiles < 1 ? 1 : tiles);
  if (one_round) return launch_early(slot_map_kernel<512, 1>, grid, 512, stream, p);
  return launch_early(slot_map_kernel<256, 4>, grid, 256, stream, p);
}

}  // namespace c128
