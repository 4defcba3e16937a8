// c128_decode_attention: attention of one new token per request over its entries of the paged FP8
// cache, on the tcgen05 tensor cores.
//
//   S = Q K^T            per tile of 64 entries: M = 64 heads, N = 64 entries, K = 512
//   P = exp2(c S - m)    c = scale * log2(e), m a running reference per head, in registers
//   O^T += K^T P^T       M = 128 columns (4 times), N = heads, K = 64 entries
//   out = O / sum P
//
// An entry is key and value, so a tile is decoded once, to bf16 in shared memory (exact: an e4m3 code
// has 4 significant bits and its scale is a power of two), and both products read it from there: as
// B with the 512 columns along K, and as A with them along M. Taking O transposed makes the heads the
// N of the second product, so its work and its TMEM columns go with the heads there are, and leaves
// 128 of the 512 columns for two S tiles. Heads are dealt out in groups of 64; a group decodes the
// cache for itself (the second group's reads hit L2).
//
// The running reference m is not the maximum itself: it is raised only when a score passes it by more
// than 2^8, because raising it means rescaling O in TMEM. P then stays below 2^8 and its sum exact
// enough in fp32, whatever the scores do.
//
// Work is dealt out in tiles: the requests' tiles, one after the other, are cut into as many equal
// runs as there are CTAs, so a long request is shared by many CTAs and a CTA takes many short ones. A
// request that is cut leaves fp32 partial results in the workspace, joined by a second kernel.
//
// Roles of the 14 warps (each wait is bounded, see c128_device.cuh):
//   0..7   decode the entries of a tile into shared memory, the next tile's bytes already in registers
//   8..11  softmax of S, rescaling of O, results
//   12     one thread issues the products and the queries' TMA loads
//   13     walks the runs: per tile the address of each entry (through the block table), prefetched
//          to L2 a few tiles ahead
#include <cuda_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "c128_device.cuh"
#include "c128_serving.h"

namespace c128 {
namespace {

constexpr int kTile = 64;           // entries per tile
constexpr int kGroup = 64;          // heads per CTA
constexpr int kChunks = kHead / 64; // 64-column chunks of 128 bytes (bf16): one swizzle atom wide
constexpr int kChunkBytes = kTile * 128;
constexpr int kTileBytes = kChunks * kChunkBytes;  // a decoded tile: 64 KiB
constexpr int kFillWarps = 8, kSoftWarps = 4;
constexpr int kMmaWarp = kFillWarps + kSoftWarps, kIndexWarp = kMmaWarp + 1;
constexpr int kDecodeThreads = 32 * (kIndexWarp + 1);
constexpr int kRing = 4;            // tiles the index warp may be ahead
constexpr float kSlack = 8.f;       // log2 units a score may pass the reference by
constexpr int kTmemCols = 512, kTmemS = 256;  // O in columns 0..255, two S tiles behind it

enum : int { kFirst = 1, kLast = 2, kEnd = 4 };

struct TileDesc {
  const uint8_t* data[kTile];    // record of each entry, NULL where there is none
  const uint8_t* scales[kTile];
  uint64_t mask;                 // entries there are
  int32_t flags, request;
  int32_t part;                  // kLast: slot of the partial result, -1 if the request is whole
  int32_t pad;
};

struct DecodeSmem {
  alignas(1024) uint8_t q[kGroup * kHead * 2];
  alignas(1024) uint8_t k[2][kTileBytes];
  alignas(1024) uint8_t p[2][kGroup * kTile * 2];
  TileDesc ring[kRing];
  alignas(16) float factor[kGroup];
  alignas(16) float inv[kGroup];
  uint64_t ring_full[kRing], ring_free[kRing];
  uint64_t k_full[2], s_full[2], s_free[2], p_full[2], pv_done[2];
  uint64_t q_full, q_free, o_free, drained;
  uint64_t soft;                 // barrier of the softmax warps
  int32_t vote[2][kSoftWarps];
  int64_t warp_sums[kDecodeThreads / 32];
  int64_t total;                 // tiles of all requests
  int64_t first_tile;            // of the run's first request: its tiles before the run
  int32_t first_request;
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(DecodeSmem) <= 232448, "shared memory of one SM");

struct Task {  // a request that CTA column c shares with the ones behind it
  int32_t request, parts;
};

// Scratch of a call: tasks, log2-sum-exps and fp32 results of partial requests. Column c of CTAs has
// two slots: 2c for the request it continues, 2c + 1 for the one it starts and does not finish.
struct Scratch {
  int columns, groups, heads;  // CTA columns, head groups, heads held per slot and group
  __host__ __device__ Scratch(int all_heads, int sms) {
    groups = (all_heads + kGroup - 1) / kGroup;
    columns = sms / groups > 0 ? sms / groups : 1;
    heads = groups > 1 ? kGroup : (all_heads + 15) / 16 * 16;
  }
  __host__ __device__ int64_t rows() const { return 2ll * columns * groups * heads; }
  __host__ __device__ int64_t lse_at() const { return (columns * static_cast<int64_t>(sizeof(Task)) + 255) / 256 * 256; }
  __host__ __device__ int64_t out_at() const { return lse_at() + (rows() * 4 + 255) / 256 * 256; }
  __host__ __device__ int64_t bytes() const { return out_at() + rows() * kHead * 4; }
  __device__ int64_t row(int slot, int group, int head) const {
    return (static_cast<int64_t>(slot) * groups + group) * heads + head;
  }
};

// A bounded wait that looks at the clock and the abort flag only now and then: reading the global
// timer takes longer than most of these waits (a try alone lets the hardware suspend the thread).
__device__ __noinline__ bool decode_wait_slow(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (abort_flag != nullptr && *abort_flag) return false;
    if (global_timer_ns() - t0 > kWaitTimeoutNs) return false;
  }
}
__device__ __forceinline__ bool decode_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  for (int i = 0; i < 4; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return decode_wait_slow(bar, parity, abort_flag);
}

// ------------------------------------------------------------------------------------ tcgen05
// Shared-memory operand with the 128-byte swizzle: the low half holds the address and the leading
// byte offset (of the next 64 rows of an M-major operand, unused for K-major), the high half the
// offset of the next 8 rows. Steps along an operand are added to the low half, in 16-byte units.
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t leading) {
  return (addr & 0x3ffff) >> 4 | leading >> 4 << 16;
}
constexpr uint32_t kDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint64_t desc64(uint32_t low) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(low), "r"(kDescHigh));
  return d;
}
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool a_mn_major) {  // bf16 x bf16 -> fp32
  return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn_major ? 1u << 15 : 0u) | static_cast<uint32_t>(n >> 3) << 17 |
         static_cast<uint32_t>(m >> 4) << 24;
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ void mma(uint32_t d, uint32_t a_low, uint32_t b_low, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(desc64(a_low)), "l"(desc64(b_low)), "r"(desc),
      "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 lanes x 64 columns: thread t gets rows t/4 and t/4 + 8, columns 8g + 2(t%4) and + 1 in x[4g ..]
__device__ __forceinline__ void tmem_ld_16x64(uint32_t addr, uint32_t (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
        "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]), "=r"(x[16]),
        "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]), "=r"(x[22]), "=r"(x[23]), "=r"(x[24]),
        "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]), "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
      : "r"(addr));
}
// 32 lanes x 16 columns, a lane's columns in one thread
__device__ __forceinline__ void tmem_ld_32x16(uint32_t addr, uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
        "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st_32x16(uint32_t addr, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]),
      "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
      : "memory");
}
__device__ __forceinline__ void load_query_box(void* dst, const CUtensorMap* map, int col, int head, int request, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(col), "r"(head), "r"(request), "r"(smem_addr(bar))
      : "memory");
}

// ------------------------------------------------------------------------------------- decoding
// Two e4m3 codes (bytes lo, lo + 1 of w) to bf16: the code's exponent and mantissa moved to the bf16
// fields give the value times 2^-120 (subnormals included, bf16 keeps them), `mul` puts 2^120 and the
// scale back.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t spread, uint32_t mul) {
  uint32_t x = (spread & 0x80008000u) | ((spread >> 4) & 0x07f007f0u), y;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(mul));
  return y;
}
// The same by way of fp32, for NaN codes and scales whose 2^(120 + e) has no bf16.
__device__ __noinline__ uint32_t codes_to_bf16_any(uint32_t two, int scale_byte) {
  float v[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t b = (two >> (8 * i)) & 0xffu, mag = b & 0x7fu;
    const float a = mag == 0x7fu ? NAN : __uint_as_float(mag << 20) * 0x1p120f;
    v[i] = ldexpf(b & 0x80u ? -a : a, scale_byte - 127);
  }
  return pack_bf16x2(v[0], v[1]);
}
constexpr int kMaxFastScale = 134;  // 2^(134 - 127 + 120) = 2^127

__device__ __forceinline__ uint4 ld16(const uint8_t* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint4 ld8x2(const uint8_t* p) {
  const uint2 a = __ldg(reinterpret_cast<const uint2*>(p)), b = __ldg(reinterpret_cast<const uint2*>(p) + 1);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ int64_t entries_of(const DecodeParams& p, int64_t r, unsigned int* err) {
  int64_t n = p.kv_lens[r];
  if (n < 0) {
    *err |= C128_DEV_BAD_LENGTH;
    n = 0;
  }
  if (n > p.columns * p.kv_bs) {
    *err |= C128_DEV_BAD_BT_COL;
    n = p.columns * p.kv_bs;
  }
  return n;
}
// A request without entries still takes a (masked) tile: its results are written like any other's.
__device__ __forceinline__ int64_t tiles_of(int64_t entries) { return entries > 0 ? (entries + kTile - 1) / kTile : 1; }

// First tile of CTA column c when `total` tiles are dealt to `columns` columns, and the column of a tile.
__device__ __forceinline__ int64_t run_begin(int64_t c, int64_t total, int64_t columns) { return c * total / columns; }
__device__ __forceinline__ int64_t column_of(int64_t tile, int64_t total, int64_t columns) {
  return ((tile + 1) * columns - 1) / total;
}

template <bool ALIGN16>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    decode_kernel(const DecodeParams p, const __grid_constant__ CUtensorMap q_map, const Scratch scratch, int box_heads) {
  extern __shared__ uint8_t smem_raw[];
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int group = blockIdx.x % scratch.groups, column = blockIdx.x / scratch.groups;
  const int heads = min(kGroup, p.heads - group * kGroup);
  const int heads16 = (heads + 15) & ~15;
  unsigned int err = 0;

  launch_dependents();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.ring_full[i], 1);
      mbar_init(&sm.ring_free[i], kFillWarps + kSoftWarps + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], kFillWarps);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], kSoftWarps);
      mbar_init(&sm.p_full[i], kSoftWarps);
      mbar_init(&sm.pv_done[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.o_free, kSoftWarps);
    mbar_init(&sm.drained, 1);
    mbar_init(&sm.soft, kSoftWarps);
    sm.abort = 0;
    sm.first_request = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (box_heads < kGroup)  // rows of absent heads, which the loads never write
    for (int i = threadIdx.x; i < kGroup * kHead * 2 / 16; i += kDecodeThreads)
      reinterpret_cast<uint4*>(sm.q)[i] = make_uint4(0, 0, 0, 0);
  async_proxy_fence();

  // The run of this column: sum the requests' tiles, then find the first and the last request.
  const int64_t per = (p.requests + kDecodeThreads - 1) / kDecodeThreads;
  const int64_t r_begin = min(threadIdx.x * per, p.requests), r_end = min(r_begin + per, p.requests);
  int64_t mine = 0;
  for (int64_t r = r_begin; r < r_end; ++r) mine += tiles_of(entries_of(p, r, &err));
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.warp_sums[warp] = incl;
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  int64_t base = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kDecodeThreads / 32; ++w) {
    const int64_t s = sm.warp_sums[w];
    if (w < warp) base += s;
    total += s;
  }
  const int64_t columns = min(static_cast<int64_t>(scratch.columns), total);
  const int64_t begin = column < columns ? run_begin(column, total, columns) : 0;
  const int64_t end = column < columns ? run_begin(column + 1, total, columns) : 0;
  Task* const tasks = reinterpret_cast<Task*>(p.workspace);
  if (column >= columns) {
    if (group == 0 && threadIdx.x == 0) tasks[column] = Task{0, 0};
  } else if (mine > 0 && base < end && base + mine > begin) {
    for (int64_t r = r_begin, at = base; r < r_end && at < end; ++r) {
      unsigned int ignore = 0;
      const int64_t n = tiles_of(entries_of(p, r, &ignore));
      if (begin >= at && begin < at + n) {
        sm.first_request = static_cast<int32_t>(r);
        sm.first_tile = begin - at;
      }
      if (group == 0 && end - 1 >= at && end - 1 < at + n) {
        const bool shared = at >= begin && at + n > end;
        tasks[column] = Task{static_cast<int32_t>(r),
                             shared ? static_cast<int32_t>(column_of(at + n - 1, total, columns)) - column + 1 : 0};
      }
      at += n;
    }
  }
  if (blockIdx.x == 0 && err) atomicOr(p.err, err);
  err = 0;
  __syncthreads();
  const uint32_t tmem = sm.tmem;
  volatile int* const abort_flag = &sm.abort;
  // A wait of a whole warp, with one answer for all its lanes; false: give up (the CTA ends).
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    const bool ok = __all_sync(0xffffffffu, decode_wait(bar, parity, abort_flag));
    if (!ok && lane == 0) {
      *abort_flag = 1;
      atomicOr(p.err, static_cast<unsigned int>(C128_DEV_TIMEOUT));
    }
    return ok;
  };

  if (column >= columns) {
    // no tiles
  } else if (warp == kIndexWarp) {
    // -------------------------------------------------------------------------- walk the run
    int64_t r = sm.first_request, tile = sm.first_tile;
    int64_t started = tile;  // the request's tile at which this run takes it up
    const uint32_t bs = static_cast<uint32_t>(p.kv_bs);
    int64_t window = r;      // lanes hold the lengths of requests window .. window + 31
    unsigned int ignore = 0;
    int64_t lens = window + lane < p.requests ? entries_of(p, window + lane, &ignore) : 0;
    int64_t n = __shfl_sync(0xffffffffu, lens, 0);
    int id[2];
    auto load_ids = [&](int64_t rr, int64_t tt, int64_t nn) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t key = tt * kTile + 32 * h + lane;
        id[h] = key < nn ? __ldg(p.table + rr * p.table_stride + static_cast<uint32_t>(key) / bs) : -1;
      }
    };
    load_ids(r, tile, n);
    int64_t left = end - begin;
    for (int i = 0; left >= 0; ++i, --left) {
      const int slot = i % kRing;
      if (i >= kRing && !warp_wait(&sm.ring_free[slot], (i / kRing - 1) & 1)) break;
      TileDesc& d = sm.ring[slot];
      if (left == 0) {
        if (lane == 0) d.flags = kEnd;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ring_full[slot]);
        break;
      }
      const int64_t tiles = tiles_of(n);
      uint64_t mask = 0;
      const uint8_t* from[2];
      const uint8_t* sc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t key = tile * kTile + 32 * h + lane;
        const bool in = key < n;
        const bool ok = in && id[h] >= 0 && id[h] < p.nkb;
        if (in && !ok) err |= C128_DEV_BAD_BLOCK;
        const uint32_t off = static_cast<uint32_t>(key) % bs;
        const uint8_t* blk = p.kc + static_cast<int64_t>(ok ? id[h] : 0) * p.kc_stride0;
        from[h] = ok ? blk + static_cast<int64_t>(off) * kTokenStride : nullptr;
        sc[h] = blk + p.kv_bs * kTokenStride + static_cast<int64_t>(off) * kScaleDim;
        mask |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << (32 * h);
      }
      const bool last_of_request = tile + 1 == tiles, last = last_of_request || left == 1;
      const int64_t here = r;
      const int flags = (tile == started ? kFirst : 0) | (last ? kLast : 0);
      const int part = started == 0 && last_of_request ? -1 : 2 * column + (started == 0 ? 1 : 0);
      // the next tile's block ids are on their way while this tile is written
      if (last_of_request) {
        ++r;
        tile = started = 0;
        if (r - window >= 32) {
          window = r;
          lens = window + lane < p.requests ? entries_of(p, window + lane, &ignore) : 0;
        }
        n = __shfl_sync(0xffffffffu, lens, static_cast<int>(r - window));
      } else {
        ++tile;
      }
      if (left > 1) load_ids(r, tile, n);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        d.data[32 * h + lane] = from[h];
        d.scales[32 * h + lane] = sc[h];
        if (from[h] != nullptr) {
          if (ALIGN16) {
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from[h]), "n"(kTokenStride) : "memory");
          } else {
#pragma unroll
            for (int b = 0; b < kTokenStride; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from[h] + b));
          }
          asm volatile("prefetch.global.L2 [%0];" ::"l"(sc[h]));
        }
      }
      if (lane == 0) {
        d.mask = mask;
        d.flags = flags;
        d.request = static_cast<int32_t>(here);
        d.part = part;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_full[slot]);
    }
    if (err) atomicOr(p.err, err);
  } else if (warp < kFillWarps) {
    // ------------------------------------------------------------------------ decode the entries
    // Four threads per entry; thread `sub` of an entry takes the 16 bytes sub, sub + 4, ...: of the
    // codes a quarter of each 64-column chunk, so load j belongs to scale j.
    const int key = 8 * warp + (lane >> 2), sub = lane & 3;
    uint4 raw[9];
    uint2 sc;
    const uint32_t row = smem_addr(sm.k[0]) + key * 128;
    const uint32_t swz = static_cast<uint32_t>(key & 7) << 4;
    const uint8_t* src = nullptr;
    const uint8_t* ssrc = nullptr;
    auto load = [&](int j) { return src == nullptr ? make_uint4(0, 0, 0, 0) : ALIGN16 ? ld16(src + 64 * j + 16 * sub) : ld8x2(src + 64 * j + 16 * sub); };
    bool more = false;
    // take tile i's addresses out of the ring
    auto fetch = [&](int i) -> bool {
      const int slot = i % kRing;
      if (!warp_wait(&sm.ring_full[slot], (i / kRing) & 1)) {
        more = false;
        return false;
      }
      more = (sm.ring[slot].flags & kEnd) == 0;
      if (more) {
        src = sm.ring[slot].data[key];
        ssrc = sm.ring[slot].scales[key];
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ring_free[slot]);
      }
      return true;
    };
    fetch(0);
    if (more) {
#pragma unroll
      for (int j = 0; j < 9; ++j) raw[j] = load(j);
      sc = src == nullptr ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2*>(ssrc));
    }
    for (int i = 0; more; ++i) {
      const int buf = i & 1;
      if (!fetch(i + 1)) break;
      const uint2 sc_now = sc;
      if (more) sc = src == nullptr ? make_uint2(0, 0) : __ldg(reinterpret_cast<const uint2*>(ssrc));
      if (i >= 2 && !warp_wait(&sm.pv_done[buf], (i / 2 - 1) & 1)) break;
      const uint32_t dst = row + buf * kTileBytes;
      const uint32_t hi = sc_now.y & 0x00ffffffu;
      const bool big = __vcmpgtu4(sc_now.x, 0x01010101u * kMaxFastScale) != 0 || __vcmpgtu4(hi, 0x01010101u * kMaxFastScale) != 0;
#pragma unroll
      for (int j = 0; j < 7; ++j) {
        const uint32_t sb = ((j < 4 ? sc_now.x : hi) >> (8 * (j & 3))) & 0xffu;
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
        uint32_t nan = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) nan |= ((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        uint32_t o[8];
        if (!big && nan == 0) {
          const uint32_t mul = (sb + 120u) * 0x00800080u;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[2 * k] = codes_to_bf16(__byte_perm(w[k], 0, 0x1404), mul);
            o[2 * k + 1] = codes_to_bf16(__byte_perm(w[k], 0, 0x3424), mul);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            o[2 * k] = codes_to_bf16_any(w[k], static_cast<int>(sb));
            o[2 * k + 1] = codes_to_bf16_any(w[k] >> 16, static_cast<int>(sb));
          }
        }
        const uint32_t at = dst + j * kChunkBytes;
        sts16(at + ((32u * sub) ^ swz), o[0], o[1], o[2], o[3]);
        sts16(at + ((32u * sub + 16u) ^ swz), o[4], o[5], o[6], o[7]);
        if (more) raw[j] = load(j);
      }
#pragma unroll
      for (int j = 7; j < 9; ++j) {  // the rope columns are bf16 already
        sts16(dst + 7 * kChunkBytes + ((64u * (j - 7) + 16u * sub) ^ swz), raw[j].x, raw[j].y, raw[j].z, raw[j].w);
        if (more) raw[j] = load(j);
      }
      async_proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[buf]);
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------------ issue the products
    // One elected thread in one branch: the compiler then keeps descriptors in uniform registers, and
    // a product issues faster than it runs (32 cycles for S, 39 to 48 for O, bound by the reads of the
    // operands from shared memory). Behind a test of the lane each took 66 to 75 cycles to issue.
    if (elect_one()) {
      const uint32_t q_at = desc_low(smem_addr(sm.q), 16), ks_at = desc_low(smem_addr(sm.k[0]), 16);
      const uint32_t kv_at = desc_low(smem_addr(sm.k[0]), kChunkBytes), p_at = desc_low(smem_addr(sm.p[0]), 16);
      constexpr uint32_t s_desc = mma_desc(kGroup, kTile, false);
      const uint32_t o_desc = mma_desc(128, heads16, true);
      int seg = -1, prev_flags = 0, prev_seg = 0;
      bool failed = false, loading = false;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (failed) return false;
        if (decode_wait(bar, parity, abort_flag)) return true;
        *abort_flag = 1;
        atomicOr(p.err, static_cast<unsigned int>(C128_DEV_TIMEOUT));
        failed = true;
        return false;
      };
      auto product_pv = [&](int i, int flags, int s) {  // O^T += K^T P^T of tile i
        const int buf = i & 1;
        if (!wait(&sm.p_full[buf], (i / 2) & 1)) return;
        if ((flags & kFirst) && s > 0 && !wait(&sm.o_free, (s - 1) & 1)) return;
        tmem_fence_after();
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks) {
            const uint32_t a = kv_at + ((buf * kTileBytes + 2 * mt * kChunkBytes + ks * 2048) >> 4);
            const uint32_t b = p_at + ((buf * (kGroup * kTile * 2) + ks * 32) >> 4);
            mma(tmem + mt * kGroup, a, b, o_desc, !(flags & kFirst) || ks > 0);
          }
        }
        mma_commit(&sm.pv_done[buf]);
      };
      int i = 0;
      for (; !failed; ++i) {
        const int slot = i % kRing, buf = i & 1;
        if (!wait(&sm.ring_full[slot], (i / kRing) & 1)) break;
        const int flags = sm.ring[slot].flags;
        if (flags & kEnd) break;
        const int request = sm.ring[slot].request;
        mbar_arrive(&sm.ring_free[slot]);
        if (flags & kFirst) {
          ++seg;
          if (seg > 0 && !wait(&sm.q_free, (seg - 1) & 1)) break;
          mbar_arrive_expect_tx(&sm.q_full, static_cast<uint32_t>(box_heads) * kHead * 2);
          for (int c = 0; c < kChunks; ++c)
            load_query_box(sm.q + c * (kGroup * 128), &q_map, 64 * c, group * kGroup, request, &sm.q_full);
          loading = true;
          if (i > 0) product_pv(i - 1, prev_flags, prev_seg);
          if (!wait(&sm.q_full, seg & 1)) break;
          loading = false;
        }
        if (!wait(&sm.k_full[buf], (i / 2) & 1)) break;
        if (i >= 2 && !wait(&sm.s_free[buf], (i / 2 - 1) & 1)) break;
        tmem_fence_after();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint32_t a = q_at + ((c * (kGroup * 128) + ks * 32) >> 4);
            const uint32_t b = ks_at + ((buf * kTileBytes + c * kChunkBytes + ks * 32) >> 4);
            mma(tmem + kTmemS + buf * kTile, a, b, s_desc, c + ks > 0);
          }
        }
        mma_commit(&sm.s_full[buf]);
        if (flags & kLast) mma_commit(&sm.q_free);
        if (!(flags & kFirst) && i > 0) product_pv(i - 1, prev_flags, prev_seg);
        prev_flags = flags;
        prev_seg = seg;
      }
      if (!failed && i > 0) product_pv(i - 1, prev_flags, prev_seg);
      // nothing may be in flight when the CTA ends
      mma_commit(&sm.drained);
      decode_wait(&sm.drained, 0, nullptr);
      if (loading) decode_wait(&sm.q_full, seg & 1, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------------------ softmax
    const int w = warp - kFillWarps;                 // TMEM lanes 32w .. 32w + 31
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const int h0 = 16 * w + (lane >> 2), h1 = h0 + 8;  // this thread's two heads of S
    const bool active = 16 * w < heads16;
    const float c2 = p.scale * kLog2e;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // Barrier of the four warps (a bounded one, so that a warp that gave up holds up no other) with
    // the OR of `pred` over them. A warp is at most one barrier ahead, hence two sets of votes.
    uint32_t soft_phase = 0;
    bool any = false;
    auto soft_sync = [&](bool pred) {
      const bool mine_ = __any_sync(0xffffffffu, pred);
      __syncwarp();
      if (lane == 0) {
        sm.vote[soft_phase][w] = mine_;
        mbar_arrive(&sm.soft);
      }
      const bool ok = warp_wait(&sm.soft, soft_phase);
      const int* v = sm.vote[soft_phase];
      any = (v[0] | v[1] | v[2] | v[3]) != 0;
      soft_phase ^= 1;
      return ok;
    };
    for (int i = 0;; ++i) {
      const int slot = i % kRing, buf = i & 1;
      if (!warp_wait(&sm.ring_full[slot], (i / kRing) & 1)) break;
      const int flags = sm.ring[slot].flags;
      if (flags & kEnd) break;
      const uint64_t mask = sm.ring[slot].mask;
      const int request = sm.ring[slot].request, part = sm.ring[slot].part;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_free[slot]);
      if (!warp_wait(&sm.s_full[buf], (i / 2) & 1)) break;
      tmem_fence_after();
      uint32_t x[32];
      tmem_ld_16x64(tmem + lanes + kTmemS + buf * kTile, x);
      tmem_wait_ld();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.s_free[buf]);
      // log2-scaled scores, -inf where there is no entry
      float top[2] = {-INFINITY, -INFINITY};
      const uint64_t bits = mask >> (2 * (lane & 3));
#pragma unroll
      for (int g = 0; g < 8; ++g) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool in = (bits >> (8 * g + (k & 1))) & 1;
          const float t = in ? __uint_as_float(x[4 * g + k]) * c2 : -INFINITY;
          x[4 * g + k] = __float_as_uint(t);
          top[k >> 1] = fmaxf(top[k >> 1], t);
        }
      }
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], 1));
        top[a] = fmaxf(top[a], __shfl_xor_sync(0xffffffffu, top[a], 2));
      }
      if (flags & kFirst) {
        m[0] = top[0], m[1] = top[1];
        l[0] = l[1] = 0.f;
      } else if (!soft_sync(active && (top[0] > m[0] + kSlack || top[1] > m[1] + kSlack))) {
        break;
      } else if (any) {
        // raise the references of all heads, and O and the sums with them
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const float to = fmaxf(m[a], top[a]);
          const float f = to == -INFINITY ? 1.f : ex2_approx(m[a] - to);
          m[a] = to;
          l[a] *= f;
          if ((lane & 3) == 0) sm.factor[a == 0 ? h0 : h1] = f;
        }
        if (!soft_sync(false)) break;
        if (!warp_wait(&sm.pv_done[(i - 1) & 1], ((i - 1) / 2) & 1)) break;
        tmem_fence_after();
        for (int mt = 0; mt < 4; ++mt) {
          for (int h = 0; h < heads16; h += 16) {
            uint32_t o[16];
            const uint32_t at = tmem + lanes + mt * kGroup + h;
            tmem_ld_32x16(at, o);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sm.factor[h + k]);
            tmem_st_32x16(at, o);
          }
        }
        tmem_wait_st();
        tmem_fence_before();
      }
      const float shift[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
      if (i >= 2 && !warp_wait(&sm.pv_done[buf], (i / 2 - 1) & 1)) break;  // the P of two tiles ago has been used
      if (active) {
        const uint32_t p_at = smem_addr(sm.p[buf]) + 4 * (lane & 3);
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          float e[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            e[k] = ex2_approx(__uint_as_float(x[4 * g + k]) - shift[k >> 1]);
            l[k >> 1] += e[k];
          }
          const uint32_t at = static_cast<uint32_t>((g ^ (h0 & 7)) << 4);  // h1 & 7 == h0 & 7
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_at + h0 * 128 + at), "r"(pack_bf16x2(e[0], e[1])) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(p_at + h1 * 128 + at), "r"(pack_bf16x2(e[2], e[3])) : "memory");
        }
        async_proxy_fence();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[buf]);
      if (!(flags & kLast)) continue;

      // ---------------------------------------------------------------------- the run's result
      const bool whole = part < 0;
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        l[a] += __shfl_xor_sync(0xffffffffu, l[a], 1);
        l[a] += __shfl_xor_sync(0xffffffffu, l[a], 2);
        const int h = a == 0 ? h0 : h1;
        const int64_t head = group * kGroup + h;
        if ((lane & 3) == 0) {
          float sum = l[a], to = shift[a], f = 1.f;
          if (whole && p.sink != nullptr && h < heads) {  // one more score, with a value of zero
            const float s = __ldg(p.sink + head) * kLog2e;
            to = fmaxf(m[a], s);
            to = to == -INFINITY ? 0.f : to;
            f = ex2_approx(shift[a] - to);
            sum = sum == 0.f ? ex2_approx(s - to) : sum * f + ex2_approx(s - to);
          }
          sm.inv[h] = l[a] == 0.f ? 0.f : f / sum;
          if (h < heads) {
            const float lse2 = sum == 0.f ? -INFINITY : to + log2f(sum);
            if (!whole)
              reinterpret_cast<float*>(p.workspace + scratch.lse_at())[scratch.row(part, group, h)] = lse2;
            else if (p.lse != nullptr)
              p.lse[request * p.lse_stride_r + head * p.lse_stride_h] = lse2 * 0.69314718055994531f;
          }
        }
      }
      if (!soft_sync(false)) break;
      if (!warp_wait(&sm.pv_done[buf], (i / 2) & 1)) break;
      tmem_fence_after();
      for (int mt = 0; mt < 4; ++mt) {
        const int col = mt * 128 + 32 * w + lane;
        for (int h = 0; h < heads; h += 16) {
          uint32_t o[16];
          tmem_ld_32x16(tmem + lanes + mt * kGroup + h, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sm.inv[h + k]);
          if (!whole) {
            float* dst = reinterpret_cast<float*>(p.workspace + scratch.out_at()) + scratch.row(part, group, h) * kHead + col;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (h + k < heads) dst[k * kHead] = __uint_as_float(o[k]);
          } else if (p.out_f32) {
            float* dst = static_cast<float*>(p.out) + request * p.out_stride_r + (group * kGroup + h) * p.out_stride_h + col;
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (h + k < heads) dst[k * p.out_stride_h] = __uint_as_float(o[k]);
          } else {
            // neighbouring lanes swap halves of a pair of heads, so that each stores two columns of one
            uint16_t* dst = static_cast<uint16_t*>(p.out) + request * p.out_stride_r +
                            (group * kGroup + h + (lane & 1)) * p.out_stride_h + (col & ~1);
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const float mine_ = __uint_as_float(lane & 1 ? o[k + 1] : o[k]);
              const float other = __shfl_xor_sync(0xffffffffu, __uint_as_float(lane & 1 ? o[k] : o[k + 1]), 1);
              if (h + k + (lane & 1) < heads)
                *reinterpret_cast<uint32_t*>(dst + k * p.out_stride_h) = lane & 1 ? pack_bf16x2(other, mine_) : pack_bf16x2(mine_, other);
            }
          }
        }
      }
      tmem_fence_before();
      if (!soft_sync(false)) break;  // sm.inv is free again
      if (lane == 0) mbar_arrive(&sm.o_free);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------------- join the partial results
// One warp per (cut request, head, quarter of the columns): out = sum_k 2^(lse_k - L) part_k.
constexpr int kJoinThreads = 256;
constexpr int kMaxColumns = 1024;

__global__ void __launch_bounds__(kJoinThreads) join_kernel(const DecodeParams p, const Scratch scratch) {
  __shared__ int s_owner[kMaxColumns];
  __shared__ int s_count;
  grid_dependency_wait();
  const Task* tasks = reinterpret_cast<const Task*>(p.workspace);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {  // the columns that start a cut request, in order
    int count = 0;
    for (int c0 = 0; c0 < scratch.columns; c0 += 32) {
      const bool has = c0 + lane < scratch.columns && tasks[c0 + lane].parts > 0;
      const unsigned vote = __ballot_sync(0xffffffffu, has);
      if (has) s_owner[count + __popc(vote & ((1u << lane) - 1))] = c0 + lane;
      count += __popc(vote);
    }
    if (lane == 0) s_count = count;
  }
  __syncthreads();
  const int64_t items = static_cast<int64_t>(s_count) * p.heads * 4;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * (kJoinThreads / 32) + warp; item < items;
       item += static_cast<int64_t>(gridDim.x) * (kJoinThreads / 32)) {
    const int quarter = static_cast<int>(item & 3);
    const int64_t head = (item >> 2) % p.heads;
    const int column = s_owner[(item >> 2) / p.heads];
    const Task t = tasks[column];
    const int group = static_cast<int>(head / kGroup), h = static_cast<int>(head % kGroup);
    const float* lse = reinterpret_cast<const float*>(p.workspace + scratch.lse_at());
    const float* part = reinterpret_cast<const float*>(p.workspace + scratch.out_at());
    auto row = [&](int k) { return scratch.row(k == 0 ? 2 * column + 1 : 2 * (column + k), group, h); };
    float top = -INFINITY;
    bool nan = false;
    for (int k = lane; k < t.parts; k += 32) {
      const float v = lse[row(k)];
      nan |= v != v;
      top = fmaxf(top, v);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    nan = __any_sync(0xffffffffu, nan);
    const float sink = p.sink != nullptr ? __ldg(p.sink + head) * kLog2e : -INFINITY;
    top = fmaxf(top, sink);
    const float shift = top == -INFINITY ? 0.f : top;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = p.sink != nullptr ? ex2_approx(sink - shift) : 0.f;
    constexpr int kFlight = 8;
    for (int k0 = 0; k0 < t.parts; k0 += kFlight) {
      float4 v[kFlight];
      float w[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        w[k] = 0.f;
        v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < t.parts) {
          const int64_t at = row(k0 + k);
          w[k] = ex2_approx(lse[at] - shift);
          v[k] = *reinterpret_cast<const float4*>(part + at * kHead + 128 * quarter + 4 * lane);
        }
      }
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        sum += w[k];
        acc.x = fmaf(w[k], v[k].x, acc.x), acc.y = fmaf(w[k], v[k].y, acc.y);
        acc.z = fmaf(w[k], v[k].z, acc.z), acc.w = fmaf(w[k], v[k].w, acc.w);
      }
    }
    if (nan) sum = NAN;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t at = t.request * p.out_stride_r + head * p.out_stride_h + 128 * quarter + 4 * lane;
    if (p.out_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.out) + at) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + at) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (p.lse != nullptr && quarter == 0 && lane == 0)
      p.lse[t.request * p.lse_stride_r + head * p.lse_stride_h] =
          sum == 0.f ? -INFINITY : (shift + log2f(sum)) * 0.69314718055994531f;
  }
}

constexpr int kDecodeSmemBytes = sizeof(DecodeSmem) + 1024;
static_assert(kDecodeSmemBytes <= 232448, "shared memory of one SM, with its alignment");

// The queries as [512, heads, requests]; a box is 64 columns of `box` heads of one request.
bool encode_query_map(const DecodeParams& p, int box, CUtensorMap* map) {
  const cuuint64_t dims[3] = {kHead, static_cast<cuuint64_t>(p.heads), static_cast<cuuint64_t>(p.requests)};
  // the stride of a dimension with one index does not matter but has to be valid
  const cuuint64_t strides[2] = {p.heads > 1 ? static_cast<cuuint64_t>(p.q_stride_h) * 2 : kHead * 2,
                                 p.requests > 1 ? static_cast<cuuint64_t>(p.q_stride_r) * 2 : kHead * 2};
  const cuuint32_t size[3] = {64, static_cast<cuuint32_t>(box), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  auto enc = tensor_map_encoder();
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, size, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t prepare_decode() {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const cudaError_t e = cudaFuncSetAttribute(decode_kernel<true>, a, kDecodeSmemBytes);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(decode_kernel<false>, a, kDecodeSmemBytes);
}

int64_t decode_workspace_bytes(int heads, int sm_count) { return Scratch(heads, sm_count).bytes(); }

cudaError_t launch_decode(const DecodeParams& p, int sm_count, cudaStream_t stream) {
  const Scratch scratch(p.heads, sm_count);
  const int box = p.heads < kGroup ? p.heads : kGroup;
  CUtensorMap map;
  if (!encode_query_map(p, box, &map)) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(scratch.columns * scratch.groups);
  const bool align16 = p.kc_stride0 % 16 == 0;  // records then start on 16 bytes, else on 8
  if (align16) decode_kernel<true><<<grid, kDecodeThreads, kDecodeSmemBytes, stream>>>(p, map, scratch, box);
  else decode_kernel<false><<<grid, kDecodeThreads, kDecodeSmemBytes, stream>>>(p, map, scratch, box);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t cut = p.requests < scratch.columns ? p.requests : scratch.columns;  // requests that can be cut
  const int64_t ctas = (cut * p.heads * 4 + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(ctas < 8 * sm_count ? ctas : 8 * sm_count));
  lc.blockDim = dim3(kJoinThreads);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  return cudaLaunchKernelEx(&lc, join_kernel, p, scratch);
}

}  // namespace c128
