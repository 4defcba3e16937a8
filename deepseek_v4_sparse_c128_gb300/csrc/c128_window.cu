// c128_window_attention where what a token sees fits into shared memory: a CTA walks consecutive tokens and keeps
// their entries decoded there, so that each entry is decoded once for all of them.
//
//   S^T = K Q^T            M = 128 entries (and the rest of them), N = rows, K = 512
//   P^T = exp2(c S^T - m)  c = scale * log2(e), m the row's largest c S^T
//   O^T = K^T P^T          M = 128 columns (4 times), N = rows, K = entries
//   out = O / sum(P as the products see it, rounded to bf16); lse = of the exact sums, in fp32
//
// An entry is key and value: both products read it as their A, with the 512 columns along K, and with them along M. An
// item is a token with its heads (up to 64 rows, padded to eights), or as many consecutive tokens as 64 rows hold. Entries
// have kSlots places of 1 KB (bf16): the `first` ones keep theirs, those behind go around a ring, where a new entry takes
// the place of one that no token sees any more. A run (consecutive positions of one request) begins with all that its
// first item sees; then an item brings an entry for each of its tokens.
//
// What bounds a run is the queries and results, 2 KB a row, and next the tensor cores' reads of shared memory: an item of
// 64 rows takes them about 3,300 cycles. So the products of one item cover what lies between those of the next: S of
// item i + 1 is issued before O of item i, whose softmax runs meanwhile; the places of entries are a few more than a token
// sees, so that the entries of item i + 1 do not wait for O of item i either (where they would, `serial` keeps the order).
// A masked entry has weight 0, and 0 times what stands there has to be 0 for every row: so an entry with a value that is
// not finite is stored as zeros and marked, and its scores are NaN for the rows that see it, and for no other.
//
// Roles of the 18 warps (each wait is bounded):
//   0..7   softmax, four warps for either half of the rows; results
//   8..15  decode entries
//   16     one thread issues the products
//   17     makes the items, reads their queries (TMA)
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "c128_step.h"
#include "c128_tensor.cuh"

namespace c128 {
namespace {

constexpr int kSlots = 136;   // entries that shared memory holds
constexpr int kMain = 128;    // of them in the first M of S; the others are its tail
constexpr int kRows = 64;
constexpr int kChunks = kHead / 64;
constexpr int kChunkBytes = kSlots * 128;  // 64 columns of all entries: rows of 128 bytes, one swizzle atom wide
constexpr int kKBytes = kChunks * kChunkBytes;
constexpr int kQChunkBytes = kRows * 128;
constexpr int kPBytes = (kSlots + 8) * 128;  // [entry][row]; K steps of 16 entries end at 144
constexpr int kSoftWarps = 8, kFillWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kFillWarps, kItemWarp = kMmaWarp + 1;
constexpr int kWindowThreads = 32 * (kItemWarp + 1);
constexpr int kRing = 4;      // items that may be on their way
constexpr int kTmemCols = 512, kTmemS = 256, kTmemTail = 320;

enum : int { kEnd = 1, kSerial = 2, kTail = 4, kStepShift = 4 };  // flags of an item; above: K steps of O
enum : uint8_t { kThere = 0, kAbsent = 1, kPoison = 2 };          // what an entry's place holds

struct Item {
  int32_t token, count;     // its first token; tokens
  int32_t row;              // their request's row of the table
  int32_t lo, hi;           // the first token sees entries lo .. hi (and `first` ones), those behind it one more each
  int32_t from, lead, news; // entries to decode: 0 .. lead - 1, and `news` from `from` on
  int32_t ring;             // where on the ring the first of them that goes there goes
  int32_t base, newest;     // the entry at place 0 of the ring when the run began; place of the last entry
  int32_t flags;
};

struct WindowPlan {
  int32_t groups, group_heads;  // head groups, heads of one
  int32_t pitch;                // rows of a token: its heads, padded to eights
  int32_t together;             // tokens of an item, at most
  int32_t columns;              // CTAs that share the tokens
  int32_t lookahead;            // entries of the next item have room beside those of this one
  uint32_t pitch_inv;           // 2^16 / pitch, rounded up
};

struct WindowSmem {
  alignas(1024) uint8_t k[kKBytes];
  alignas(1024) uint8_t zeros[1024];  // where the last K step of the last chunk reads on
  alignas(1024) uint8_t q[kRows * kHead * 2];
  alignas(1024) uint8_t p[kPBytes];
  alignas(16) float by_max[2][4][kRows];         // of even and odd items: 32 entries each
  alignas(16) float sums[2][4][kRows], rounded[2][4][kRows];
  alignas(16) float ref[2][kRows];
  alignas(16) float inv[kRows];
  int64_t at[kRows];                  // where a row's results go, -1: nowhere
  Item ring[kRing];
  uint64_t ring_full[kRing], ring_free[kRing];
  uint64_t k_full[2], o_full[2];      // of even and odd items
  uint64_t set[2];                    // barriers of the softmax warps of either half
  uint64_t q_full, q_free, s_full, s_free, p_full, o_free, drained;
  uint8_t state[kSlots];
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(WindowSmem) <= 232448, "shared memory of one SM");

__device__ __forceinline__ void load_query_rows(void* dst, const CUtensorMap* map, int col, int head, int token, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_addr(dst)),
      "l"(map), "r"(col), "r"(head), "r"(token), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_query_rows(const CUtensorMap* map, int col, int head, int token) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global [%0, {%1, %2, %3}];" ::"l"(map), "r"(col), "r"(head), "r"(token) : "memory");
}

// Values of eight rows in each lane (row 8g + 2 (lane % 4) + e in v[2g + e]) to one, over the eight lanes with the same
// rows: lane / 4's bits choose the row, the highest g's high bit.
template <typename F>
__device__ __forceinline__ float reduce_rows(const float (&v)[8], int lane, F op) {
  float a[4], b[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool hi = lane & 16;
    a[k] = op(hi ? v[k + 4] : v[k], __shfl_xor_sync(0xffffffffu, hi ? v[k] : v[k + 4], 16));
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const bool hi = lane & 8;
    b[k] = op(hi ? a[k + 2] : a[k], __shfl_xor_sync(0xffffffffu, hi ? a[k] : a[k + 2], 8));
  }
  const bool hi = lane & 4;
  return op(hi ? b[1] : b[0], __shfl_xor_sync(0xffffffffu, hi ? b[0] : b[1], 4));
}

// Four threads per entry; thread `sub` has the 16 bytes sub, sub + 4, ...: of the codes a quarter of each 64-column
// chunk, so load j belongs to scale j.
struct Quarter {
  uint4 raw[9];
  uint2 scales;
  template <bool ALIGN16>
  __device__ __forceinline__ void load(const uint8_t* data, const uint8_t* sc, int sub) {
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      if (data == nullptr) raw[j] = make_uint4(0, 0, 0, 0);
      else raw[j] = ALIGN16 ? ld16(data + 16 * sub + 64 * j) : ld8x2(data + 16 * sub + 64 * j);
    }
    scales = data == nullptr ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu) : ld8(sc);
  }
  __device__ __forceinline__ float scale(int j) const { return scale_of(((j < 4 ? scales.x : scales.y) >> (8 * (j & 3))) & 0xffu); }
  // Chunk j as bf16
  __device__ __forceinline__ void decode(int j, uint32_t (&o)[8]) const {
    const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
    const float s = scale(j);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[2 * k] = codes_to_bf16(static_cast<uint16_t>(w[k]), s);
      o[2 * k + 1] = codes_to_bf16(static_cast<uint16_t>(w[k] >> 16), s);
    }
  }
  // Whether a value is not finite: a code of NaN, a bf16 or (scales from 2^120 on) a product without room.
  __device__ __forceinline__ bool not_finite() const {
    uint32_t codes = 0, halves = 0, large = 0;
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) codes |= (w[k] & 0x7f7f7f7fu) + 0x01010101u;
      large |= (((j < 4 ? scales.x : scales.y) >> (8 * (j & 3))) & 0xffu) >= 247u;
    }
#pragma unroll
    for (int j = 7; j < 9; ++j) {
      const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) halves |= (w[k] & 0x7fff7fffu) + 0x00800080u;
    }
    if (large) {
#pragma unroll 1
      for (int j = 0; j < 7; ++j) {
        uint32_t o[8];
        uint4 r = raw[0];
#pragma unroll
        for (int i = 1; i < 7; ++i)
          if (i == j) r = raw[i];
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[2 * k] = codes_to_bf16(static_cast<uint16_t>(w[k]), scale(j));
          o[2 * k + 1] = codes_to_bf16(static_cast<uint16_t>(w[k] >> 16), scale(j));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) halves |= (o[k] & 0x7fff7fffu) + 0x00800080u;
      }
    }
    return ((codes & 0x80808080u) | (halves & 0x80008000u)) != 0;
  }
};

template <bool ALIGN16>
__global__ void __launch_bounds__(kWindowThreads, 1)
    window_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ WindowPlan plan) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  WindowSmem& sm = *reinterpret_cast<WindowSmem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int column = blockIdx.x / plan.groups, group = blockIdx.x - column * plan.groups;
  const int head0 = group * plan.group_heads, heads = min(plan.group_heads, p.heads - head0);
  const int first = p.first, circle = kSlots - first, window = static_cast<int>(p.window);
  const int rows = plan.together > 1 ? plan.together * plan.pitch : heads;
  const int rows16 = (rows + 15) & ~15;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.ring_full[i], 1);
      mbar_init(&sm.ring_free[i], kSoftWarps + kFillWarps + 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.k_full[i], kFillWarps);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, kSoftWarps);
    mbar_init(&sm.p_full, kSoftWarps);
    mbar_init(&sm.o_free, kSoftWarps);
    mbar_init(&sm.drained, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.set[i], kSoftWarps / 2);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // Places without an entry, and weights of those that there never are, have to be finite from the start.
  for (int i = threadIdx.x; i < (kKBytes + 1024) / 16; i += kWindowThreads) reinterpret_cast<uint4*>(sm.k)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < 1024 / 16; i += kWindowThreads) reinterpret_cast<uint4*>(sm.p + kSlots * 128)[i] = make_uint4(0, 0, 0, 0);
  async_proxy_fence();  // (to the products, behind the barrier below)
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)), "n"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  launch_dependents();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  grid_dependency_wait();  // what the kernels before this one wrote is read from here on
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);
  volatile int* const abort_flag = &sm.abort;
  // A wait of a whole warp; as in the decode attention's kernel, one that runs out sets the abort flag, every wait then
  // returns at once, and the warps run on to the end, which item_flags shows them. No result is stored then.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    if (!decode_wait(bar, parity, abort_flag)) *abort_flag = 1;
    __syncwarp();
  };
  auto item_flags = [&](int i) {
    warp_wait(&sm.ring_full[i % kRing], (i / kRing) & 1);
    const int flags = sm.ring[i % kRing].flags;
    return *abort_flag ? kEnd : flags;
  };
  auto free_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ring_free[i % kRing]);
  };

  if (warp == kItemWarp) {
    // -------------------------------------------------------------------------- items and queries
    const int64_t begin = p.requests * column / plan.columns, end = p.requests * (column + 1) / plan.columns;
    const uint32_t q_bytes = static_cast<uint32_t>(kChunks * plan.together * plan.pitch * 128);
    unsigned int err = 0;
    int64_t batch = begin;  // lanes hold tokens batch .. batch + 31
    int lo = 0, hi = 0, req = 0;
    unsigned live = 0, goes_on = 0;  // tokens that are not skipped; those that follow the one before
    int64_t last_pos = -1;           // of the token before the batch
    int last_req = -1;
    auto load_batch = [&] {
      const int64_t t = batch + lane;
      int64_t pos = -1;
      bool ok = false;
      if (t < end) {
        pos = p.positions[t];
        req = p.token_req[t];
        ok = pos >= 0 && p.slots[t] >= 0;
        if (ok && (req < 0 || req >= p.table_rows)) ok = false, err |= C128_DEV_BAD_REQ;
        if (ok && pos >= p.most) err |= C128_DEV_BAD_BT_COL;
      }
      if (!ok) pos = -1;
      hi = static_cast<int>(min(pos, static_cast<int64_t>(p.most) - 1));
      lo = static_cast<int>(min(max(pos + 1 - window, static_cast<int64_t>(0)), static_cast<int64_t>(p.most)));
      int64_t pos_before = __shfl_up_sync(0xffffffffu, pos, 1);
      int req_before = __shfl_up_sync(0xffffffffu, req, 1);
      if (lane == 0) pos_before = last_pos, req_before = last_req;
      live = __ballot_sync(0xffffffffu, ok);
      goes_on = __ballot_sync(0xffffffffu, ok && pos_before >= 0 && pos == pos_before + 1 && req == req_before && pos < p.most);
      last_pos = __shfl_sync(0xffffffffu, pos, 31);
      last_req = __shfl_sync(0xffffffffu, req, 31);
    };
    if (begin < end) load_batch();
    int base = 0, newest = -1, seen_to = -1;  // the run's
    bool stalled = p.stall && blockIdx.x == 0;
    int i = 0, loads = 0;
    int64_t t = begin;
    for (; !stalled; ++i) {
      while (t < end) {  // the next token that is not skipped
        if (t - batch >= 32) {
          batch += 32;
          load_batch();
        }
        const unsigned rest = live >> (t - batch);
        if (rest != 0) {
          t += __ffs(rest) - 1;
          break;
        }
        t = batch + 32;
      }
      const int slot = i % kRing;
      if (i >= kRing) warp_wait(&sm.ring_free[slot], (i / kRing - 1) & 1);
      if (t >= end || *abort_flag) {
        if (lane == 0) {
          sm.ring[slot].flags = kEnd;
          mbar_arrive(&sm.ring_full[slot]);
        }
        break;
      }
      const int j = static_cast<int>(t - batch);
      const unsigned behind = ~(j < 31 ? goes_on >> (j + 1) : 0u);
      const int count = min(__ffs(behind), plan.together);
      Item it;
      it.token = static_cast<int>(t);
      it.count = count;
      it.row = __shfl_sync(0xffffffffu, req, j);
      it.lo = __shfl_sync(0xffffffffu, lo, j);
      it.hi = __shfl_sync(0xffffffffu, hi, j);
      const int last = it.hi + count - 1;
      const bool fresh = i == 0 || !(goes_on >> j & 1);
      if (fresh) {
        it.lead = min(first, it.lo);
        it.from = it.lo;
        base = max(first, it.lo);
        it.ring = 0;
        newest = max(last - base, -1);  // (-1: the ring is empty)
      } else {
        it.lead = 0;
        it.from = seen_to + 1;
        it.ring = it.from < first ? 0 : newest + 1 == circle ? 0 : newest + 1;
        newest += last - max(it.from, first) + 1 > 0 ? last - max(it.from, first) + 1 : 0;
        if (newest >= circle) newest -= circle;
      }
      it.news = max(last - it.from + 1, 0);
      it.base = base;
      it.newest = newest;
      seen_to = last;
      const int used = last >= base ? first + min(last - base + 1, circle) : min(first, last + 1);
      it.flags = (fresh || !plan.lookahead ? kSerial : 0) | (used > kMain ? kTail : 0) | max((used + 15) / 16, 1) << kStepShift;
      if (lane == 0) {
        sm.ring[slot] = it;
        mbar_arrive(&sm.ring_full[slot]);
        if (i > 0)
          for (int c = 0; c < kChunks; ++c) prefetch_query_rows(&q_map, 64 * c, head0, it.token);
      }
      __syncwarp();
      t += count;
      // its queries, when S of the item before has been taken
      if (i > 0) warp_wait(&sm.q_free, (i - 1) & 1);
      if (*abort_flag) break;
      loads = i + 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.q_full, q_bytes);
        for (int c = 0; c < kChunks; ++c) load_query_rows(sm.q + c * kQChunkBytes, &q_map, 64 * c, head0, it.token, &sm.q_full);
      }
      __syncwarp();
    }
    if (err) atomicOr(p.err, err);
    if (loads > 0) decode_wait(&sm.q_full, (loads - 1) & 1, nullptr);  // nothing may be in flight when the CTA ends
    __syncwarp();
  } else if (warp >= kSoftWarps && warp < kMmaWarp) {
    // ------------------------------------------------------------------------ decode the entries
    const int sub = lane & 3, mine = 8 * (warp - kSoftWarps) + (lane >> 2);
    const uint32_t k_at = smem_addr(sm.k);
    const Divisor bs = p.kv_div;
    unsigned int err = 0;
    for (int i = 0;; ++i) {
      const int flags = item_flags(i);
      if (flags & kEnd) break;
      const Item it = sm.ring[i % kRing];
      free_item(i);
      const int all = it.lead + it.news;
      bool waited = false;
      for (int e0 = 0; e0 < all || !waited; e0 += 8 * kFillWarps) {
        const int e = e0 + mine;
        const bool in = e < all;
        const int entry = e < it.lead ? e : it.from + e - it.lead;
        const uint8_t* data = nullptr;
        const uint8_t* sc = nullptr;
        if (in) {
          const uint32_t block = divide(entry, bs), off = entry - block * bs.value;
          const int id = __ldcg(p.table + it.row * p.table_stride + block);
          if (id >= 0 && id < p.nkb) {
            const uint8_t* blk = p.kc + static_cast<int64_t>(id) * p.kc_stride0;
            data = blk + static_cast<int64_t>(off) * kTokenStride;
            sc = blk + p.kv_bs * kTokenStride + static_cast<int64_t>(off) * kScaleDim;
          } else {
            err |= C128_DEV_BAD_BLOCK;
          }
        }
        Quarter x;
        x.load<ALIGN16>(data, sc, sub);
        bool poison = x.not_finite();
        poison |= __shfl_xor_sync(0xffffffffu, static_cast<int>(poison), 1) != 0;
        poison |= __shfl_xor_sync(0xffffffffu, static_cast<int>(poison), 2) != 0;
        if (!waited) {  // the places are free
          if (i > 0 && (flags & kSerial)) warp_wait(&sm.o_full[(i - 1) & 1], ((i - 1) >> 1) & 1);
          else if (i > 1) warp_wait(&sm.o_full[i & 1], ((i - 2) >> 1) & 1);
          waited = true;
        }
        if (in) {
          int place = entry;
          if (entry >= first) {
            place = it.ring + entry - max(it.from, first);
            place = first + (place >= circle ? place - circle : place);
          }
          if (sub == 0) sm.state[place] = data == nullptr ? kAbsent : poison ? kPoison : kThere;
          const uint32_t row = k_at + place * 128, swz = static_cast<uint32_t>(place & 7) << 4;
          const uint32_t dst0 = row + ((32u * sub) ^ swz), dst1 = row + ((32u * sub + 16u) ^ swz), dst_rope = row + 7 * kChunkBytes + ((16u * sub) ^ swz);
#pragma unroll
          for (int j = 0; j < 7; ++j) {
            uint32_t o[8];
            x.decode(j, o);
            if (poison) {
#pragma unroll
              for (int k = 0; k < 8; ++k) o[k] = 0;
            }
            sts16(dst0 + j * kChunkBytes, o[0], o[1], o[2], o[3]);
            sts16(dst1 + j * kChunkBytes, o[4], o[5], o[6], o[7]);
          }
          if (poison) x.raw[7] = x.raw[8] = make_uint4(0, 0, 0, 0);
          sts16(dst_rope, x.raw[7].x, x.raw[7].y, x.raw[7].z, x.raw[7].w);
          sts16(dst_rope ^ 64u, x.raw[8].x, x.raw[8].y, x.raw[8].z, x.raw[8].w);
        }
        __syncwarp();
      }
      async_proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.k_full[i & 1]);
    }
    if (err) atomicOr(p.err, err);
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------------ issue the products
    if (elect_one()) {
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (decode_wait(bar, parity, abort_flag)) return true;
        *abort_flag = 1;
        return false;
      };
      const uint32_t q_at = desc_low(smem_addr(sm.q), 16), ks_at = desc_low(smem_addr(sm.k), 16);
      const uint32_t kv_at = desc_low(smem_addr(sm.k), kChunkBytes), p_at = desc_low(smem_addr(sm.p), 16);
      const uint32_t desc_s = mma_desc(kMain, rows16, false), desc_tail = mma_desc(64, rows16, false), desc_o = mma_desc(128, rows16, true);
      auto product_s = [&](uint32_t d, uint32_t row0, uint32_t desc) {
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma(d, desc64(ks_at + ((row0 * 128 + c * kChunkBytes + ks * 32) >> 4)), desc64(q_at + ((c * kQChunkBytes + ks * 32) >> 4)), desc, c + ks > 0);
        }
      };
      auto product_o = [&](int i, int steps) {  // of item i
        if (!wait(&sm.p_full, i & 1)) return false;
        if (i > 0 && !wait(&sm.o_free, (i - 1) & 1)) return false;
        tmem_fence_after();
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll 1
          for (int ks = 0; ks < steps; ++ks)
            mma(tmem + mt * kRows, desc64(kv_at + ((2 * mt * kChunkBytes + ks * 2048) >> 4)), desc64(p_at + (ks * 2048 >> 4)), desc_o, ks > 0);
        }
        mma_commit(&sm.o_full[i & 1]);
        return true;
      };
      int steps = 0;
      for (int i = 0;; ++i) {
        const int slot = i % kRing;
        if (!wait(&sm.ring_full[slot], (i / kRing) & 1)) break;
        const int flags = sm.ring[slot].flags;
        mbar_arrive(&sm.ring_free[slot]);
        if (i > 0 && (flags & (kEnd | kSerial)) && !product_o(i - 1, steps)) break;
        if (flags & kEnd) break;
        if (!wait(&sm.q_full, i & 1) || !wait(&sm.k_full[i & 1], (i >> 1) & 1)) break;
        if (i > 0 && !wait(&sm.s_free, (i - 1) & 1)) break;
        tmem_fence_after();
        product_s(tmem + kTmemS, 0, desc_s);
        if (flags & kTail) product_s(tmem + kTmemTail, kMain, desc_tail);
        mma_commit(&sm.s_full);
        mma_commit(&sm.q_free);
        if (i > 0 && !(flags & kSerial) && !product_o(i - 1, steps)) break;
        steps = flags >> kStepShift;
      }
      mma_commit(&sm.drained);
      decode_wait(&sm.drained, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------- softmax and results
    const int w = warp & 3, set = warp >> 2, own = 32 * set;  // TMEM lanes 32w .., rows own .. own + 31
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const int r0 = own + 2 * (lane & 3);                      // this thread's rows: r0 and r0 + 1, and on in steps of 8
    const int reduced = own + 8 * (lane >> 4 << 1 | (lane >> 3 & 1)) + 2 * (lane & 3) + (lane >> 2 & 1);  // reduce_rows' row
    const float c2 = p.scale * kLog2e;
    const bool busy = own < rows16;
    uint32_t set_phase = 0;
    auto set_sync = [&] {  // bounded, as every wait: a warp that has seen the abort flag does not come
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.set[set]);
      warp_wait(&sm.set[set], set_phase);
      set_phase ^= 1;
    };
    // the results of item i
    auto results = [&](int i) {
      warp_wait(&sm.o_full[i & 1], (i >> 1) & 1);
      const Item& it = sm.ring[i % kRing];
      if (busy && !*abort_flag) {
        tmem_fence_after();
        const int row = own + lane, token = static_cast<int>(row * plan.pitch_inv >> 16), h = row - token * plan.pitch;
        const bool there = token < it.count && h < heads;
        const float (&s)[4][kRows] = sm.sums[i & 1];
        const float (&r)[4][kRows] = sm.rounded[i & 1];
        const float own_sum = (s[0][row] + s[1][row]) + (s[2][row] + s[3][row]);
        const float rounded = (r[0][row] + r[1][row]) + (r[2][row] + r[3][row]), ref = sm.ref[i & 1][row];
        float sum = own_sum, to = ref, share = own_sum == 0.f ? 0.f : 1.f;
        if (p.sink != nullptr && there) {  // one more score, with a value of zero
          const float sink = __ldcg(p.sink + head0 + h) * kLog2e;
          to = own_sum == 0.f ? (sink == -INFINITY ? 0.f : sink) : fmaxf(ref, sink);
          const float entries = own_sum == 0.f ? 0.f : own_sum * ex2_approx(ref - to);
          sum = entries + ex2_approx(sink - to);
          if (own_sum != 0.f) share = entries / sum;
        }
        // (the four warps of a set write the same)
        sm.inv[row] = share == 0.f ? 0.f : share / rounded;
        const int64_t out_token = static_cast<int64_t>(it.token) + token;
        sm.at[row] = there ? out_token * p.out_stride_r + (head0 + h) * p.out_stride_h : -1;
        if (w == 0 && there && p.lse != nullptr)
          p.lse[out_token * p.lse_stride_r + (head0 + h) * p.lse_stride_h] =
              sum == 0.f ? -INFINITY : (to + log2f(sum)) * 0.69314718055994531f;
        __syncwarp();
#pragma unroll 1
        for (int part = 0; part < 8; ++part) {  // 16 rows of 128 columns each
          const int mt = part >> 1, row0 = own + 16 * (part & 1);
          if (row0 >= rows) continue;
          uint32_t o[16];
          tmem_ld_32x16(tmem + lanes + mt * kRows + row0, o);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            const float4 f = *reinterpret_cast<const float4*>(&sm.inv[row0 + k]);
            o[k] = __float_as_uint(__uint_as_float(o[k]) * f.x), o[k + 1] = __float_as_uint(__uint_as_float(o[k + 1]) * f.y);
            o[k + 2] = __float_as_uint(__uint_as_float(o[k + 2]) * f.z), o[k + 3] = __float_as_uint(__uint_as_float(o[k + 3]) * f.w);
          }
          const int col = mt * 128 + 32 * w + lane;
          if (p.out_f32) {
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int64_t at = sm.at[row0 + k];
              if (at >= 0) static_cast<float*>(p.out)[at + col] = __uint_as_float(o[k]);
            }
          } else {
            // neighbouring lanes swap halves of a pair of rows, so that each stores two columns of one
            const uint32_t halves = lane & 1 ? 0x3276 : 0x5410;
#pragma unroll
            for (int k = 0; k < 16; k += 2) {
              const uint32_t two = pack_bf16x2(__uint_as_float(o[k]), __uint_as_float(o[k + 1]));
              const uint32_t both = __byte_perm(two, __shfl_xor_sync(0xffffffffu, two, 1), halves);
              const int64_t at = sm.at[row0 + k + (lane & 1)];
              if (at >= 0) *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + at + (col & ~1)) = both;
            }
          }
        }
        tmem_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_free);
      free_item(i);
    };

    int i = 0;
    for (;; ++i) {
      const int flags = item_flags(i);
      if (flags & kEnd) break;
      const Item& it = sm.ring[i % kRing];
      const bool serial = flags & kSerial, tail = (flags & kTail) && w == 0;
      if (i > 0 && serial) {
        warp_wait(&sm.p_full, (i - 1) & 1);  // (its sums are all there)
        results(i - 1);
      }
      // What this thread's entries are: their position, or out of sight (a position behind all). The tail's are 128 ..
      // 135, in the first 16 lanes of TMEM.
      int pos[5];
      bool poison[5];
      const int last = it.hi + it.count - 1;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        const int place = k < 4 ? 32 * w + 8 * k + (lane >> 2) : kMain + (lane >> 2);
        int d = it.newest - (place - first);
        if (d < 0) d += circle;
        pos[k] = place < first ? place : last - d;
        if (place >= first && pos[k] < it.base) pos[k] = 0x7fffffff;
        // (what other items' entries leave there is not looked at: their positions are out of sight)
        poison[k] = false;
      }
      // Rows of one group of 8 are of one token; its lowest and highest entry.
      int lo[4], hi[4];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int token = static_cast<int>((own + 8 * g) * plan.pitch_inv >> 16);
        hi[g] = it.hi + token;
        lo[g] = token == 0 ? it.lo : max(hi[g] - window + 1, 0);
      }
      warp_wait(&sm.s_full, i & 1);
      tmem_fence_after();
      if (busy) {
        bool any_poison = false;
#pragma unroll
        for (int k = 0; k < 5; ++k) {
          const int place = k < 4 ? 32 * w + 8 * k + (lane >> 2) : kMain + (lane >> 2);
          const uint8_t state = sm.state[place];
          if (state == kAbsent) pos[k] = 0x7fffffff;
          poison[k] = state == kPoison;
          any_poison |= poison[k];
        }
        uint32_t x[2][16], y[16];
        tmem_ld_scores<32>(tmem + lanes + kTmemS + own, x[0]);
        tmem_ld_scores<32>(tmem + lanes + (16u << 16) + kTmemS + own, x[1]);
        if (tail) tmem_ld_scores<32>(tmem + lanes + kTmemTail + own, y);
        tmem_wait_ld();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free);
        // v[k][2g + e]: entry k, row r0 + 8g + e; -inf where the row does not see the entry
        float v[5][8], top[8];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
#pragma unroll
          for (int k = 0; k < 5; ++k) {
            const bool sees = pos[k] <= hi[g] && (pos[k] >= lo[g] || pos[k] < first) && (k < 4 || tail);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float s = __uint_as_float(k < 4 ? x[k >> 1][4 * g + 2 * (k & 1) + e] : y[4 * g + e]);
              v[k][2 * g + e] = sees ? __fmul_rn(s, c2) : -INFINITY;
              if (any_poison && poison[k] && sees) v[k][2 * g + e] = NAN;
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(fmaxf(v[0][2 * g + e], v[1][2 * g + e]), fmaxf(v[2][2 * g + e], v[3][2 * g + e]));
            top[2 * g + e] = fmaxf(m, v[4][2 * g + e]);
          }
        }
        sm.by_max[i & 1][w][reduced] = reduce_rows(top, lane, [](float a, float b) { return fmaxf(a, b); });
        set_sync();
        float sum[8], rounded[8];
        uint32_t packed[5][4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float2 m[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) m[k] = *reinterpret_cast<const float2*>(&sm.by_max[i & 1][k][r0 + 8 * g]);
          float ref[2] = {fmaxf(fmaxf(m[0].x, m[1].x), fmaxf(m[2].x, m[3].x)), fmaxf(fmaxf(m[0].y, m[1].y), fmaxf(m[2].y, m[3].y))};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (ref[e] == -INFINITY) ref[e] = 0.f;
            sum[2 * g + e] = rounded[2 * g + e] = 0.f;
          }
          if (w == 0 && lane < 4) *reinterpret_cast<float2*>(&sm.ref[i & 1][r0 + 8 * g]) = make_float2(ref[0], ref[1]);
#pragma unroll
          for (int k = 0; k < 5; ++k) {
            const float a = ex2_approx(__fsub_rn(v[k][2 * g], ref[0])), b = ex2_approx(__fsub_rn(v[k][2 * g + 1], ref[1]));
            packed[k][g] = pack_bf16x2(a, b);
            sum[2 * g] += a, sum[2 * g + 1] += b;
            rounded[2 * g] += __uint_as_float(packed[k][g] << 16), rounded[2 * g + 1] += __uint_as_float(packed[k][g] & 0xffff0000u);
          }
        }
        const float sum1 = reduce_rows(sum, lane, [](float a, float b) { return a + b; });
        const float rounded1 = reduce_rows(rounded, lane, [](float a, float b) { return a + b; });
        // the weights of the item before have been used
        if (i > 0) {
          warp_wait(&sm.o_full[(i - 1) & 1], ((i - 1) >> 1) & 1);
          warp_wait(&sm.p_full, (i - 1) & 1);  // (and its sums are all there)
        }
        sm.sums[i & 1][w][reduced] = sum1;
        sm.rounded[i & 1][w][reduced] = rounded1;
        const uint32_t swz = static_cast<uint32_t>(lane >> 2) << 4;  // of all its entries
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t at = smem_addr(sm.p) + (32 * w + (lane >> 2)) * 128 + 4 * (lane & 3) + ((16u * (own / 8 + g)) ^ swz);
#pragma unroll
          for (int k = 0; k < 4; ++k) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + k * 1024), "r"(packed[k][g]) : "memory");
          if (w == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + kMain * 128), "r"(packed[4][g]) : "memory");
        }
        async_proxy_fence();
      } else {
        if (lane == 0) mbar_arrive(&sm.s_free);
        if (i > 0) {
          warp_wait(&sm.o_full[(i - 1) & 1], ((i - 1) >> 1) & 1);
          warp_wait(&sm.p_full, (i - 1) & 1);
        }
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full);
      if (i > 0 && !serial) results(i - 1);
    }
    if (i > 0) {
      warp_wait(&sm.p_full, (i - 1) & 1);
      results(i - 1);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) atomicOr(p.err, static_cast<unsigned int>(C128_DEV_TIMEOUT));
  if (warp == kMmaWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

const void* window_kernel_for(bool align16) {
  return align16 ? reinterpret_cast<const void*>(window_kernel<true>) : reinterpret_cast<const void*>(window_kernel<false>);
}

// The queries as [512, heads, tokens]; a box is 64 columns of the heads of an item's tokens.
bool encode_query_rows(const DecodeParams& p, const WindowPlan& plan, CUtensorMap* map) {
  const cuuint64_t dims[3] = {kHead, static_cast<cuuint64_t>(p.heads), static_cast<cuuint64_t>(p.requests)};
  const cuuint64_t strides[2] = {p.heads > 1 ? static_cast<cuuint64_t>(p.q_stride_h) * 2 : kHead * 2,
                                 p.requests > 1 ? static_cast<cuuint64_t>(p.q_stride_r) * 2 : kHead * 2};
  const cuuint32_t size[3] = {64, static_cast<cuuint32_t>(plan.pitch), static_cast<cuuint32_t>(plan.together)};
  const cuuint32_t step[3] = {1, 1, 1};
  auto enc = tensor_map_encoder();
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, size, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool window_fits(const DecodeParams& p) { return p.window + p.first <= kSlots; }

cudaError_t prepare_window() {
  cudaError_t e = cudaSuccess;
  for (int align16 = 0; align16 < 2; ++align16)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(window_kernel_for(align16 != 0), cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(WindowSmem));
  return e;
}

cudaError_t launch_window(const DecodeParams& p, int sm_count, cudaStream_t stream) {
  const int64_t T = p.requests;
  WindowPlan plan;
  // Smaller head groups while there are SMs for all of them: the fewer rows, the sooner an item is done.
  int group = kRows;
  while (group > 16 && T * ((p.heads + group / 2 - 1) / (group / 2)) <= sm_count) group /= 2;
  plan.groups = (p.heads + group - 1) / group;
  plan.group_heads = group < p.heads ? group : p.heads;
  plan.pitch = (plan.group_heads + 7) / 8 * 8;
  plan.pitch_inv = (65536 + plan.pitch - 1) / plan.pitch;
  const int room = kSlots - p.first - static_cast<int>(p.window) + 1;  // entries that a run may bring before O is done with those they replace
  int64_t together = plan.groups > 1 ? 1 : kRows / plan.pitch;
  if (together > room) together = room;
  if (together > (T + sm_count - 1) / sm_count) together = (T + sm_count - 1) / sm_count;
  plan.together = static_cast<int32_t>(together);
  plan.lookahead = 2 * plan.together <= room ? 1 : 0;
  const int64_t most = sm_count / plan.groups > 0 ? sm_count / plan.groups : 1;
  plan.columns = static_cast<int32_t>(T < most ? T : most);
  CUtensorMap map;
  if (!encode_query_rows(p, plan, &map)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(plan.columns * plan.groups));
  lc.blockDim = dim3(kWindowThreads);
  lc.dynamicSmemBytes = sizeof(WindowSmem);
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  void* args[] = {const_cast<DecodeParams*>(&p), &map, &plan};
  return cudaLaunchKernelExC(&lc, window_kernel_for(p.kc_stride0 % 16 == 0), args);
}

}  // namespace c128
