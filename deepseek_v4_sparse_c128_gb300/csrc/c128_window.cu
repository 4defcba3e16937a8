// c128_window_attention where what a token sees fits into shared memory: a CTA walks consecutive tokens and keeps
// their entries decoded there, so that each entry is decoded once for all of them.
//
//   S^T = K Q^T            M = 128 entries (and the rest of them), N = rows, K = 512
//   P^T = exp2(c S^T - m) / l   c = scale * log2(e), m the row's largest c S^T, l the sum (and the sink's share)
//   O^T = K^T P^T          M = 128 columns (4 times), N = rows, K = entries; the result (of fp32 results: see below)
//
// An entry is key and value: both products read it as their A, with the 512 columns along K, and with them along M. An
// item is a token with its heads (up to 64 rows, padded to eights), or as many consecutive tokens as 64 rows hold. Entries
// have kSlots places of 1 KB (bf16): the `first` ones keep theirs, those behind go around a ring, where a new entry takes
// the place of one that no token sees any more. A run (consecutive positions of one request) begins with all that its
// first item sees; then an item brings an entry for each of its tokens.
//
// Measured, device time per call: 5,119 tokens of 64 heads, window 128 and 4 first entries, 156 us (as decode attention, token
// by token, 341 us); 200 requests of one token each, 24.2 us; one token 9.2 us. With few heads an item's chain of waits is the
// same, and two tokens at most share one: 16 heads 92 us, 1 head 86.
// The least that a run takes is its queries and results, 2 KB a row (100 us of the 156); next are the tensor cores, which
// work 3,900 of the 8,900 cycles of an item of 64 rows, and the 16,600 instructions of its warps, half the issue slots. No unit
// is full: an item's stages wait for one another, over one set of weights and one O, which is what TMEM's 512 columns
// and shared memory leave room for. So the products of one item cover what lies between those of the next: S of
// item i + 1 is issued before O of item i, whose softmax runs meanwhile; the places of entries are a few more than a token
// sees, so that the entries of item i + 1 do not wait for O of item i either (where they would, `serial` keeps the order).
// A masked entry has weight 0, and 0 times what stands there has to be 0 for every row: so an entry with a value that is
// not finite is stored as zeros and marked, and its scores are NaN for the rows that see it, and for no other.
//
// Weights are rounded to bf16 for the second product (2^-8 of each at most). For bf16 results they are divided by their sum,
// which is in fp32 and of the exact weights, before that: so O is the result, a result of one entry is that entry, and nothing is
// left to do between TMEM and memory but to round and store. For fp32 results they are rounded as they are, the largest 1, and O
// is multiplied by the entries' share of all weight over the sum of the rounded ones (as in decode attention), so that their
// rounding is felt against the other entries' only: the error against 64 bits is 0.0008 instead of 0.0016 (2-norm), the 5,119
// tokens take 180 us instead of 183. bf16 results would be 0.0018 off instead of 0.0023, where their own rounding alone is
// 0.0017, but the factors' loads and the second sums took 172 us instead of 155.
//
// Roles of the 20 warps (five to a scheduler leave them 96 registers; each wait is bounded):
//   0..7   softmax, four warps for either half of the rows
//   8..15  results, four warps for either half of the rows
//          (all of these decode entries at the start of a run, and store the last item's results: one token 9.7 us without that)
//   16     one thread issues the products
//   17     makes the items
//   18     decodes entries
//   19     reads the queries (TMA)
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "c128_step.h"
#include "c128_tensor.cuh"

namespace c128 {
namespace {

constexpr int kSlots = 136;   // entries that shared memory holds, beside 64 rows of queries and weights: 227 KB
constexpr int kMain = 128;    // of them in the first M of S; the others are its tail
constexpr int kRows = 64;
constexpr int kChunks = kHead / 64;
constexpr int kChunkBytes = kSlots * 128;  // 64 columns of all entries: rows of 128 bytes, one swizzle atom wide
constexpr int kKBytes = kChunks * kChunkBytes;
constexpr int kQChunkBytes = kRows * 128;
constexpr int kPBytes = (kSlots + 8) * 128;  // [entry][row]; K steps of 16 entries end at 144
constexpr int kSoftWarps = 8, kOutWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kOutWarps, kItemWarp = kMmaWarp + 1, kDecodeWarp = kMmaWarp + 2, kQueryWarp = kMmaWarp + 3;
constexpr int kHelpers = kSoftWarps + kOutWarps;  // decode entries at the start of a run, beside the decoding warp
static_assert(8 * (kHelpers + 1) >= kSlots, "eight entries each");
constexpr int kWindowThreads = 32 * (kQueryWarp + 1);
constexpr int kRing = 4;      // items that may be on their way
constexpr int kTmemCols = 512, kTmemS = 256, kTmemTail = 320;

enum : int { kEnd = 1, kFresh = 2, kSerial = 4, kTail = 8, kStepShift = 4 };  // flags of an item; above: K steps of O
enum : uint8_t { kThere = 0, kAbsent = 1, kPoison = 2 };          // what an entry's place holds

struct Item {
  int32_t token, count;     // its first token; tokens
  int32_t row;              // their request's row of the table
  int32_t hi, last;         // the first token's position; the last entry that there is for them
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
  int32_t stride;               // from a column's token to its next: 1, or (items of one token) 0, 1 or all columns as the tokens show
  int32_t lookahead;            // an item's entries have room beside those of so many items, itself among them
  uint32_t pitch_inv;           // 2^16 / pitch, rounded up
};

struct WindowSmem {
  alignas(1024) uint8_t k[kKBytes];
  alignas(1024) uint8_t zeros[1024];  // where the last K step of the last chunk reads on
  alignas(1024) uint8_t q[kRows * kHead * 2];
  alignas(1024) uint8_t p[kPBytes];
  alignas(16) float by_warp[3][4][kRows];  // maxima, sums, and sums of rounded weights, of 32 entries each
  alignas(16) float ref[kRows], share[kRows];  // less the largest score; 1 / l
  alignas(16) float factor[kRing][kRows];      // of fp32 results
  Item ring[kRing];
  uint64_t ring_full[kRing], ring_free[kRing];
  uint64_t k_full[kRing], o_full[kRing];
  uint64_t p_full[2];                 // of even and odd items
  uint64_t k_help;                    // the first entries of a run
  uint64_t q_full[2], q_free[2];      // of either half of the columns
  uint64_t set[2];                    // barriers of the softmax warps of either half
  uint64_t o_part[4], o_free[4];      // by 128 columns: O is there; it has been read
  uint64_t s_full, s_free, drained;
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

// The bounded wait of this kernel. Tries that let the thread rest: most warps wait most of the time, and each try passes
// through the shared memory that the products' operands need. Short, since there are many of them.
constexpr uint32_t kTries = 50000;  // of up to 20 us each: about a second
__device__ __forceinline__ bool wait_for(volatile int* abort_flag, uint64_t* bar, uint32_t parity) {
  uint32_t left = kTries;
#pragma unroll 1
  while (!mbar_try_wait_suspend(bar, parity)) {
    if (*abort_flag || --left == 0) return false;
  }
  return true;
}
// Of a whole warp: as in the decode attention's kernel, one that runs out sets the abort flag, every wait then returns at
// once, and the warps run on to the end, which the items' flags show them. No result is stored then.
__device__ __forceinline__ void warp_wait(volatile int* abort_flag, uint64_t* bar, uint32_t parity) {
  if (!wait_for(abort_flag, bar, parity)) *abort_flag = 1;
  __syncwarp();
}

// Where entry e of those that an item brings is in the cache (NULL: nowhere), and its place.
struct Source {
  const uint8_t* data;
  const uint8_t* scales;
  int place;
  __device__ __forceinline__ Source(const DecodeParams& p, const Item& it, int e) : data(nullptr), scales(nullptr) {
    const Divisor bs = p.kv_div;
    const int entry = e < it.lead ? e : it.from + e - it.lead, circle = kSlots - p.first;
    const uint32_t block = divide(entry, bs), off = entry - block * bs.value;
    const int id = __ldcg(p.table + it.row * p.table_stride + block);
    if (id >= 0 && id < p.nkb) {
      const uint8_t* blk = p.kc + id * p.kc_stride0;
      data = blk + static_cast<int64_t>(off) * kTokenStride;
      scales = blk + p.kv_bs * kTokenStride + static_cast<int64_t>(off) * kScaleDim;
    } else {
      atomicOr(p.err, static_cast<unsigned int>(C128_DEV_BAD_BLOCK));
    }
    place = entry;
    if (entry >= p.first) {
      place = it.ring + entry - max(it.from, p.first);
      place = p.first + (place >= circle ? place - circle : place);
    }
  }
};
// 16 codes to bf16
__device__ __forceinline__ void decode_codes(uint4 r, uint32_t scale_byte, uint32_t (&o)[8]) {
  const float s = scale_of(scale_byte);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    o[2 * k] = codes_to_bf16(static_cast<uint16_t>(w[k]), s);
    o[2 * k + 1] = codes_to_bf16(static_cast<uint16_t>(w[k] >> 16), s);
  }
}
// Whether one of the bf16 is not finite shows in bits 15 and 31.
__device__ __forceinline__ uint32_t not_finite(const uint32_t (&o)[8]) {
  uint32_t most = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) most |= (o[k] & 0x7fff7fffu) + 0x00800080u;
  return most & 0x80008000u;
}

// The entries that item i brings to its run, one after the other by all lanes of a warp: lanes 0 .. 27 have 16 codes each,
// lanes 28 .. 31 two times 8 rope values. Stored once O has been through the item `back` items before, which was the last to
// see what they replace. (O may be on its way through later ones, so what is there has to be finite at any time.)
template <bool ALIGN16>
__device__ __forceinline__ void decode_next(const DecodeParams& p, WindowSmem& sm, int i, int back) {
  const Item& it = sm.ring[i % kRing];
  const int lane = threadIdx.x & 31, all = it.news;
  const bool rope = lane >= 28;
#pragma unroll 1
  for (int e = 0; e < all; ++e) {  // (an item that goes on with a run brings one at least: its own)
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    uint32_t scale = 127;
    const Source src(p, it, e);
    if (src.data != nullptr) {
      const uint8_t* from = src.data + 16 * lane;
      a = ALIGN16 ? ld16(from) : ld8x2(from);
      if (rope) b = ALIGN16 ? ld16(from + 64) : ld8x2(from + 64);
      else asm("ld.global.cg.u8 %0, [%1];" : "=r"(scale) : "l"(src.scales + (lane >> 2)));
    }
    if (e == 0 && i >= back) warp_wait(&sm.abort, &sm.o_full[(i - back) % kRing], ((i - back) / kRing) & 1);
    uint32_t o[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (!rope) decode_codes(a, scale, o);
    const bool poison = __any_sync(0xffffffffu, not_finite(o) != 0);
    if (poison) {
#pragma unroll
      for (int k = 0; k < 8; ++k) o[k] = 0;
    }
    const uint32_t swz = static_cast<uint32_t>(src.place & 7) << 4, unit = rope ? 16u * (lane - 28) : 32u * (lane & 3);
    const uint32_t at = smem_addr(sm.k) + src.place * 128 + (rope ? 7 : lane >> 2) * kChunkBytes;
    sts16(at + (unit ^ swz), o[0], o[1], o[2], o[3]);
    sts16(at + ((unit + (rope ? 64u : 16u)) ^ swz), o[4], o[5], o[6], o[7]);
    if (lane == 0) sm.state[src.place] = src.data == nullptr ? kAbsent : poison ? kPoison : kThere;
  }
  async_proxy_fence();
  __syncwarp();
}

// The entries that a run begins with, once O has been through the item before: eight to a warp, each by four threads, which
// have the 16 bytes sub, sub + 4, ... of it (of the codes a quarter of each 64 columns, so piece j belongs to scale j).
template <bool ALIGN16>
__device__ __forceinline__ void decode_first(const DecodeParams& p, WindowSmem& sm, int i, int index) {
  const Item& it = sm.ring[i % kRing];
  const int lane = threadIdx.x & 31, sub = lane & 3, e = 8 * index + (lane >> 2);
  const bool in = e < it.lead + it.news;
  const uint8_t* data = nullptr;
  int place = 0;
  uint4 raw[9];
  uint2 scales = make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu);
#pragma unroll
  for (int j = 0; j < 9; ++j) raw[j] = make_uint4(0, 0, 0, 0);
  if (in) {
    const Source src(p, it, e);
    data = src.data, place = src.place;
    if (data != nullptr) {
#pragma unroll
      for (int j = 0; j < 9; ++j) raw[j] = ALIGN16 ? ld16(data + 16 * sub + 64 * j) : ld8x2(data + 16 * sub + 64 * j);
      scales = ld8(src.scales);
    }
  }
  __syncwarp();
  if (i > 0) warp_wait(&sm.abort, &sm.o_full[(i - 1) % kRing], ((i - 1) / kRing) & 1);
  if (__any_sync(0xffffffffu, in)) {
    const uint32_t row = smem_addr(sm.k) + place * 128, swz = static_cast<uint32_t>(place & 7) << 4;
    const uint32_t rope[8] = {raw[7].x, raw[7].y, raw[7].z, raw[7].w, raw[8].x, raw[8].y, raw[8].z, raw[8].w};  // bf16 already
    if (in) {
      const uint32_t at = row + 7 * kChunkBytes;
      sts16(at + ((16u * sub) ^ swz), rope[0], rope[1], rope[2], rope[3]);
      sts16(at + ((16u * sub + 64u) ^ swz), rope[4], rope[5], rope[6], rope[7]);
    }
    uint32_t poison = not_finite(rope);
#pragma unroll
    for (int j = 0; j < 7; ++j) {
      uint32_t o[8];
      decode_codes(raw[j], ((j < 4 ? scales.x : scales.y) >> (8 * (j & 3))) & 0xffu, o);
      if (in) {
        const uint32_t at = row + j * kChunkBytes;
        sts16(at + ((32u * sub) ^ swz), o[0], o[1], o[2], o[3]);
        sts16(at + ((32u * sub + 16u) ^ swz), o[4], o[5], o[6], o[7]);
      }
      poison |= not_finite(o);
    }
    // An entry with a value that is not finite (a code of NaN, a bf16 that is not, a product without room): zeros, by each
    // thread where it has stored itself, since nothing orders its stores and those of another one.
    poison |= __shfl_xor_sync(0xffffffffu, poison, 1);
    poison |= __shfl_xor_sync(0xffffffffu, poison, 2);
    if (in && poison) {
#pragma unroll 1
      for (int j = 0; j < 16; ++j)
        sts16(row + (j >> 1) * kChunkBytes + ((j < 14 ? 32u * sub + 16u * (j & 1) : 16u * sub + 64u * (j & 1)) ^ swz), 0, 0, 0, 0);
    }
    if (in && sub == 0) sm.state[place] = data == nullptr ? kAbsent : poison ? kPoison : kThere;
  }
  async_proxy_fence();
  __syncwarp();
}

// 32 rows of one column of O, as they are stored: bf16 of two rows each, or fp32, times the rows' factors.
template <bool OUT_F32>
struct Packed {
  uint32_t x[OUT_F32 ? 32 : 16];
  __device__ __forceinline__ Packed(const uint32_t (&o)[32], const float* factor) {
    if constexpr (OUT_F32) {
#pragma unroll
      for (int k = 0; k < 32; k += 4) {
        const float4 f = *reinterpret_cast<const float4*>(factor + k);
        const float2 a = __fmul2_rn(make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])), make_float2(f.x, f.y));
        const float2 b = __fmul2_rn(make_float2(__uint_as_float(o[k + 2]), __uint_as_float(o[k + 3])), make_float2(f.z, f.w));
        x[k] = __float_as_uint(a.x), x[k + 1] = __float_as_uint(a.y), x[k + 2] = __float_as_uint(b.x), x[k + 3] = __float_as_uint(b.y);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = pack_bf16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
    }
  }
};
// Where a warp's 32 rows and 32 columns of 128 go. Eight rows are of one token: where the first of them that this lane stores
// goes, from the item's first token on. (Of bf16 a lane stores every other row of pairs of columns.)
template <bool OUT_F32>
struct OutRows {
  int64_t at[4], step;  // elements; bytes from a row to the next that this lane stores
  __device__ __forceinline__ OutRows(const DecodeParams& p, const WindowPlan& plan, int head0, int own, int w, int lane) {
    const int odd = OUT_F32 ? 0 : lane & 1;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int token = static_cast<int>((own + 8 * g) * plan.pitch_inv >> 16), h0 = own + 8 * g - token * plan.pitch;
      at[g] = token * p.out_stride_r + (head0 + h0 + odd) * p.out_stride_h + 32 * w + (OUT_F32 ? lane : lane & ~1);
    }
    step = p.out_stride_h * 4;  // one row of fp32, two of bf16
    asm volatile("" : "+l"(step));
  }
  // Of an item: where its first token's row is, and how many rows there are from `at` on.
  __device__ __forceinline__ int64_t item(const DecodeParams& p, const WindowPlan& plan, const Item& it, int heads, int own, int lane,
                                          int (&limit)[4]) const {
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int token = static_cast<int>((own + 8 * g) * plan.pitch_inv >> 16), h0 = own + 8 * g - token * plan.pitch;
      limit[g] = token < it.count ? heads - h0 - (OUT_F32 ? 0 : lane & 1) : 0;
    }
    return it.token * p.out_stride_r;
  }
  __device__ __forceinline__ void store(const DecodeParams& p, int64_t from, const int (&limit)[4], const Packed<OUT_F32>& v, int lane) const {
    const uint32_t halves = lane & 1 ? 0x3276 : 0x5410;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      char* dst = static_cast<char*>(p.out) + (from + at[g]) * (OUT_F32 ? 4 : 2);
#pragma unroll
      for (int k = 0; k < (OUT_F32 ? 8 : 4); ++k) {
        uint32_t x = v.x[(OUT_F32 ? 8 : 4) * g + k];
        // neighbouring lanes swap halves of a pair of rows, so that each stores two columns of one
        if constexpr (!OUT_F32) x = __byte_perm(x, __shfl_xor_sync(0xffffffffu, x, 1), halves);
        if ((OUT_F32 ? k : 2 * k) < limit[g]) *reinterpret_cast<uint32_t*>(dst) = x;
        dst += step;
        asm volatile("" : "+l"(dst));  // (a running sum: a product of 64 bits for each row takes five times the instructions)
      }
    }
  }
};

template <bool ALIGN16, bool OUT_F32>
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
      mbar_init(&sm.ring_free[i], kSoftWarps + kOutWarps + 3);
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.o_full[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.p_full[i], kSoftWarps);
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.q_free[i], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.s_free, kSoftWarps);
    mbar_init(&sm.k_help, kHelpers);
    mbar_init(&sm.drained, 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.set[i], kSoftWarps / 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.o_part[i], 1);
      mbar_init(&sm.o_free[i], kOutWarps);
    }
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
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) { c128::warp_wait(abort_flag, bar, parity); };
  auto item_flags = [&](int i) {
    warp_wait(&sm.ring_full[i % kRing], (i / kRing) & 1);
    const int flags = sm.ring[i % kRing].flags;
    return *abort_flag ? kEnd : flags;
  };
  auto free_item = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.ring_free[i % kRing]);
  };

  int last = -1;  // the last item, of which the softmax warps, which are done by then, store half of the results

  if (warp == kItemWarp) {
    // --------------------------------------------------------------------------------- the items
    const unsigned share = static_cast<unsigned>(p.requests) / static_cast<unsigned>(plan.columns);  // tokens of a column, the first `extra` one more
    const int extra = static_cast<int>(p.requests) - static_cast<int>(share) * plan.columns;
    const int64_t in_order = static_cast<int64_t>(share) * column + min(column, extra);
    int stride = plan.stride;
    int64_t begin = in_order;
    const int64_t end = share + (column < extra ? 1 : 0);  // `t` counts the column's tokens up to here
    unsigned int err = 0;
    int64_t batch = 0;  // lanes hold tokens batch .. batch + 31
    int lo = 0, hi = 0, req = 0;
    unsigned live = 0, goes_on = 0;  // tokens that are not skipped; those that follow the one before
    int64_t last_pos = -1;           // of the token before the batch
    int last_req = -1;
    auto load_batch = [&] {
      const int64_t t = begin + (batch + lane) * stride;
      int64_t pos = -1;
      bool ok = false;
      if (batch + lane < end) {
        pos = p.positions[t];
        req = p.token_req[t];
        ok = pos >= 0 && p.slots[t] >= 0;
        if (ok && (req < 0 || req >= p.table_rows)) ok = false, err |= C128_DEV_BAD_REQ;
        if (ok && pos >= p.most) err |= C128_DEV_BAD_BT_COL;
      }
      if (!ok) pos = -1;
      // (A token behind the table begins a run, and goes alone: of the entries that it brings it sees all.)
      hi = static_cast<int>(min(pos, static_cast<int64_t>(p.most)));
      lo = static_cast<int>(min(max(pos - (window - 1), static_cast<int64_t>(0)), static_cast<int64_t>(p.most)));
      int64_t pos_before = __shfl_up_sync(0xffffffffu, pos, 1);
      int req_before = __shfl_up_sync(0xffffffffu, req, 1);
      if (lane == 0) pos_before = last_pos, req_before = last_req;
      live = __ballot_sync(0xffffffffu, ok);
      goes_on = __ballot_sync(0xffffffffu, ok && pos_before >= 0 && pos == pos_before + 1 && req == req_before && pos < p.most);
      last_pos = __shfl_sync(0xffffffffu, pos, 31);
      last_req = __shfl_sync(0xffffffffu, req, 31);
    };
    if (stride == 0) {
      // Some tokens and those behind them, the same for all CTAs: where most follow one another they go in order, else in turn
      // (as which this CTA's are on their way meanwhile).
      const int64_t t = (p.requests - 1) * lane / 32;
      const int64_t pos0 = p.positions[t], pos1 = p.positions[t + 1], slot0 = p.slots[t], slot1 = p.slots[t + 1];
      const int req0 = p.token_req[t], req1 = p.token_req[t + 1];
      stride = plan.columns, begin = column;
      load_batch();
      const bool live0 = pos0 >= 0 && slot0 >= 0, follows = live0 && slot1 >= 0 && pos1 == pos0 + 1 && req1 == req0;
      if (2 * __popc(__ballot_sync(0xffffffffu, follows)) > __popc(__ballot_sync(0xffffffffu, live0))) {
        stride = 1, begin = in_order, last_pos = -1, last_req = -1;
        load_batch();
      }
    } else if (end > 0) {
      load_batch();
    }
    int base = 0, newest = -1, seen_to = -1;  // the run's
    bool stalled = p.stall && blockIdx.x == 0;
    int64_t t = 0;
    for (int i = 0; !stalled; ++i) {
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
      it.token = static_cast<int>(begin + t * stride);
      it.count = count;
      it.row = __shfl_sync(0xffffffffu, req, j);
      const int lo_j = __shfl_sync(0xffffffffu, lo, j);
      it.hi = __shfl_sync(0xffffffffu, hi, j);
      const int last = min(it.hi + (count - 1), p.most - 1);
      it.last = last;
      const bool fresh = i == 0 || !(goes_on >> j & 1);
      if (fresh) {
        it.lead = min(first, lo_j);
        it.from = lo_j;
        base = max(first, lo_j);
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
      it.flags = (fresh ? kFresh : 0) | (fresh || plan.lookahead < 2 ? kSerial : 0) | (used > kMain ? kTail : 0) | max((used + 15) / 16, 1) << kStepShift;
      if (lane == 0) {
        sm.ring[slot] = it;
        mbar_arrive(&sm.ring_full[slot]);
      }
      __syncwarp();
      t += count;
    }
    if (err) atomicOr(p.err, err);
  } else if (warp == kQueryWarp) {
    // -------------------------------------------------------------------------------- the queries
    const uint32_t q_bytes = static_cast<uint32_t>(kChunks / 2 * plan.together * plan.pitch * 128);
    int loads = 0;
    for (int i = 0;; ++i) {
      if (item_flags(i) & kEnd) break;
      const int token = sm.ring[i % kRing].token;
      free_item(i);
      if (i > 0 && lane < kChunks) prefetch_query_rows(&q_map, 64 * lane, head0, token);
      // each half of the columns when S of the item before has been through it
#pragma unroll 1
      for (int half = 0; half < 2 && !*abort_flag; ++half) {
        if (i > 0) warp_wait(&sm.q_free[half], (i - 1) & 1);
        if (*abort_flag) break;
        ++loads;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full[half], q_bytes);
          for (int c = kChunks / 2 * half; c < kChunks / 2 * (half + 1); ++c)
            load_query_rows(sm.q + c * kQChunkBytes, &q_map, 64 * c, head0, token, &sm.q_full[half]);
        }
        __syncwarp();
      }
      if (*abort_flag) break;
    }
    for (int k = max(loads - 2, 0); k < loads; ++k) decode_wait(&sm.q_full[k & 1], k >> 1 & 1, nullptr);  // nothing may be in flight when the CTA ends
    __syncwarp();
  } else if (warp == kDecodeWarp || (warp >= kSoftWarps && warp < kMmaWarp)) {
    // ------------------------------------------------------------------- entries and results
    const int w = warp & 3, own = 32 * ((warp >> 2) & 1);  // of results: TMEM lanes 32w .., rows own .. own + 31
    const bool decodes = warp == kDecodeWarp;
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const bool busy = own < rows16;
    const OutRows<OUT_F32> to(p, plan, head0, own, w, lane);
    auto results = [&](int i) {
      const Item& it = sm.ring[i % kRing];
      int limit[4];
      const int64_t row0 = to.item(p, plan, it, heads, own, lane, limit);
      uint32_t o[32];
      if constexpr (OUT_F32) warp_wait(&sm.p_full[i & 1], (i >> 1) & 1);  // (with the factors)
      warp_wait(&sm.o_part[0], i & 1);
      tmem_fence_after();
      tmem_ld_32x32(tmem + lanes + own, o);
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {  // 128 columns, of them 32 to a warp, of 32 rows
        tmem_wait_ld();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free[mt]);
        const bool more = mt + 1 < 4;
        if (more) {
          warp_wait(&sm.o_part[mt + 1], i & 1);
          tmem_fence_after();
        }
        const Packed<OUT_F32> packed(o, sm.factor[i % kRing] + own);
        if (more) tmem_ld_32x32(tmem + lanes + (mt + 1) * kRows + own, o);  // on its way as these are stored
        if (busy && !*abort_flag) to.store(p, row0 + 128 * mt, limit, packed, lane);
      }
      free_item(i);
    };
    for (int i = 0;; ++i) {
      const int flags = item_flags(i);
      const bool fresh = flags & kFresh, end = flags & kEnd;
      if (!end && (decodes || fresh)) {
        if (fresh) decode_first<ALIGN16>(p, sm, i, decodes ? kHelpers : warp);
        else decode_next<ALIGN16>(p, sm, i, plan.lookahead);
        if (lane == 0) mbar_arrive(decodes ? &sm.k_full[i % kRing] : &sm.k_help);
      }
      if (decodes && !end) free_item(i);
      if (end) {
        last = i - 1;
        break;
      }
      if (!decodes && i > 0) {
        results(i - 1);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------------------ issue the products
    if (elect_one()) {
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (wait_for(abort_flag, bar, parity)) return true;
        *abort_flag = 1;
        return false;
      };
      const uint32_t q_at = desc_low(smem_addr(sm.q), 16), ks_at = desc_low(smem_addr(sm.k), 16);
      const uint32_t kv_at = desc_low(smem_addr(sm.k), kChunkBytes), p_at = desc_low(smem_addr(sm.p), 16);
      const uint32_t desc_s = mma_desc(kMain, rows16, false), desc_tail = mma_desc(64, rows16, false), desc_o = mma_desc(128, rows16, true);
      auto half_of_s = [&](int half, bool tail) {
        tmem_fence_after();
#pragma unroll 1
        for (int c = kChunks / 2 * half; c < kChunks / 2 * (half + 1); ++c) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma(tmem + kTmemS, desc64(ks_at + ((c * kChunkBytes + ks * 32) >> 4)), desc64(q_at + ((c * kQChunkBytes + ks * 32) >> 4)), desc_s, c + ks > 0);
          if (!tail) continue;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            mma(tmem + kTmemTail, desc64(ks_at + ((kMain * 128 + c * kChunkBytes + ks * 32) >> 4)), desc64(q_at + ((c * kQChunkBytes + ks * 32) >> 4)), desc_tail,
                c + ks > 0);
        }
        mma_commit(&sm.q_free[half]);
      };
      auto product_o = [&](int i, int steps) {  // of item i
        if (!wait(&sm.p_full[i & 1], (i >> 1) & 1)) return false;
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {  // as the results of the item before leave it
          if (i > 0 && !wait(&sm.o_free[mt], (i - 1) & 1)) return false;
          tmem_fence_after();
#pragma unroll 1
          for (int ks = 0; ks < steps; ++ks)
            mma(tmem + mt * kRows, desc64(kv_at + ((2 * mt * kChunkBytes + ks * 2048) >> 4)), desc64(p_at + (ks * 2048 >> 4)), desc_o, ks > 0);
          mma_commit(&sm.o_part[mt]);
        }
        mma_commit(&sm.o_full[i % kRing]);
        return true;
      };
      int steps = 0, helped = 0;
      for (int i = 0;; ++i) {
        const int slot = i % kRing;
        if (!wait(&sm.ring_full[slot], (i / kRing) & 1)) break;
        const int flags = sm.ring[slot].flags;
        mbar_arrive(&sm.ring_free[slot]);
        // S of this item before O of the one before, or (serial) behind it
        if (i > 0 && (flags & (kEnd | kSerial)) && !product_o(i - 1, steps)) break;
        if (flags & kEnd) break;
        if (i > 0 && !wait(&sm.s_free, (i - 1) & 1)) break;
        if (!wait(&sm.q_full[0], i & 1)) break;
        if (!wait(&sm.k_full[i % kRing], (i / kRing) & 1)) break;
        if (flags & kFresh) {
          if (!wait(&sm.k_help, helped & 1)) break;
          ++helped;
        }
        half_of_s(0, flags & kTail);
        if (!wait(&sm.q_full[1], i & 1)) break;
        half_of_s(1, flags & kTail);
        mma_commit(&sm.s_full);
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
    // the row that this lane has the statistics of: its token and head in any item, and the head's sink
    const int my_row = own + lane, my_token = static_cast<int>(my_row * plan.pitch_inv >> 16), my_head = my_row - my_token * plan.pitch;
    const float sink = p.sink != nullptr && my_head < heads ? __ldcg(p.sink + head0 + my_head) * kLog2e : -INFINITY;
    uint32_t set_phase = 0;
    int helped = 0;
    auto set_sync = [&] {  // bounded, as every wait: a warp that has seen the abort flag does not come
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.set[set]);
      warp_wait(&sm.set[set], set_phase);
      set_phase ^= 1;
    };
    for (int i = 0;; ++i) {
      const int flags = item_flags(i);
      if (flags & kEnd) {
        last = i - 1;
        break;
      }
      const Item& it = sm.ring[i % kRing];
      const bool tail = (flags & kTail) && w == 0;
      if (flags & kFresh) {
        decode_first<ALIGN16>(p, sm, i, warp);
        if (lane == 0) mbar_arrive(&sm.k_help);
      }
      warp_wait(&sm.k_full[i % kRing], (i / kRing) & 1);
      if (flags & kFresh) {
        warp_wait(&sm.k_help, helped & 1);
        ++helped;
      }
      float total = 0.f, base2 = 0.f;  // of this lane's row: the sum of weights (the sink's too) is total * 2^base2
      if (busy) {
        // This thread's entries are 32w + lane / 4 and on in steps of 8, and of the tail (in the first 16 lanes of TMEM) one.
        // A score is at most `most`: -inf where the row does not see the entry, else +inf (which a NaN becomes, and in the
        // difference from the largest NaN again). `plus` is NaN for an entry that is not finite, else 0.
        float most[5][4], plus[5];
        int ahead[5];  // positions from the entry to the first token
        unsigned reach[5];
#pragma unroll
        for (int k = 0; k < 5; ++k) {
          const int place = k < 4 ? 32 * w + 8 * k + (lane >> 2) : kMain + (lane >> 2);
          int d = it.newest - (place - first);
          if (d < 0) d += circle;
          const int pos = place < first ? place : it.last - d;
          const uint8_t state = sm.state[place];
          ahead[k] = it.hi - pos;
          // it is seen from that many positions on, from its own; 0: there is none (a token behind the table has first entries up to
          // the table's end only; what stands in the places of the others, and in `state`, is of no entry)
          reach[k] = state == kAbsent || (place < first ? place > it.last : pos < it.base) ? 0u : place < first ? 0x80000000u : window;
          plus[k] = state == kPoison ? NAN : 0.f;
        }
        if (plan.together == 1) {
#pragma unroll
          for (int k = 0; k < 5; ++k)
            most[k][0] = most[k][1] = most[k][2] = most[k][3] = static_cast<unsigned>(ahead[k]) < reach[k] ? INFINITY : -INFINITY;
        } else {
#pragma unroll
          for (int g = 0; g < 4; ++g) {  // eight rows are of one token
            const int token = static_cast<int>((own + 8 * g) * plan.pitch_inv >> 16);
#pragma unroll
            for (int k = 0; k < 5; ++k) most[k][g] = static_cast<unsigned>(ahead[k]) + token < reach[k] ? INFINITY : -INFINITY;
          }
        }
        warp_wait(&sm.s_full, i & 1);
        tmem_fence_after();
        float2 v[5][4];  // scores of rows r0 + 8g and + 1 in v[..][g]
        {
          uint32_t x[2][16], y[16];
          tmem_ld_scores<32>(tmem + lanes + kTmemS + own, x[0]);
          tmem_ld_scores<32>(tmem + lanes + (16u << 16) + kTmemS + own, x[1]);
          if (tail) tmem_ld_scores<32>(tmem + lanes + kTmemTail + own, y);
          tmem_wait_ld();
          auto score = [&](uint32_t a, uint32_t b, int k, int g) {
            const float2 t = __ffma2_rn(make_float2(__uint_as_float(a), __uint_as_float(b)), make_float2(c2, c2), make_float2(plus[k], plus[k]));
            return make_float2(fminf(t.x, most[k][g]), fminf(t.y, most[k][g]));
          };
#pragma unroll
          for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k][g] = score(x[k >> 1][4 * g + 2 * (k & 1)], x[k >> 1][4 * g + 2 * (k & 1) + 1], k, g);
          }
          if (tail) {
#pragma unroll
            for (int g = 0; g < 4; ++g) v[4][g] = score(y[4 * g], y[4 * g + 1], 4, g);
          }
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.s_free);
        float top[8];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          top[2 * g] = fmaxf(fmaxf(v[0][g].x, v[1][g].x), fmaxf(v[2][g].x, v[3][g].x));
          top[2 * g + 1] = fmaxf(fmaxf(v[0][g].y, v[1][g].y), fmaxf(v[2][g].y, v[3][g].y));
        }
        if (tail) {
#pragma unroll
          for (int g = 0; g < 4; ++g) top[2 * g] = fmaxf(top[2 * g], v[4][g].x), top[2 * g + 1] = fmaxf(top[2 * g + 1], v[4][g].y);
        }
        sm.by_warp[0][w][reduced] = reduce_rows(top, lane, [](float a, float b) { return fmaxf(a, b); });
        set_sync();
        // (the four warps of a set make and write the same, here and below)
        const float largest = fmaxf(fmaxf(sm.by_warp[0][0][my_row], sm.by_warp[0][1][my_row]), fmaxf(sm.by_warp[0][2][my_row], sm.by_warp[0][3][my_row]));
        const float m = largest == -INFINITY ? 0.f : largest;  // (of a row that sees nothing)
        sm.ref[my_row] = -m;
        __syncwarp();
        float2 sum[4] = {};
        auto weigh = [&](int k, int g, float2 ref) {
          const float2 t = __fadd2_rn(v[k][g], ref);
          v[k][g] = make_float2(ex2_approx(t.x), ex2_approx(t.y));
          sum[g] = k == 0 ? v[k][g] : __fadd2_rn(sum[g], v[k][g]);
        };
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float2 ref = *reinterpret_cast<const float2*>(&sm.ref[r0 + 8 * g]);
#pragma unroll
          for (int k = 0; k < 4; ++k) weigh(k, g, ref);
          if (tail) weigh(4, g, ref);
        }
        const float sums8[8] = {sum[0].x, sum[0].y, sum[1].x, sum[1].y, sum[2].x, sum[2].y, sum[3].x, sum[3].y};
        auto add = [](float a, float b) { return a + b; };
        sm.by_warp[1][w][reduced] = reduce_rows(sums8, lane, add);
        uint32_t packed[5][4];
        if constexpr (OUT_F32) {  // the weights as they are, and the sums of what the product sees of them
          float rounded[8] = {};
          auto pack = [&](int k, int g) {
            packed[k][g] = pack_bf16x2(v[k][g].x, v[k][g].y);
            rounded[2 * g] += __uint_as_float(packed[k][g] << 16), rounded[2 * g + 1] += __uint_as_float(packed[k][g] & 0xffff0000u);
          };
#pragma unroll
          for (int g = 0; g < 4; ++g) {
#pragma unroll
            for (int k = 0; k < 4; ++k) pack(k, g);
            if (tail) pack(4, g);
          }
          sm.by_warp[2][w][reduced] = reduce_rows(rounded, lane, add);
        }
        set_sync();
        {
          const float own_sum = (sm.by_warp[1][0][my_row] + sm.by_warp[1][1][my_row]) + (sm.by_warp[1][2][my_row] + sm.by_warp[1][3][my_row]);
          float sum = own_sum, to = m, share = 1.f;
          if (p.sink != nullptr) {  // one more score, with a value of zero
            to = own_sum == 0.f ? (sink == -INFINITY ? 0.f : sink) : fmaxf(m, sink);
            share = own_sum == 0.f ? 0.f : ex2_approx(m - to);
            sum = own_sum * share + ex2_approx(sink - to);
          }
          total = sum, base2 = to;
          if constexpr (OUT_F32) {
            const float rounded = (sm.by_warp[2][0][my_row] + sm.by_warp[2][1][my_row]) + (sm.by_warp[2][2][my_row] + sm.by_warp[2][3][my_row]);
            // (What stood there has been used: S of this item came behind O of the last but one, which waited for results that
            // come behind those.)
            if (w == 0) sm.factor[i % kRing][my_row] = own_sum == 0.f ? 0.f : __fdividef(own_sum * share, sum * rounded);
          } else {
            sm.share[my_row] = own_sum == 0.f ? 0.f : __fdividef(share, sum);
          }
          __syncwarp();
        }
        if constexpr (!OUT_F32) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const float2 share = *reinterpret_cast<const float2*>(&sm.share[r0 + 8 * g]);
            auto pack = [&](int k) {
              const float2 t = __fmul2_rn(v[k][g], share);
              packed[k][g] = pack_bf16x2(t.x, t.y);
            };
#pragma unroll
            for (int k = 0; k < 4; ++k) pack(k);
            if (tail) pack(4);
          }
        }
        // the weights of the item before have been used
        if (i > 0) warp_wait(&sm.o_full[(i - 1) % kRing], ((i - 1) / kRing) & 1);
        const uint32_t swz = static_cast<uint32_t>(lane >> 2) << 4;  // of all its entries
        const uint32_t p_at = smem_addr(sm.p) + (32 * w + (lane >> 2)) * 128 + 4 * (lane & 3);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t at = p_at + ((16u * (own / 8 + g)) ^ swz);
#pragma unroll
          for (int k = 0; k < 4; ++k) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + k * 1024), "r"(packed[k][g]) : "memory");
          if (tail) asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + kMain * 128), "r"(packed[4][g]) : "memory");
        }
        async_proxy_fence();
      } else {
        warp_wait(&sm.s_full, i & 1);
        if (lane == 0) mbar_arrive(&sm.s_free);
        if (i > 0) warp_wait(&sm.o_full[(i - 1) % kRing], ((i - 1) / kRing) & 1);
      }
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full[i & 1]);
      if (busy && w == 0 && my_token < it.count && my_head < heads && p.lse != nullptr && !*abort_flag)
        p.lse[(static_cast<int64_t>(it.token) + my_token) * p.lse_stride_r + (head0 + my_head) * p.lse_stride_h] =
            total == 0.f ? -INFINITY : (base2 + log2f(total)) * 0.69314718055994531f;
      free_item(i);
    }
  }
  if (warp < kMmaWarp && last >= 0) {
    const int w = warp & 3, own = 32 * ((warp >> 2) & 1);
    const bool soft = warp < kSoftWarps;  // (these wait for all of O: only of that have they seen every phase)
    const OutRows<OUT_F32> to(p, plan, head0, own, w, lane);
    int limit[4];
    const int64_t row0 = to.item(p, plan, sm.ring[last % kRing], heads, own, lane, limit);
    if constexpr (OUT_F32) warp_wait(&sm.p_full[last & 1], (last >> 1) & 1);
    if (soft) warp_wait(&sm.o_full[last % kRing], (last / kRing) & 1);
#pragma unroll 1
    for (int mt = soft ? 2 : 0, end = mt + 2; mt < end; ++mt) {
      if (!soft) warp_wait(&sm.o_part[mt], last & 1);
      tmem_fence_after();
      uint32_t o[32];
      tmem_ld_32x32(tmem + (static_cast<uint32_t>(32 * w) << 16) + mt * kRows + own, o);
      tmem_wait_ld();
      if (own < rows16 && !*abort_flag) to.store(p, row0 + 128 * mt, limit, Packed<OUT_F32>(o, sm.factor[last % kRing] + own), lane);
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

const void* window_kernel_for(bool align16, bool out_f32) {
  if (out_f32) return align16 ? reinterpret_cast<const void*>(window_kernel<true, true>) : reinterpret_cast<const void*>(window_kernel<false, true>);
  return align16 ? reinterpret_cast<const void*>(window_kernel<true, false>) : reinterpret_cast<const void*>(window_kernel<false, false>);
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

bool window_fits(int64_t window, int64_t first) { return window + first <= kSlots; }

cudaError_t prepare_window() {
  cudaError_t e = cudaSuccess;
  for (int variant = 0; variant < 4; ++variant)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(window_kernel_for((variant & 1) != 0, (variant & 2) != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               sizeof(WindowSmem));
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
  if (together > room / 2) together = room / 2 > 0 ? room / 2 : 1;  // (so that entries of one item do not wait for O of the one before)
  if (together > (T + sm_count - 1) / sm_count) together = (T + sm_count - 1) / sm_count;
  const int64_t most = sm_count / plan.groups > 0 ? sm_count / plan.groups : 1;
  plan.columns = static_cast<int32_t>(T < most ? T : most);
  // A decode step's tokens are dealt out in turn, so that a batch padded at its end is shared by all CTAs (130 requests padded to 256
  // tokens 13.8 us, in order 21.1); others in order, for the entries that neighbours share (200 requests of two tokens each, 16
  // heads, 20.3 us, in turn 27.0). With less than two tokens to a row of the table the step can be either (a table may have rows
  // for more requests than there are in the step: 5,119 tokens of 5 of its 4,096 rows in turn 248 us, in order 157), and the
  // tokens decide; their items are of one token then.
  plan.stride = T > plan.columns && T < 2 * p.table_rows ? 0 : 1;
  if (plan.stride == 0) together = 1;
  plan.together = static_cast<int32_t>(together);
  plan.lookahead = room / plan.together < kRing ? room / plan.together : kRing;
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
  return cudaLaunchKernelExC(&lc, window_kernel_for(p.kc_stride0 % 16 == 0, p.out_f32 != 0), args);
}

}  // namespace c128
