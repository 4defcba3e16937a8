// c128_decode_attention: attention of one new token per request over its entries of the paged FP8
// cache, on the tcgen05 tensor cores.
//
//   S^T = K Q^T            per tile of 64 entries: M = 64 entries, N = heads, K = 512
//   P^T = exp2(c S^T - m)  c = scale * log2(e), m a running reference per head
//   O^T += K^T P^T         M = 128 columns (4 times), N = heads, K = 64 entries
//   L += 1 P^T             the sums of P as the products see it, rounded to bf16: M = 64 rows of ones
//   out = O / L
//
// An entry is key and value, so a tile is decoded once, to bf16 in shared memory (exact: an e4m3 code
// has 4 significant bits and its scale is a power of two), and both products read it from there as
// their A: with the 512 columns along K, and with them along M. Taking both products transposed makes
// the heads their N, so their work, their reads of shared memory (which bound them) and their TMEM
// columns go with the heads there are, and leaves room for two S tiles beside O. It also leaves the
// softmax next to nothing to exchange: a thread holds two entries and some heads, and keeps its own
// sums to the end. Heads are dealt out in groups of 64; a group decodes the cache for itself (the
// second group's reads hit L2).
//
// P is rounded to bf16 (2^-8), and O is divided by the sums of the rounded weights: then a weight's
// rounding is felt only against the other entries', not at all with a single one. lse is of the exact
// sums, in fp32. (Two sums in the softmax warps' registers took 10 % longer than the product with ones.)
//
// The running reference m need not be the maximum: P, its sums and O are floating point, so a common
// factor costs no precision while the products stay inside the range. So m is 0 where that does, that is where
// every head has a weight within 2^+-32 of 1 in the first tile, none passes 2^32, and no value passes 2^64 (2^31
// entries of that are 2^127). Else it is raised or lowered to the maximum so far, O in TMEM rescaled with it: then
// no weight of this tile is above 1. Values that large are looked for where they pass through registers, in the scale
// bytes and the rope columns. (At the other end a head's weights reach down to 2^-32, and values below 2^-92 can get
// lost: a look for those as well took 3 % of a tile's time, and is not worth it.)
//
// Work is dealt out in tiles: the requests' tiles, one after the other, are cut into as many equal
// runs as there are CTAs, so a long request is shared by many CTAs and a CTA takes many short ones. (What
// a run has of one request is called a stretch here.) A request that is cut leaves fp32 partial results in
// the workspace, joined by a second kernel.
//
// Measured, device time per call with the join: 8 requests of up to 65,536 entries, 16 heads (173 MB) 64.0 us,
// 2.70 TB/s; 48 of up to 8,192, 128 heads 60.2 us; 64 of up to 1,024, 64 heads 27.7 us; one of 1,024 12.4 us. A
// tile takes an SM 1.47 us (16 heads) or 1.87 (64). Its stages wait for one another over two buffers; decoding is the
// longest of them, on a shared memory of which the products' operands take half the bandwidth and come first. With
// references other than 0 (scores of a deviation of 20) 69.6, 82.0, 36.1 and 13.5 us.
//
// Roles of the 19 warps (each wait is bounded; five warps to a scheduler leave them 96 registers, and a
// spill would be a trip to L2, beside the little L1 that the tiles leave):
//   0..7   decode the entries of a tile, in registers until the buffer has room, the next tile's bytes
//          on their way meanwhile. Tiles pass to S in halves of the columns and come back from O in
//          quarters
//   8..15  softmax, four warps for either half of the heads; rescaling of O; results
//   16, 17 one thread each issues the first product (and the queries' TMA loads) and the second. Two,
//          so that either waits for its own operands: one thread that looks for whichever is ready
//          first takes a third of all issued instructions, and holds up the warps beside it
//   18     walks the runs: per tile the address of each entry (through the block table), prefetched
//          to L2 a few tiles ahead
#include <cuda_runtime.h>

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
constexpr int kQuarters = 4;        // of a tile's columns: 128 each, an M of the second product
constexpr int kFillWarps = 8;       // decode a tile
constexpr int kAhead = 3;           // of a tile's 7 chunks of codes, decoded before the buffer has room for them
// Eight softmax warps, half the heads each: with four, which left 128 registers to all, a tile took 0.25 us
// (16 heads) or 0.5 us (64) longer. Sixteen decoding warps, a set for alternate tiles or for either half
// of the columns, took 0.1 to 0.6 us longer: seven warps to a scheduler have 72 registers, and spill. (With
// four softmax warps and the registers dealt out so that nothing spilled: 0.2 us longer.)
constexpr int kSoftWarps = 8;
constexpr int kSoftWarp = kFillWarps, kMmaWarp = kSoftWarp + kSoftWarps, kIndexWarp = kMmaWarp + 2;
constexpr int kDecodeThreads = 32 * (kIndexWarp + 1);
constexpr int kStaged = 2;          // of the 9 16-byte pieces that a decoding thread has on their way: the rope values
constexpr int kStageBytes = kFillWarps * 32 * 16;
constexpr int kRing = 4;            // tiles the index warp may be ahead
constexpr float kHigh = 0x1p32f, kLow = 0x1p-32f;  // weights may be up to, and one in the first tile has to be over
constexpr int kTmemCols = 512, kTmemS = 256, kTmemL = 384;  // O in columns 0..255, two S tiles and L behind it

enum : int { kFirst = 1, kLast = 2, kEnd = 4, kRunShift = 3 };  // of its stretch of one request's tiles; above, the stretch's number mod 4

// In the place of a part's log-sum-exp: the part's CTA gave up. (None comes out so: a reference or a sum that is infinite makes NaN.)
constexpr float kNotThere = INFINITY;

struct Task {  // a request that a CTA starts and leaves to the columns behind it, if parts > 0
  int32_t request, parts, column, group_heads;
};

// How a call's heads and scratch are laid out for head groups of `group` heads (16, 32 or 64). CTA
// column c of every group has two slots for partial results: 2c for the request it continues, 2c + 1
// for the one it starts and does not finish.
struct Layout {
  int groups, columns, heads, ctas;  // head groups, CTA columns, heads held per slot and group
  Layout() = default;
  Layout(int all_heads, int sms, int group) {
    groups = (all_heads + group - 1) / group;
    columns = sms / groups;  // 0: no such groups on this GPU, but for the largest
    if (columns == 0 && group == kGroup) columns = 1;
    heads = groups > 1 ? group : (all_heads + 15) / 16 * 16;
    ctas = sms > columns * groups ? sms : columns * groups;
  }
  __host__ __device__ int64_t rows() const { return 2ll * columns * groups * heads; }
  __host__ __device__ int64_t lse_at() const { return (ctas * static_cast<int64_t>(sizeof(Task)) + 255) / 256 * 256; }
  __host__ __device__ int64_t out_at() const { return lse_at() + (rows() * 4 + 255) / 256 * 256; }
  // smaller groups need no more than the largest
  __host__ __device__ int64_t bytes() const { return out_at() + rows() * kHead * 4; }
  __device__ int64_t row(int slot, int group, int head) const {
    return (static_cast<int64_t>(slot) * groups + group) * heads + head;
  }
  // A partial result is kept as the threads that make and join it hold it: per 32 columns and 4 heads
  // 32 x 4 floats, column by column. Where `row` starts its 512 x heads floats, the block of `cols32`
  // and `head4`:
  __device__ int64_t block(int slot, int group, int cols32, int head4) const {
    return row(slot, group, 0) * kHead + (static_cast<int64_t>(cols32) * (heads / 4) + head4) * 128;
  }
};

struct Layouts {  // made on the host: their divisions would stand in front of the kernel's work
  Layout of[3];  // for groups of 16, 32 and 64 heads
};

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
  alignas(128) uint32_t ones[512];    // 64 x 16 of bf16, in any order
  alignas(16) uint8_t stage[kStaged][kStageBytes];
  TileDesc ring[kRing];
  alignas(16) float ref[kGroup];      // the running references m
  alignas(16) float factor[kGroup];   // what O is rescaled by
  alignas(16) float sums[kGroup];     // L
  alignas(16) float inv[2][kGroup];   // 1 / L (with a sink: the entries' share / L), of even and odd stretches
  float by_warp[4][kGroup];           // maxima or sums of 16 entries each
  uint64_t ring_full[kRing], ring_free[kRing];
  uint64_t k_full[2][2];              // half of a tile's columns decoded
  uint64_t k_free[2][kQuarters];      // O has taken the quarter (the last: O is done)
  uint64_t s_full[2], s_free[2], p_full[2];
  uint64_t q_full, q_free, o_free, drained;
  uint64_t inv_full[2];          // `inv` and `done` of a stretch are there
  uint64_t soft;                 // barrier of the softmax warps
  volatile int32_t off[2];       // 1 + the tile whose P in this buffer was made with a reference that is off, or will be
  int32_t done_request[2], done_part[2];
  int warp_sums[32];
  int32_t first_request, first_tile, first_entries;  // where the column's run begins, and that request's entries
  int32_t end_request, end_tile;  // and the tile behind its end
  Layout lay;                    // read back where results are written, to keep registers free
  int32_t group, group_heads;
  uint32_t tmem;
  volatile int abort;
};
static_assert(sizeof(DecodeSmem) <= 232448, "shared memory of one SM");

// The bounded wait of this kernel, inline and on the SM's clock: a call would have to keep the many
// values that live across it out of registers, and the global timer takes longer than most waits. (Tries
// without a time hint: a tile takes 4 % less.)
constexpr uint32_t kWaitCycles = 2000000000u;  // about a second; the 32-bit clock wraps after two
__device__ __forceinline__ bool decode_wait(uint64_t* bar, uint32_t parity, const volatile int* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = clock();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (abort_flag != nullptr && *abort_flag) return false;
    if (static_cast<uint32_t>(clock()) - t0 > kWaitCycles) return false;
  }
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
__host__ __device__ constexpr uint32_t mma_desc(int m, int n, bool mn_major) {  // bf16 x bf16 -> fp32
  return 1u << 4 | 1u << 7 | 1u << 10 | (mn_major ? 3u << 15 : 0u) | static_cast<uint32_t>(n >> 3) << 17 |
         static_cast<uint32_t>(m >> 4) << 24;
}
template <int V>
struct Const {
  static constexpr int value = V;
};
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(e));
  return e != 0;
}
// An unswizzled K-major operand of 16 columns: 8 rows of 16 bytes, the same 128 bytes on for the other 8 columns, 256
// bytes on for the next 8 rows.
__device__ __forceinline__ uint64_t desc_plain(uint32_t addr) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"((addr & 0x3ffff) >> 4 | 128u >> 4 << 16), "r"(256u >> 4 | 1u << 14));
  return d;
}
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d), "l"(a), "l"(b), "r"(desc),
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
// 16 lanes x N columns: thread t gets rows t/4 and t/4 + 8, columns 8g + 2(t%4) and + 1 in x[4g ..]
template <int N>
__device__ __forceinline__ void tmem_ld_scores(uint32_t addr, uint32_t (&x)[N / 2]) {
  if constexpr (N == 32) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]),
          "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15])
        : "r"(addr));
  } else if constexpr (N == 16) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7])
                 : "r"(addr));
  } else {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                 : "r"(addr));
  }
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
// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
// Two e4m3 codes times a power of two to bf16x2, by way of fp16 (exact, NaN stays NaN) and fp32. About
// 50 cycles of a scheduler per 16 codes and warp; moving the bits into bf16 fields and multiplying
// there took 85, most of it half-rate integer operations, NaN codes aside.
__device__ __forceinline__ uint32_t codes_to_bf16(uint16_t two, float scale) {
  uint32_t h;
  float2 v;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  v = mul2(v, make_float2(scale, scale));
  return pack_bf16x2(v.x, v.y);
}
// The larger magnitudes of two pairs of bf16 (under either sign).
__device__ __forceinline__ uint32_t larger2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// Whether a value is beyond what a reference of 0 allows: one of 7 scale bytes at 176 (the largest code gives 2^57.8) or
// above, or one of two bf16 magnitudes at 2^64. The low bits of a field plus a constant carry into its highest.
__device__ __forceinline__ bool too_large(uint2 scales, uint32_t values) {
  const uint32_t a = ((scales.x & 0x7f7f7f7fu) + 0x50505050u) & scales.x, b = ((scales.y & 0x007f7f7fu) + 0x00505050u) & scales.y & 0x00ffffffu;
  const uint32_t v = (values & 0x7fff7fffu) + (0x80008000u - 0x5f805f80u);
  return (((a | b) & 0x80808080u) | (v & 0x80008000u)) != 0;
}
// 2^(byte - 127): the byte is the float's exponent field (0: the subnormal 2^-127).
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }

// Read once and past L1, whose memory the tiles and the products use (0.2 us a tile less than with
// L1::no_allocate).
__device__ __forceinline__ uint4 ld16(const uint8_t* p) {
  uint4 v;
  asm("ld.global.cg.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 ld8(const uint8_t* p) {
  uint2 v;
  asm("ld.global.cg.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 ld8x2(const uint8_t* p) {
  const uint2 a = ld8(p), b = ld8(p + 8);
  return make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void sts16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// Entries of request r (p.most: what its table row holds, at most INT_MAX).
__device__ __forceinline__ int entries_of(const DecodeParams& p, int64_t r, unsigned int* err) {
  const int n = p.kv_lens[r];
  if (n < 0) *err |= C128_DEV_BAD_LENGTH;
  if (n > p.most) *err |= C128_DEV_BAD_BT_COL;
  return max(min(n, p.most), 0);
}
// A request without entries still takes a (masked) tile: its results are written like any other's.
__device__ __forceinline__ int tiles_of(int entries) { return max((entries >> 6) + ((entries & 63) != 0), 1); }
static_assert(kTile == 64, "tiles_of");

// The requests' tiles one after the other, kRunCost units between two requests, are dealt to the CTA
// columns in equal runs: storing the results of a request takes a CTA about as long as a tile (2 us of
// 64 heads), and every run ends with that. (The units of all requests are less than 2^31.)
// `total` units go to `columns`, the first `extra` of them one more than the rest. A cut that falls between
// requests, or would fall within `snap` tiles of a request's begin or end, is made there: a cut request
// costs its partial results (2 KB per head and part, written and read again), about what a tile or two take.
// (A cost of 2: 64 x 1,024 entries 4 % slower, 48 x 8,192 4 % faster; snap of 1 or 3: up to 6 % slower.)
constexpr int kRunCost = 1;  // not 0: a cut at the end of one request would be in none
constexpr int kSnap = 2;
struct Deal {
  int share, extra, snap;
  __device__ Deal(int total, int columns) {
    share = static_cast<unsigned>(total) / static_cast<unsigned>(columns);
    extra = total - share * columns;
    snap = min(share / 2, kSnap);
  }
  __device__ int begin(int column) const { return share * column + min(column, extra); }
  __device__ int column_of(int tile) const {
    const int longer = extra * (share + 1);
    const int t = tile < longer ? tile : tile - longer, d = tile < longer ? share + 1 : share;
    const int q = static_cast<unsigned>(t) / static_cast<unsigned>(d);
    return tile < longer ? q : extra + q;
  }
};

// A stretch's results: O of all heads times 1 / sum, to the output or the workspace. The softmax and the
// decoding warps share the work, four warps (`rank`) to each quarter of the TMEM lanes.
__device__ __forceinline__ void store_results(DecodeSmem& sm, const DecodeParams& p, int heads, int rank, int odd) {
  int tid = threadIdx.x;
  asm volatile("" : "+r"(tid));  // keeps what follows from being computed ahead, and in registers, in the callers' loops
  const int warp = tid >> 5, lane = tid & 31, heads16 = (heads + 15) & ~15;
  const int64_t request = sm.done_request[odd];
  const int part = sm.done_part[odd];
  tmem_fence_after();
  const int quarter = warp & 3, group0 = sm.group * sm.group_heads;
  const uint32_t o_at = sm.tmem + (static_cast<uint32_t>(32 * quarter) << 16);
#pragma unroll 1
  for (int item = rank; item < heads16 / 4; item += (kFillWarps + kSoftWarps) / 4) {  // 16 heads of 128 columns each
    const int mt = item & 3, h = (item >> 2) * 16;
    const int col = mt * 128 + 32 * quarter + lane;
    uint32_t o[16];
    tmem_ld_32x16(o_at + mt * kGroup + h, o);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; k += 4) {
      const float4 f = *reinterpret_cast<const float4*>(&sm.inv[odd][h + k]);
      o[k] = __float_as_uint(__uint_as_float(o[k]) * f.x), o[k + 1] = __float_as_uint(__uint_as_float(o[k + 1]) * f.y);
      o[k + 2] = __float_as_uint(__uint_as_float(o[k + 2]) * f.z), o[k + 3] = __float_as_uint(__uint_as_float(o[k + 3]) * f.w);
    }
    if (part >= 0) {
      uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<float*>(p.workspace + sm.lay.out_at()) +
                                            sm.lay.block(part, sm.group, 4 * mt + quarter, h / 4)) + lane;
#pragma unroll
      for (int k = 0; k < 4; ++k) dst[32 * k] = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
      continue;
    }
    const int64_t row = request * p.out_stride_r + (group0 + h) * p.out_stride_h;
    if (p.out_f32) {
      float* dst = static_cast<float*>(p.out) + row + col;
#pragma unroll
      for (int k = 0; k < 16; ++k, dst += p.out_stride_h)
        if (h + k < heads) *dst = __uint_as_float(o[k]);
    } else {
      // neighbouring lanes swap halves of a pair of heads, so that each stores two columns of one
      uint16_t* dst = static_cast<uint16_t*>(p.out) + row + (lane & 1) * p.out_stride_h + (col & ~1);
      const uint32_t halves = lane & 1 ? 0x3276 : 0x5410;
#pragma unroll
      for (int k = 0; k < 16; k += 2, dst += 2 * p.out_stride_h) {
        const uint32_t two = pack_bf16x2(__uint_as_float(o[k]), __uint_as_float(o[k + 1]));
        const uint32_t both = __byte_perm(two, __shfl_xor_sync(0xffffffffu, two, 1), halves);
        if (h + k + (lane & 1) < heads) *reinterpret_cast<uint32_t*>(dst) = both;
      }
    }
  }
  tmem_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.o_free);
}

// The end of a CTA whose wait ran out. What it has in the workspace may be of any call: its parts are marked, and the
// requests that they are of are not joined.
__device__ __noinline__ void give_up(const DecodeSmem& sm, uint8_t* workspace, int all_heads, unsigned int* err) {
  if (threadIdx.x == 0) atomicOr(err, static_cast<unsigned int>(C128_DEV_TIMEOUT));
  const int column = blockIdx.x / sm.lay.groups, heads = min(sm.group_heads, all_heads - sm.group * sm.group_heads);
  float* lse = reinterpret_cast<float*>(workspace + sm.lay.lse_at());
  for (int i = threadIdx.x; i < 2 * heads; i += kDecodeThreads)
    lse[sm.lay.row(2 * column + (i >= heads), sm.group, i >= heads ? i - heads : i)] = kNotThere;
}

constexpr int kBoxHeads = 16;  // heads of a TMA load of queries

template <bool ALIGN16, int HEADS>
__global__ void __launch_bounds__(kDecodeThreads, 1)
    decode_kernel(const __grid_constant__ DecodeParams p, const __grid_constant__ CUtensorMap q_map, const __grid_constant__ Layouts layouts) {
  constexpr int kOwn = HEADS / 2;  // heads of four softmax warps
  extern __shared__ uint8_t smem_raw[];
  DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t{1023});
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned int err = 0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.ring_full[i], 1);
      mbar_init(&sm.ring_free[i], kFillWarps + kSoftWarps + 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 2; ++k) mbar_init(&sm.k_full[i][k], kFillWarps);
      for (int k = 0; k < kQuarters; ++k) mbar_init(&sm.k_free[i][k], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.s_free[i], kSoftWarps);
      mbar_init(&sm.p_full[i], kSoftWarps);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_free, 1);
    mbar_init(&sm.o_free, kSoftWarps + kFillWarps);
    mbar_init(&sm.inv_full[0], kSoftWarps);
    mbar_init(&sm.inv_full[1], kSoftWarps);
    mbar_init(&sm.soft, kSoftWarps);
    sm.off[0] = sm.off[1] = 0;
    mbar_init(&sm.drained, 2);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (threadIdx.x < 512) sm.ones[threadIdx.x] = 0x3f803f80u;
  async_proxy_fence();  // (to the products, behind the barriers below)
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem)),
                 "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  launch_dependents();
  // This CTA's place for each size of head groups: its division is done before there is anything to read.
  constexpr int kSizes = HEADS == 16 ? 1 : HEADS == 32 ? 2 : 3;
  int most_columns[kSizes], column_for[kSizes], group_for[kSizes];
#pragma unroll
  for (int k = 0; k < kSizes; ++k) {
    const unsigned groups = layouts.of[k].groups;
    most_columns[k] = layouts.of[k].columns;
    column_for[k] = static_cast<int>(blockIdx.x / groups);
    group_for[k] = static_cast<int>(blockIdx.x - column_for[k] * groups);
  }
  const int requests = static_cast<int>(p.requests);
  grid_dependency_wait();  // what the kernels before this one wrote is read from here on
  // Sum the requests' units (each thread a stretch of requests)...
  const unsigned per = (static_cast<unsigned>(requests) + kDecodeThreads - 1) / kDecodeThreads;
  const int r_begin = min(threadIdx.x * per, static_cast<unsigned>(requests)), r_end = min(r_begin + per, static_cast<unsigned>(requests));
  const int n_begin = r_begin < r_end ? entries_of(p, r_begin, &err) : 0;
  int mine = r_begin < r_end ? tiles_of(n_begin) + kRunCost : 0;
  for (int r = r_begin + 1; r < r_end; ++r) mine += tiles_of(entries_of(p, r, &err)) + kRunCost;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.warp_sums[warp] = incl;
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  int warps = lane < kDecodeThreads / 32 ? sm.warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, warps, o);
    if (lane >= o) warps += u;
  }
  const int total = __shfl_sync(0xffffffffu, warps, 31) - kRunCost;  // none behind the last request
  const int tiles = total - (requests - 1) * kRunCost;
  const int base = __shfl_sync(0xffffffffu, warps, warp) - __shfl_sync(0xffffffffu, incl, 31) + incl - mine;
  // ...choose the head groups: smaller ones while there are CTAs for a tile each, since the fewer
  // heads a CTA has, the sooner it has loaded their queries and stored their results...
  int size = kSizes - 1, most = most_columns[kSizes - 1], column = column_for[kSizes - 1], group = group_for[kSizes - 1];
#pragma unroll
  for (int k = kSizes - 2; k >= 0; --k)
    if (tiles <= most_columns[k]) size = k, most = most_columns[k], column = column_for[k], group = group_for[k];
  const int group_heads = 16 << size;
  const int heads = min(group_heads, p.heads - group * group_heads);
  const int heads16 = (heads + 15) & ~15;
  // ...and find this column's run: its first request, and whether its last one goes on behind it.
  const int columns = min(most, total);
  const bool idle = column >= columns;
  const Deal deal(total, columns);
  const int cut0 = idle ? 0 : deal.begin(column), cut1 = idle ? 0 : deal.begin(column + 1);
  Task* const task = reinterpret_cast<Task*>(p.workspace) + blockIdx.x;
  if (threadIdx.x == 32 * kMmaWarp) {
    sm.lay = layouts.of[size];
    sm.group = group;
    sm.group_heads = group_heads;
    if (idle) *task = Task{0, 0, 0, 0};
  }
  if (!idle && mine > 0 && base <= cut1 && base + mine > cut0) {
    int at = base;
    for (int r = r_begin; r < r_end && at <= cut1; ++r) {
      unsigned int ignore = 0;
      const int entries = r == r_begin ? n_begin : entries_of(p, r, &ignore), end = at + tiles_of(entries), next = end + kRunCost;
      const bool holds0 = cut0 >= at && cut0 < next, holds1 = cut1 >= at && cut1 < next;
      auto on = [&](int cut) { return cut >= end || (cut - at > deal.snap && end - cut <= deal.snap); };
      auto back = [&](int cut) { return cut < end && cut - at <= deal.snap; };
      if (holds0) {
        const bool begins = on(cut0);  // with the next request
        sm.first_request = begins ? r + 1 : r;
        sm.first_tile = begins || back(cut0) ? 0 : cut0 - at;
        sm.first_entries = !begins ? entries : r + 1 < requests ? entries_of(p, r + 1, &ignore) : 0;
      }
      if (holds1) {
        // cut inside: does the request begin in this column? Then this column's task is to join it,
        // with every column that has a cut of it as its begin
        const bool inside = !on(cut1) && !back(cut1);
        sm.end_request = on(cut1) ? r + 1 : r;
        sm.end_tile = inside ? cut1 - at : 0;
        *task = Task{r,
                     inside && back(cut0) && group == 0 ? deal.column_of(end - deal.snap - 1) - column + 1 : 0, column, group_heads};
      }
      at = next;
    }
  }
  if (blockIdx.x == 0 && err) atomicOr(p.err, err);
  err = 0;
  __syncthreads();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);  // known to be the same in the whole warp
  volatile int* const abort_flag = &sm.abort;
  // A wait of a whole warp. One that runs out sets the abort flag, and with that set every wait returns
  // at once: the warps then run on as ever, on whatever they find, to the end that `tile_flags` shows them,
  // and no result is stored: the flag is looked at behind the last wait that a result depends on. So no lane or warp
  // leaves a path that others count on it for, without asking all lanes after every wait whether to go on (that took 6 %
  // of a tile's time).
  auto warp_wait = [&](uint64_t* bar, uint32_t parity) {
    if (!decode_wait(bar, parity, abort_flag)) *abort_flag = 1;
    __syncwarp();
  };
  auto tile_flags = [&](int i) {
    warp_wait(&sm.ring_full[i % kRing], (i / kRing) & 1);
    const int flags = sm.ring[i % kRing].flags;
    return *abort_flag ? kEnd : flags;
  };

  if (idle) {
    // no tiles
  } else if (warp == kIndexWarp) {
    // -------------------------------------------------------------------------- walk the run
    int64_t r = sm.first_request;
    int tile = sm.first_tile, n = sm.first_entries;
    const int end_tile = sm.end_tile;
    const int64_t end_request = sm.end_request;
    bool ends = r == end_request && tile == end_tile;  // the run, here
    int started = tile;  // the request's tile at which this run takes it up
    const Divisor bs = p.kv_div;
    int64_t window = r;      // lanes hold the lengths of requests window .. window + 31
    unsigned int ignore = 0;
    int id[2];
    // Entries are fewer than 2^31, so an index past them does not wrap in 32 unsigned bits. (Not as read-only data: this
    // kernel may have started before the one that writes the table has ended.)
    auto load_ids = [&] {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t key = static_cast<uint32_t>(tile) * kTile + 32 * h + lane;
        id[h] = key < static_cast<uint32_t>(n) ? __ldcg(p.table + r * p.table_stride + divide(key, bs)) : -1;
      }
    };
    int stretch = 0;
    if (!ends) load_ids();
    int lens = window + lane < p.requests ? entries_of(p, window + lane, &ignore) : 0;
    for (int i = 0; !(p.stall && blockIdx.x == 0); ++i) {
      const int slot = i % kRing;
      if (i >= kRing) warp_wait(&sm.ring_free[slot], (i / kRing - 1) & 1);
      TileDesc& d = sm.ring[slot];
      if (ends) {
        if (lane == 0) {
          d.flags = kEnd;
          mbar_arrive(&sm.ring_full[slot]);
        }
        break;
      }
      const int tiles = tiles_of(n);
      uint64_t mask = 0;
      const uint8_t* from[2];
      const uint8_t* sc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t key = static_cast<uint32_t>(tile) * kTile + 32 * h + lane;
        const bool in = key < static_cast<uint32_t>(n);
        const bool ok = in && id[h] >= 0 && id[h] < p.nkb;
        if (in && !ok) err |= C128_DEV_BAD_BLOCK;
        const uint32_t off = key - divide(key, bs) * bs.value;
        const uint8_t* blk = p.kc + static_cast<int64_t>(ok ? id[h] : 0) * p.kc_stride0;
        from[h] = ok ? blk + static_cast<int64_t>(off) * kTokenStride : nullptr;
        sc[h] = blk + p.kv_bs * kTokenStride + static_cast<int64_t>(off) * kScaleDim;
        d.data[32 * h + lane] = from[h];
        d.scales[32 * h + lane] = sc[h];
        mask |= static_cast<uint64_t>(__ballot_sync(0xffffffffu, ok)) << (32 * h);
      }
      const bool last_of_request = tile + 1 == tiles;
      if (lane == 0) {
        d.mask = mask;
        d.flags = (tile == started ? kFirst : 0) | (last_of_request || (r == end_request && tile + 1 == end_tile) ? kLast : 0) | (stretch & 3) << kRunShift;
        d.request = static_cast<int32_t>(r);
        d.part = started == 0 && last_of_request ? -1 : 2 * column + (started == 0 ? 1 : 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_full[slot]);
      // Into L2, line by line (a bulk prefetch is one operation per lane, some 40 cycles each).
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (from[h] != nullptr) {
#pragma unroll
          for (int b = 0; b < kTokenStride; b += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(from[h] + b));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(sc[h]));
        }
      }
      if (last_of_request) {
        ++stretch;
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
      ends = r == end_request && tile == end_tile;
      if (!ends) load_ids();
    }
    if (err) atomicOr(p.err, err);
  } else if (warp < kSoftWarp) {
    // ------------------------------------------------------------------------ decode the entries
    // (Results are stored in two places of this code, not three, for the sake of the instruction cache.)
    // Four threads per entry; thread `sub` of an entry takes the 16 bytes sub, sub + 4, ...: of the
    // codes a quarter of each 64-column chunk, so load j belongs to scale j.
    const int key = 8 * warp + (lane >> 2), sub = lane & 3;
    // where its first 16 bytes go: decoded codes to two places of a chunk, rope values to one
    const uint32_t row = smem_addr(sm.k[0]) + key * 128, swz = static_cast<uint32_t>(key & 7) << 4;
    const uint32_t dst0 = row + ((32u * sub) ^ swz), dst1 = row + ((32u * sub + 16u) ^ swz);
    const uint32_t dst_rope = row + 7 * kChunkBytes + ((16u * sub) ^ swz);
    // Loads on their way, a tile ahead: codes to registers; rope values, which are only moved, by way of shared
    // memory, as far as there is room (with all nine in registers, which spilled, a tile took 5 % longer; with all nine
    // in shared memory, where fewer heads leave room, 3 %).
    constexpr int kInRegs = 9 - kStaged;
    uint4 raw[kInRegs];
    const uint32_t stage = smem_addr(sm.stage[0]) + threadIdx.x * 16;
    auto stage_at = [&](int j) { return stage + (j - kInRegs) * kStageBytes; };
    uint2 sc;
    const uint8_t* src = nullptr;
    const uint8_t* ssrc = nullptr;
    int flags = kEnd;
    auto load = [&](int j) {
      if (j >= kInRegs) {
        const uint8_t* from = src == nullptr ? p.workspace : src + 64 * j;
        const uint32_t bytes = src == nullptr ? 0 : ALIGN16 ? 16 : 8;  // 0: zeros, and nothing is read
        if constexpr (ALIGN16) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(stage_at(j)), "l"(from), "r"(bytes) : "memory");
        } else {
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(stage_at(j)), "l"(from), "r"(bytes) : "memory");
          asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(stage_at(j) + 8), "l"(from + (bytes ? 8 : 0)), "r"(bytes) : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      } else if (src == nullptr) {
        raw[j] = make_uint4(0, 0, 0, 0);
      } else {
        raw[j] = ALIGN16 ? ld16(src + 64 * j) : ld8x2(src + 64 * j);
      }
    };
    auto take = [&](int j) {
      if (j < kInRegs) return raw[j];
      uint4 v;
      asm volatile("cp.async.wait_group %0;" ::"n"(kStaged - 1) : "memory");  // the oldest, of this thread's own
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(stage_at(j)) : "memory");
      return v;
    };
    auto load_scales = [&] { sc = src == nullptr ? make_uint2(0x7f7f7f7fu, 0x7f7f7f7fu) : ld8(ssrc); };
    // take tile i's addresses out of the ring
    auto fetch = [&](int i) {
      const int slot = i % kRing;
      flags = tile_flags(i);
      src = sm.ring[slot].data[key];
      ssrc = sm.ring[slot].scales[key];
      if (flags & kEnd) src = nullptr;
      if (src != nullptr) src += 16 * sub;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ring_free[slot]);
    };
    // the results of the stretch that tile i ended
    auto results = [&](int i, int flags_i) {
      const int stretch = flags_i >> kRunShift;
      warp_wait(&sm.k_free[i & 1][kQuarters - 1], (i / 2) & 1);
      // (that of the stretch after next needs a tile of these warps, so the parity means this one)
      warp_wait(&sm.inv_full[stretch & 1], stretch >> 1 & 1);
      if (!*abort_flag) store_results(sm, p, heads, 2 + warp / 4, stretch & 1);
    };
    fetch(0);
    load_scales();
    // in the order of their use, as the loop has them
#pragma unroll
    for (int j = 0; j < 4; ++j) load(j);
    load(7);
    load(8);
#pragma unroll
    for (int j = 4; j < 7; ++j) load(j);
    int done1 = 0, done2 = 0;  // flags of the tile before this one, and of the one before it
    int i = 0;
    for (; !(flags & kEnd); ++i) {
      // the buffer is free when O has taken the tile two before; if that ended a run, its results come first
      if (done2 & kLast) results(i - 2, done2);
      const int buf = i & 1;
      done2 = done1;
      done1 = flags;
      const uint2 now = sc;
      auto decode = [&](int j, uint32_t (&o)[8]) {
        const float scale = scale_of(((j < 4 ? now.x : now.y) >> (8 * (j & 3))) & 0xffu);
        const uint4 r = take(j);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          o[2 * k] = codes_to_bf16(static_cast<uint16_t>(w[k]), scale);
          o[2 * k + 1] = codes_to_bf16(static_cast<uint16_t>(w[k] >> 16), scale);
        }
        load(j);  // of the next tile
      };
      auto store = [&](int j, const uint32_t (&o)[8]) {
        const uint32_t at = buf * kTileBytes + j * kChunkBytes;
        sts16(dst0 + at, o[0], o[1], o[2], o[3]);
        sts16(dst1 + at, o[4], o[5], o[6], o[7]);
      };
      auto await_room = [&](int quarter) {
        if (i >= 2) warp_wait(&sm.k_free[buf][quarter], (i / 2 - 1) & 1);
      };
      auto publish = [&](int half) {
        async_proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.k_full[buf][half]);
      };
      fetch(i + 1);
      load_scales();
      // As much as there are registers for is decoded before its room in the buffer is free.
      uint32_t o[kAhead][8];
      constexpr auto at = [](int j) { return (j & 3) % kAhead; };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) decode(j, o[j]);
      await_room(1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j >= kAhead) decode(j, o[at(j)]);
        store(j, o[at(j)]);
      }
      publish(0);
      await_room(3);
      uint32_t large = 0;
#pragma unroll
      for (int j = 7; j < 9; ++j) {  // the rope columns are bf16 already; the sooner the next ones are on their way, the better
        const uint4 r = take(j);
        sts16((dst_rope + buf * kTileBytes) ^ (64u * (j - 7)), r.x, r.y, r.z, r.w);
        load(j);
        large = larger2(larger2(large, larger2(r.x, r.y)), larger2(r.z, r.w));
      }
      // (What stands there is of tile i - 2, whose last P has been used.)
      if (too_large(now, large)) sm.off[buf] = i + 1;
#pragma unroll
      for (int j = 4; j < 4 + kAhead; ++j) decode(j, o[at(j)]);
#pragma unroll
      for (int j = 4; j < 7; ++j) {
        if (j >= 4 + kAhead) decode(j, o[at(j)]);
        store(j, o[at(j)]);
      }
      publish(1);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // nothing may be in flight when the CTA ends
#pragma unroll 1
    for (int k = 2; k > 0; --k) {  // the last two tiles'
      if (done2 & kLast) results(i - k, done2);
      done2 = done1;
    }
  } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
    // ------------------------------------------------------------------------ issue the products
    // One elected thread in one branch: the compiler then keeps descriptors in uniform registers, and
    // a product issues faster than it runs (23 to 32 cycles for S, 39 to 48 for O, bound by the reads of
    // the operands from shared memory). Behind a test of the lane each took 66 to 75 cycles to issue.
    // The loops are short, and the same for both buffers: five warps with five programs share a scheduler's
    // instruction cache, and with this code unrolled and twice a tile took 5 % longer.
    if (elect_one()) {
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        if (decode_wait(bar, parity, abort_flag)) return true;
        *abort_flag = 1;
        return false;
      };
      const uint32_t k_at = smem_addr(sm.k[0]);
      if (warp == kMmaWarp) {
        const uint32_t q_at = desc_low(smem_addr(sm.q), 16), ks_at = desc_low(k_at, 16);
        const uint32_t desc = mma_desc(kTile, heads16, false);
        const int boxes = heads16 / kBoxHeads;
        const uint32_t box_bytes = static_cast<uint32_t>(min(p.heads, kBoxHeads)) * 128;
        auto half_of_s = [&](int buf, auto which) {
          constexpr int half = decltype(which)::value;
          tmem_fence_after();
#pragma unroll 1
          for (int k = 0; k < kChunks / 2; ++k) {
            constexpr int c0 = half * (kChunks / 2);
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
              const uint32_t a = ks_at + ((buf * kTileBytes + (c0 + k) * kChunkBytes + ks * 32) >> 4);
              const uint32_t b = q_at + (((c0 + k) * (kGroup * 128) + ks * 32) >> 4);
              mma(tmem + kTmemS + buf * kGroup, desc64(a), desc64(b), desc, half + k + ks > 0);
            }
          }
        };
        int seg = -1;  // requests begun
        bool loading = false;
        for (int i = 0;; ++i) {
          const int slot = i % kRing, buf = i & 1;
          if (!wait(&sm.ring_full[slot], (i / kRing) & 1)) break;
          const int flags = sm.ring[slot].flags, request = sm.ring[slot].request;
          if (flags & kEnd) break;
          mbar_arrive(&sm.ring_free[slot]);
          if (flags & kFirst) {
            if (++seg > 0 && !wait(&sm.q_free, (seg - 1) & 1)) break;
            mbar_arrive_expect_tx(&sm.q_full, static_cast<uint32_t>(boxes * kChunks) * box_bytes);
            for (int b = 0; b < boxes; ++b)
              for (int c = 0; c < kChunks; ++c)
                load_query_box(sm.q + c * (kGroup * 128) + b * (kBoxHeads * 128), &q_map, 64 * c,
                               group * group_heads + b * kBoxHeads, request, &sm.q_full);
            loading = true;
          }
          if (i >= 2 && !wait(&sm.s_free[buf], (i / 2 - 1) & 1)) break;
          if (loading) {
            if (!wait(&sm.q_full, seg & 1)) break;
            loading = false;
          }
          if (!wait(&sm.k_full[buf][0], (i / 2) & 1)) break;
          half_of_s(buf, Const<0>());
          if (!wait(&sm.k_full[buf][1], (i / 2) & 1)) break;
          half_of_s(buf, Const<1>());
          mma_commit(&sm.s_full[buf]);
          if (flags & kLast) mma_commit(&sm.q_free);
        }
        if (loading) decode_wait(&sm.q_full, seg & 1, nullptr);  // nothing may be in flight when the CTA ends
      } else {
        const uint32_t kv_at = desc_low(k_at, kChunkBytes), p_at = desc_low(smem_addr(sm.p[0]), 16);
        const uint32_t desc = mma_desc(128, heads16, true), desc_ones = mma_desc(64, heads16, false) | 1u << 16;  // (of P the other way around)
        const uint64_t ones = desc_plain(smem_addr(sm.ones));
        auto product_o = [&](int buf, bool first) {
          tmem_fence_after();
#pragma unroll
          for (int mt = 0; mt < kQuarters; ++mt) {
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks) {
              const uint32_t a = kv_at + ((buf * kTileBytes + 2 * mt * kChunkBytes + ks * 2048) >> 4);
              const uint32_t b = p_at + ((buf * (kGroup * kTile * 2) + ks * 2048) >> 4);
              mma(tmem + mt * kGroup, desc64(a), desc64(b), desc, !first || ks > 0);
            }
            if (mt == kQuarters - 1) {
#pragma unroll
              for (int ks = 0; ks < kTile / 16; ++ks)
                mma(tmem + kTmemL, ones, desc64(p_at + ((buf * (kGroup * kTile * 2) + ks * 2048) >> 4)), desc_ones, !first || ks > 0);
            }
            mma_commit(&sm.k_free[buf][mt]);
          }
        };
        int seg = -1;
        uint32_t phase = 0;  // of p_full, bit b of buffer b
        for (int i = 0;; ++i) {
          const int slot = i % kRing, buf = i & 1;
          if (!wait(&sm.ring_full[slot], (i / kRing) & 1)) break;
          const int flags = sm.ring[slot].flags;
          if (flags & kEnd) break;
          mbar_arrive(&sm.ring_free[slot]);
          if (!wait(&sm.p_full[buf], phase >> buf & 1)) break;
          phase ^= 1u << buf;
          if (sm.off[buf] == i + 1) {  // that was made with references that are off: another comes
            if (!wait(&sm.p_full[buf], phase >> buf & 1)) break;
            phase ^= 1u << buf;
          }
          // the results of the run before are out of O
          if ((flags & kFirst) && ++seg > 0 && !wait(&sm.o_free, (seg - 1) & 1)) break;
          product_o(buf, flags & kFirst);
        }
      }
      mma_commit(&sm.drained);
      decode_wait(&sm.drained, 0, nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------------------ softmax
    const int w = warp & 3;                          // TMEM lanes 32w .. 32w + 31
    const int own = (warp - kSoftWarp) / 4 * kOwn;   // this warp's first head
    const bool lead = own == 0;
    const uint32_t lanes = static_cast<uint32_t>(32 * w) << 16;
    const int key0 = 16 * w + (lane >> 2), key1 = key0 + 8;  // this thread's two entries of a tile
    const int h0 = own + 2 * (lane & 3);  // and its heads: h0 and h0 + 1, and on in steps of 8
    const float c2 = p.scale * kLog2e;
    float2 l[kOwn / 8];            // its sums: of heads h0 + 8g and + 1 in l[g]
    bool zero = true, fresh = true;  // the references are 0; the run has had no entry yet
    uint32_t soft_phase = 0, p_phase = 0;  // p_phase: bit b of buffer b
    auto soft_sync = [&] {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.soft);
      warp_wait(&sm.soft, soft_phase);
      soft_phase ^= 1;
    };
    for (int i = 0;; ++i) {
      const int slot = i % kRing, buf = i & 1;
      const int flags = tile_flags(i);
      const uint64_t mask = sm.ring[slot].mask;
      if (flags & kEnd) break;
      // the P of two tiles ago has been used
      if (i >= 2) warp_wait(&sm.k_free[buf][kQuarters - 1], (i / 2 - 1) & 1);
      const bool in0 = mask >> key0 & 1, in1 = mask >> key1 & 1;
      const bool first = flags & kFirst;
      const uint32_t s_at = tmem + lanes + kTmemS + buf * kGroup;
      if (first) {
        fresh = zero = true;
#pragma unroll
        for (int g = 0; g < kOwn / 8; ++g) l[g] = make_float2(0.f, 0.f);
      }
      warp_wait(&sm.s_full[buf], (i / 2) & 1);
      tmem_fence_after();
      // P with the references as they are; a warp that finds one off leaves word before it arrives. The
      // second product looks there when all have arrived, and so do the warps: then once more, and only
      // once, with new references. (A vote before the arrival took 5 % of a tile's time.)
      float2 sums[kOwn / 8];
      for (bool again = false;; again = true) {
        bool off = false;
        const bool any = fresh && __any_sync(0xffffffffu, in0 || in1);  // else no entry here speaks for a head
        const uint32_t p_at = smem_addr(sm.p[buf]) + key0 * 128 + 4 * (lane & 3);
        const uint32_t swz = static_cast<uint32_t>(key0 & 7) << 4;  // key1 & 7 is the same
        // The sums of a thread's two weights stand for the higher of the two in these checks.
        float high = 0.f;
        if (own < heads16) {
          uint32_t x[kOwn / 2];
          tmem_ld_scores<kOwn>(s_at + own, x);  // scores of absent heads are there, and not used
          tmem_wait_ld();
          uint32_t packed[kOwn / 4];
          const float2 scale = make_float2(c2, c2);
#pragma unroll
          for (int g = 0; g < kOwn / 8; ++g) {
            // log2-scaled scores over the reference, -inf where there is no entry
            const uint32_t* y = x + 4 * g;
            float2 t0 = mul2(make_float2(__uint_as_float(y[0]), __uint_as_float(y[1])), scale);
            float2 t1 = mul2(make_float2(__uint_as_float(y[2]), __uint_as_float(y[3])), scale);
            if (!zero) {
              // the product is rounded before the difference, as a reference is: the highest is then 0 exactly
              const float2 ref = *reinterpret_cast<const float2*>(&sm.ref[h0 + 8 * g]);
              t0 = make_float2(__fsub_rn(t0.x, ref.x), __fsub_rn(t0.y, ref.y));
              t1 = make_float2(__fsub_rn(t1.x, ref.x), __fsub_rn(t1.y, ref.y));
            }
            if (!in0) t0 = make_float2(-INFINITY, -INFINITY);
            if (!in1) t1 = make_float2(-INFINITY, -INFINITY);
            const float2 e0 = make_float2(ex2_approx(t0.x), ex2_approx(t0.y));
            const float2 e1 = make_float2(ex2_approx(t1.x), ex2_approx(t1.y));
            sums[g] = add2(e0, e1);
            packed[2 * g] = pack_bf16x2(e0.x, e0.y);
            packed[2 * g + 1] = pack_bf16x2(e1.x, e1.y);
            float2 s = sums[g];
            if (heads < own + kOwn) {  // absent heads pass any check
              if (h0 + 8 * g >= heads) s.x = 1.f;
              if (h0 + 8 * g + 1 >= heads) s.y = 1.f;
            }
            high = fmaxf(high, fmaxf(s.x, s.y));
            if (any) {
              const unsigned four = 0x11111111u << (lane & 3);  // the lanes that hold these heads
              off |= (__ballot_sync(0xffffffffu, s.x > kLow) & four) == 0;
              off |= (__ballot_sync(0xffffffffu, s.y > kLow) & four) == 0;
            }
          }
#pragma unroll
          for (int g = 0; g < kOwn / 8; ++g) {
            const uint32_t at = p_at + ((16u * (own / 8 + g)) ^ swz);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(packed[2 * g]) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(packed[2 * g + 1]) : "memory");
          }
        }
        off |= high > kHigh;
        if (off && !again) sm.off[buf] = i + 1;
        tmem_fence_before();
        async_proxy_fence();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[buf]);
        warp_wait(&sm.p_full[buf], p_phase >> buf & 1);
        p_phase ^= 1u << buf;
        if (again || sm.off[buf] != i + 1) break;
        tmem_fence_after();
        // New references: the maxima so far of all heads. O and the sums are rescaled to them.
        if (own < heads16) {
          uint32_t x[kOwn / 2];
          tmem_ld_scores<kOwn>(s_at + own, x);
          tmem_wait_ld();
#pragma unroll
          for (int g = 0; g < kOwn / 8; ++g) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float top = fmaxf(in0 ? __fmul_rn(__uint_as_float(x[4 * g + c]), c2) : -INFINITY,
                                in1 ? __fmul_rn(__uint_as_float(x[4 * g + 2 + c]), c2) : -INFINITY);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
              if (lane < 4) sm.by_warp[w][h0 + 8 * g + c] = top;
            }
          }
        }
        soft_sync();
        float to[kGroup / 32];  // two heads per lane of every warp
        float f[kGroup / 32];
#pragma unroll
        for (int a = 0; a < kGroup / 32; ++a) {
          const int h = 32 * a + lane;
          const float top = fmaxf(fmaxf(sm.by_warp[0][h], sm.by_warp[1][h]), fmaxf(sm.by_warp[2][h], sm.by_warp[3][h]));
          const float was = zero ? 0.f : sm.ref[h];
          // without an entry so far sums and O are 0; a head of which all scores are -inf keeps its reference
          to[a] = top == -INFINITY ? was : fresh ? top : fmaxf(top, was);
          f[a] = fresh ? 1.f : ex2_approx(was - to[a]);
        }
        soft_sync();  // all have read the old ones
        if (lead && w == 0) {
#pragma unroll
          for (int a = 0; a < kGroup / 32; ++a) sm.ref[32 * a + lane] = to[a], sm.factor[32 * a + lane] = f[a];
        }
        if (!first) warp_wait(&sm.k_free[(i - 1) & 1][kQuarters - 1], ((i - 1) / 2) & 1);
        soft_sync();
#pragma unroll
        for (int g = 0; g < kOwn / 8; ++g) {
          l[g].x *= sm.factor[h0 + 8 * g];
          l[g].y *= sm.factor[h0 + 8 * g + 1];
        }
        if (!first) {
          tmem_fence_after();
#pragma unroll 1
          for (int mt = 0; mt < 5; ++mt) {  // O and L
#pragma unroll 1
            for (int h = lead ? 0 : 16; h < heads16; h += 32) {
              uint32_t o[16];
              const uint32_t at = tmem + lanes + (mt < 4 ? mt * kGroup : kTmemL) + h;
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
        zero = fresh = false;
      }
      fresh = fresh && mask == 0;
#pragma unroll
      for (int g = 0; g < kOwn / 8; ++g) l[g] = add2(l[g], sums[g]);  // of absent heads: unused
      const int request = sm.ring[slot].request, part = sm.ring[slot].part;
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.s_free[buf]);
        mbar_arrive(&sm.ring_free[slot]);
      }
      if (!(flags & kLast)) continue;

      // ---------------------------------------------------------------------- the run's result
      const bool whole = part < 0;
      const int group0 = sm.group * sm.group_heads;  // the first head of this CTA
#pragma unroll
      for (int g = 0; g < kOwn / 8; ++g) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float sum = e ? l[g].y : l[g].x;
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
          if (lane < 4) sm.by_warp[w][h0 + 8 * g + e] = sum;
        }
      }
      soft_sync();
      // lse, while the last product runs, and what the entries have of all weight (the sink's too) into `inv`: the
      // stretch before the last, which had this one, is stored, since the last one's O was done when these warps stored it
      const int stretch = flags >> kRunShift, odd = stretch & 1;
      if (lead && w < 2 && 32 * w + lane < heads) {
        const int h = 32 * w + lane;
        const int64_t head = group0 + h;
        const float own = (sm.by_warp[0][h] + sm.by_warp[1][h]) + (sm.by_warp[2][h] + sm.by_warp[3][h]), ref = zero ? 0.f : sm.ref[h];
        float sum = own, to = ref, share = own == 0.f ? 0.f : 1.f;
        if (whole && p.sink != nullptr) {  // one more score, with a value of zero
          const float s = __ldcg(p.sink + head) * kLog2e;
          // (with nothing else in the sum, or if it is far above the rest, the result is 0 and lse the sink's)
          to = own == 0.f ? (s == -INFINITY ? 0.f : s) : fmaxf(ref, s);
          const float entries = own == 0.f ? 0.f : own * ex2_approx(ref - to);
          sum = entries + ex2_approx(s - to);
          if (own != 0.f) share = entries / sum;
        }
        sm.inv[odd][h] = share;
        const float lse2 = sum == 0.f ? -INFINITY : to + log2f(sum);
        if (!*abort_flag) {
          if (!whole)
            reinterpret_cast<float*>(p.workspace + sm.lay.lse_at())[sm.lay.row(part, sm.group, h)] = lse2;
          else if (p.lse != nullptr)
            p.lse[request * p.lse_stride_r + head * p.lse_stride_h] = lse2 * 0.69314718055994531f;
        }
      }
      if (lead && w == 0 && lane == 0) sm.done_request[odd] = request, sm.done_part[odd] = part;
      warp_wait(&sm.k_free[buf][kQuarters - 1], (i / 2) & 1);
      if (lead && w < 2 && 32 * w < heads16) {
        tmem_fence_after();
#pragma unroll 1
        for (int h = 32 * w; h < min(heads16, 32 * w + 32); h += 16) {  // every row of L is the same
          uint32_t x[16];
          tmem_ld_32x16(tmem + lanes + kTmemL + h, x);
          tmem_wait_ld();
          if (lane == 0) {
#pragma unroll
            for (int k = 0; k < 16; k += 4) *reinterpret_cast<uint4*>(&sm.sums[h + k]) = make_uint4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          }
        }
        __syncwarp();
        if (32 * w + lane < heads && sm.inv[odd][32 * w + lane] != 0.f) sm.inv[odd][32 * w + lane] /= sm.sums[32 * w + lane];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.inv_full[odd]);
      warp_wait(&sm.inv_full[odd], stretch >> 1 & 1);
      if (!*abort_flag) store_results(sm, p, heads, lead ? 0 : 1, odd);
    }
  }
  tmem_fence_before();
  __syncthreads();
  if (*abort_flag) give_up(sm, p.workspace, p.heads, p.err);
  if (warp == kMmaWarp) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols) : "memory");
  }
}

// ------------------------------------------------------------------- join the partial results
// out = sum_k 2^(lse_k - L) part_k, in the layout of the parts: a warp takes four heads and 32 or 128
// columns of a cut request, 16 bytes per lane, part and 32 columns. What it takes is the trips to L2 one
// behind the other: who has been cut, that task, and then the parts' statistics and values at once. One
// request in 16 parts takes 3.4 us, 64 requests in about 200 parts of 64 heads (26 MB) 6.
constexpr int kJoinThreads = 128;
constexpr int kJoinPerSm = 4;  // CTAs that fit (registers)
constexpr int kMaxCtas = 1024;

__device__ __forceinline__ float4 ld16_if(bool p, const float* from) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t@p ld.global.v4.f32 {%0, %1, %2, %3}, [%5];\n}"
               : "+f"(v.x), "+f"(v.y), "+f"(v.z), "+f"(v.w)
               : "r"(static_cast<uint32_t>(p)), "l"(from));
  return v;
}

// Heads head .. head + 3, columns 32 * block .. of BLOCKS blocks.
template <int BLOCKS>
__device__ __forceinline__ void join_columns(const DecodeParams& p, const Layout& lay, const Task t, int head, int block) {
  constexpr int kFlight = 16 / BLOCKS;  // parts whose values are on their way at once
  const int lane = threadIdx.x & 31;
  const int size = t.group_heads >> 5, group = head >> (4 + size), h = head & (t.group_heads - 1);
  // (at most 2 * 1024 * 64 rows of 512 floats: in 32 bits)
  const int first = ((2 * t.column + 1) * lay.groups + group) * lay.heads, step = 2 * lay.groups * lay.heads;
  auto row = [&](int k) { return first + k * step - (k > 0 ? lay.groups * lay.heads : 0); };  // slots 2c + 1, 2c + 2, 2c + 4, ...
  const float* lse = reinterpret_cast<const float*>(p.workspace + lay.lse_at());
  const float* part = reinterpret_cast<const float*>(p.workspace + lay.out_at()) + (block * (lay.heads / 4) + h / 4) * 128 + 4 * lane;
  float4 v[kFlight][BLOCKS];
  auto load = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) v[u][b] = ld16_if(k0 + u < t.parts, part + row(k0 + u) * kHead + b * (lay.heads * 32));
  };
  load(0);
  // the parts' statistics: lane = 4 * part + head within eight parts, reduced over the parts
  const int hh = lane & 3;
  const bool real = head + hh < p.heads;
  auto lse_of = [&](int k) { return k < t.parts && real ? lse[row(k) + h + hh] : -INFINITY; };
  const float sink = p.sink != nullptr && real ? __ldcg(p.sink + head + hh) * kLog2e : -INFINITY;
  float top = -INFINITY;
  bool nan = false;
  for (int k = lane >> 2; k < t.parts; k += 8) {
    const float x = lse_of(k);
    nan |= x != x;
    top = fmaxf(top, x);
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    nan |= __shfl_xor_sync(0xffffffffu, static_cast<int>(nan), o) != 0;
  }
  const unsigned gone = __ballot_sync(0xffffffffu, top == kNotThere);  // bit e: of head e, and on in steps of 4
  top = fmaxf(top, sink);
  const float shift = nan ? NAN : top == -INFINITY ? 0.f : top;
  float acc[BLOCKS][4] = {};
  float sum = lane < 4 ? ex2_approx(sink - shift) : 0.f;  // lane 4k + hh: of head hh, some of the parts
#pragma unroll 1
  for (int k0 = 0; k0 < t.parts; k0 += kFlight) {
    if (k0 > 0) load(k0);
    float w[(kFlight + 7) / 8];
#pragma unroll
    for (int j = 0; j < (kFlight + 7) / 8; ++j) {
      w[j] = ex2_approx(lse_of(k0 + 8 * j + (lane >> 2)) - shift);
      if (kFlight >= 8 || (lane >> 2) < kFlight) sum += w[j];
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = __shfl_sync(0xffffffffu, w[u / 8], 4 * (u % 8) + e);
#pragma unroll
      for (int b = 0; b < BLOCKS; ++b) {
        acc[b][0] = fmaf(f[0], v[u][b].x, acc[b][0]), acc[b][1] = fmaf(f[1], v[u][b].y, acc[b][1]);
        acc[b][2] = fmaf(f[2], v[u][b].z, acc[b][2]), acc[b][3] = fmaf(f[3], v[u][b].w, acc[b][3]);
      }
    }
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float f = __shfl_sync(0xffffffffu, inv, e);
    if (head + e >= p.heads) break;
    if (gone >> e & 1) continue;
    const int64_t at = t.request * p.out_stride_r + (head + e) * p.out_stride_h + 32 * block + lane;
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      const float x = acc[b][e] * f;
      if (p.out_f32) static_cast<float*>(p.out)[at + 32 * b] = x;
      else static_cast<uint16_t*>(p.out)[at + 32 * b] = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
    }
  }
  if (p.lse != nullptr && block == 0 && lane < 4 && real && !(gone >> lane & 1))
    p.lse[t.request * p.lse_stride_r + (head + lane) * p.lse_stride_h] =
        sum == 0.f ? -INFINITY : (shift + log2f(sum)) * 0.69314718055994531f;
}

__global__ void __launch_bounds__(kJoinThreads, kJoinPerSm) join_kernel(const DecodeParams p, const __grid_constant__ Layouts layouts) {
  launch_dependents();
  grid_dependency_wait();
  const Task* tasks = reinterpret_cast<const Task*>(p.workspace);
  const int lane = threadIdx.x & 31;
  // The CTAs that start a cut request: lane w has those of 32 w .. 32 w + 31, and how many come before.
  const int ctas = layouts.of[2].ctas;
  unsigned votes = 0;
  static_assert(kMaxCtas <= 32 * 32, "a word of votes for each lane");
#pragma unroll 1
  for (int w0 = 0; 32 * w0 < ctas; w0 += 5) {  // 160 CTAs at once
    bool has[5];
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const int c = 32 * (w0 + k) + lane;
      has[k] = c < ctas && tasks[c].parts > 0;
    }
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const unsigned vote = __ballot_sync(0xffffffffu, has[k]);
      if (lane == w0 + k) votes = vote;
    }
  }
  int behind = __popc(votes);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, behind, o);
    if (lane >= o) behind += u;
  }
  const int count = __shfl_sync(0xffffffffu, behind, 31), before = behind - __popc(votes);
  const int heads4 = (p.heads + 3) / 4;
  const int warps = gridDim.x * (kJoinThreads / 32);
  // Few: a warp for each 32 columns. Many: 128 columns, so that with the few parts of each there is enough on
  // its way, and a request's statistics are made less often.
  const bool many = count * heads4 * 16 > warps;
  const unsigned per_head4 = many ? 4 : 16, items = count * heads4 * per_head4;
#pragma unroll 1
  for (unsigned item = blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5); item < items; item += warps) {
    const unsigned rest = item / per_head4, block = item - rest * per_head4;
    const int n = rest / static_cast<unsigned>(heads4), head4 = rest - n * heads4;
    // the n-th of those CTAs
    const int word = __ffs(__ballot_sync(0xffffffffu, before <= n && n < behind)) - 1;
    const unsigned bits = __shfl_sync(0xffffffffu, votes, word);
    const int rank = n - __shfl_sync(0xffffffffu, before, word);
    const int bit = __ffs(__ballot_sync(0xffffffffu, (bits >> lane & 1) && __popc(bits & ((1u << lane) - 1)) == rank)) - 1;
    const Task t = tasks[32 * word + bit];
    const Layout& lay = layouts.of[t.group_heads >> 5];  // 16, 32, 64 -> 0, 1, 2
    if (many) join_columns<4>(p, lay, t, 4 * head4, 4 * block);
    else join_columns<1>(p, lay, t, 4 * head4, block);
  }
}

constexpr int kDecodeSmemBytes = sizeof(DecodeSmem) + 1024;
static_assert(kDecodeSmemBytes <= 232448, "shared memory of one SM, with its alignment");

// The queries as [512, heads, requests]; a box is 64 columns of 16 heads of one request.
bool encode_query_map(const DecodeParams& p, CUtensorMap* map) {
  const cuuint64_t dims[3] = {kHead, static_cast<cuuint64_t>(p.heads), static_cast<cuuint64_t>(p.requests)};
  // the stride of a dimension with one index does not matter but has to be valid
  const cuuint64_t strides[2] = {p.heads > 1 ? static_cast<cuuint64_t>(p.q_stride_h) * 2 : kHead * 2,
                                 p.requests > 1 ? static_cast<cuuint64_t>(p.q_stride_r) * 2 : kHead * 2};
  const cuuint32_t size[3] = {64, static_cast<cuuint32_t>(p.heads < kBoxHeads ? p.heads : kBoxHeads), 1};
  const cuuint32_t step[3] = {1, 1, 1};
  auto enc = tensor_map_encoder();
  return enc != nullptr &&
         enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(p.q), dims, strides, size, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

namespace {
// The kernel for caches whose records start on 16 or 8 bytes, and for all heads in one group of 16 or
// 32 (which frees registers) or in groups of up to 64.
const void* decode_kernel_for(bool align16, int heads) {
  if (heads <= 16) return reinterpret_cast<const void*>(align16 ? decode_kernel<true, 16> : decode_kernel<false, 16>);
  if (heads <= 32) return reinterpret_cast<const void*>(align16 ? decode_kernel<true, 32> : decode_kernel<false, 32>);
  return reinterpret_cast<const void*>(align16 ? decode_kernel<true, 64> : decode_kernel<false, 64>);
}
}  // namespace

cudaError_t prepare_decode() {
  cudaError_t e = cudaSuccess;
  for (int heads = 16; heads <= 64; heads *= 2)
    for (int align16 = 0; align16 < 2; ++align16)
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(decode_kernel_for(align16 != 0, heads), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kDecodeSmemBytes);
  return e;
}

int64_t decode_workspace_bytes(int heads, int sm_count) { return Layout(heads, sm_count, kGroup).bytes(); }

cudaError_t launch_decode(const DecodeParams& p, int sm_count, cudaStream_t stream) {
  CUtensorMap map;
  if (!encode_query_map(p, &map)) return cudaErrorInvalidValue;
  Layouts layouts;
  for (int i = 0; i < 3; ++i) layouts.of[i] = Layout(p.heads, sm_count, 16 << i);
  const int ctas = layouts.of[2].ctas;
  if (ctas > kMaxCtas) return cudaErrorInvalidValue;
  const bool align16 = p.kc_stride0 % 16 == 0;  // records then start on 16 bytes, else on 8
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(static_cast<unsigned>(ctas));
  lc.blockDim = dim3(kDecodeThreads);
  lc.dynamicSmemBytes = kDecodeSmemBytes;
  lc.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = 1;
  void* args[] = {const_cast<DecodeParams*>(&p), &map, &layouts};
  const cudaError_t e = cudaLaunchKernelExC(&lc, decode_kernel_for(align16, p.heads), args);
  if (e != cudaSuccess) return e;
  const int64_t cut = p.requests < ctas ? p.requests : ctas;  // requests that can be cut
  const int64_t join_ctas = (cut * ((p.heads + 3) / 4) * 16 + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  lc.gridDim = dim3(static_cast<unsigned>(join_ctas < kJoinPerSm * sm_count ? join_ctas : kJoinPerSm * sm_count));
  lc.blockDim = dim3(kJoinThreads);
  lc.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&lc, join_kernel, p, layouts);
}

}  // namespace c128
