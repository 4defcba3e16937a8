/*
 * libc128compress — GB300 (sm_103a) DeepSeek-V4 C128 sparse-attention KV compressor.
 *
 * One stream-ordered call, compress_norm_rope_store(), does for every active token
 *   1. window gather: the 128 state-cache rows p-127 .. p of the token's request, found through
 *      the paged block table (state block size 8, so 16 whole blocks);
 *   2. a per-column softmax of score (row columns 512..1023) over those 128 rows and the
 *      softmax-weighted sum of kv (row columns 0..511): compressed[512], fp32;
 *   3. RMSNorm with weight rms_w and eps;
 *   4. FP8 e4m3 quantisation of the 448 "nope" columns with one UE8M0 (power-of-two) scale per
 *      64 columns, and interleaved-pair (GPT-J) RoPE of the 64 rope columns, stored as bf16;
 *   5. the paged k_cache store at kv_slot_mapping[t].
 * It follows the fused Triton kernel _fused_kv_compress_norm_rope_insert_sparse_attn and its
 * launcher compress_norm_rope_store_triton on the API page of
 * vllm.models.deepseek_v4.common.ops.fused_compress_quant_cache (sections "Gather state cache
 * entries", "Softmax + weighted sum", "RMSNorm", "KV cache pointers", "FP8 UE8M0 quant",
 * "GPT-J RoPE"), in the C128 layout of vLLM PR #44230 "optimize the compressor 128 split cutedsl
 * kernel" (Summary: head 512, state width 512, compress ratio 128, no overlap, state block 8;
 * Changes: reject unsupported layouts and kv_cache_block_size != k_cache.shape[1]).
 *
 * Arithmetic (where the pages leave precision open): the softmax and weighted sum run in fp32
 * (within 1e-5 relative / 1e-6 absolute of the exact value); from compressed[] on, every step is
 * a fixed IEEE computation, so the bytes are a pure function of compressed[]:
 *   var = RN32(exact(sum c^2) / 512); rrms = RN32(1 / sqrt(double(RN32(var + eps))));
 *   normed = RN32(RN32(c * rrms) * w); nope: bf16 round, absmax (floor RN32(1e-4)),
 *   e = ceil(log2(RN32(absmax * RN32(1/448)))), q = e4m3_rn_satfinite(clamp(x * 2^-e, +-448)),
 *   scale byte = clamp(e + 127, 0, 255), 8th scale byte 0; rope: e' = RN32(RN32(e*C) - RN32(o*S)),
 *   o' = RN32(RN32(o*C) + RN32(e*S)), each stored as bf16 (round to nearest even).
 *
 * A token is active iff slot_mapping[t] >= 0, positions[t] >= 0, (positions[t] + 1) % 128 == 0
 * and kv_slot_mapping[t] >= 0. Inactive tokens write nothing; no byte of k_cache outside the
 * 576 token bytes and 8 scale bytes of an active token's slot is touched.
 *
 * All tensors are caller-owned device memory described by c128_tensor_t (strides in elements).
 * The call is asynchronous on `stream`: it never synchronises the host with the GPU and never
 * reads device memory back to the host.
 * It uses a per-(device, stream) workspace owned by the library (a 256-byte header with the
 * sticky device error bits, then one int32 per token). The first call on a stream, and any call
 * with more tokens than that workspace holds, grows it stream-ordered: a new buffer from the
 * device's default memory pool (cudaMallocAsync on `stream`), the header copied device-to-device
 * on `stream`, the old buffer returned with cudaFreeAsync on `stream`. Nothing waits on the host.
 * A stream that is being captured into a CUDA graph cannot grow its workspace: such a call
 * returns C128_ERR_CAPTURE and enqueues nothing, so call c128_reserve_workspace with the largest
 * batch before capturing. A graph keeps the workspace it was captured with; a later call on the
 * same stream that grows the workspace frees that buffer, so reserve enough before capturing a
 * graph that will be replayed. Calls on the same stream are serialised by the stream; calls on
 * different streams use different workspaces. c128_release_stream returns one stream's workspace
 * (call it before destroying the stream). Two active tokens naming the same kv slot race
 * (undefined which one lands); this is not checked.
 */
#ifndef C128COMPRESS_H
#define C128COMPRESS_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same object as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* c128_stream_t;

/* Element types of c128_tensor_t. */
enum {
    C128_I32 = 1,
    C128_I64 = 2,
    C128_F32 = 3,
    C128_U8 = 4,
    C128_BF16 = 5,
};

/* A strided view of caller-owned device memory. shape/stride beyond ndim are ignored. */
typedef struct c128_tensor {
    void* data;          /* device pointer (may be NULL only when the tensor is empty) */
    int32_t dtype;       /* one of C128_I32, C128_I64, C128_F32, C128_U8, C128_BF16 */
    int32_t ndim;        /* 1 .. 4 */
    int64_t shape[4];
    int64_t stride[4];   /* in elements */
} c128_tensor_t;

/* Return codes. Every error is detected on the host before anything is launched, except
 * C128_ERR_CUDA (a CUDA call or launch failed) and C128_ERR_NOMEM (workspace allocation);
 * C128_ERR_CAPTURE is also returned before anything is enqueued. */
enum {
    C128_OK = 0,
    C128_ERR_NULL_PTR = 1,     /* a descriptor, or the data of a non-empty tensor, is NULL */
    C128_ERR_DTYPE = 2,        /* wrong element type */
    C128_ERR_SHAPE = 3,        /* wrong rank / extent, or token counts disagree */
    C128_ERR_STRIDE = 4,       /* innermost dimension not contiguous, or an unusable stride */
    C128_ERR_ALIGN = 5,        /* state_cache or k_cache base/stride not aligned (see below) */
    C128_ERR_UNSUPPORTED = 6,  /* not the C128 layout: state block != 8, row != 1024, head != 512 */
    C128_ERR_ARG = 7,          /* kv_block_size < 1 or != k_cache.shape[1]; too many tokens */
    C128_ERR_CUDA = 8,
    C128_ERR_NOMEM = 9,
    C128_ERR_TOO_MANY_TOKENS = 10, /* c128_compress_norm_rope_store_noalloc: T > C128_NOALLOC_MAX_TOKENS */
    C128_ERR_CAPTURE = 11,     /* the stream is being captured and its workspace would have to grow */
};

/* Device-side error bits (OR-ed into the stream's workspace, sticky until cleared).
 * An active token whose indices fall outside the given tensors is skipped (writes nothing)
 * and reports one of the first five bits; a bounded wait that ran out reports TIMEOUT. */
enum {
    C128_DEV_BAD_REQ = 1,        /* token_to_req_indices[t] outside [0, block_table.shape[0]) */
    C128_DEV_BAD_BT_COL = 2,     /* positions[t] / 8 >= block_table.shape[1] */
    C128_DEV_BAD_BLOCK = 4,      /* a window block id outside [0, state_cache.shape[0]) */
    C128_DEV_BAD_COS_ROW = 8,    /* window start (p/128)*128 >= cos_sin_cache.shape[0] */
    C128_DEV_BAD_KV_SLOT = 16,   /* kv_slot_mapping[t] >= k_cache.shape[0] * kv_block_size */
    C128_DEV_TIMEOUT = 32,       /* a pipeline wait exceeded its time limit; the kernel gave up */
    C128_DEV_NO_FREE_BLOCK = 64, /* c128_extend_block_tables: the list of free blocks ran out */
    C128_DEV_BAD_LENGTH = 128,   /* a length, count or block total that cannot be (see each call) */
};

/*
 * compress_norm_rope_store — the whole C128 compressor path for one batch of tokens.
 *
 *   token_to_req_indices [T]               int32  request of each token (contiguous)
 *   positions            [T]               int64  absolute position of each token (contiguous)
 *   slot_mapping         [T]               int64  state-cache slot; < 0 marks a padded token
 *   block_table          [R, MB]           int32  state-cache block ids per request; row stride
 *                                                 stride[0] >= MB, stride[1] == 1
 *   state_cache          [NB, 8, 1024]     fp32   row = kv[0:512] | score[512:1024];
 *                                                 stride[2] == 1, stride[1] >= 1024,
 *                                                 data 16-byte aligned, stride[0] and stride[1]
 *                                                 multiples of 4 elements
 *   rms_w                [512]             fp32   RMSNorm weight (contiguous)
 *   eps                                    fp32   RMSNorm epsilon
 *   cos_sin_cache        [MP, 64]          fp32   cos in [0, 32), sin in [32, 64) of row
 *                                                 (p / 128) * 128; stride[1] == 1
 *   k_cache              [NKB, bs, W>=584] uint8  written in place: block b holds bs token
 *                                                 records of 576 bytes (448 e4m3 + 64 bf16 rope)
 *                                                 at b*stride[0] + off*576, then bs x 8 scale
 *                                                 bytes (7 UE8M0 + a zero pad) at
 *                                                 b*stride[0] + bs*576 + off*8; W*bs >= bs*584,
 *                                                 data 16-byte aligned, stride[0] a multiple of 8
 *   kv_slot_mapping      [T]               int64  k_cache slot (block*bs + offset); < 0: no store
 *   kv_block_size                                 must equal k_cache.shape[1]
 *   stream                                        CUDA stream the work is enqueued on
 *
 * Returns C128_OK or a C128_ERR_* code (nothing is launched on an error). T == 0 is a no-op.
 */
int compress_norm_rope_store(const c128_tensor_t* token_to_req_indices,
                             const c128_tensor_t* positions,
                             const c128_tensor_t* slot_mapping,
                             const c128_tensor_t* block_table,
                             const c128_tensor_t* state_cache,
                             const c128_tensor_t* rms_w,
                             float eps,
                             const c128_tensor_t* cos_sin_cache,
                             const c128_tensor_t* k_cache,
                             const c128_tensor_t* kv_slot_mapping,
                             int64_t kv_block_size,
                             c128_stream_t stream);

/*
 * Test of the failure handling, for tests only. Runs compress_norm_rope_store on the same
 * arguments (C128 layout), except that CTA 0 arms the first stage of its first window and never
 * copies into it (the one-CTA-per-token kernel up to 8 tokens per SM, where CTA 0 has a window only
 * if token 0 is active; the compress kernel above).
 * Every wait in the kernels is bounded (1 s), so the consumers of that stage give up, the CTA
 * stops, and the kernel ends with C128_DEV_TIMEOUT in the device error bits (read them with
 * c128_device_errors) instead of hanging; the CUDA context stays usable. Other CTAs store their
 * windows as usual; CTA 0's windows are not stored. Takes about two seconds of GPU time. Returns
 * C128_ERR_ARG when the batch has no more tokens than the GPU has SMs (such batches run the
 * cluster-split kernel, which is not set up for this test), else the codes of
 * compress_norm_rope_store.
 */
int c128_debug_stall_first_window(const c128_tensor_t* token_to_req_indices,
                                  const c128_tensor_t* positions,
                                  const c128_tensor_t* slot_mapping,
                                  const c128_tensor_t* block_table,
                                  const c128_tensor_t* state_cache,
                                  const c128_tensor_t* rms_w,
                                  float eps,
                                  const c128_tensor_t* cos_sin_cache,
                                  const c128_tensor_t* k_cache,
                                  const c128_tensor_t* kv_slot_mapping,
                                  int64_t kv_block_size,
                                  c128_stream_t stream);

/*
 * Same as compress_norm_rope_store, and also writes the fp32 compressed vector (the softmax-
 * weighted sum, before RMSNorm) of every token it stores to comp_out [T, 512] fp32 (contiguous,
 * 16-byte aligned). Rows of other tokens are left as they were. For tests and diagnostics: it
 * exposes the quantity the byte-exact epilogue is a function of.
 */
int c128_compress_norm_rope_store_debug(const c128_tensor_t* token_to_req_indices,
                                        const c128_tensor_t* positions,
                                        const c128_tensor_t* slot_mapping,
                                        const c128_tensor_t* block_table,
                                        const c128_tensor_t* state_cache,
                                        const c128_tensor_t* rms_w,
                                        float eps,
                                        const c128_tensor_t* cos_sin_cache,
                                        const c128_tensor_t* k_cache,
                                        const c128_tensor_t* kv_slot_mapping,
                                        int64_t kv_block_size,
                                        const c128_tensor_t* comp_out,
                                        c128_stream_t stream);

/*
 * c128_compress_norm_rope_store_noalloc — the same operation, for callers that cannot allocate.
 * The pages have no counterpart to this entry point; it exists for the library's users.
 *
 * compress_norm_rope_store keeps its list of active tokens in a workspace that it allocates with
 * cudaMalloc on the first call on a stream and whenever a larger batch arrives. Some callers may
 * not allocate device memory once they are running: a serving engine that hands all free memory
 * to its KV caches at start-up and must never see an allocation (or its implicit device
 * synchronisation) on the decode path, code running inside a memory-pool or allocator callback,
 * or a host that enforces a fixed device-memory budget. This entry point allocates nothing.
 *
 * Its scratch (a 256-byte header, the token list and the planning pass's per-chunk counts) is one
 * static device array for C128_NOALLOC_MAX_TOKENS tokens (256 KiB + 384 B) in the library image;
 * every GPU that loads the library holds it until the process exits. The first call on each
 * device looks up that array's
 * device address (cudaGetSymbolAddress, with that device current) and caches it; make that first
 * call before any stream capture. Arguments, layout and results are exactly those of
 * compress_norm_rope_store; T > C128_NOALLOC_MAX_TOKENS returns C128_ERR_TOO_MANY_TOKENS without
 * launching anything. All calls share the one array: each call clears the counters it needs,
 * and calls that can overlap on the GPU (different streams, or different host threads) race and
 * corrupt each other's work. Device error bits of these calls are not readable through
 * c128_device_errors (tokens with out-of-range indices are still skipped).
 */
#define C128_NOALLOC_MAX_TOKENS 65536
int c128_compress_norm_rope_store_noalloc(const c128_tensor_t* token_to_req_indices,
                                          const c128_tensor_t* positions,
                                          const c128_tensor_t* slot_mapping,
                                          const c128_tensor_t* block_table,
                                          const c128_tensor_t* state_cache,
                                          const c128_tensor_t* rms_w,
                                          float eps,
                                          const c128_tensor_t* cos_sin_cache,
                                          const c128_tensor_t* k_cache,
                                          const c128_tensor_t* kv_slot_mapping,
                                          int64_t kv_block_size,
                                          c128_stream_t stream);

/*
 * compress_norm_rope_store_ex — the same op for the other configurations of the fused kernels
 * on the API page (one launcher, compress_norm_rope_store_triton, serves all three):
 *
 *   C128_FORMAT_SPARSE_FP8    _fused_kv_compress_norm_rope_insert_sparse_attn: head 512, rope 64;
 *                             448 e4m3 + 64 bf16 rope (576 B) then 8 scale bytes per slot
 *   C128_FORMAT_INDEXER_FP8   _fused_kv_compress_norm_rope_insert_indexer_attn: head 128, rope 64;
 *                             RoPE of the last 32 pairs first, bf16 round, one absmax block:
 *                             128 e4m3 bytes per slot, then one fp32 scale 2^e (4 B) per slot
 *   C128_FORMAT_INDEXER_MXFP4 _fused_kv_compress_norm_rope_insert_indexer_mxfp4_attn: head 128;
 *                             RoPE, bf16 round, per 32 values e = ceil(log2(absmax/6)) (absmax
 *                             floor 6*2^-126, e clamped to [-127,127]), E2M1 codes of x*2^-e
 *                             (round to nearest even, saturating), pair j in byte j with the even
 *                             value in the low nibble: 64 bytes per slot, then 4 UE8M0 bytes (e+127)
 *
 * with compress ratio `compress_ratio` (a power of two; window end: (p+1) % ratio == 0) and, when
 * `overlap` is 1, windows of 2*ratio rows whose newer `ratio` rows read kv and score at +head_dim
 * (the C4 layout); rows at negative positions take no weight. A state row is kv[state_width]
 * followed by score[state_width] (state_width >= (1+overlap)*head_dim, a multiple of 4), blocks of
 * any number of rows (state_cache [NB, block, 2*state_width]); cos/sin come from row
 * (p / ratio) * ratio. k_cache blocks hold bs token records then bs scale records, as above.
 * comp_out, if not NULL, receives the fp32 compressed vectors ([T, head_dim], contiguous, 16-byte
 * aligned) of stored tokens.
 * The k_cache block stride (stride[0], bytes) must be a multiple of 8 for the sparse format, 4 for
 * the indexer FP8 format and 2 for MXFP4 (the widest store of each), which the natural layout
 * bs x record bytes always is.
 * Everything else is as for compress_norm_rope_store; the C128 configuration (512, 64, 128, 0, 512,
 * sparse) runs the same kernels as compress_norm_rope_store when its state block is any multiple
 * of 8 rows.
 * Returns C128_ERR_NULL_PTR for a NULL config and C128_ERR_UNSUPPORTED for a configuration outside
 * the ones above (another head or rope size, a head that does not match the format, a ratio that
 * is not a power of two or makes windows longer than 256 rows, overlap other than 0 or 1, a state
 * width below (1 + overlap) * head_dim or not a multiple of 4); the tensor checks and their codes
 * are those of compress_norm_rope_store, with head_dim in place of 512.
 * Kernels: the C128 configuration with a state block that is a multiple of 8 rows runs the C128
 * kernels; windows of at most 8 rows stream through a shared-memory ring (many windows per SM);
 * longer head-128 windows whose state block is a multiple of 8 rows stream in 8-row tiled loads;
 * the rest run a gather kernel. All of them are CUDA-graph capturable.
 */
enum {
    C128_FORMAT_SPARSE_FP8 = 0,
    C128_FORMAT_INDEXER_FP8 = 1,
    C128_FORMAT_INDEXER_MXFP4 = 2,
};
typedef struct c128_config {
    int32_t head_dim;        /* 512 (sparse format) or 128 (indexer formats) */
    int32_t rope_head_dim;   /* 64 */
    int32_t compress_ratio;  /* power of two; (1 + overlap) * ratio <= 256 */
    int32_t overlap;         /* 0 or 1 */
    int32_t state_width;     /* kv columns of a state row; as many score columns follow */
    int32_t cache_format;    /* C128_FORMAT_* */
} c128_config_t;
int compress_norm_rope_store_ex(const c128_config_t* config,
                                const c128_tensor_t* token_to_req_indices,
                                const c128_tensor_t* positions,
                                const c128_tensor_t* slot_mapping,
                                const c128_tensor_t* block_table,
                                const c128_tensor_t* state_cache,
                                const c128_tensor_t* rms_w,
                                float eps,
                                const c128_tensor_t* cos_sin_cache,
                                const c128_tensor_t* k_cache,
                                const c128_tensor_t* kv_slot_mapping,
                                int64_t kv_block_size,
                                const c128_tensor_t* comp_out,
                                c128_stream_t stream);

/*
 * The same test for the other configurations (tests only): compress_norm_rope_store_ex with the
 * small-window kernel (windows of at most 8 rows) leaving the stage of the first listed window
 * unfilled, or the indexer kernel (head-128 windows of more than 8 rows) leaving CTA 0's first
 * stage unfilled, with the same outcome:
 * C128_DEV_TIMEOUT in the device error bits, the other CTAs' windows stored, the context usable.
 * Configurations served by the gather kernel (no copy warp) run normally. Returns the codes of
 * compress_norm_rope_store_ex.
 */
int c128_debug_stall_first_window_ex(const c128_config_t* config,
                                     const c128_tensor_t* token_to_req_indices,
                                     const c128_tensor_t* positions,
                                     const c128_tensor_t* slot_mapping,
                                     const c128_tensor_t* block_table,
                                     const c128_tensor_t* state_cache,
                                     const c128_tensor_t* rms_w,
                                     float eps,
                                     const c128_tensor_t* cos_sin_cache,
                                     const c128_tensor_t* k_cache,
                                     const c128_tensor_t* kv_slot_mapping,
                                     int64_t kv_block_size,
                                     c128_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * Around the compressor: the block tables and per-token arrays its call takes, made on the GPU from
 * the requests' lengths, and the attention of a decode step over the cache it writes. The calls
 * follow the rules above: caller-owned tensors, host checks that return C128_ERR_* before anything
 * is launched, asynchronous on `stream` and capturable, device error bits in the stream's workspace
 * (read with c128_device_errors; a stream without a workspace gets one, so the first call on a
 * stream that is being captured returns C128_ERR_CAPTURE unless c128_reserve_workspace came before).
 * All tensors live on the current device. Unless a call says otherwise, an output overlaps no input
 * and no other output, and (C128_ERR_STRIDE) the rows of an output do not overlap one another: those of
 * one dimension lie between two neighbours of the other.
 */

/*
 * c128_extend_block_tables — give every request the blocks that its length now needs, from a list
 * of free blocks. With entries(n) = floor(n / compress_ratio) and needed = ceil(entries(seq_lens[r])
 * / block_size), request r gets max(0, needed - held[r]) blocks; the requests are served in order:
 *   block_table[r, held[r] + j] = free_blocks[taken + (blocks given to requests before r) + j]
 * and held_out[r] = max(held[r], needed), taken_out = taken + (all blocks given). compress_ratio is
 * 1 for the state cache and the compressor's ratio for the k_cache.
 *
 *   seq_lens    [R]      int32   length of each request
 *   held        [R]      int32   blocks it holds already
 *   block_table [R, MB]  int32   in place; stride[1] == 1, stride[0] >= MB. Entries other than the
 *                                ones given are left as they were
 *   free_blocks [F]      int32   block ids, F < 2^31 - 1
 *   taken       [1]      int64   ids of free_blocks given away already
 *   held_out    [R]      int32   may be `held` itself (else: no overlap)
 *   taken_out   [1]      int64   may be `taken` itself
 *
 * Device error bits: C128_DEV_NO_FREE_BLOCK - the list ran out: the first request that it cannot
 * serve in full and every later one that needs blocks get none and keep their count;
 * C128_DEV_BAD_BT_COL - a request needs more than MB blocks (it gets none, the others are served);
 * C128_DEV_BAD_LENGTH - a negative length (counts as 0) or held count (the request gets none), or
 * taken outside [0, F] (nobody gets any).
 * Results do not depend on scheduling: the same inputs give the same tables.
 */
int c128_extend_block_tables(const c128_tensor_t* seq_lens, const c128_tensor_t* held,
                             const c128_tensor_t* block_table, const c128_tensor_t* free_blocks,
                             const c128_tensor_t* taken, int32_t compress_ratio, int64_t block_size,
                             const c128_tensor_t* held_out, const c128_tensor_t* taken_out,
                             c128_stream_t stream);

/*
 * c128_build_slot_maps — the per-token arrays of one step. Request r has seq_lens[r] tokens, the
 * last query_lens[r] of them new; the step's tokens are those of request 0, then of request 1, ...
 * Token i of request r sits at position p = seq_lens[r] - query_lens[r] + i and gets
 *   token_to_req_indices = r, positions = p,
 *   slot_mapping = state_table[r, p / state_block] * state_block + p % state_block,
 *   kv_slot_mapping = the same of entry p / compress_ratio in kv_table with kv_block_size where p
 *                     ends a window ((p + 1) % compress_ratio == 0), -1 elsewhere.
 * Rows of the per-token arrays behind the last token (a batch padded to a captured size) get request
 * 0, position 0 and slots -1, which compress_norm_rope_store skips.
 *
 *   seq_lens, query_lens [R] int32; state_table [R, MBs], kv_table [R, MBk] int32 (rows may be
 *   padded); query_start [R + 1] int32: the index of each request's first token, and their number;
 *   token_to_req_indices [T] int32; positions, slot_mapping, kv_slot_mapping [T] int64; kv_lens [R]
 *   int32: floor(seq_lens[r] / compress_ratio), the entries of the request's cache once the step's
 *   windows are stored. T < 2^31 - 1.
 *
 * Device error bits: C128_DEV_BAD_LENGTH - a negative length (counts as 0), query_lens[r] >
 * seq_lens[r] (tokens at negative positions get slots -1), or more tokens than T (those behind are
 * dropped); C128_DEV_BAD_BT_COL - a position behind the end of its table (slot -1);
 * C128_DEV_BAD_BLOCK - a negative block id where one is needed (slot -1).
 */
int c128_build_slot_maps(const c128_tensor_t* seq_lens, const c128_tensor_t* query_lens,
                         const c128_tensor_t* state_table, int64_t state_block,
                         const c128_tensor_t* kv_table, int64_t kv_block_size, int32_t compress_ratio,
                         const c128_tensor_t* query_start, const c128_tensor_t* token_to_req_indices,
                         const c128_tensor_t* positions, const c128_tensor_t* slot_mapping,
                         const c128_tensor_t* kv_slot_mapping, const c128_tensor_t* kv_lens,
                         c128_stream_t stream);

/*
 * c128_decode_attention — attention of one new token per request over its entries of the paged
 * k_cache, in the layout that the C128_FORMAT_SPARSE_FP8 compressor stores. Entry j is the vector
 * k_j of 512 values that its record stands for: e4m3 code x 2^(scale byte - 127) for the 448 "nope"
 * columns, the bf16 values for the 64 rope columns. It is key and value at once, for all heads:
 *   s_hj = scale * <q[r,h], k_j>,  j = 0 .. kv_lens[r] - 1
 *   lse[r,h] = log(sum_j exp(s_hj) + exp(sink[h]))       (the sink term only if `sink` is given)
 *   out[r,h] = sum_j exp(s_hj - lse[r,h]) k_j
 * A request without entries gets zeros and an lse of sink[h], or -inf without a sink.
 *
 *   q           [R, H, 512]   bf16   stride[2] == 1, other strides >= 512 and multiples of 8, data
 *                                    16-byte aligned; 1 <= H <= 1024
 *   k_cache     [NKB, bs, W]  uint8  as for compress_norm_rope_store; kv_block_size == bs
 *   block_table [R, MB]       int32  k_cache block of entries b*bs .. b*bs + bs - 1 of request r
 *   kv_lens     [R]           int32  entries of each request; bytes behind them are never used
 *   scale                     fp32   finite, times log2(e) too
 *   sink        [H]           fp32   may be NULL
 *   out         [R, H, 512]   bf16 or fp32, strides as for q (fp32: multiples of 4)
 *   lse         [R, H]        fp32   positive strides; may be NULL
 *   workspace   [n]           uint8  at least c128_decode_attention_workspace bytes, 256-byte
 *                                    aligned; scratch of this call: calls that can overlap on the
 *                                    GPU need one each (so do graphs that are replayed at once)
 *
 * Products take bf16 operands (the entries are exact in bf16 for scale bytes 8 .. 246; the softmax
 * weights are rounded to bf16) and add up in fp32. out is divided by the sums of the rounded weights, so
 * that of one entry is that entry; lse is of the exact ones, in fp32. The sums are relative to the largest
 * weight where they have to be: an entry may be of any magnitude, as long as the largest times the
 * number of entries stays below 2^128, but values below 2^-92 can count as 0.
 * Device error bits: C128_DEV_BAD_BT_COL - kv_lens[r] > MB*bs (the entries behind are left out);
 * C128_DEV_BAD_BLOCK - a block id outside [0, NKB) (its entries are left out); C128_DEV_BAD_LENGTH
 * - a negative kv_lens[r] (counts as 0); C128_DEV_TIMEOUT - a wait inside the kernel ran out: some of
 * the results are not there, and each value of out and lse is the result or what it was before.
 * R * (MB*bs / 64 + 2) < 2^31, else C128_ERR_ARG.
 */
int c128_decode_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                          const c128_tensor_t* block_table, const c128_tensor_t* kv_lens, float scale,
                          const c128_tensor_t* sink, const c128_tensor_t* out, const c128_tensor_t* lse,
                          const c128_tensor_t* workspace, c128_stream_t stream);

/*
 * Test of the failure handling, for tests only: c128_decode_attention, except that CTA 0 never learns of
 * its tiles. Every wait of that kernel is bounded (about 1 s), so CTA 0 gives up and ends with
 * C128_DEV_TIMEOUT in the device error bits, and stores nothing; requests (or heads) that it shares with
 * other CTAs are left as they were too, all others are computed as usual. The context stays usable.
 */
int c128_debug_stall_decode_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache,
                                      int64_t kv_block_size, const c128_tensor_t* block_table,
                                      const c128_tensor_t* kv_lens, float scale, const c128_tensor_t* sink,
                                      const c128_tensor_t* out, const c128_tensor_t* lse,
                                      const c128_tensor_t* workspace, c128_stream_t stream);

/* Bytes of workspace that c128_decode_attention needs on the current device for `num_heads` heads, whatever the
 * requests and their lengths. */
int c128_decode_attention_workspace(int64_t num_heads, int64_t* bytes);

/*
 * c128_merge_attention — join attentions of the same queries over different sets of entries (the
 * parts of a cache, or the compressed cache and the window of recent tokens) by their log-sum-exp:
 *   lse[r,h] = log(sum_p exp(part_lse[p,r,h])),
 *   out[r,h] = sum_p exp(part_lse[p,r,h] - lse[r,h]) part_out[p,r,h].
 * A part whose lse is -inf saw nothing and its part_out is not used, whatever it holds; where every
 * part is so, out is 0 and lse -inf. At most one part may have had a sink.
 *
 *   part_out [P, R, H, 512] bf16 or fp32, stride[3] == 1, rows 16-byte aligned, P >= 1
 *   part_lse [P, R, H]      fp32, any positive strides
 *   out      [R, H, 512]    bf16 or fp32 (fp32 sums, rounded once), stride[2] == 1, rows 16-byte
 *                           aligned. May be one of the parts (part_out[p], same type and strides)
 *   lse      [R, H]         fp32, positive strides; may be NULL, or the part_lse[p] of that part
 */
int c128_merge_attention(const c128_tensor_t* part_out, const c128_tensor_t* part_lse,
                         const c128_tensor_t* out, const c128_tensor_t* lse, c128_stream_t stream);

/* ------------------------------------------------------------------------------------------------
 * Around the attention of recent tokens: what makes a step's queries and the entries of its tokens, the
 * rotations that carry their positions, and the attention over the last tokens. The rules are those of
 * the calls above. A token with slot_mapping[t] < 0 or positions[t] < 0 (a batch padded to a captured size)
 * is skipped: its rows are left as they were. So is a token whose indices do not fit, which is reported.
 */

/*
 * c128_rope_t — how far each pair of columns turns with a position. Pair i of the R / 2 has the step
 * f_i = theta^(-2i/R) radians per position, changed by the scaling:
 *   C128_ROPE_PLAIN   f_i
 *   C128_ROPE_LINEAR  f_i / factor
 *   C128_ROPE_YARN    f_i (1 - g_i) + f_i / factor g_i, as the YaRN paper has it ("NTK by parts"): with
 *                     pair(b) = R ln(original_positions / (2 pi b)) / (2 ln theta), the pair that turns b
 *                     times over the original positions, low = max(floor(pair(beta_fast)), 0), high =
 *                     min(ceil(pair(beta_slow)), R - 1), g_i = (i - low) / max(high - low, 0.001) cut
 *                     to [0, 1]
 * `magnitude` multiplies every cosine and sine (YaRN's attention factor; 1 for none).
 * A step over 2^20 turns per position, which a tiny factor makes, is refused (C128_ERR_ARG).
 */
enum {
    C128_ROPE_PLAIN = 0,
    C128_ROPE_LINEAR = 1,
    C128_ROPE_YARN = 2,
};
typedef struct c128_rope {
    double theta;              /* > 1 */
    double factor;             /* > 0; plain: not used */
    double original_positions; /* the rest but magnitude: yarn only. > 0 */
    double beta_fast, beta_slow; /* > 0 */
    double magnitude;          /* finite */
    int32_t scaling;           /* C128_ROPE_* */
    int32_t reserved;          /* 0 */
} c128_rope_t;

/*
 * c128_build_cos_sin — the table that the other calls take as cos_sin_cache: row j holds the cosines of
 * position first_position + j's R / 2 angles, then their sines.
 *
 *   cos_sin_cache [MP, R] fp32  stride[1] == 1, stride[0] >= R; R even, 2 .. 512
 *   first_position        0 <= first_position, first_position + MP <= 2^32
 *
 * Angles are kept as 64-bit fractions of a turn, which whole turns drop out of without rounding, so the product
 * of position and step adds no error. The steps are made in double, and their rounding grows with the position: an
 * angle is within 2^-30 + 2^-46 * (its turns, scaled or not, whichever are more) of position * step, so 2^-29.3 for
 * the first pair at position 2^18 and 2^-16.6 at 2^32; and each value is within 2^-22 of its own size for that angle.
 */
int c128_build_cos_sin(const c128_rope_t* rope, int64_t first_position, const c128_tensor_t* cos_sin_cache,
                       c128_stream_t stream);

/*
 * c128_rotate — turn columns first_column .. first_column + R - 1 of every head by its token's position:
 *   (u, v) -> (u cos - v sin, v cos + u sin)     inverse: (u cos + v sin, v cos - u sin)
 * where (u, v) are columns 2i and 2i + 1 of those (C128_ROPE_PAIRS) or i and i + R/2 (C128_ROPE_HALVES).
 * The other columns are copied, or stay where `out` is `x` itself. The inverse takes the position out of
 * attention results, which carry it because entries are values too.
 *
 *   x             [T, H, D]  bf16 or fp32, stride[2] == 1, other strides >= D
 *   positions     [T]        int64; < 0: the token is skipped
 *   cos_sin_cache [MP, R]    fp32, as c128_build_cos_sin makes it; R even, 2 .. D - first_column
 *   out           [T, H, D]  type as x; x itself (with its strides), else no overlap
 *
 * Sums in fp32 (each product rounded), rounded once to the type. H * D < 2^31, T < 2^31.
 * Device error bits: C128_DEV_BAD_COS_ROW - positions[t] >= MP (the token is skipped).
 */
enum {
    C128_ROPE_PAIRS = 0,
    C128_ROPE_HALVES = 1,
};
int c128_rotate(const c128_tensor_t* x, const c128_tensor_t* positions, const c128_tensor_t* cos_sin_cache,
                int64_t first_column, int32_t layout, int32_t inverse, const c128_tensor_t* out,
                c128_stream_t stream);

/*
 * c128_norm_rope_store — a step's queries and keys: each head of q, and the key, is normalised (RMSNorm
 * over its 512 values, times a weight if there is one) and its last 64 columns, pairs of neighbours, are
 * turned by the token's position; the key becomes an entry of the paged cache, in the layout that the
 * C128_FORMAT_SPARSE_FP8 compressor stores and c128_window_attention reads.
 *   n = x * rrms * w, rrms = 1 / sqrt(mean(x^2) + eps);  (e, o) -> (e cos - o sin, o cos + e sin)
 * Queries: the mean of squares in fp32, n and the rotation in fp32, rounded once to q_out's type. Keys:
 * every step as compress_norm_rope_store has it behind compressed[] (at the top of this file), with k's
 * row in its place and the position's own row of cos_sin_cache: the bytes are a pure function of the row.
 * (Of a row with an infinity or NaN, values that are NaN get the code of NaN.)
 *
 *   positions     [T]           int64
 *   slot_mapping  [T]           int64  cache slot (block*bs + offset) of the token; < 0: skipped. Two
 *                                      tokens with the same slot race
 *   cos_sin_cache [MP, 64]      fp32   cos in [0, 32), sin in [32, 64) of row positions[t]; stride[1] == 1
 *   q             [T, H, 512]   bf16 or fp32, stride[2] == 1, other strides >= 512, rows 16-byte aligned;
 *                               NULL (and q_out): no queries
 *   q_w           [512]         fp32, 16-byte aligned; NULL: no weight
 *   q_out         [T, H, 512]   bf16 or fp32, strides as for q; may be q itself (same type and strides)
 *   k             [T, 512]      bf16 or fp32, stride[1] == 1, rows 16-byte aligned; NULL (and k_cache): no keys
 *   k_w           [512]         fp32, 16-byte aligned; NULL: no weight
 *   k_cache       [NKB, bs, W]  uint8  as for compress_norm_rope_store; kv_block_size == bs. Only the 584
 *                               bytes of a token's slot are written
 *
 * T * (ceil(H / 4) + 1) < 2^31. q and k may differ in type.
 * Device error bits: C128_DEV_BAD_COS_ROW - positions[t] >= MP; C128_DEV_BAD_KV_SLOT - slot_mapping[t] >=
 * NKB*bs (with keys). The token is skipped, its queries too.
 */
int c128_norm_rope_store(const c128_tensor_t* positions, const c128_tensor_t* slot_mapping, float eps,
                         const c128_tensor_t* cos_sin_cache, const c128_tensor_t* q, const c128_tensor_t* q_w,
                         const c128_tensor_t* q_out, const c128_tensor_t* k, const c128_tensor_t* k_w,
                         const c128_tensor_t* k_cache, int64_t kv_block_size, c128_stream_t stream);

/*
 * c128_window_attention — attention of a step's tokens to the last entries before them and a few first ones,
 * over the paged cache that c128_norm_rope_store fills (an entry per position). The token at position p of
 * its request sees entry j of that request where
 *   j <= p  and  (j > p - window  or  j < first)
 * and with those, k_j, scale, sink, lse and out are as for c128_decode_attention. A step's tokens may be one of
 * each request or many, in any order; entries of the step's own tokens have to be in the cache. lse lets the
 * result be merged with that of c128_decode_attention over the compressed cache (c128_merge_attention; the sink in
 * one of them only).
 *
 * Where window + first <= 136 a kernel keeps the entries of consecutive tokens in shared memory: in a step of which most
 * tokens follow one another they are decoded once for all of them. There, for bf16 results, the softmax weights are divided
 * by their sum (and the sink's share) before they are rounded to bf16, so that of one entry out is that entry; for fp32
 * results out is divided by the sums of the rounded weights, as for c128_decode_attention, which halves its error. lse is of
 * the exact sums, in fp32. Larger windows run as c128_decode_attention does, a token at a time; with up to 16 heads, and
 * three tokens to a row of the table or more, tokens that follow one another (four at most, between multiples of four) are
 * taken together. (So there a step wants the table's rows of its own requests, a slice, rather than those of all that there
 * may be.)
 * An entry that holds NaN makes out and lse of the tokens that see it NaN, and of no others; so does an infinity, or the
 * formula's value is stored.
 *
 *   q                    [T, H, 512]   bf16   as for c128_decode_attention
 *   k_cache              [NKB, bs, W]  uint8  kv_block_size == bs
 *   block_table          [R, MB]       int32  k_cache block of entries b*bs .. b*bs + bs - 1 of a request. Blocks
 *                                             that hold no entry that a token sees are not read (-1, say)
 *   token_to_req_indices [T]           int32
 *   positions            [T]           int64
 *   slot_mapping         [T]           int64  only its sign is used: < 0, the token is skipped
 *   window                             1 <= window < 2^31
 *   first                              0 <= first < 2^31
 *   scale, sink [H], out [T, H, 512], lse [T, H]: as for c128_decode_attention
 *   workspace            [n]           uint8  c128_window_attention_workspace bytes (0 of a short window: nothing is read or
 *                                             written), else as for c128_decode_attention. With up to 16 heads fewer
 *                                             will do, c128_decode_attention_workspace bytes: every token goes alone then
 *
 * The rows of out and lse of skipped tokens are left as they were.
 * Device error bits: C128_DEV_BAD_REQ - token_to_req_indices[t] outside [0, R) (the token is skipped);
 * C128_DEV_BAD_BT_COL - positions[t] >= MB*bs (the entries behind are left out); C128_DEV_BAD_BLOCK - a block id
 * outside [0, NKB) where one is needed (its entries are left out); C128_DEV_TIMEOUT as for c128_decode_attention.
 * T * (min(MB*bs, window + first) / 64 + 2) < 2^31, else C128_ERR_ARG.
 */
int c128_window_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                          const c128_tensor_t* block_table, const c128_tensor_t* token_to_req_indices,
                          const c128_tensor_t* positions, const c128_tensor_t* slot_mapping, int64_t window,
                          int64_t first, float scale, const c128_tensor_t* sink, const c128_tensor_t* out,
                          const c128_tensor_t* lse, const c128_tensor_t* workspace, c128_stream_t stream);

/* Bytes of workspace for c128_window_attention on the current device, whatever the tokens: 0 where window + first <= 136. */
int c128_window_attention_workspace(int64_t num_heads, int64_t window, int64_t first, int64_t* bytes);

/*
 * Test of the failure handling, for tests only: c128_window_attention, except that CTA 0 never learns of its tokens. Its
 * waits run out (after about a second), it ends with C128_DEV_TIMEOUT in the device error bits and stores nothing, and
 * what it would have stored is left as it was. The context stays usable.
 */
int c128_debug_stall_window_attention(const c128_tensor_t* q, const c128_tensor_t* k_cache, int64_t kv_block_size,
                                      const c128_tensor_t* block_table, const c128_tensor_t* token_to_req_indices,
                                      const c128_tensor_t* positions, const c128_tensor_t* slot_mapping,
                                      int64_t window, int64_t first, float scale, const c128_tensor_t* sink,
                                      const c128_tensor_t* out, const c128_tensor_t* lse,
                                      const c128_tensor_t* workspace, c128_stream_t stream);

/* Human-readable name of a return code (static string, never NULL). */
const char* c128_status_string(int status);

/* Make the workspace of (current device, stream) hold at least max_tokens tokens, growing it
 * stream-ordered as described at the top (cudaMallocAsync / device-to-device header copy /
 * cudaFreeAsync on `stream`, no host synchronisation). Returns C128_ERR_CAPTURE if it would have
 * to grow while `stream` is being captured, C128_ERR_NOMEM if the pool has no room. */
int c128_reserve_workspace(int64_t max_tokens, c128_stream_t stream);

/* Return the workspace and kernel-timer events of (current device, stream) to the library: the
 * workspace is freed with cudaFreeAsync on `stream`, after the work already enqueued there, and
 * the stream's sticky device error bits go with it. Call it before destroying a stream the
 * library was used on (a later call on a stream with the same handle starts a fresh workspace).
 * Does not synchronise. Returns C128_ERR_CAPTURE (and releases nothing) while `stream` is being
 * captured. */
int c128_release_stream(c128_stream_t stream);

/* Synchronise `stream`, store the device error bits (C128_DEV_*) of its workspace in *bits,
 * and clear them when `clear` is non-zero. A stream never used reports 0. */
int c128_device_errors(c128_stream_t stream, uint32_t* bits, int clear);

/* Kernel timer. Between begin and end, every call on `stream` records a CUDA event pair around
 * its compress kernel (the dominant kernel; the planning kernel is outside the pair). end()
 * synchronises the stream and returns the summed kernel time in ms and the number of launches.
 * While the timer runs the compress kernel does not overlap the planning kernel. */
int c128_kernel_timer_begin(c128_stream_t stream);
int c128_kernel_timer_end(c128_stream_t stream, double* total_ms, int64_t* launches);

/* Static launch facts of the compress kernel on the current device. */
typedef struct c128_info {
    int32_t sm_count;        /* streaming multiprocessors */
    int32_t threads;         /* threads per CTA of the compress kernel */
    int32_t smem_bytes;      /* dynamic shared memory per CTA */
    int32_t stages;          /* shared-memory ring depth, 32 KiB (one state block) per stage */
    int32_t ctas_per_sm;     /* resident CTAs per SM */
    int32_t plan_tokens_per_cta;
    int32_t wait_timeout_ms; /* limit of every pipeline wait */
    int32_t version;
} c128_info_t;
int c128_get_info(c128_info_t* info);

/* Read-bandwidth probe (a measurement helper; the pages have no counterpart). It streams `bytes`
 * of the device buffer `buf` once with plain 16-byte loads and XORs every 32-bit word into the
 * device word *xor_out (atomicXor per warp: zero it first and it ends as the XOR of the buffer's
 * words, which proves every byte was read). The compressor's kernels read far more than they
 * write, so this read rate, taken in the same process, is the denominator beside the copy
 * bandwidth for their reported bandwidth fraction.
 *   threads_per_cta   32..1024, a multiple of 32
 *   ctas_per_sm       1..32, with threads_per_cta x ctas_per_sm <= 2048; the grid is #SM x the
 *                     smaller of ctas_per_sm and the CTAs that fit on an SM at once (so all are
 *                     resident), fewer when the buffer holds less than one load per thread
 *   loads_in_flight   16-byte loads each thread issues before it uses them: 1, 2, 4 or 8
 * `buf` 16-byte aligned, `bytes` a multiple of 16; both pointers are caller-owned device memory
 * and nothing is allocated. Stream-ordered and asynchronous. Returns C128_ERR_ARG (bad sizes or
 * launch shape), C128_ERR_NULL_PTR, C128_ERR_ALIGN or C128_ERR_CUDA; bytes == 0 is a no-op. */
int c128_read_probe(const void* buf, int64_t bytes, int32_t threads_per_cta, int32_t ctas_per_sm,
                    int32_t loads_in_flight, uint32_t* xor_out, c128_stream_t stream);

/* Free every workspace and timer the library holds, on every device it was used on
 * (synchronises those devices). */
int c128_release_all(void);

#ifdef __cplusplus
}
#endif
#endif /* C128COMPRESS_H */
