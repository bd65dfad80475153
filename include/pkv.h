/*
 * pkv.h -- C ABI of libpkv: the per-pass hot path of a continuous-batching engine on one GB300 (sm_103a):
 * append this pass's K/V into a block-paged cache, then run causal grouped-query attention for a ragged
 * batch of decode rows (one new token) and chunked-prefill rows (many new tokens).
 *
 * Sources (web pages, cited by title and section):
 *   [CB]  "Continuous Batching Is Not a Bigger Batch" (deepconcepts.dev)
 *   [SB]  "Static batching" (danielfleming.xyz)
 *   [SC]  "Saturation and Capacity" (doublewordai inference-lab)
 *   [ABL] "An advertised batch limit proves nothing until sampled" (a8q9.cn)
 *
 * Conventions for every call below
 *   - Device pointers are owned by the caller (e.g. torch tensors).  The library never allocates device
 *     memory; where it needs scratch, the caller passes a workspace sized by a *_bytes query.
 *   - GPU work is enqueued asynchronously on `stream` (a cudaStream_t passed as void*; NULL = legacy
 *     default stream).  A call returns before its kernels finish.
 *   - The pool's device is the current device in every call that launches (PKV_ERR_INVALID_ARG otherwise).
 *   - Argument and shape errors are detected on the host and returned BEFORE anything is launched;
 *     pkv_last_error() then holds a message (thread-local, valid until the next call on the thread).
 *   - Contents of device metadata (block ids, slots, lengths) cannot be checked on the host without a
 *     sync.  Kernels bounds-check every index they derive from them: an out-of-range value is skipped
 *     (never dereferenced) and recorded in the pool's device error word, read by pkv_pool_check().
 *   - PKV_VALIDATE=1 in the environment (read at every call): the calls below also copy the device metadata
 *     they are given (query_start_loc, context_lens, block tables up to each row's context, slots) to the
 *     host after synchronizing the stream, and refuse a bad pass before launching anything --
 *     PKV_ERR_INVALID_ARG for rows (query_start_loc not running from 0 to num_tokens without decreasing, or
 *     not 1 <= q_len <= ctx <= max_blocks_per_seq * block_size), PKV_ERR_OUT_OF_RANGE for block ids and
 *     slots.  A plan issued under PKV_VALIDATE=1 also remembers a hash of the context_lens and
 *     query_start_loc contents; a pkv_attention / pkv_attention_append on that workspace whose metadata
 *     contents differ (same pointers, rewritten in place without a new plan) is refused with
 *     PKV_ERR_INVALID_ARG.  A debugging aid: it costs a synchronization and copies per call, and is skipped
 *     while the stream is being captured into a graph.
 *   - No call traps the device, and no kernel waits on another grid.
 *   - A pool handle is used by one host thread at a time: it remembers the plan issued on each of its 32
 *     most recently planned workspaces and, on an 8-bit or 4-bit cache, the tensor map of the last workspace's fp16
 *     shadow.  Different pools are independent; pkv_last_error is per thread.
 *   - Supported shapes: fp16 Q and K/V inputs; an fp16, 8-bit (E4M3) or 4-bit cache; head_dim 64, 128 or 256;
 *     block_size 16; num_q_heads a multiple of num_kv_heads with a group of 1, 2, 4, 6 or 8 query heads
 *     per KV head; for attention at most 256 KV heads.  Others: PKV_ERR_UNSUPPORTED.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,   /* null pointer, negative size, inconsistent shapes, misaligned buffer */
  PKV_ERR_OUT_OF_RANGE = 2,  /* layer, request id or size outside what the object was built for    */
  PKV_ERR_UNSUPPORTED = 3,   /* shape the kernels are not built for                                   */
  PKV_ERR_CUDA = 4,          /* a CUDA runtime call failed; pkv_last_error() has cudaGetErrorString  */
  PKV_ERR_NO_BLOCKS = 5,     /* scheduler: pool cannot hold a request even when empty                 */
  PKV_ERR_NOT_FOUND = 6      /* scheduler: unknown request id                                         */
} pkv_status;

/* Device error word bits (pkv_pool_check). */
#define PKV_DEVERR_SLOT_RANGE   0x1  /* an append or gather: slot outside [-1, num_blocks*block_size) */
#define PKV_DEVERR_BLOCK_RANGE  0x2  /* attention or a block call: block id outside [0, num_blocks)   */
#define PKV_DEVERR_ROW_META     0x4  /* row with q_len < 1, q_len > ctx, or ctx > max_blocks*bs; a fork's rows */
#define PKV_DEVERR_QSL          0x8  /* query_start_loc not monotone / not ending at num_tokens       */
#define PKV_DEVERR_WAIT_TIMEOUT 0x10 /* an on-chip barrier wait gave up (should never happen)          */

/* ------------------------------------------------------------------------------------------------
 * Cache pool
 *
 * [CB] "What the scheduler does on one step" / "Where the batch size actually comes from": every
 * sequence holds one key and one value per token per layer, allocated on demand in 16-token blocks;
 * grouped-query attention keeps num_kv_heads < num_q_heads.  [SB] "Ragged batches": a paged layout
 * stores only real tokens.
 *
 * Layout of the caller's buffer (row-major), kv_dtype = PKV_KV_F16:
 *     cache[num_layers][2 (K, V)][num_blocks][num_kv_heads][block_size][head_dim]   fp16
 * followed by a 256-byte status area (the device error word).  One (block, kv head) is a contiguous
 * run of block_size*head_dim*2 bytes, which the kernels move with single bulk copies.
 * Bytes per token of context = 2 * num_layers * num_kv_heads * head_dim * 2 ([CB], same section).
 *
 * kv_dtype = PKV_KV_E4M3, the 8-bit cache.  [CB] "Checking it on a real system": when the cache is
 * what limits the batch, quantize it; [ABL] "Context math sets the ceiling the fields ignore": 8-bit KV
 * is half the raw bytes of fp16, with scales on top.  Every cached row (one token's head_dim values of
 * one KV head, K and V separately) is stored as E4M3 codes (OCP 8-bit floating point: bias 7, no
 * infinities, largest magnitude 448) and one power-of-two scale 2^e, kept as the byte e + 127; e is the
 * smallest integer with max|x| <= 448 * 2^e (0 for an all-zero row), and each code is x / 2^e rounded to
 * the nearest E4M3 value, ties to even.  Nothing is clipped; attention reads code * 2^e exactly.
 *     codes [num_layers][2 (K, V)][num_blocks][num_kv_heads][block_size][head_dim]   uint8
 *     scales[num_layers][num_blocks][num_kv_heads][2 (K, V)][block_size]              uint8
 * then the status area (at the next 256-byte boundary).  A (block, kv head) run of codes is
 * block_size*head_dim bytes; its K and V scales are one 32-byte record.  Bytes per token of context =
 * 2 * num_layers * num_kv_heads * (head_dim + 1).  K and V inputs must be finite.
 *
 * kv_dtype = PKV_KV_INT4, the 4-bit cache.  [ABL], same section, sizes a window's cache at 4 bits next to 8.  32
 * consecutive values of a cached row (one token's head_dim values of one KV head, K and V separately) share a scale s: the
 * smallest number of at most 8 significant bits, and a multiple of 2^-24, that is no less than a seventh of their largest
 * magnitude, but at most 9344 (a seventh of 65408, as which larger magnitudes count), kept in fp16 (0 for 32 zeros).  Each
 * value is held as the integer nearest to x / s, ties to even, which is in -7 .. 7; nothing is clipped.  It stands
 * for code * s, which is an fp16 number: attention, in every path, and pkv_gather read exactly that.  A (block, KV head) is
 * one record of 18 * head_dim bytes, codes stored plus 8 and two to a byte, the lower half first:
 *     records[num_layers][num_blocks][num_kv_heads]:
 *         K codes [head_dim / 32][block_size][16]  uint8
 *         V codes [head_dim / 32][block_size][16]  uint8
 *         scales  [block_size][2 (K, V)][head_dim / 32]  fp16
 * then the status area.  Bytes per token of context = 2 * num_layers * num_kv_heads * (head_dim / 2 + head_dim / 16):
 * 0.56 of the 8-bit cache's, 0.28 of fp16's.  K and V inputs must be finite.
 * ---------------------------------------------------------------------------------------------- */
#define PKV_KV_F16  0
#define PKV_KV_E4M3 1
#define PKV_KV_INT4 4

typedef struct {
  int32_t num_layers;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;    /* tokens per block; must be 16 */
  int32_t num_blocks;    /* physical blocks per layer    */
  int32_t split_blocks;  /* blocks per split-K partition of a decode row, at most 32, which 0 selects (4-bit: 256, 128) */
  int32_t kv_dtype;      /* PKV_KV_F16 (0), PKV_KV_E4M3 or PKV_KV_INT4 */
} pkv_config;

typedef struct pkv_pool pkv_pool;

/* Bytes the caller must provide to pkv_pool_init for this configuration (cache + status area),
 * or 0 if the configuration is invalid. */
size_t pkv_pool_bytes(const pkv_config* cfg);

/* Wrap caller-owned device memory `dev_cache` (>= pkv_pool_bytes(cfg) bytes, 256-byte aligned) as a
 * pool.  Zeroes the status area (synchronously, on the legacy default stream); the cache contents
 * are left as they are.  *out receives a host handle; free it with pkv_pool_destroy. */
pkv_status pkv_pool_init(const pkv_config* cfg, void* dev_cache, size_t bytes, pkv_pool** out);

/* Frees the host handle only; the device buffer stays the caller's. */
void pkv_pool_destroy(pkv_pool* pool);

/* Device address of layer `layer`'s K (kv = 0) or V (kv = 1) pool [num_blocks][Hkv][bs][d] (fp16 values,
 * or E4M3 codes for an 8-bit cache; for a 4-bit cache the K or V codes of the layer's first record, of records
 * 18 * d bytes apart); NULL on a bad argument. */
void* pkv_pool_layer_ptr(const pkv_pool* pool, int32_t layer, int32_t kv);

/* Device address of layer `layer`'s scale bytes [num_blocks][Hkv][2 (K, V)][bs] of an 8-bit cache, or of the scales
 * of the layer's first record of a 4-bit cache; NULL for an fp16 cache or a bad argument. */
void* pkv_pool_scales_ptr(const pkv_pool* pool, int32_t layer);

/* Synchronously read the device error word (PKV_DEVERR_* bits) into *bits, then clear it if `clear`.
 * Waits for all work on the legacy default stream's device.  While PKV_DEVERR_WAIT_TIMEOUT is set,
 * attention launches return without work; after clearing it, issue a new pkv_attention_plan before
 * the next pkv_attention (the interrupted launch may have left split counters mid-count). */
pkv_status pkv_pool_check(pkv_pool* pool, int32_t* bits, int32_t clear);

/* ------------------------------------------------------------------------------------------------
 * Slot mapping (device)
 *
 * [CB] "What the scheduler does on one step": a row's new tokens are the positions from
 * num_computed_tokens up; blocks are allocated as tokens are computed.  Token i of row b sits at
 * absolute position p = context_lens[b] - q_len_b + i and writes slot
 *     block_tables[b][p / block_size] * block_size + p % block_size.
 *
 * block_tables    int32 [num_seqs][max_blocks_per_seq]   device
 * context_lens    int32 [num_seqs]  cached + new tokens   device
 * query_start_loc int32 [num_seqs + 1], [0] = 0, [num_seqs] = num_tokens   device
 * slot_mapping    int64 [num_tokens] output               device
 * Rows whose metadata is out of range get slot -1 and set PKV_DEVERR_ROW_META / _BLOCK_RANGE.
 * ---------------------------------------------------------------------------------------------- */
pkv_status pkv_slot_mapping(pkv_pool* pool, const int32_t* block_tables, int32_t max_blocks_per_seq,
                            const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
                            int32_t num_tokens, int64_t* slot_mapping, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Append (kv_append)
 *
 * [CB] opening section and "The allocator is the other half": each computed token's key and value
 * are stored in the cache so later passes need not recompute them; storage is the token's slot in a
 * 16-token block.  Copies k[t], v[t] ([num_kv_heads][head_dim] fp16 each) of `layer` into slot
 * slot_mapping[t] for t < num_tokens; a slot of -1 is skipped (padding); any other out-of-range slot
 * is skipped and sets PKV_DEVERR_SLOT_RANGE.  fp16 cache: a bit copy, no arithmetic.  8-bit cache: each
 * (token, KV head) row of K and of V is quantized as the pool section describes (codes and scale byte,
 * bit-exact); the 4-bit cache likewise (codes and scales, bit-exact).  Duplicate slots in one call race (last writer unspecified).
 *
 * k, v          fp16 [num_tokens][num_kv_heads][head_dim]   device, 16-byte aligned
 * slot_mapping  int64 [num_tokens]                          device
 * ---------------------------------------------------------------------------------------------- */
pkv_status pkv_append(pkv_pool* pool, int32_t layer, const void* k, const void* v,
                      const int64_t* slot_mapping, int32_t num_tokens, void* stream);

/* Reads cached rows back as values, whatever the cache holds them in: k_out[t], v_out[t] ([num_kv_heads][head_dim] fp16
 * each) become what slot slot_mapping[t] of `layer` stands for, for t < num_tokens -- the bits of an fp16 cache, code
 * times scale of a 4-bit one, code times scale of an 8-bit one (exact where that is an fp16 number, else rounded to one;
 * within 3 % of the fp16 maximum it saturates to +-65504).  The way out of a pool into another one, of another
 * format or another engine's, by an append.  Where the slot is -1 the outputs are left as they were; any other
 * out-of-range slot likewise, and sets PKV_DEVERR_SLOT_RANGE.  A slot may be named more than once.
 *
 * slot_mapping  int64 [num_tokens]                          device
 * k_out, v_out  fp16 [num_tokens][num_kv_heads][head_dim]   device, 16-byte aligned, apart from one another */
pkv_status pkv_gather(pkv_pool* pool, int32_t layer, const int64_t* slot_mapping, int32_t num_tokens, void* k_out,
                      void* v_out, void* stream);

/* ------------------------------------------------------------------------------------------------
 * Ragged paged attention
 *
 * [CB] "What the scheduler does on one step": one pass mixes decode rows (one new token) and
 * chunked-prefill rows (up to the token budget of new prompt tokens), with no separate prefill phase.
 * Row b owns query tokens query_start_loc[b] .. query_start_loc[b+1]-1 (q_len_b of them) and
 * context_lens[b] keys, this pass's appended tokens included.  Query i of the row is at absolute
 * position ctx_b - q_len_b + i and attends causally to keys 0 .. ctx_b - q_len_b + i.  Query head h
 * reads KV head h / (num_q_heads / num_kv_heads).  Scores are scaled by 1/sqrt(head_dim); scores, the softmax's maximum
 * and sum and the accumulation in fp32; each softmax weight (before its division by the sum) is rounded to fp16 for its
 * product with V on the tensor cores, and the output once to fp16 (both round-to-nearest-even).
 *
 * Use: size a workspace with pkv_attention_workspace_bytes, call pkv_attention_plan once per pass
 * (after the metadata is on the device), then pkv_attention once per layer.  A plan stays valid
 * for every pkv_attention call with the same workspace and metadata pointers and sizes until the
 * next pkv_attention_plan on that workspace; changing the metadata CONTENTS requires a new plan.
 * pkv_attention refuses (PKV_ERR_INVALID_ARG) a call whose workspace/metadata pointers or sizes
 * differ from the last plan issued on `workspace` (and, under PKV_VALIDATE=1, one whose metadata
 * contents changed).  Plans live per workspace: planning one workspace leaves the plans of the
 * pool's other workspaces valid (double-buffered passes), up to the 32 most recently planned
 * workspaces per pool.  Plans and calls on one workspace must be ordered on one stream (or
 * synchronised by the caller).
 * Calls on one stream see the cache as the calls before them left it, whatever an append between the plan and the
 * attention wrote; cached rows that the caller's own kernels write are written before the plan.
 *
 * The result is independent of the batch: a row's split-K partition depends only on its own
 * context length, so a row gives bit-identical output alone or in any batch, in any row order.
 *
 * 8-bit cache: attention reads the dequantized values code * 2^e exactly (scales applied in fp32).  Rows
 * with 16 or more new tokens first have their blocks dequantized into an fp16 shadow
 * inside the workspace, read by the tensor-core tile kernel; values within 3 % of the fp16 maximum saturate
 * there.  pkv_attention_workspace_bytes then includes room for min(num_blocks, R * max_blocks_per_seq)
 * shadow blocks, R the most rows of 16+ new tokens the pass can hold.  Rows may share blocks (forks of a prompt that is
 * still being computed): that many hold them all.
 *
 * Scores are fp32.  Rows with 16 or more new tokens take scores, times log2(e) / sqrt(head_dim), of up to 2^27 in magnitude;
 * the decode path takes any.
 *
 * 4-bit cache: attention reads the values code * s exactly; scores are scaled by group in fp32, and each softmax
 * weight is rounded to fp16.  Rows with 16 or more new tokens take the same fp16 shadow, with the same workspace.
 *
 * Rows are there to be attended: each has a new token.  A pass with rows that have none is reported
 * (PKV_DEVERR_ROW_META) and its other rows get their results by the decode path, however long; one whose
 * query_start_loc does not run from 0 to num_tokens (PKV_DEVERR_QSL) gets none.
 *
 * q                fp16 [num_tokens][num_q_heads][head_dim]   device, 16-byte aligned
 * block_tables     int32 [num_seqs][max_blocks_per_seq]       device
 * context_lens     int32 [num_seqs]                           device
 * query_start_loc  int32 [num_seqs + 1]                       device
 * out              fp16 [num_tokens][num_q_heads][head_dim]   device (may not alias q)
 * workspace        device, >= pkv_attention_workspace_bytes(...) bytes, 256-byte aligned
 * ---------------------------------------------------------------------------------------------- */
size_t pkv_attention_workspace_bytes(const pkv_pool* pool, int32_t num_seqs, int32_t num_tokens,
                                     int32_t max_blocks_per_seq);

pkv_status pkv_attention_plan(pkv_pool* pool, const int32_t* context_lens, const int32_t* query_start_loc,
                              int32_t num_seqs, int32_t num_tokens, int32_t max_blocks_per_seq,
                              void* workspace, size_t workspace_bytes, void* stream);

pkv_status pkv_attention(pkv_pool* pool, int32_t layer, const void* q, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* context_lens,
                         const int32_t* query_start_loc, int32_t num_seqs, int32_t num_tokens, void* out,
                         void* workspace, size_t workspace_bytes, void* stream);

/* kv_append and attention of one layer in one call: the same result -- cache contents and output --
 * as pkv_append(pool, layer, k, v, slot_mapping, num_tokens) followed by pkv_attention(...) with the
 * other arguments, under the same plan.  When no row of the pass can take the prefill path (every row
 * has fewer than 16 new tokens; the host checks num_tokens - num_seqs < 15), the append runs inside
 * the decode launch: tiles take this pass's keys and values from k / v directly (on an 8-bit
 * or 4-bit cache, quantized exactly as the append would store them), and each token is written to the cache by the warp
 * whose block holds its position, so no separate append precedes the attention.  Otherwise (and on an
 * 8-bit or 4-bit cache whenever a row may have 16 or more new tokens) this is the append launch followed by the
 * attention launches.  Tokens of rows
 * whose metadata is rejected (PKV_DEVERR_ROW_META) are not appended on the fused path.
 *
 * k, v             fp16 [num_tokens][num_kv_heads][head_dim]   device, 16-byte aligned
 * slot_mapping     int64 [num_tokens]                          device (-1: skip the token)
 * (everything else as pkv_attention) */
pkv_status pkv_attention_append(pkv_pool* pool, int32_t layer, const void* q, const void* k, const void* v,
                                const int64_t* slot_mapping, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                const int32_t* context_lens, const int32_t* query_start_loc, int32_t num_seqs,
                                int32_t num_tokens, void* out, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ------------------------------------------------------------------------------------------------
 * Attention behind a sliding window, with sinks
 *
 * As pkv_attention, but a query at position p sees only the keys k <= p of its row with k > p - window (the last
 * `window` ones, its own among them) or k < sinks (the row's first tokens, which stay visible however far the
 * window has moved).  The pages attend a row's whole context; this bounds what a long row reads and
 * what it must hold.
 *
 * Use: size the workspace with pkv_attention_window_workspace_bytes and plan the pass with
 * pkv_attention_window_plan instead of pkv_attention_plan; then call pkv_attention or pkv_attention_append as ever:
 * the plan on their workspace carries the window.  A model with windowed and full layers plans two workspaces.
 * Everything said of pkv_attention_plan holds, and:
 *   - context_lens still count the whole row, and block tables still have an entry for every 16 tokens.  Entries
 *     of blocks that no new token of the row sees -- every key at or past the sinks, and in front of
 *     the window of the row's first new token -- are never read: they may be -1 and the blocks freed (by the
 *     caller: the host scheduler below keeps the blocks of a request's whole context).
 *   - Keys and values that a query does not see have no part in its result, whatever they hold, with one
 *     exception: in a row of 16 or more new tokens, a non-finite value (of V) that is seen by one of the row's
 *     queries may reach the row's other queries.
 *   - A row whose contexts the window holds whole gives the bits of a plan without one (at head_dim 64 only with 16 or
 *     more new tokens: shorter rows there sum their blocks in pairs).
 *   - pkv_attention_noalloc knows no window: it attends whole contexts.
 * window >= 1, sinks >= 0 (else PKV_ERR_INVALID_ARG, and 0 bytes). */
size_t pkv_attention_window_workspace_bytes(const pkv_pool* pool, int32_t num_seqs, int32_t num_tokens,
                                            int32_t max_blocks_per_seq, int32_t window, int32_t sinks);
pkv_status pkv_attention_window_plan(pkv_pool* pool, const int32_t* context_lens, const int32_t* query_start_loc,
                                     int32_t num_seqs, int32_t num_tokens, int32_t max_blocks_per_seq,
                                     int32_t window, int32_t sinks, void* workspace, size_t workspace_bytes,
                                     void* stream);

/* Allocation-free attention.  The pages have no counterpart to this call; it exists for callers that
 * cannot give the library a workspace -- an engine whose device memory is already carved up by its
 * own allocator, or code that must not call cudaMalloc (a device-wide synchronisation) mid-pass.
 *
 * Does what pkv_attention_plan followed by pkv_attention does, with the same arguments minus the
 * workspace, and gives the same result.  The split-K scratch lives in one array of
 * PKV_NOALLOC_SCRATCH_BYTES compiled into libpkv, held on every device that loads the library until
 * the process exits; the library allocates nothing.  A pass whose scratch
 * (pkv_attention_workspace_bytes for the same sizes) exceeds that limit is refused with
 * PKV_ERR_OUT_OF_RANGE before anything is launched.
 *
 * The first call in a device's context looks up the array's device address (cudaGetSymbolAddress) with
 * that device current -- the pool's device must be the current device -- so make that first call
 * before any stream capture: a first call made while `stream` is capturing is refused with
 * PKV_ERR_INVALID_ARG.  The address is cached per (device, context), so a context re-created after
 * cudaDeviceReset looks it up again.  Every call shares the one array and leaves its contents behind;
 * nothing in it has to start at zero, but two calls whose kernels can overlap on the GPU (different
 * streams with no ordering between them) race on it.  Every refusal (sizes, the 8-bit cache's prefill
 * limits, the capture rule) comes before anything is launched. */
#define PKV_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)
pkv_status pkv_attention_noalloc(pkv_pool* pool, int32_t layer, const void* q, const int32_t* block_tables,
                                 int32_t max_blocks_per_seq, const int32_t* context_lens,
                                 const int32_t* query_start_loc, int32_t num_seqs, int32_t num_tokens, void* out,
                                 void* stream);

/* ------------------------------------------------------------------------------------------------
 * Rotary positions and the append in one call
 *
 * A model with rotary positions turns pair i of every query and key head by the angle position * f_i
 * before the key is cached.  The pages have no counterpart (their rows are positions in a cache); these
 * calls put the rotation next to pkv_append, so that keys are rotated on their way into their slots and
 * queries on their way into the packed rows pkv_attention reads.
 *
 * Of each head's head_dim values the first rot_dim are rotated, the others pass through.  Pair i
 * (0 <= i < rot_dim / 2) is values (i, i + rot_dim / 2) with PKV_ROPE_HALF and (2i, 2i + 1) with
 * PKV_ROPE_INTERLEAVED:
 *     a' = output_scale * (a cos - b sin),   b' = output_scale * (b cos + a sin).
 * Frequencies f_i = base^(-2i / rot_dim), then for long contexts, with t_i = original_context * f_i / (2 pi)
 * the pair's turns over the original context:
 *     PKV_ROPE_SCALE_NONE    f_i
 *     PKV_ROPE_SCALE_LINEAR  f_i / factor
 *     PKV_ROPE_SCALE_BANDS   f_i (w + (1 - w) / factor), w = clamp((t_i - low_turns) / (high_turns - low_turns), 0, 1)
 *     PKV_ROPE_SCALE_RAMP    f_i (w + (1 - w) / factor), w = 1 - clamp((i - lo) / max(hi - lo, 0.001), 0, 1), where
 *                            pair(t) = rot_dim ln(original_context / (2 pi t)) / (2 ln base),
 *                            lo = max(floor(pair(high_turns)), 0), hi = min(ceil(pair(low_turns)), rot_dim - 1)
 * Angles are reduced modulo a turn exactly: f_i (computed in 64-bit floating point) over 2 pi is held as a 64-bit
 * binary fraction, and its product with the position wraps.  For frequencies up to 1 the fraction is off by less than
 * 2^-53: 2^-22 turns at any int32 position, 2^-33 below a million tokens.  cos, sin and the rotation are fp32; each result
 * is rounded once to fp16.  Frequencies and output_scale have to be finite (in 64 and 32 bits; else PKV_ERR_INVALID_ARG).
 * ---------------------------------------------------------------------------------------------- */
#define PKV_ROPE_HALF         0
#define PKV_ROPE_INTERLEAVED  1
#define PKV_ROPE_SCALE_NONE   0
#define PKV_ROPE_SCALE_LINEAR 1
#define PKV_ROPE_SCALE_BANDS  2
#define PKV_ROPE_SCALE_RAMP   3

typedef struct {
  int32_t head_dim;         /* 64, 128 or 256                                                          */
  int32_t rot_dim;          /* values rotated, a multiple of 16 up to head_dim; 0 = head_dim             */
  int32_t layout;           /* PKV_ROPE_HALF or PKV_ROPE_INTERLEAVED                                     */
  int32_t scaling;          /* PKV_ROPE_SCALE_*                                                          */
  double base;              /* > 1                                                                       */
  double factor;            /* > 0 (unused with PKV_ROPE_SCALE_NONE)                                     */
  double original_context;  /* > 0 (bands, ramp)                                                         */
  double low_turns;         /* bands, ramp: 0 < low_turns < high_turns; both 0 = 1 and 4 (bands), 1 and 32 (ramp) */
  double high_turns;
  double output_scale;      /* factor on the rotated values; 0 = 1                                       */
} pkv_rope_config;

typedef struct pkv_rope pkv_rope;

/* A host handle holding the frequencies (no device memory).  Any number of pools and threads may use one. */
pkv_status pkv_rope_create(const pkv_rope_config* cfg, pkv_rope** out);
void pkv_rope_destroy(pkv_rope* rope);

/* The first n of the rot_dim / 2 frequencies, in radians a token, into out (may be NULL); returns rot_dim / 2. */
int32_t pkv_rope_frequencies(const pkv_rope* rope, double* out, int32_t n);

/* Absolute positions of a pass's tokens: token i of row b gets context_lens[b] - q_len_b + i (arguments as
 * pkv_slot_mapping).  Tokens of a row whose metadata is out of range get 0 and set PKV_DEVERR_ROW_META. */
pkv_status pkv_positions(pkv_pool* pool, const int32_t* context_lens, const int32_t* query_start_loc,
                         int32_t num_seqs, int32_t num_tokens, int32_t* positions, void* stream);

/* For every token t < num_tokens: q[t] rotated into q_out[t], k[t] rotated and v[t] as it is into slot
 * slot_mapping[t] of `layer`, as pkv_append would store them (8-bit cache: quantized from the rotated key
 * rounded to fp16, bit for bit what a rotation followed by pkv_append stores).  A slot of -1 is skipped (its
 * query is rotated all the same); any other out-of-range slot is skipped and sets PKV_DEVERR_SLOT_RANGE.
 * Duplicate slots in one call race (last writer unspecified).  (A 4-bit cache quantizes the rounded rotated key, as an 8-bit
 * one does.)
 *
 * q, k, v       fp16, token t's heads at t * {q,k,v}_stride values from the pointer, [heads][head_dim] within a
 *               token: separate tensors, or slices of one packed projection.  16-byte aligned; strides multiples of 8 and
 *               at least heads * head_dim.  q may be NULL (and then q_out): keys and values alone.
 * positions     int32 [num_tokens]   device; any value (negative ones turn backwards)
 * slot_mapping  int64 [num_tokens]   device
 * q_out         fp16 [num_tokens][num_q_heads][head_dim], 16-byte aligned; may be q itself when q_stride is
 *               num_q_heads * head_dim; must not overlap q, k or v otherwise */
pkv_status pkv_rope_append(pkv_pool* pool, int32_t layer, const pkv_rope* rope, const void* q, int64_t q_stride,
                           const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                           const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens, void* q_out,
                           void* stream);

/* pkv_rope_append with a norm of every head in front of its rotation: with x a query or key head of head_dim values,
 *     y = x / sqrt(mean(x^2) + eps) * (weight_offset + w)
 * takes the place of x, w being q_weight for query heads and k_weight for key heads.  All in fp32 -- the mean square, the
 * product and the rotation of its first rot_dim values -- and rounded once to fp16; an 8-bit or 4-bit cache quantizes that.
 * Values (v) are appended as they are.  Everything else as pkv_rope_append, and:
 *
 * rope                NULL: no rotation (positions are then not read, and may be NULL)
 * q_weight, k_weight  fp16 [head_dim], device, 16-byte aligned; NULL: the query (key) heads are not normalised.  Not both
 *                     NULL
 * eps                 finite, at least 1e-30
 * weight_offset       at most 1e20 in magnitude; 0 for weights as they are, 1 for weights kept as their distance from one */
pkv_status pkv_norm_rope_append(pkv_pool* pool, int32_t layer, const pkv_rope* rope, const void* q_weight,
                                const void* k_weight, float eps, float weight_offset, const void* q, int64_t q_stride,
                                const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                const int32_t* positions, const int64_t* slot_mapping, int32_t num_tokens, void* q_out,
                                void* stream);

/* ------------------------------------------------------------------------------------------------
 * Copying, forking and compacting blocks (device, every layer)
 *
 * [CB] "The allocator is the other half": requests hold blocks, and a freed block is another's.  These calls
 * move what blocks hold: K and V of every layer and, on an 8-bit or 4-bit cache, the scales, bit for bit.
 * ---------------------------------------------------------------------------------------------- */

/* pairs int32 [num_pairs][2] (source, destination), device: block `destination` becomes a copy of block
 * `source`.  A pair with a -1 in it is skipped (padding); any other id outside [0, num_blocks) skips the
 * pair and sets PKV_DEVERR_BLOCK_RANGE.  A source may be copied to several destinations; a block that is a
 * destination must be in no other pair (its contents would depend on the order of the copies; under PKV_VALIDATE=1
 * such a list is refused with PKV_ERR_INVALID_ARG). */
pkv_status pkv_copy_blocks(pkv_pool* pool, const int32_t* pairs, int32_t num_pairs, void* stream);

/* Rows that continue from a common prefix (several samples of one prompt, a beam's branches).
 * forks int32 [num_forks][3] (parent row, child row, block), device.  For each fork, with c = context_lens[parent]:
 *     the child's table row becomes the parent's first c / 16 entries (shared blocks), then, if c % 16 > 0,
 *     `block`, then -1;  context_lens[child] = c;  the c % 16 tokens of the parent's last block are copied into
 *     `block`, whose other rows are left as they were.
 * The two rows then append without seeing each other: only full blocks are shared.  With c % 16 = 0 `block` is
 * not used and may be -1.  A fork with a row outside [0, num_seqs), parent = child, or a context
 * outside [0, 16 * max_blocks_per_seq] does nothing and sets PKV_DEVERR_ROW_META; one whose partial block or `block` is
 * out of range does nothing and sets PKV_DEVERR_BLOCK_RANGE.  A fork whose parent row is -1 is skipped (padding).
 * Several forks may share a parent; a child must be in no other fork of the call, and a `block` in no other fork
 * nor in use (under PKV_VALIDATE=1 a repeated child or block, or a child that is a parent, is refused).
 *
 * block_tables int32 [num_seqs][max_blocks_per_seq], context_lens int32 [num_seqs]   device, updated in place */
pkv_status pkv_fork_rows(pkv_pool* pool, int32_t* block_tables, int32_t max_blocks_per_seq, int32_t* context_lens,
                         int32_t num_seqs, const int32_t* forks, int32_t num_forks, void* stream);

/* Moves the blocks in use to the front of the pool, so that what is free is one range.  In use is every
 * block named in block_tables [num_seqs][max_blocks_per_seq] (entries of -1 name none; a block in several rows
 * counts once; any other id outside [0, num_blocks) names none and sets PKV_DEVERR_BLOCK_RANGE).  With n
 * blocks in use, the k-th lowest used block of those at n or above is copied to the k-th lowest unused block
 * below n; the others stay.  Written, all on the device:
 *     new_tables  int32 [num_seqs][max_blocks_per_seq]  block_tables with every used block's new id (other
 *                                                       entries as they were); may be block_tables itself, and
 *                                                       must not overlap it otherwise
 *     remap       int32 [num_blocks]                    a used block's new id, -1 for an unused one
 *     num_live    int32 [1]                             n: blocks n .. num_blocks - 1 are free now
 * Every table of the pool's requests must be in the call: a block named in none is free, and may be overwritten.
 * Blocks moved away from keep their contents.
 * workspace    device, >= pkv_compact_workspace_bytes(pool) bytes, 256-byte aligned; two calls on one workspace must
 *              be ordered by the caller */
size_t pkv_compact_workspace_bytes(const pkv_pool* pool);
pkv_status pkv_compact(pkv_pool* pool, const int32_t* block_tables, int32_t max_blocks_per_seq, int32_t num_seqs,
                       int32_t* new_tables, int32_t* remap, int32_t* num_live, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Test hook, off by default: refused with PKV_ERR_UNSUPPORTED unless PKV_TEST_HOOKS=1 is in the environment.
 * The pages have no counterpart; it exercises the failure path of [ABL] "Counting jobs while they run" (a
 * job must not be left holding the device).  Launches one kernel whose thread waits on an on-chip barrier
 * that never completes, through the same bounded wait every attention kernel uses, with the time limit
 * shortened to limit_ns (1 .. 1e8); when the wait gives up it sets PKV_DEVERR_WAIT_TIMEOUT in the pool's
 * error word and returns.  Afterwards attention launches on the pool do no work until pkv_pool_check
 * clears the bit and the pass is planned again. */
pkv_status pkv_debug_expire_wait(pkv_pool* pool, int64_t limit_ns, void* stream);

/* Number of kernel launches the last successful call on `pool` that launches any enqueued (for accounting; host-side
 * counter). */
int32_t pkv_last_launch_count(const pkv_pool* pool);

/* Message for the last failed call on this thread ("" if none). */
const char* pkv_last_error(void);

/* ------------------------------------------------------------------------------------------------
 * Host reference scheduler (generates the per-pass batches; never on the timed path)
 *
 * [CB] "What the scheduler does on one step": schedule() runs once per pass.  Phase one walks running
 * requests in arrival order; each wants num_tokens - num_computed_tokens (1 when decoding, the rest of
 * the prompt when prefilling) capped by the token budget (chunked prefill).  Blocks are allocated for
 * them; on failure the newest running request is popped, its blocks freed, its status set PREEMPTED,
 * num_computed_tokens reset to 0 and it is prepended to the waiting queue; retry.  If the popped
 * request is the one being scheduled, phase one stops.  Phase two (only when the pass preempted
 * nobody) admits from the waiting queue's head while the budget lasts and fewer than max_num_seqs
 * run; an unallocatable head stops admission for the pass.  [SC] "Runtime capacity control":
 * max_num_seqs gates admission only and must be >= 1; lowering it drains, never evicts.  [ABL]
 * "Counting jobs while they run": a cancelled request must free its memory (pkv_sched_abort).
 * A pass that computes a request's last known token yields one output token; at max_output outputs
 * the request finishes and frees its blocks in the same pass (freed blocks join the free list's tail).
 * ---------------------------------------------------------------------------------------------- */
typedef struct {
  int32_t max_num_seqs;   /* >= 1                                    */
  int32_t token_budget;   /* new tokens per pass, >= 1               */
  int32_t block_size;     /* tokens per block, >= 1                  */
  int32_t num_blocks;     /* physical blocks in the pool             */
} pkv_sched_config;

typedef struct pkv_sched pkv_sched;

/* One pass's ragged batch.  All arrays are HOST memory owned by the scheduler, valid until the next
 * pkv_sched_step / pkv_sched_destroy.  Rows are in scheduling order (running first, then admitted). */
typedef struct {
  int32_t num_seqs;
  int32_t num_tokens;
  int32_t max_blocks_per_seq;       /* width of block_tables: max blocks held by a scheduled row (>= 1) */
  const int64_t* req_ids;           /* [num_seqs]                                   */
  const int32_t* q_lens;            /* [num_seqs]                                   */
  const int32_t* context_lens;      /* [num_seqs]  num_computed before + q_len       */
  const int32_t* query_start_loc;   /* [num_seqs + 1]                               */
  const int32_t* block_tables;      /* [num_seqs][max_blocks_per_seq], -1 padded     */
  const int64_t* slot_mapping;      /* [num_tokens]                                 */
  int32_t num_preempted;
  const int64_t* preempted;         /* in pop order (newest first)                  */
  int32_t num_admitted;
  const int64_t* admitted;
  int32_t num_finished;
  const int64_t* finished;
} pkv_step;

typedef struct {
  int64_t steps;
  int64_t preemptions;
  int64_t recomputed_tokens;        /* num_computed_tokens discarded by preemption */
  int64_t recomputed_prompt_tokens; /* the prompt part of it                       */
  int64_t max_batch;                /* most rows in one pass                       */
  int64_t batch_sum;                /* sum of rows over passes (mean = /steps)     */
  int64_t tokens_scheduled;
  int32_t running;
  int32_t waiting;
  int32_t free_blocks;
  int64_t live_tokens;              /* summed over passes, after each pass: tokens running requests hold */
  int64_t held_slots;               /* summed over passes: slots of the blocks running requests hold    */
  int64_t prefix_hit_tokens;        /* recompute refunded by prefix caching                            */
} pkv_sched_stats;

/* Block allocation policies and units of scheduling (pkv_sched_set_policy).  [CB] "The allocator is
 * the other half": on demand (the default) allocates a request's blocks as its tokens are computed and
 * preempts when the pool runs out; RESERVE (Orca) admits a request only if its worst case fits --
 * ceil((prompt_len + declared_output) / block_size) free blocks, all taken at admission and returned when
 * it finishes -- so it never preempts, at the price of holding cache for output the client only claimed.
 * [CB] "The boundary: when this is worth nothing": UNIT_PASS re-decides membership every pass (continuous
 * batching, the default); UNIT_REQUEST is static batching: a batch forms when nothing runs, takes members
 * until the first pass in which one of them finishes, and then runs to its slowest member. */
#define PKV_ALLOC_ON_DEMAND 0
#define PKV_ALLOC_RESERVE   1
#define PKV_UNIT_PASS       0
#define PKV_UNIT_REQUEST    1

/* free_order: the initial free list ([num_blocks] distinct ids in [0, num_blocks)), or NULL for
 * 0..num_blocks-1.  Copied. */
pkv_status pkv_sched_create(const pkv_sched_config* cfg, const int32_t* free_order, pkv_sched** out);
void pkv_sched_destroy(pkv_sched* s);
/* Arrival: appended to the waiting queue.  Duplicate live ids: PKV_ERR_INVALID_ARG.  A request that
 * could never fit the pool (ceil((prompt_len + max_output) / block_size) > num_blocks):
 * PKV_ERR_NO_BLOCKS. */
pkv_status pkv_sched_add(pkv_sched* s, int64_t req_id, int32_t prompt_len, int32_t max_output);
/* As pkv_sched_add, with the output the client declares (>= max_output; RESERVE reserves for it).  A
 * request whose reservation could never fit the pool: PKV_ERR_NO_BLOCKS. */
pkv_status pkv_sched_add_declared(pkv_sched* s, int64_t req_id, int32_t prompt_len, int32_t max_output,
                                  int32_t declared_output);
/* Choose the policies; only before the first request is added (PKV_ERR_INVALID_ARG afterwards). */
pkv_status pkv_sched_set_policy(pkv_sched* s, int32_t alloc, int32_t unit);
/* Prefix caching of recompute after preemption ([CB] "What the scheduler does on one step": the recompute
 * "is partly refundable" when the freed blocks were not evicted by the time the request comes back).  A
 * preempted request's full blocks stay registered while they sit in the free list (returned last block
 * first, so its prefix is evicted last); handing a block out evicts it.  On readmission the request takes
 * back the longest still-registered prefix of its blocks, leaving at least one token to compute, and only
 * the rest is recomputed (pkv_step rows then start past the reused blocks).  On demand only (a reserving
 * scheduler never preempts); set before the first request is added. */
pkv_status pkv_sched_set_prefix_caching(pkv_sched* s, int32_t enable);
/* Run one pass; fills *out (num_seqs may be 0 when nothing is left to do). */
pkv_status pkv_sched_step(pkv_sched* s, pkv_step* out);
pkv_status pkv_sched_abort(pkv_sched* s, int64_t req_id);
/* Continue running request parent_id as child_id as well, between passes: the child has the parent's prompt,
 * outputs so far and computed tokens, and runs from the next pass on to max_output outputs in all (more than the
 * parent has).  They share the parent's full blocks, counted: a shared block is freed with its last holder.  If the
 * parent's computed tokens end inside a block, *block is the child's own block for them, whose rows have to be copied
 * before the next pass (pkv_fork_rows, or pkv_copy_blocks), else -1.  On demand and UNIT_PASS only
 * (PKV_ERR_UNSUPPORTED).  Refused, with nothing changed: an unknown parent (PKV_ERR_NOT_FOUND), one that is
 * not running or a child id in use (PKV_ERR_INVALID_ARG), max_num_seqs requests running already
 * (PKV_ERR_OUT_OF_RANGE), no free block or a child that could never fit (PKV_ERR_NO_BLOCKS).  A preempted request
 * that shared blocks keeps none of them registered for prefix caching; the statistics count a shared block for each
 * of its holders. */
pkv_status pkv_sched_fork(pkv_sched* s, int64_t parent_id, int64_t child_id, int32_t max_output, int32_t* block);
/* Every running request's blocks (reserved ones included), for pkv_compact: returns the number of running requests and
 * sets *width (may be NULL) to the most blocks one holds (at least 1); if block_tables is non-NULL and
 * max_rows and max_blocks_per_seq hold them, fills block_tables [rows][max_blocks_per_seq] (-1 padded) and req_ids
 * [rows] (may be NULL). */
int32_t pkv_sched_tables(const pkv_sched* s, int32_t max_rows, int32_t max_blocks_per_seq, int64_t* req_ids,
                         int32_t* block_tables, int32_t* width);
/* Take over a compaction's remap (host copy, [num_blocks]): every held block b becomes remap[b], the others are free in
 * ascending order, and prefix caching forgets what free blocks held.  A remap that does not give every held block a
 * block of its own is refused (PKV_ERR_INVALID_ARG) with nothing changed. */
pkv_status pkv_sched_remap(pkv_sched* s, const int32_t* remap);
pkv_status pkv_sched_set_max_num_seqs(pkv_sched* s, int32_t max_num_seqs);
void pkv_sched_get_stats(const pkv_sched* s, pkv_sched_stats* out);
/* 1 when no request is running or waiting. */
int32_t pkv_sched_done(const pkv_sched* s);
/* Current free list (head first) copied into out[0 .. min(n, free)-1]; returns the free count. */
int32_t pkv_sched_free_list(const pkv_sched* s, int32_t* out, int32_t n);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
