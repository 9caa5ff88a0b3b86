/*
 * pkv.h -- C ABI of the GB300 (sm_103a) paged KV-cache decode library, libpkv.so.
 *
 * What it computes.  A KV cache kept as a pool of fixed-size physical blocks of
 * 16 tokens; each sequence owns a block table mapping its logical block i to a
 * physical block ("Series 03: why the KV cache eats memory, and how
 * PagedAttention pages it", sections 3.1-3.3).  A decode step appends the new
 * token's K and V rows to the cache and then lets the token's query attend over
 * every cached row of its sequence ("KV Cache, the memory notepad of LLM
 * inference", sections 二 and 三):
 *      out[b, h] = sum_j softmax_j(scale * <q[b, h], K_j>) V_j,   j < context_lens[b]
 * where K_j / V_j of KV head g = h / G (G = num_q_heads / num_kv_heads, the GQA
 * group of the same page's section 六) are found through the block table.  An
 * E4M3 (8-bit float) cache stores code = E4M3(fl32(x / scale[g])) with one fp32
 * scale per KV head and dequantises before the arithmetic ("KV cache capacity
 * planning, from the budget to task-level regression", sections 4 and 5).
 *
 * Data layout (all row-major, C order):
 *   k_cache, v_cache   [num_blocks, num_kv_heads, block_size, head_dim]; K and V
 *                      are separate buffers ("What a KV cache is and why it is
 *                      the crux of LLM inference", section 3.1); one
 *                      (block, head) slab of 16 rows is contiguous.
 *   slot               physical row index = block_id * block_size + offset.
 *   block_tables       int32 [batch, max_blocks_per_seq]; entries past
 *                      ceil(context_len / block_size) are never read.
 *   q, out             [batch, num_q_heads, head_dim] in the 16-bit dtype.
 *   k_new, v_new       [num_tokens, num_kv_heads, head_dim].
 *
 * Conventions.
 *   - Ownership: every buffer is allocated and owned by the caller.  Device
 *     pointers must stay valid until the stream work they feed completes.  The
 *     library allocates no device memory and keeps no device state.
 *   - Execution: launches are asynchronous on `stream` (a cudaStream_t passed
 *     as void*; NULL = the legacy default stream).  The returned status only
 *     reports argument validation and launch errors.
 *   - Alignment: every device pointer is 16-byte aligned; head_dim is 64 or 128
 *     and block_size is 16 (anything else returns PKV_ERR_UNSUPPORTED).
 *   - Device-detected errors (a block id outside [0, num_blocks), a slot past
 *     the pool, a context longer than its table or than max_context_len, an
 *     internal wait that timed out) make the kernel skip the access and, when
 *     `err_flag` (a device int32, nullable) is given, store the first error
 *     code there.  No kernel traps.  The caller synchronises and reads it.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,  /* bad pointer, size or shape                      */
  PKV_ERR_UNSUPPORTED = 2,  /* valid but not built: head_dim, group, block size */
  PKV_ERR_NO_BLOCKS = 3,    /* the host block pool has no free block            */
  PKV_ERR_OOB = 4,          /* (device) block id / slot / length out of range   */
  PKV_ERR_CUDA = 5,         /* a CUDA runtime call failed                        */
  PKV_ERR_WORKSPACE = 6,    /* workspace missing or smaller than required        */
  PKV_ERR_TIMEOUT = 7       /* (device) a bounded internal wait expired          */
} pkv_status;

typedef enum { PKV_F16 = 0, PKV_BF16 = 1 } pkv_dtype;

/* Library version (major * 10000 + minor * 100 + patch). */
int pkv_version(void);

/* Static text for a status code. */
const char* pkv_status_string(int status);

/* The CUDA runtime call that made the calling thread's last PKV_ERR_CUDA
 * (name, error name and text); "" when none has failed.  Thread-local. */
const char* pkv_last_error(void);

/* ---------------------------------------------------------------------------
 * Slot mapping.  For token t of sequence b = seq_idx[t] (or b = t when seq_idx
 * is NULL) at logical position p = positions[t] + position_offset:
 *     slot_mapping[t] = block_tables[b][p / block_size] * block_size + p % block_size
 * (the block-table lookup of "Series 03 ...", section 3.1).  p < 0 gives -1 (a
 * padding token).  A table entry outside [0, num_blocks) or p past the table
 * gives -1 and PKV_ERR_OOB in err_flag.  Decode: positions = context_lens with
 * position_offset = -1 (the last position).  All pointers are device memory.
 * ------------------------------------------------------------------------- */
pkv_status pkv_slot_mapping(const int32_t* block_tables, int max_blocks_per_seq, int64_t num_blocks,
                            const int32_t* seq_idx, const int32_t* positions, int32_t position_offset,
                            int64_t num_tokens, int block_size, int64_t* slot_mapping, int32_t* err_flag,
                            void* stream);

/* ---------------------------------------------------------------------------
 * Append ("KV Cache, the memory notepad ...", section 三: each step appends the
 * new token's K/V to the cache).  Copies k_new[t, h, :] to
 * k_cache[s / block_size, h, s % block_size, :] with s = slot_mapping[t], and
 * the same for V; a bit-exact copy.  s < 0 skips the token; s >= num_blocks *
 * block_size is skipped and reported as PKV_ERR_OOB.  dtype is the element type
 * of k_new, v_new and the caches.
 * ------------------------------------------------------------------------- */
pkv_status pkv_kv_append(const void* k_new, const void* v_new, const int64_t* slot_mapping, int64_t num_tokens,
                         void* k_cache, void* v_cache, int64_t num_blocks, int num_kv_heads, int head_dim,
                         int block_size, pkv_dtype dtype, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * E4M3 append ("KV cache capacity planning ...", section 4: FP8 E4M3 storage
 * with a per-attention-head scale).  Stores
 *     code = E4M3_RN_satfinite(fl32(x) / k_scale[h])
 * (IEEE fp32 division, round to nearest even, magnitudes above 448 clamp to
 * 448) for every element x of k_new (in_dtype) into the uint8 cache, and the
 * same for V with v_scale.  k_scale, v_scale: device float32 [num_kv_heads].
 * Slots as in pkv_kv_append.
 * ------------------------------------------------------------------------- */
pkv_status pkv_kv_append_fp8(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                             int64_t num_tokens, uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                             const float* k_scale, const float* v_scale, int num_kv_heads, int head_dim,
                             int block_size, pkv_dtype in_dtype, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * E5M2 append ("KV cache capacity planning ...", section 4: the second FP8
 * format it names, with the wider exponent range and the lower precision; the
 * OCP 8-bit floating point specification of its reference list: bias 15, two
 * mantissa bits, largest finite value 57344).  Stores
 *     code = E5M2_RN_satfinite(fl32(x) / k_scale[h])
 * (IEEE fp32 division, round to nearest even, magnitudes above 57344 --
 * infinities included -- clamp to 57344, NaN stores a NaN code) for every
 * element x of k_new (in_dtype) into the uint8 cache, and the same for V with
 * v_scale.  Arguments, layout and errors as in pkv_kv_append_fp8.
 * ------------------------------------------------------------------------- */
pkv_status pkv_kv_append_e5m2(const void* k_new, const void* v_new, const int64_t* slot_mapping,
                              int64_t num_tokens, uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks,
                              const float* k_scale, const float* v_scale, int num_kv_heads, int head_dim,
                              int block_size, pkv_dtype in_dtype, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Workspace for decode attention, in bytes, on the current CUDA device.  The
 * decode splits the work over the flattened (sequence, KV head, block) space;
 * pieces of a sequence handled by different thread blocks leave fp32 partial
 * results (running max, sum, unnormalised output) that a combine kernel merges
 * by log-sum-exp.  partition_tokens = 0 sizes the balanced split (one equal
 * share per resident thread block); > 0 (a multiple of block_size) sizes a
 * split into fixed partitions of that many tokens of the flattened space, an
 * equal number of consecutive partitions per resident thread block (the
 * partitions of one sequence and KV head that one thread block holds are
 * merged as it streams them, so each pair leaves one partial per thread block
 * it meets).  Returns 0 on invalid arguments or when the device cannot be
 * queried.
 * ------------------------------------------------------------------------- */
size_t pkv_decode_workspace_bytes(int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                  int max_blocks_per_seq, int max_context_len, int partition_tokens);

/* ---------------------------------------------------------------------------
 * Paged decode attention, 16-bit cache.  For every sequence b and query head h:
 *     out[b, h] = sum_{j < n} softmax_j(scale * <q[b, h], K_j>) V_j
 * with n = context_lens[b] and K_j = k_cache[block_tables[b][j / 16], h / G,
 * j % 16, :] (V likewise).  Softmax arithmetic is fp32 with the running
 * maximum subtracted; out is rounded to dtype (nearest even).  n = 0 gives
 * out[b, :, :] = 0.  One thread block serves all G query heads of a KV head,
 * so each KV byte is read from HBM once.
 *   q, k_cache, v_cache, out      dtype (F16 / BF16), layouts above.
 *   block_tables, context_lens    device int32.
 *   max_context_len               an upper bound of context_lens (sizes the
 *                                 partition split; longer contexts are clamped
 *                                 and reported as PKV_ERR_OOB).
 *   partition_tokens              0 = balanced split; > 0 see the workspace query.
 *   workspace, workspace_bytes    caller-owned device scratch of at least
 *                                 pkv_decode_workspace_bytes(...); its contents
 *                                 need no initialisation and are overwritten.
 *                                 Two calls running at the same time on the GPU
 *                                 must not share a workspace.
 * Requirements: num_q_heads % num_kv_heads == 0 with G in {1, 2, 4, 8};
 * head_dim in {64, 128}; block_size == 16.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_attention(const void* q, const void* k_cache, const void* v_cache,
                                      const int32_t* block_tables, const int32_t* context_lens, int batch,
                                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                      int max_blocks_per_seq, int64_t num_blocks, int max_context_len,
                                      float scale, void* out, pkv_dtype dtype, int partition_tokens,
                                      void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Paged decode attention without a workspace argument, for callers that
 * cannot allocate device memory: a plugin or C host program whose host
 * application owns every device allocation and exposes no allocator, or a
 * latency-critical loop where cudaMalloc / cudaFree (which synchronise the
 * device) are not allowed.  The pages have no counterpart: this is a calling
 * convention, not part of the method.
 *
 * Computes exactly what pkv_paged_decode_attention computes (same arguments,
 * minus workspace / workspace_bytes).  The scratch is one file-scope device
 * array of PKV_NOALLOC_SCRATCH_BYTES bytes that every GPU loading the library
 * holds until the process exits.  This function allocates nothing.
 *   - Limit: a call whose pkv_decode_workspace_bytes(...) exceeds
 *     PKV_NOALLOC_SCRATCH_BYTES (16 MiB) is refused with PKV_ERR_WORKSPACE.
 *     Either split needs about 5 MB at most on a 152-SM GPU (head_dim 128,
 *     group 8) plus 8 bytes per sequence, so calls of up to about a million
 *     sequences fit.
 *   - Set-up: every call looks up the array's device address on the current
 *     device (cudaGetSymbolAddress, which allocates nothing), so the address
 *     is right after a cudaDeviceReset too.  The first call on a device also
 *     loads the library's device code there: make that first call before any
 *     stream capture.
 *   - Argument errors are reported as pkv_paged_decode_attention reports
 *     them (batch 0 included); only a size check comes first.
 *   - Sharing: every call on a device uses the same array and it keeps the
 *     last call's contents; the kernel writes each scratch word before reading
 *     it, so nothing needs clearing.  Calls that overlap on the GPU (other
 *     streams, or other host threads) race on the scratch: serialise them.
 * ------------------------------------------------------------------------- */
#define PKV_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u)

pkv_status pkv_paged_decode_attention_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_tables, const int32_t* context_lens, int batch,
                                              int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                              int max_blocks_per_seq, int64_t num_blocks, int max_context_len,
                                              float scale, void* out, pkv_dtype dtype, int partition_tokens,
                                              int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Paged decode attention over an E4M3 cache (uint8 codes) with per-KV-head
 * scales: K_j and V_j above are replaced by E4M3(code) * k_scale[g] and
 * E4M3(code) * v_scale[g], dequantised in registers before the arithmetic
 * ("KV cache capacity planning ...", section 5).  q and out use q_dtype.  All
 * other arguments as in pkv_paged_decode_attention.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_attention_fp8(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                          const float* k_scale, const float* v_scale,
                                          const int32_t* block_tables, const int32_t* context_lens, int batch,
                                          int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                          int max_blocks_per_seq, int64_t num_blocks, int max_context_len,
                                          float scale, void* out, pkv_dtype q_dtype, int partition_tokens,
                                          void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                          void* stream);

/* ---------------------------------------------------------------------------
 * Paged decode attention over an E5M2 cache (uint8 codes, as stored by
 * pkv_kv_append_e5m2) with per-KV-head scales: K_j and V_j are
 * E5M2(code) * k_scale[g] and E5M2(code) * v_scale[g], dequantised in
 * registers before the arithmetic ("KV cache capacity planning ...", sections
 * 4 and 5).  Arguments as in pkv_paged_decode_attention_fp8.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_attention_e5m2(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                           const float* k_scale, const float* v_scale,
                                           const int32_t* block_tables, const int32_t* context_lens, int batch,
                                           int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                           int max_blocks_per_seq, int64_t num_blocks, int max_context_len,
                                           float scale, void* out, pkv_dtype q_dtype, int partition_tokens,
                                           void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                           void* stream);

/* ---------------------------------------------------------------------------
 * One whole decode step in a single decode launch (plus the partial merge):
 * for every sequence b, append k_new[b] / v_new[b] at position
 * p = context_lens[b] - 1 (slot = block_tables[b][p / 16] * 16 + p % 16,
 * written to slot_mapping_out[b] when that pointer is not NULL; -1 for an
 * empty context or an out-of-range table entry), then attend
 * over the context_lens[b] tokens.  Same results as pkv_slot_mapping +
 * pkv_kv_append + pkv_paged_decode_attention, bit for bit.
 *   k_new, v_new    device [batch, num_kv_heads, head_dim] in dtype.
 *   k_cache, v_cache written (the new rows) and read.
 * The new row's slot must belong to sequence b alone (not a block shared with
 * another table), as for any append.  Other arguments as in
 * pkv_paged_decode_attention.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_step(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                                 const int32_t* block_tables, const int32_t* context_lens, int batch,
                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                 int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale,
                                 void* out, pkv_dtype dtype, int partition_tokens, int64_t* slot_mapping_out,
                                 void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * The same fused step over an E4M3 cache: the new rows (q_dtype) are stored as
 * E4M3_RN_satfinite(fl32(x) / scale[h]) exactly as pkv_kv_append_fp8 stores
 * them, and attention uses those codes, as pkv_paged_decode_attention_fp8.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_step_fp8(const void* q, const void* k_new, const void* v_new, uint8_t* k_cache,
                                     uint8_t* v_cache, const float* k_scale, const float* v_scale,
                                     const int32_t* block_tables, const int32_t* context_lens, int batch,
                                     int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                     int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale,
                                     void* out, pkv_dtype q_dtype, int partition_tokens, int64_t* slot_mapping_out,
                                     void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * The same fused step over an E5M2 cache: the new rows (q_dtype) are stored as
 * pkv_kv_append_e5m2 stores them, and attention uses those codes, as
 * pkv_paged_decode_attention_e5m2.  Arguments as in pkv_paged_decode_step_fp8.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_step_e5m2(const void* q, const void* k_new, const void* v_new, uint8_t* k_cache,
                                      uint8_t* v_cache, const float* k_scale, const float* v_scale,
                                      const int32_t* block_tables, const int32_t* context_lens, int batch,
                                      int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                      int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale,
                                      void* out, pkv_dtype q_dtype, int partition_tokens, int64_t* slot_mapping_out,
                                      void* workspace, size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * One whole decode step from HOST buffers: copies q, k_new, v_new,
 * block_tables and context_lens from (preferably pinned) host memory into the
 * caller's device staging buffers, runs pkv_paged_decode_step (slots of the
 * new tokens into d_slots, append, attention) and copies out back to host
 * memory, all enqueued on `stream`.  The caller synchronises the stream before reading h_out.
 *   h_*        host pointers; shapes as above with num_tokens = batch.
 *   d_*        device staging buffers of the same sizes; d_slots is int64 [batch].
 *   caches     device, persistent across steps.
 * ------------------------------------------------------------------------- */
pkv_status pkv_decode_step_host(const void* h_q, const void* h_k_new, const void* h_v_new,
                                const int32_t* h_block_tables, const int32_t* h_context_lens, void* h_out,
                                void* d_q, void* d_k_new, void* d_v_new, int32_t* d_block_tables,
                                int32_t* d_context_lens, int64_t* d_slots, void* d_out, void* k_cache,
                                void* v_cache, int batch, int num_q_heads, int num_kv_heads, int head_dim,
                                int block_size, int max_blocks_per_seq, int64_t num_blocks, int max_context_len,
                                float scale, pkv_dtype dtype, int partition_tokens, void* workspace,
                                size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * INT8 KV cache with per-block min-max scaling ("What a KV cache is ...",
 * section 3.3: q = round((k - k_min) / (k_max - k_min) * 255), two scalars
 * per block).  Codes are uint8, num_blocks x num_kv_heads slabs of 16 x
 * head_dim bytes.  A K slab holds the 16 rows in order, [16][head_dim].  A V
 * slab is the same with head_dim 64; with head_dim 128 it is stored
 * transposed, [128][16], and the 16 columns of a row hold tokens 0 1 8 9 2 3
 * 10 11 4 5 12 13 6 7 14 15 (column c: token 2 (c / 4) + c % 2 +
 * 8 ((c / 2) % 2)), the order in which the decode kernel's tensor-core
 * consumer multiplies them (so it needs no transpose).  The
 * scalars are per (block, KV head) for K and for V, stored as float
 * [num_blocks, num_kv_heads, 4] = (k_min, k_max, v_min, v_max) (16-byte
 * aligned).  Encoding: float32 in the formula's order with IEEE rounding,
 * round half to even, clamped to [0, 255]; max == min gives 0; rows of a
 * block that hold no token have code 0 and do not enter min / max.
 * Decoding: x = min + q (max - min) / 255.
 *
 * pkv_kv_quantize_int8: quantise 16-bit pools k_src / v_src [num_blocks,
 * num_kv_heads, 16, head_dim] of src_dtype; rows_used (device int32
 * [num_blocks], nullable = 16 each) gives the rows of each block that hold
 * tokens.
 * pkv_kv_append_int8: write token t's rows k_new / v_new [T, num_kv_heads,
 * head_dim] (in_dtype) at slot_mapping[t] (< 0 skips; past the pool:
 * PKV_ERR_OOB) and re-quantise rows 0..slot % 16 of that block: the old codes
 * are decoded in float32 as min + ((q * (max - min)) / 255), min / max are
 * taken again over those rows and the new one, and all of them are encoded
 * again.  The tokens of one call must lie in distinct blocks; k_cache, v_cache
 * and slab_params must be 16-byte aligned (PKV_ERR_INVALID_ARG otherwise).
 * pkv_paged_decode_attention_int8: pkv_paged_decode_attention over such a
 * cache; dequantisation happens in registers as k_min sum(q) + dk (q . codes)
 * per score and v_min sum(p) + dv (p . codes) per output.  q_dtype is the type
 * of q and out.
 * ------------------------------------------------------------------------- */
pkv_status pkv_kv_quantize_int8(const void* k_src, const void* v_src, uint8_t* k_cache, uint8_t* v_cache,
                                float* slab_params, const int32_t* rows_used, int64_t num_blocks, int num_kv_heads,
                                int head_dim, int block_size, pkv_dtype src_dtype, int32_t* err_flag, void* stream);
pkv_status pkv_kv_append_int8(const void* k_new, const void* v_new, const int64_t* slot_mapping, int64_t num_tokens,
                              uint8_t* k_cache, uint8_t* v_cache, float* slab_params, int64_t num_blocks,
                              int num_kv_heads, int head_dim, int block_size, pkv_dtype in_dtype, int32_t* err_flag,
                              void* stream);
pkv_status pkv_paged_decode_attention_int8(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                           const float* slab_params, const int32_t* block_tables,
                                           const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads,
                                           int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                           int max_context_len, float scale, void* out, pkv_dtype q_dtype,
                                           int partition_tokens, void* workspace, size_t workspace_bytes,
                                           int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Multi-layer cache and whole-step launch ("What a KV cache is ...", section
 * 2.2: one preallocated cache of shape (num_blocks, num_layers, H_kv,
 * block_size, head_dim) for the whole model, so one block id addresses a token
 * range in every layer).  k_cache / v_cache are [num_blocks, num_layers,
 * num_kv_heads, 16, head_dim] (16-bit, 16-byte aligned); block tables and
 * lengths are shared by all layers.
 *
 * pkv_paged_decode_step_layer: pkv_paged_decode_step on layer `layer` of such a
 * cache (0 <= layer < num_layers; PKV_ERR_INVALID_ARG otherwise).
 *
 * pkv_step_graph_create: capture one decode step over all num_layers layers --
 * for each layer l the fused step with q + l * batch * num_q_heads * head_dim,
 * k_new / v_new + l * batch * num_kv_heads * head_dim and out + l * batch *
 * num_q_heads * head_dim elements (q, out [num_layers, batch, Hq, D]; k_new,
 * v_new [num_layers, batch, Hkv, D]), one workspace reused layer after layer --
 * into a CUDA graph.  The graph holds these pointers: later launches read
 * whatever the buffers hold then.  pkv_step_graph_launch replays it on
 * `stream` (one host call per model step); pkv_step_graph_destroy frees it.
 * Errors: PKV_ERR_INVALID_ARG for a null handle or bad sizes, PKV_ERR_CUDA if
 * capture or instantiation fails (pkv_last_error names the call).
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_step_layer(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                       void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
                                       int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                       int max_blocks_per_seq, int64_t num_blocks, int num_layers, int layer,
                                       int max_context_len, float scale, void* out, pkv_dtype dtype,
                                       int partition_tokens, int64_t* slot_mapping_out, void* workspace,
                                       size_t workspace_bytes, int32_t* err_flag, void* stream);

typedef struct pkv_step_graph pkv_step_graph;

pkv_status pkv_step_graph_create(pkv_step_graph** graph, const void* q, const void* k_new, const void* v_new,
                                 void* k_cache, void* v_cache, const int32_t* block_tables,
                                 const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads,
                                 int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                 int num_layers, int max_context_len, float scale, void* out, pkv_dtype dtype,
                                 int partition_tokens, int64_t* slot_mapping_out, void* workspace,
                                 size_t workspace_bytes, int32_t* err_flag);
pkv_status pkv_step_graph_launch(pkv_step_graph* graph, void* stream);
void pkv_step_graph_destroy(pkv_step_graph* graph);

/* ---------------------------------------------------------------------------
 * The INT8 decode step: for every sequence b, the new rows k_new[b] /
 * v_new[b] (q_dtype, [batch, num_kv_heads, head_dim]) go to position
 * p = context_lens[b] - 1 (slot written to slot_mapping_out[b] when not NULL;
 * -1 for an empty context or an out-of-range table entry, which also records
 * PKV_ERR_OOB) and rows 0..p % 16 of that block are re-quantised as
 * pkv_kv_append_int8 does; then the attention of
 * pkv_paged_decode_attention_int8 runs over the context_lens[b] tokens.  The
 * same codes, scalars, slots and outputs as pkv_slot_mapping +
 * pkv_kv_append_int8 + pkv_paged_decode_attention_int8, bit for bit, in three
 * launches (append with the slots from the table, decode, combine) that
 * overlap: the decode kernel starts while the append runs and waits for it
 * before reading the cache.  The new row's block must belong to sequence b
 * alone.  Other arguments as in pkv_paged_decode_attention_int8.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_step_int8(const void* q, const void* k_new, const void* v_new, uint8_t* k_cache,
                                      uint8_t* v_cache, float* slab_params, const int32_t* block_tables,
                                      const int32_t* context_lens, int batch, int num_q_heads, int num_kv_heads,
                                      int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                      int max_context_len, float scale, void* out, pkv_dtype q_dtype,
                                      int partition_tokens, int64_t* slot_mapping_out, void* workspace,
                                      size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Rotary positions, fused with the append.  The first rot_dim elements of
 * every query and key head are rot_dim / 2 pairs -- elements (2 i, 2 i + 1) in
 * the interleaved layout, (i, i + rot_dim / 2) in the half one -- and pair
 * (x, y) number i of a token at position p becomes
 *     (a (x cos t - y sin t), a (x sin t + y cos t)),   t = p f_i
 * with a = amplitude; the elements from rot_dim on pass through.
 *
 * pkv_rope_plan (host, no CUDA call) lays out the frequencies of
 *     f_i = base^(-2 i / rot_dim),   i < rot_dim / 2
 * scaled for a context longer than original_context:
 *   PKV_ROPE_NONE        as they are
 *   PKV_ROPE_LINEAR      f_i / factor
 *   PKV_ROPE_BASE        base replaced by base factor^(rot_dim / (rot_dim - 2))
 *   PKV_ROPE_RAMP        f_i (1 - w_i) + f_i / factor w_i, where w_i rises
 *                        from 0 to 1 over the pairs between the one that makes
 *                        high_turns full turns in original_context positions
 *                        (rounded down) and the one that makes low_turns
 *                        (rounded up); amplitude 0.1 ln(factor) + 1
 *   PKV_ROPE_WAVELENGTH  f_i w + f_i / factor (1 - w), w = (n - low_turns) /
 *                        (high_turns - low_turns) clamped to [0, 1], n the
 *                        full turns of f_i in original_context positions
 * into turns[rot_dim / 2] (host): f_i / (2 pi), full turns per position, in
 * units of 2^-64 (rounded).  A position times it, modulo 2^64, is the angle
 * modulo one turn, so far positions lose nothing but p times f_i's rounding.
 * amplitude: 1 but for PKV_ROPE_RAMP.  The caller copies turns to the device
 * once.
 * PKV_ERR_INVALID_ARG: an odd or non-positive rot_dim, base <= 1, factor < 1,
 * low_turns <= 0 or high_turns <= low_turns (where they are used).
 *
 * pkv_rope_append: q_out[t] takes the turned q[t]; the cache slot
 * slot_mapping[t] (as in pkv_kv_append) takes the turned k_new[t] and v_new[t]
 * as it is.  The rotation is fp32 and each turned element is rounded once, to
 * dtype or to the cache's FP8 format (fl32(x) / scale[h] as
 * pkv_kv_append_fp8 / _e5m2; v rows are stored bit for bit as those calls
 * store them).
 *   q, k_new, v_new    dtype; token t's heads, [H, head_dim] contiguous, start
 *                      t * stride elements from the pointer, so they may be
 *                      slices of one projection's output.  Strides: multiples
 *                      of 8, at least H head_dim.
 *   q_out              as q, with its own stride; q_out == q with the same
 *                      stride turns q in place.  Other overlaps, of it or of
 *                      the caches with an input, are undefined.
 *   positions          device int32 [T]; a negative one marks a padding token,
 *                      for which nothing is written.
 *   slot_mapping       device int64 [T]; negative: no append for the token (q
 *                      is turned all the same); past the pool: skipped and
 *                      PKV_ERR_OOB in err_flag.  The slots of one call are
 *                      distinct.
 *   turns, amplitude   from pkv_rope_plan, turns in device memory.
 * q and q_out may both be NULL (append only), or k_new and v_new (turn q only;
 * the caches and slots are then not used).  rot_dim: a multiple of 16 up to
 * head_dim (else PKV_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------- */
typedef enum { PKV_ROPE_HALF = 0, PKV_ROPE_INTERLEAVED = 1 } pkv_rope_layout;
typedef enum {
  PKV_ROPE_NONE = 0,
  PKV_ROPE_LINEAR = 1,
  PKV_ROPE_BASE = 2,
  PKV_ROPE_RAMP = 3,
  PKV_ROPE_WAVELENGTH = 4
} pkv_rope_scaling;

pkv_status pkv_rope_plan(int rot_dim, double base, pkv_rope_scaling scaling, double factor, double original_context,
                         double low_turns, double high_turns, uint64_t* turns, float* amplitude);

pkv_status pkv_rope_append(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride, const void* v_new,
                           int64_t v_stride, const int32_t* positions, const int64_t* slot_mapping,
                           int64_t num_tokens, const uint64_t* turns, int rot_dim, pkv_rope_layout layout,
                           float amplitude, void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache,
                           int64_t num_blocks, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                           pkv_dtype dtype, int32_t* err_flag, void* stream);
pkv_status pkv_rope_append_fp8(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                               const void* v_new, int64_t v_stride, const int32_t* positions,
                               const int64_t* slot_mapping, int64_t num_tokens, const uint64_t* turns, int rot_dim,
                               pkv_rope_layout layout, float amplitude, void* q_out, int64_t q_out_stride,
                               uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks, const float* k_scale,
                               const float* v_scale, int num_q_heads, int num_kv_heads, int head_dim,
                               int block_size, pkv_dtype dtype, int32_t* err_flag, void* stream);
pkv_status pkv_rope_append_e5m2(const void* q, int64_t q_stride, const void* k_new, int64_t k_stride,
                                const void* v_new, int64_t v_stride, const int32_t* positions,
                                const int64_t* slot_mapping, int64_t num_tokens, const uint64_t* turns, int rot_dim,
                                pkv_rope_layout layout, float amplitude, void* q_out, int64_t q_out_stride,
                                uint8_t* k_cache, uint8_t* v_cache, int64_t num_blocks, const float* k_scale,
                                const float* v_scale, int num_q_heads, int num_kv_heads, int head_dim,
                                int block_size, pkv_dtype dtype, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Block-sparse decode: attention over the blocks of a long context that a
 * cheap score picks for each (sequence, KV head).
 *
 * pkv_kv_block_bounds: bounds[id, h] = the elementwise minimum, then maximum,
 * of the rows of block id that hold tokens ([num_blocks, num_kv_heads, 2,
 * head_dim] of dtype, exact; a NaN key element gives NaN), for the blocks of
 * every sequence that hold its last new_lens[b] tokens: the new ones after an
 * append, whose first block may have held older rows as well.  new_lens NULL:
 * all blocks of the context.  max_new_len: an upper bound of new_lens (of
 * context_lens when NULL); it sizes the launch (0: nothing is done), and blocks
 * past it are left as they are and reported as PKV_ERR_OOB.  _fp8 / _e5m2: over
 * codes; the bounds are the codes' values, before the per-head scale, in
 * bounds_dtype (exact in both).  A block that two sequences share must hold the
 * same rows for both (full, or equal lengths).  Bounds of other blocks stay.
 *
 * pkv_block_scores: for i < ceil(context_lens[b] / 16), with (lo, hi) the
 * bounds of block_tables[b][i],
 *     scores[b, g, i] = scale k_scale[g] max_h sum_d max(q_d lo_d, q_d hi_d)
 * over the query heads h of KV head g: no token of the block has a larger
 * scaled logit for any of them.  fp32 [batch, num_kv_heads,
 * max_blocks_per_seq]; entries past the context stay as they are.  k_scale:
 * device [num_kv_heads], NULL = 1.  scale >= 0.  Elements must be finite for
 * a defined score; a NaN or an infinity in q or the bounds gives NaN or an
 * infinity.  A table entry outside the pool scores -infinity and reports
 * PKV_ERR_OOB.  max_context_len as in pkv_paged_decode_attention.
 *
 * pkv_select_blocks: the blocks to attend to, ascending, in selected [batch,
 * num_kv_heads, budget] int32: every block when there are at most budget of
 * them, else the first num_first, the last num_last and the highest-scoring
 * others (ties to the lowest index; NaN above +infinity, -0 equal to +0);
 * entries behind the list are -1.  num_first + num_last <= budget.  scores:
 * any fp32 [batch, num_kv_heads, max_blocks_per_seq].
 *
 * pkv_paged_decode_attention_sparse[_fp8 / _e5m2]: pkv_paged_decode_attention
 * over the tokens of the listed blocks only: of selected[b, g] the first
 * min(budget, ceil(context_lens[b] / 16)) entries count, in any order; a
 * negative entry is skipped, one listed twice counts twice, one behind the
 * context is skipped and reported as PKV_ERR_OOB.  The context's last block
 * contributes its tokens only.  No tokens listed gives out = 0.
 *   workspace   at least pkv_decode_workspace_bytes(batch, num_q_heads,
 *               num_kv_heads, head_dim, budget, 16 budget, 0).
 * ------------------------------------------------------------------------- */
pkv_status pkv_kv_block_bounds(const void* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                               const int32_t* new_lens, int max_new_len, int batch, int num_kv_heads, int head_dim,
                               int block_size, int max_blocks_per_seq, int64_t num_blocks, void* bounds,
                               pkv_dtype dtype, int32_t* err_flag, void* stream);
pkv_status pkv_kv_block_bounds_fp8(const uint8_t* k_cache, const int32_t* block_tables, const int32_t* context_lens,
                                   const int32_t* new_lens, int max_new_len, int batch, int num_kv_heads,
                                   int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
                                   void* bounds, pkv_dtype bounds_dtype, int32_t* err_flag, void* stream);
pkv_status pkv_kv_block_bounds_e5m2(const uint8_t* k_cache, const int32_t* block_tables,
                                    const int32_t* context_lens, const int32_t* new_lens, int max_new_len, int batch,
                                    int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                                    int64_t num_blocks, void* bounds, pkv_dtype bounds_dtype, int32_t* err_flag,
                                    void* stream);
pkv_status pkv_block_scores(const void* q, const void* bounds, const int32_t* block_tables,
                            const int32_t* context_lens, const float* k_scale, int batch, int num_q_heads,
                            int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                            int64_t num_blocks, int max_context_len, float scale, float* scores, pkv_dtype dtype,
                            int32_t* err_flag, void* stream);
pkv_status pkv_select_blocks(const float* scores, const int32_t* context_lens, int batch, int num_kv_heads,
                             int block_size, int max_blocks_per_seq, int num_first, int num_last, int budget,
                             int32_t* selected, int32_t* err_flag, void* stream);
pkv_status pkv_paged_decode_attention_sparse(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, const int32_t* context_lens,
                                             const int32_t* selected, int budget, int batch, int num_q_heads,
                                             int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq,
                                             int64_t num_blocks, float scale, void* out, pkv_dtype dtype,
                                             void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                             void* stream);
pkv_status pkv_paged_decode_attention_sparse_fp8(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                 const float* k_scale, const float* v_scale,
                                                 const int32_t* block_tables, const int32_t* context_lens,
                                                 const int32_t* selected, int budget, int batch, int num_q_heads,
                                                 int num_kv_heads, int head_dim, int block_size,
                                                 int max_blocks_per_seq, int64_t num_blocks, float scale, void* out,
                                                 pkv_dtype q_dtype, void* workspace, size_t workspace_bytes,
                                                 int32_t* err_flag, void* stream);
pkv_status pkv_paged_decode_attention_sparse_e5m2(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                  const float* k_scale, const float* v_scale,
                                                  const int32_t* block_tables, const int32_t* context_lens,
                                                  const int32_t* selected, int budget, int batch, int num_q_heads,
                                                  int num_kv_heads, int head_dim, int block_size,
                                                  int max_blocks_per_seq, int64_t num_blocks, float scale, void* out,
                                                  pkv_dtype q_dtype, void* workspace, size_t workspace_bytes,
                                                  int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Decode attention for sequences that share a prefix ("Series 03 ...", section
 * 3.3: shared prompts keep one copy of their blocks): the result of
 * pkv_paged_decode_attention, with the prefix's K and V read once per group
 * and KV head instead of once per sequence.  The sequences are cut into
 * consecutive groups, group j being sequences group_starts[j] ..
 * group_starts[j + 1] - 1 (group_starts[0] = 0, group_starts[num_groups] =
 * batch; a group may be empty or a single sequence), and the first
 * prefix_lens[j] / 16 (rounded down) entries of their block table rows are the
 * same ids; the remaining tokens are each sequence's own.  A sequence shorter
 * than its group's whole shared blocks is attended to through its own row
 * alone (so a padding sequence of length 0 gives 0 and its row is not read);
 * the prefix is read through the row of the first sequence that covers it.
 *   group_starts, prefix_lens   device int32 [num_groups + 1], [num_groups].
 *   max_prefix_len              an upper bound of prefix_lens; it sizes the
 *                               launch only.
 *   scale                       > 0.
 *   workspace                   at least pkv_prefix_workspace_bytes(...), no
 *                               initialisation needed; not shared by calls
 *                               that run at the same time.
 * The weights are multiplied in 16 bits as there, fp16 ones rounded once (and
 * the normaliser sums the rounded ones); bf16 ones, and fp16 ones with one query
 * head per KV head, as two parts (exact to 2^-16).
 * 16-bit caches; at most 1024 groups, and a batch whose counts (16 bytes a
 * sequence) fit one thread block's shared memory, as 10,000 sequences always do
 * (PKV_ERR_UNSUPPORTED beyond, with nothing launched).  Group
 * starts that are not as described report PKV_ERR_OOB in err_flag, and the
 * outputs are then unspecified.  Other arguments, requirements and errors as
 * in pkv_paged_decode_attention.
 * ------------------------------------------------------------------------- */
size_t pkv_prefix_workspace_bytes(int batch, int num_groups, int num_q_heads, int num_kv_heads, int head_dim,
                                  int max_blocks_per_seq, int max_context_len, int max_prefix_len);
pkv_status pkv_paged_decode_attention_prefix(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, const int32_t* context_lens,
                                             const int32_t* group_starts, const int32_t* prefix_lens,
                                             int num_groups, int batch, int num_q_heads, int num_kv_heads,
                                             int head_dim, int block_size, int max_blocks_per_seq,
                                             int64_t num_blocks, int max_context_len, int max_prefix_len,
                                             float scale, void* out, pkv_dtype dtype, void* workspace,
                                             size_t workspace_bytes, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Decode attention to the first num_sinks and the last `window` tokens of each
 * context: pkv_paged_decode_attention with token j of n = context_lens[b] seen
 * only where j < num_sinks or j >= n - window (so a window of at least n is the
 * dense decode).  Blocks that hold no such token are not looked up and not
 * read: their table entries may be anything and their memory may have been
 * given back.  K and V rows that are not seen may hold anything.
 *   window      >= 1; num_sinks >= 0 (else PKV_ERR_INVALID_ARG).
 *   workspace   at least pkv_decode_workspace_bytes(batch, num_q_heads,
 *               num_kv_heads, head_dim, max_blocks_per_seq, n, 0), the same for
 *               every n.
 * Other arguments, requirements and errors as in pkv_paged_decode_attention and
 * its FP8 forms (a context longer than the table is cut to it and reported).
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_decode_attention_window(const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, const int32_t* context_lens, int batch,
                                             int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                             int max_blocks_per_seq, int64_t num_blocks, int window, int num_sinks,
                                             float scale, void* out, pkv_dtype dtype, void* workspace,
                                             size_t workspace_bytes, int32_t* err_flag, void* stream);
pkv_status pkv_paged_decode_attention_window_fp8(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                 const float* k_scale, const float* v_scale,
                                                 const int32_t* block_tables, const int32_t* context_lens, int batch,
                                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                                 int max_blocks_per_seq, int64_t num_blocks, int window,
                                                 int num_sinks, float scale, void* out, pkv_dtype q_dtype,
                                                 void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                                 void* stream);
pkv_status pkv_paged_decode_attention_window_e5m2(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                                  const float* k_scale, const float* v_scale,
                                                  const int32_t* block_tables, const int32_t* context_lens, int batch,
                                                  int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                                  int max_blocks_per_seq, int64_t num_blocks, int window,
                                                  int num_sinks, float scale, void* out, pkv_dtype q_dtype,
                                                  void* workspace, size_t workspace_bytes, int32_t* err_flag,
                                                  void* stream);

/* ---------------------------------------------------------------------------
 * The same rule for the tokens of a prompt chunk (the windowed form of
 * pkv_paged_prefill_attention, without its clusters): the n_b = cu_seqlens[b +
 * 1] - cu_seqlens[b] new tokens of sequence b are its last n_b positions, already
 * in the cache; token i, at position p = context_lens[b] - n_b + i, sees position
 * j where j <= p and (j < num_sinks or j > p - window).  q and out are
 * [num_tokens, num_q_heads, head_dim]; 16-bit caches, head_dim 64 or 128, scale >
 * 0.  Blocks that hold no key of a new token's are not looked up and not read.  K
 * and V of positions that a token does not see change nothing for it, whatever
 * bits they hold; an element of V that is not finite gives an output that is not
 * finite where it is seen.  Weights in 16 bits as in the drafted tokens' attention
 * below (fp16 ones rounded once, as in pkv_paged_prefill_attention, with one query
 * head per KV head too).  max_query_len: an upper bound of n_b.  Outputs of tokens
 * behind the last sequence are not written, and their q changes nothing.  Device
 * errors (PKV_ERR_OOB; the sequence is skipped, its outputs stay as they are):
 * offsets that do not ascend within [0, num_tokens], more tokens than
 * max_query_len or than the context has, a context longer than its table.  A table
 * entry outside the pool reads as zeros and is reported.
 * ------------------------------------------------------------------------- */
pkv_status pkv_paged_prefill_attention_window(const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_tables, const int32_t* context_lens,
                                              const int32_t* cu_seqlens, int64_t num_tokens, int batch,
                                              int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                              int max_blocks_per_seq, int64_t num_blocks, int max_query_len,
                                              int window, int num_sinks, float scale, void* out, pkv_dtype dtype,
                                              int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Drafted tokens: one pass over several candidate continuations of each
 * sequence, and the move of the accepted ones.  The n_b = cu_nodes[b + 1] -
 * cu_nodes[b] drafted tokens of sequence b (tokens cu_nodes[b] .. cu_nodes[b + 1]
 * - 1 of a batch's num_tokens) are its last n_b cached ones: context_lens[b]
 * counts them, and token i of them is cached at position base + i, base =
 * context_lens[b] - n_b.  cu_nodes: device int32 [batch + 1], cu_nodes[0] >= 0,
 * cu_nodes[batch] <= num_tokens; a sequence may have none.  What belongs to
 * tokens behind the last sequence is not written, and changes nothing whatever it
 * holds (rows of q there may be read).
 *
 * pkv_tree_plan: the tokens of a sequence form a tree whose root is the
 * context's last token: parents[t] (device int32 [num_tokens]) is the index of
 * token t's parent within its sequence, before its own (-1: the root).  With a
 * token's ancestors in the tree,
 *     tree_mask[t]     bit j of word j / 64: token j of the sequence is t itself
 *                      or an ancestor of it ([num_tokens, mask_words] uint64;
 *                      mask_words <= 4, else PKV_ERR_UNSUPPORTED)
 *     positions[t]     base + the number of its ancestors (int32; its rotary
 *                      position; NULL: not wanted)
 *     slot_mapping[t]  the slot of position base + i, as pkv_slot_mapping (int64;
 *                      NULL: not wanted, and block_tables is not used)
 * Device errors (PKV_ERR_OOB): offsets that are not as described (the sequence
 * is skipped); more tokens than 64 mask_words or than the context has (mask 0,
 * position and slot -1); a parent that is not before its token (taken as -1); a
 * table entry outside the pool (slot -1).
 *
 * pkv_paged_tree_attention[_fp8 / _e5m2]: token i of sequence b sees the base
 * tokens before the drafted ones and the drafted tokens j with bit j of its row
 * of tree_mask set -- any set of them, ancestors or not, itself or not; bits from
 * n_b on are not used:
 *     out[t, h] = sum_j softmax_j(scale <q[t, h], K_j>) V_j over those j
 * (0 where it sees none).  K and V rows of the drafted tokens are read from the
 * cache like the others.  A drafted token's K and V change nothing for the rows
 * that do not see it, whatever bits they hold; an element of V that is not finite
 * gives an output that is not finite where it is seen.
 *   q, out               [num_tokens, num_q_heads, head_dim].
 *   max_nodes            an upper bound of n_b, at most 64 mask_words.
 *   max_context_len      an upper bound of context_lens; it sizes the launch only.
 *   scale                > 0.
 *   workspace            at least pkv_tree_workspace_bytes(...), no
 *                        initialisation needed; not shared by calls that run at
 *                        the same time.
 * Weights are multiplied in 16 bits: over fp16 and FP8 caches as fp16 rounded
 * once (and the normaliser sums the rounded ones; weights below 2^-21 of their
 * row's largest to the nearest multiple of 2^-31 of it at worst), or, with one
 * query head per KV head, as two fp16 parts; over bf16 caches as two parts (exact
 * to 2^-16).  q meets FP8 keys as a sum of FP8 values: exact for
 * elements down to 2^-9 (bf16) or 2^-6 (fp16) of their row's largest, smaller ones off
 * by at most 2^-17 of that one; in a row where that concerns an eighth of the elements or
 * more, exact down to 2^-13, and off by at most 2^-21 (bf16) or 2^-24 (fp16).  At most 1024 sequences, num_blocks *
 * num_kv_heads < 2^27 (PKV_ERR_UNSUPPORTED beyond).  Device errors (PKV_ERR_OOB; the
 * sequence is skipped, its outputs stay as they are): offsets that are not as described, more
 * tokens than max_nodes or than the context has, a context longer than its table.
 * A table entry outside the pool reads as zeros and is reported.  Other arguments
 * and requirements as in pkv_paged_decode_attention and its FP8 forms.
 *
 * pkv_tree_commit: the drafted tokens that were accepted become the context's
 * next ones.  accepted[b] (device int32 [batch, max_accept], max_accept <= 1024)
 * lists them, strictly ascending indices within the sequence, up to its first
 * negative entry; K and V of the k-th of them move from position base +
 * accepted[b][k] to base + k, in every head (bit for bit, any type of elt_bytes 1
 * or 2; a layer-major cache [num_blocks, num_layers, H_kv, 16, head_dim] is passed
 * with num_kv_heads = num_layers * H_kv).  Other rows stay as they are.  new_lens
 * (device int32 [batch], nullable; no part of context_lens: PKV_ERR_INVALID_ARG)
 * takes base + the number of accepted tokens.  The blocks from position base on
 * belong to the sequence alone.  Device errors (PKV_ERR_OOB; nothing of the
 * sequence moves and new_lens[b] stays): a list that does not ascend or passes
 * the sequence's tokens, offsets or lengths that are not as described, a table
 * entry outside the pool where a row comes from or goes to.
 * ------------------------------------------------------------------------- */
pkv_status pkv_tree_plan(const int32_t* parents, const int32_t* cu_nodes, const int32_t* block_tables,
                         const int32_t* context_lens, int batch, int64_t num_tokens, int mask_words, int block_size,
                         int max_blocks_per_seq, int64_t num_blocks, uint64_t* tree_mask, int32_t* positions,
                         int64_t* slot_mapping, int32_t* err_flag, void* stream);
size_t pkv_tree_workspace_bytes(int batch, int64_t num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                                int max_nodes);
pkv_status pkv_paged_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, const int32_t* context_lens, const int32_t* cu_nodes,
                                    const uint64_t* tree_mask, int mask_words, int max_nodes, int64_t num_tokens,
                                    int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                    int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale,
                                    void* out, pkv_dtype dtype, void* workspace, size_t workspace_bytes,
                                    int32_t* err_flag, void* stream);
pkv_status pkv_paged_tree_attention_fp8(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                        const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                        const int32_t* context_lens, const int32_t* cu_nodes,
                                        const uint64_t* tree_mask, int mask_words, int max_nodes, int64_t num_tokens,
                                        int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                        int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale,
                                        void* out, pkv_dtype q_dtype, void* workspace, size_t workspace_bytes,
                                        int32_t* err_flag, void* stream);
pkv_status pkv_paged_tree_attention_e5m2(const void* q, const uint8_t* k_cache, const uint8_t* v_cache,
                                         const float* k_scale, const float* v_scale, const int32_t* block_tables,
                                         const int32_t* context_lens, const int32_t* cu_nodes,
                                         const uint64_t* tree_mask, int mask_words, int max_nodes, int64_t num_tokens,
                                         int batch, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                         int max_blocks_per_seq, int64_t num_blocks, int max_context_len, float scale,
                                         void* out, pkv_dtype q_dtype, void* workspace, size_t workspace_bytes,
                                         int32_t* err_flag, void* stream);
pkv_status pkv_tree_commit(void* k_cache, void* v_cache, const int32_t* block_tables, const int32_t* context_lens,
                           const int32_t* cu_nodes, const int32_t* accepted, int max_accept, int batch,
                           int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int64_t num_blocks,
                           int elt_bytes, int32_t* new_lens, int32_t* err_flag, void* stream);

/* ---------------------------------------------------------------------------
 * Host-side block pool ("Series 03 ...", sections 3.2-3.3; "What a KV cache
 * is ...", section 3.2): a preallocated set of block ids handed out on demand,
 * with reference counts for blocks shared by several block tables.  Policy: a
 * LIFO free list whose first allocations return 0, 1, 2, ...; a block freed by
 * its last decref is the next one handed out.  Not thread-safe.
 * ------------------------------------------------------------------------- */
typedef struct pkv_pool pkv_pool;

/* NULL on invalid arguments or host allocation failure. */
pkv_pool* pkv_pool_create(int64_t num_blocks, int block_size);
void pkv_pool_destroy(pkv_pool* pool);
/* PKV_ERR_NO_BLOCKS when the pool is empty ("What a KV cache is ...", 4.2). */
pkv_status pkv_pool_alloc(pkv_pool* pool, int32_t* block_id);
/* PKV_ERR_INVALID_ARG for an id that is not allocated. */
pkv_status pkv_pool_incref(pkv_pool* pool, int32_t block_id);
pkv_status pkv_pool_decref(pkv_pool* pool, int32_t block_id);
int64_t pkv_pool_num_free(const pkv_pool* pool);
int32_t pkv_pool_refcount(const pkv_pool* pool, int32_t block_id);   /* -1 for a bad id */
/* Blocks needed for n tokens: ceil(n / block_size) ("Series 03 ...", 3.2). */
int64_t pkv_blocks_needed(int64_t num_tokens, int block_size);

/* ---------------------------------------------------------------------------
 * Copy-on-write ("Series 03 ...", section 3.3: the branches of a beam search,
 * or parallel samples, share the prefix blocks without copying; when a branch
 * writes its first token of its own into a shared block, a new block is taken,
 * the old contents are copied into it and the token is written there, while
 * the other branches keep the old block).
 *
 * pkv_pool_cow: make block_id private before a write.  Reference count 1:
 * *out_id = block_id, nothing changes.  Otherwise a fresh block is taken
 * (reference count 1), block_id loses one reference and *out_id is the new
 * id; the caller points its table at it and copies block_id into it
 * (pkv_copy_blocks) before writing.  PKV_ERR_NO_BLOCKS (nothing changed) when
 * the pool is empty, PKV_ERR_INVALID_ARG for an id that is not allocated.
 * ------------------------------------------------------------------------- */
pkv_status pkv_pool_cow(pkv_pool* pool, int32_t block_id, int32_t* out_id);

/* Host side of one decode step over tables that may share blocks.  For each
 * sequence b the step's token sits at position p = context_lens[b] - 1 (the
 * length after the append; 0 means no token for b).  Entry i = p / block_size
 * of row b of block_tables ([batch, max_blocks_per_seq], host memory):
 *   - negative: the sequence grows into a new block; a fresh block is taken
 *     and stored there;
 *   - a shared block: pkv_pool_cow, the new id is stored and the pair
 *     (old, new) is appended to src_blocks / dst_blocks (host arrays of
 *     capacity batch);
 *   - a private block: nothing.
 * Sequences are taken in order b = 0, 1, ..., so when several rows share one
 * block, all but the last of them copy and the last writes in place.
 * *num_pairs receives the number of copies.  All-or-nothing: when the pool
 * cannot supply every block the step needs, PKV_ERR_NO_BLOCKS and nothing
 * changes.  PKV_ERR_INVALID_ARG for p past the row or an entry that is not an
 * allocated block.
 * ------------------------------------------------------------------------- */
pkv_status pkv_prepare_append(pkv_pool* pool, int32_t* block_tables, int batch, int max_blocks_per_seq,
                              const int32_t* context_lens, int32_t* src_blocks, int32_t* dst_blocks,
                              int32_t* num_pairs);

/* Block copy on the device (the data movement of copy-on-write): for each
 * i < num_pairs, physical block dst_blocks[i] of k_cache and of v_cache takes
 * the contents of block src_blocks[i], all heads and all rows; a bit-exact
 * copy of num_kv_heads * block_size * head_dim elements of elt_bytes bytes
 * (2 for fp16/bf16 caches, 1 for E4M3) per block and cache.  src_blocks and
 * dst_blocks are device int32 arrays.  A pair with an id outside
 * [0, num_blocks) is skipped and reported as PKV_ERR_OOB in err_flag.  The
 * destinations must be distinct and none may be a source (the pairs
 * pkv_prepare_append returns are); otherwise the result is undefined.
 * ------------------------------------------------------------------------- */
pkv_status pkv_copy_blocks(const int32_t* src_blocks, const int32_t* dst_blocks, int64_t num_pairs, void* k_cache,
                           void* v_cache, int64_t num_blocks, int num_kv_heads, int head_dim, int block_size,
                           int elt_bytes, int32_t* err_flag, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
