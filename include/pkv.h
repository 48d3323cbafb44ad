/*
 * pkv.h -- C ABI of libpkv.so: attention over a paged KV cache on GB300 (sm_103a).
 *
 * The three operations are the attention block of a nano-vLLM style engine,
 * as the pages walk through it:
 *   - "vLLM 学习笔记 02：nano-vllm 源码逐段精读", layers/attention.py listing
 *     (store_kvcache, then flash_attn_varlen_func for prefill or
 *     flash_attn_with_kvcache for decode) and engine/model_runner.py listing
 *     (how slot_mapping, cu_seqlens, block_tables and context_lens are built);
 *   - "Nano-vLLM代码手撕笔记", sections "请求执行 – 输入序列预处理与context构建"
 *     and "请求执行 – run model" (the same steps with a worked example).
 *
 * Conventions shared by every entry point
 *   - Element type: bf16 for q, k, v, caches and outputs; the *_f16 entry
 *     points take IEEE fp16 for all of them instead (the experiment code in
 *     "Nano-vLLM代码手撕笔记", section "目录结构概览", builds the engine with
 *     dtype=torch.float16). Arithmetic is fp32 for both. pkv_store_kvcache
 *     copies 16-bit patterns and serves both types. Index arrays int32.
 *   - Supported shape: head_dim = 128, block_size = 256; prefill and decode
 *     also need num_kv_heads = 8 and num_heads = 16 (Qwen3-0.6B attention:
 *     16 query heads grouped 2 per kv head). Query head h reads kv head
 *     h / (num_heads / num_kv_heads).
 *   - Cache layout: k_cache, v_cache are [num_blocks, 256, num_kv_heads, 128]
 *     contiguous; token slot s is the row starting at element s*num_kv_heads*128.
 *   - Pointers are DEVICE pointers owned by the caller unless stated. The
 *     library allocates no memory, never synchronises a stream (except
 *     pkv_device_error) and launches only on the stream it is given, so every
 *     compute call can be captured in a CUDA graph.
 *   - Return value: PKV_OK (0) or a negative PKV_ERR_* detected on the host
 *     before anything is launched (then nothing is launched). Launch failures
 *     return PKV_ERR_CUDA.
 *   - Problems only visible on the device (a slot or block id outside the
 *     pool, inconsistent cu_seqlens, a context longer than max_context_len)
 *     never cause an out-of-bounds access: the offending work is skipped and a
 *     bit is OR-ed into a per-device error word that pkv_device_error reads.
 *     Outputs touched by skipped work are unspecified.
 *   - Every device-side wait is bounded in time; a wait that runs out sets
 *     PKV_DEVERR_TIMEOUT and the kernel returns instead of hanging.
 */
#ifndef PKV_H_
#define PKV_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Host-side status codes. */
#define PKV_OK 0
#define PKV_ERR_NULL_POINTER (-1)      /* a required pointer is NULL */
#define PKV_ERR_UNSUPPORTED (-2)       /* head_dim/block_size/head counts outside the call's supported shape */
#define PKV_ERR_BAD_STRIDE (-3)        /* a row stride smaller than the row */
#define PKV_ERR_ALIGNMENT (-4)         /* pointer or stride not 16-byte aligned where a kernel needs it */
#define PKV_ERR_WORKSPACE (-5)         /* workspace NULL or smaller than the *_workspace_bytes query */
#define PKV_ERR_BAD_SIZE (-6)          /* a negative count or a size beyond the library's limits */
#define PKV_ERR_CUDA (-7)              /* a CUDA call or kernel launch failed */
#define PKV_ERR_DEVICE (-8)            /* current device is not a compute capability 10.3 GPU */
#define PKV_ERR_SCRATCH_LIMIT (-9)     /* pkv_decode_noalloc: the sizes need more than its built-in scratch */

/* Device-side error bits (pkv_device_error). */
#define PKV_DEVERR_BAD_SLOT 0x1u       /* slot_mapping entry not -1 and outside [0, num_slots) */
#define PKV_DEVERR_BAD_BLOCK 0x2u      /* block_tables entry outside [0, num_blocks) where it is read */
#define PKV_DEVERR_BAD_SEQLEN 0x4u     /* cu_seqlens not monotone, seqlen_k < seqlen_q, lengths above the
                                          declared maxima, or a context longer than the block table */
#define PKV_DEVERR_TIMEOUT 0x8u        /* a bounded device wait ran out */

/* Human-readable text for a PKV_* status. Never NULL. */
const char* pkv_status_string(int status);

/* Library version: major*10000 + minor*100 + patch. */
int pkv_version(void);

/*
 * pkv_store_kvcache -- store_kvcache from layers/attention.py
 * ("vLLM 学习笔记 02：nano-vllm 源码逐段精读"; explained in
 * "Nano-vLLM代码手撕笔记", section "请求执行 – run model").
 *
 * For each token i < num_tokens with slot = slot_mapping[i] != -1:
 *   k_cache[slot, :, :] = k[i, :, :]   and   v_cache[slot, :, :] = v[i, :, :]
 * (num_kv_heads*head_dim elements each, a bit-exact copy). Tokens with
 * slot -1 (padding) are skipped.
 *
 *   k, v            [num_tokens, num_kv_heads, head_dim] 16-bit elements
 *                   (bf16 or fp16: the copy is bit-exact either way); heads and
 *                   dims contiguous within a row, rows k_row_stride /
 *                   v_row_stride ELEMENTS apart (>= num_kv_heads*head_dim;
 *                   e.g. 4096 for views of a fused qkv projection).
 *   k_cache,v_cache [num_slots, num_kv_heads, head_dim], same type, contiguous
 *                   (num_slots = num_blocks * block_size).
 *   slot_mapping    [num_tokens] int32.
 * Any head_dim and num_kv_heads are accepted. When every pointer is 16-byte
 * aligned and both row strides and the row length are multiples of 8
 * elements, 16-byte vector copies are used; otherwise 2-byte copies.
 * Duplicate slots in one call race (the pages never produce them); k/v must
 * not overlap the caches. Slots outside [0, num_slots) set PKV_DEVERR_BAD_SLOT.
 */
int pkv_store_kvcache(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride,
                      void* k_cache, void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                      int32_t num_kv_heads, int32_t head_dim, int64_t num_slots, cudaStream_t stream);

/*
 * pkv_prefill_varlen -- causal variable-length prefill attention, the
 * flash_attn_varlen_func call of layers/attention.py with causal=True.
 *
 * Sequence b owns query rows [cu_seqlens_q[b], cu_seqlens_q[b+1]) of q and
 * Lk_b = cu_seqlens_k[b+1] - cu_seqlens_k[b] keys. Query row i of sequence b
 * sits at position Lk_b - Lq_b + i (prefix-cache hits and chunked prefill put
 * the new tokens at the end, engine/model_runner.py prepare_prefill) and
 * attends to keys 0..that position:
 *   out[row, h, :] = softmax(softmax_scale * q[row, h, :] . K[0..p, h/G, :]^T) V[0..p, h/G, :]
 * with fp32 logits and accumulation, bf16 output.
 *
 * Key source:
 *   block_tables != NULL  (prefix-cache mode): key t of sequence b is slot
 *     block_tables[b*block_table_stride + t/256]*256 + t%256 of k_cache/v_cache
 *     ([num_blocks, 256, 8, 128]). The caller runs pkv_store_kvcache for the
 *     new tokens first, on the same stream, as layers/attention.py does.
 *     Entries past ceil(Lk_b/256) are never read.
 *   block_tables == NULL  (no prefix hit): key t of sequence b is row
 *     cu_seqlens_k[b] + t of k/v ([total_k, 8, 128], rows kv_row_stride
 *     elements apart); k_cache/v_cache are ignored.
 *
 *   q    [total_q, 16, 128] bf16, rows q_row_stride elements apart.
 *   out  [total_q, 16, 128] bf16 contiguous; every row of every sequence written.
 *   total_q, total_k  row counts of q and of contiguous k/v (the tensors'
 *        first dimension; total_k is ignored in prefix-cache mode). Tiles are
 *        fetched by tensor-memory-access copies, which need the exact extent.
 *   cu_seqlens_q/k [num_seqs+1] int32, max_seqlen_q/k their largest lengths;
 *        cu_seqlens_q[num_seqs] <= total_q and, in contiguous mode,
 *        cu_seqlens_k[num_seqs] <= total_k.
 * q, k, v, k_cache, v_cache must be 16-byte aligned and their row strides
 * multiples of 8 elements (tensor-memory-access rules).
 *
 * workspace: NULL, or a tile plan -- workspace_bytes/4 int32 items written by
 *   pkv_prefill_plan for these cu_seqlens and copied to device memory (4-byte
 *   aligned, workspace_bytes a multiple of 4, at most 2^28 items). Without a
 *   plan every (128-row query tile, sequence) pair up to max_seqlen_q is
 *   launched, longest key ranges first, and the tiles past a sequence's end
 *   exit at once; with a plan exactly the plan's items are launched, in its
 *   order. Items past a sequence's end are skipped, items naming a sequence
 *   >= num_seqs are skipped and set PKV_DEVERR_BAD_SEQLEN (a stale plan gives
 *   missing rows, never an out-of-bounds access); results are identical with
 *   and without a plan.
 */
int pkv_prefill_varlen(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                       int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                       int32_t num_blocks,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t max_seqlen_q,
                       int32_t max_seqlen_k, const int32_t* block_tables, int32_t block_table_stride,
                       int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                       int32_t block_size, float softmax_scale, void* out, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/*
 * pkv_prefill_varlen_f16 -- pkv_prefill_varlen with IEEE fp16 q, k, v,
 * caches and output (fp32 logits and accumulation; P is rounded to fp16
 * for the probability-times-value product). Arguments, layouts and errors
 * as for pkv_prefill_varlen.
 */
int pkv_prefill_varlen_f16(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                           int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                           int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                           int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                           int32_t block_table_stride, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                           int32_t head_dim, int32_t block_size, float softmax_scale, void* out, void* workspace,
                           size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes pkv_prefill_varlen(_f16) needs for these sizes (0: none;
 * an optional tile plan may be passed in its place). */
size_t pkv_prefill_workspace_bytes(int32_t num_seqs, int32_t max_seqlen_q, int32_t num_heads);

/*
 * pkv_prefill_plan -- host-side tile plan for pkv_prefill_varlen(_f16), built
 * once per engine step from the host copies of the step's cu_seqlens (the
 * pages' prepare_prefill builds them on the host) and reused by every layer.
 *
 * Writes one int32 per (128-row query tile qt, sequence b) pair that holds
 * query rows, encoded (qt << 16) | b, ordered by the number of 128-key tiles
 * the query tile attends to, most first (ties: lower b, then higher qt), so the
 * longest tiles start first. h_cu_seqlens_q / h_cu_seqlens_k: [num_seqs+1]
 * host arrays. h_items: host output with room for `capacity` items; the
 * number needed is sum over b of ceil(Lq_b / 128) <= total_q/128 + num_seqs.
 * Returns the number of items (>= 0), or PKV_ERR_NULL_POINTER, or
 * PKV_ERR_BAD_SIZE (num_seqs outside [0, 65535], lengths not monotone or
 * Lk_b < Lq_b, a sequence of 2^22 or more query rows, or capacity too small).
 */
int32_t pkv_prefill_plan(const int32_t* h_cu_seqlens_q, const int32_t* h_cu_seqlens_k, int32_t num_seqs,
                         int32_t* h_items, int32_t capacity);

/*
 * pkv_decode -- single-query GQA decode attention over the paged cache, the
 * flash_attn_with_kvcache(q.unsqueeze(1), k_cache, v_cache,
 * cache_seqlens=context_lens, block_table=block_tables, causal=True) call of
 * layers/attention.py.
 *
 * For sequence b and query head h, with ctx = context_lens[b] (the length
 * including the token just stored, engine/model_runner.py prepare_decode):
 *   out[b, h, :] = softmax(softmax_scale * q[b, h, :] . K_b[0..ctx-1]^T) V_b[0..ctx-1]
 * where key t of sequence b is slot block_tables[b*block_table_stride + t/256]*256
 * + t%256 of the kv head h/2. Rows with ctx == 0 (graph padding) get zeros.
 * Entries of block_tables past ceil(ctx/256) are never read (they may be -1
 * or stale).
 *
 *   q       [num_seqs, 16, 128] bf16, rows q_row_stride elements apart (>= 2048).
 *   out     [num_seqs, 16, 128] bf16 contiguous.
 *   max_context_len  upper bound on every context_lens[b] (e.g. max_model_len
 *           when the call is captured in a graph and replayed with new lengths);
 *           sizes the split-KV grid. Longer contexts set PKV_DEVERR_BAD_SEQLEN
 *           and give zeros.
 *   workspace  >= pkv_decode_workspace_bytes(num_seqs, num_heads, max_context_len)
 *           bytes of device memory, ZERO-FILLED ONCE before its first use; every
 *           call leaves it ready for the next. Calls that share a workspace
 *           must not overlap in time (same stream, or ordered).
 */
int pkv_decode(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
               int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
               const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
               int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
               void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * pkv_store_decode -- store_kvcache fused into the decode step
 * (layers/attention.py runs store_kvcache, then flash_attn_with_kvcache, on
 * the same slot_mapping; "vLLM 学习笔记 02：nano-vllm 源码逐段精读").
 *
 * Same result as pkv_store_kvcache(k, k_row_stride, v, v_row_stride, k_cache,
 * v_cache, slot_mapping, num_seqs, ...) followed by pkv_decode(...), in one
 * launch: the CTA that streams sequence b's last block first writes the new
 * K/V row there. It requires what engine/model_runner.py prepare_decode
 * produces: slot_mapping[b] is -1 (padding, nothing stored) or the slot of
 * position context_lens[b]-1 of sequence b. Any other slot is not stored and
 * sets PKV_DEVERR_BAD_SLOT.
 *   k, v  [num_seqs, 8, 128] bf16, rows k_row_stride / v_row_stride elements
 *         apart, 16-byte aligned, strides multiples of 8 elements.
 * Every other argument is as for pkv_decode.
 */
int pkv_store_decode(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                     int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                     int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                     const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                     int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                     void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * pkv_decode_f16 / pkv_store_decode_f16 -- pkv_decode and pkv_store_decode
 * with IEEE fp16 q, k, v, caches and output (fp32 arithmetic). Arguments,
 * layouts, workspace and errors as for the bf16 calls; a workspace may be
 * shared between bf16 and fp16 calls under the same ordering rule.
 */
int pkv_decode_f16(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                   int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                   const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                   int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                   void* workspace, size_t workspace_bytes, cudaStream_t stream);
int pkv_store_decode_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                         int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                         int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                         const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                         void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes pkv_decode, pkv_store_decode and their _f16 forms need for these sizes. */
size_t pkv_decode_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t max_context_len);

/*
 * pkv_decode_noalloc -- pkv_decode for callers that cannot allocate device
 * memory. The pages have no counterpart to this entry point: it exists for
 * users of this library, not for the method.
 *
 * Who needs it: an engine that sized its KV-cache pool to take all device
 * memory left after start-up, a plug-in whose host process owns the only
 * device allocator, or a latency-critical loop that must not call cudaMalloc
 * because it can synchronise the device. None of them can hand pkv_decode a
 * workspace.
 *
 * Same arguments and result as pkv_decode (bf16 only; there is no fp16 form),
 * without the workspace: the split-KV scratch lives in a fixed array of
 * PKV_DECODE_NOALLOC_SCRATCH_BYTES that is part of the library's device
 * image, reserved on every GPU that loads the library and held until the
 * process exits. The call allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library routine).
 *   - Limit: sizes with pkv_decode_workspace_bytes(num_seqs, num_heads,
 *     max_context_len) > PKV_DECODE_NOALLOC_SCRATCH_BYTES are rejected with
 *     PKV_ERR_SCRATCH_LIMIT before anything is launched (e.g. 256 sequences
 *     with max_context_len 4096 fit; 512 sequences fit up to 2048). Every
 *     other argument error pkv_decode reports is reported too, also before
 *     anything is queued on the stream.
 *   - The call passes the kernel the array's device address, which it asks
 *     the runtime for (cudaGetSymbolAddress) with the calling thread's device
 *     current, and caches per device and context. The first call on each
 *     device makes that lookup: make it before any stream capture.
 *   - Every call shares the one array and leaves its contents behind; each
 *     call first clears (cudaMemsetAsync on `stream`) the part that must start
 *     at zero. Calls whose execution overlaps on the GPU (different streams
 *     without ordering, or several host threads) race on the array and give
 *     wrong results: order them.
 */
#define PKV_DECODE_NOALLOC_SCRATCH_BYTES (64u * 1024u * 1024u)
int pkv_decode_noalloc(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                       int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                       const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                       void* out, cudaStream_t stream);

/*
 * ---- The 4-bit paged cache ----
 *
 * The pages keep K and V in the cache as 16-bit rows. These entry points have
 * no counterpart there: they hold the same paged cache in 4 bits per element
 * plus a scale and a minimum per 32 elements (5 bits in all), 3.2 times the
 * tokens in the same memory, with the same slots, block tables and lengths.
 *
 * Format. A row (one token, one kv head, 128 dims, of K or of V) is 4 groups
 * of 32 dims. A group keeps, in fp16, s = (max - min) / 15 and z = min; a dim
 * keeps the code c = (x - z) / s rounded half to even and clamped to 0..15 (0
 * where s is 0), and stands for s * c + z. |x| > 65504 counts as 65504. A
 * group that holds a NaN or an infinity has s = z = NaN: it reads back as NaN
 * and takes part in attention as NaN.
 *
 * Layout. k_cache and v_cache are uint8 [num_blocks, num_kv_heads, 16, 1280],
 * contiguous and 16-byte aligned: a 256-token block of a head is 16 tiles of
 * 16 tokens, a tile is 16 x 64 bytes of codes, then 16 x 4 x (s, z) fp16.
 *   K code row: the 32-bit word at byte 16 t + 4 j holds dims 32 j + 8 t + p in
 *     bits 4p..4p+3 (p = 0..7; j, t = 0..3).
 *   V code row: the 8-byte chunk r (0..7) lies at chunk place
 *     r ^ (token & 4); its 16-bit field j holds dims 32 j + 4 r + p in bits
 *     4p..4p+3 (p = 0..3).
 * Slot s is token s % 256 of block s / 256, as in the 16-bit cache. A cache
 * needs no initialisation: only stored tokens are read (bytes of others may be
 * fetched, but never reach a result).
 *
 * Supported: head_dim 128, block_size 256, any num_kv_heads; for attention one
 * or an even number of query heads to a kv head (prefill: an even number), up
 * to 8192 heads. The rows
 * (q, k, v, out) are bf16, or fp16 for the *_f16 names; the cache is the same
 * for both. Sizes of 0 are no-ops.
 */

/*
 * pkv_store_kvcache_q4 -- pkv_store_kvcache into the 4-bit cache: rows
 * k[i], v[i] are quantised into slot slot_mapping[i] (-1: skipped).
 *   k, v  [num_tokens, num_kv_heads, 128], heads and dims contiguous, rows
 *         k_row_stride / v_row_stride elements apart; any 2-byte alignment
 *         (16-byte vectors where pointers and strides allow it).
 * A row's bytes belong to that row alone, so tokens of one call may share a
 * block or a tile. Duplicate slots in one call race. Slots outside the pool set
 * PKV_DEVERR_BAD_SLOT and are skipped.
 */
int pkv_store_kvcache_q4(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, void* k_cache,
                         void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int32_t num_blocks, cudaStream_t stream);
int pkv_store_kvcache_q4_f16(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, void* k_cache,
                             void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int32_t block_size, int32_t num_blocks, cudaStream_t stream);

/*
 * pkv_load_kvcache_q4 -- reads slots back: k[i], v[i] = the values that slot
 * slot_mapping[i] stands for, rounded to the element type (fp16: saturated at
 * 65504). Rows whose slot is -1, or outside the pool (PKV_DEVERR_BAD_SLOT),
 * are left as they were. Slots may repeat (a shared prefix).
 *   k, v  [num_tokens, num_kv_heads, 128] contiguous, 16-byte aligned.
 */
int pkv_load_kvcache_q4(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, void* k,
                        void* v, cudaStream_t stream);
int pkv_load_kvcache_q4_f16(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, void* k,
                            void* v, cudaStream_t stream);

/*
 * pkv_decode_q4 -- pkv_decode over the 4-bit cache: attention of one query row
 * per sequence over the values that its cached tokens stand for (the codes are
 * used exactly; p times a row's scale is rounded to fp16 for the product with
 * V's codes, sums and maxima are fp32). Arguments and errors as for pkv_decode
 * but for the caches, the head counts and the workspace:
 *   workspace  >= pkv_decode_q4_workspace_bytes(num_seqs, num_heads,
 *         num_kv_heads, max_context_len) bytes, ZERO-FILLED ONCE before its
 *         first use and used for these calls only, always with the same
 *         workspace_bytes; every call leaves it ready for the next one, of any
 *         sizes and head counts that it is large enough for. Calls that share
 *         it (two captured graphs, say) must not overlap in time. The exception
 *         is a call that sets PKV_DEVERR_TIMEOUT: it leaves the workspace marked,
 *         and later calls on it write nothing and set PKV_DEVERR_TIMEOUT again
 *         until it has been zero-filled once more.
 * How a sequence is split over the GPU follows from the call's context lengths
 * alone, and the partial results are joined in chunk order, so equal calls give
 * equal bits.
 */
int pkv_decode_q4(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache, int32_t num_blocks,
                  const int32_t* block_tables, int32_t block_table_stride, const int32_t* context_lens,
                  int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  int32_t max_context_len, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream);
int pkv_decode_q4_f16(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                      int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                      const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * pkv_store_decode_q4 -- pkv_store_kvcache_q4 of the step's new rows, then
 * pkv_decode_q4, in one launch, with the same results. As for
 * pkv_store_decode, slot_mapping[b] is -1 (nothing stored) or the slot of
 * position context_lens[b] - 1; any other slot is not stored and sets
 * PKV_DEVERR_BAD_SLOT. k, v 16-byte aligned, row strides multiples of 8.
 */
int pkv_store_decode_q4(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                        int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                        int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                        const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream);
int pkv_store_decode_q4_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                            int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                            int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                            const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                            void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * pkv_prefill_varlen_q4 -- pkv_prefill_varlen in prefix-cache mode with every
 * key and value (cached prefix and new tokens, which the caller stores first
 * on the same stream) taken from the 4-bit cache. Keys are rounded to the
 * element type as pkv_load_kvcache_q4 rounds them, values and p to fp16 (more
 * exact than bf16, whichever the element type is); sums and maxima are fp32. The
 * result is, up to those roundings, that of loading the rows and attending to
 * them contiguously, without the load. A call of few query tiles splits their
 * keys over up to 8 CTAs, whose fp32 partial results are added in key order; how
 * follows from the call's sizes alone (the bounds of the lengths, the block
 * table's width and the number of a plan's items among them), so equal calls give
 * equal bits, and calls with and without a plan may differ by the order of those
 * sums. A group of V that
 * reads back as NaN gives NaN in its 32 dims to the rows that may attend to it,
 * and to no others.
 * Arguments, errors and the optional tile plan in `workspace` are as for
 * pkv_prefill_varlen. A plan spares the places past a sequence's end, which
 * counts where the lengths differ widely (one prompt of 4096 beside 20 of 10: 112
 * us without, 77 with it). Long prompts of like lengths are better off without:
 * two CTAs then share the widening of their keys, which a plan's items do not
 * (5000 tokens after 7001: 321 us without, 356 with it). Rows of q and out that
 * belong to no sequence, or with a plan to none of its tiles, are left as they
 * were.
 */
int pkv_prefill_varlen_q4(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache,
                          const void* v_cache, int32_t num_blocks, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                          const int32_t* block_tables, int32_t block_table_stride, int32_t num_seqs,
                          int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          float softmax_scale, void* out, const void* workspace, size_t workspace_bytes,
                          cudaStream_t stream);
int pkv_prefill_varlen_q4_f16(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache,
                          const void* v_cache, int32_t num_blocks, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                          const int32_t* block_tables, int32_t block_table_stride, int32_t num_seqs,
                          int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          float softmax_scale, void* out, const void* workspace, size_t workspace_bytes,
                          cudaStream_t stream);

/* Workspace bytes pkv_decode_q4, pkv_store_decode_q4 and their _f16 forms need (0 for sizes they refuse). */
size_t pkv_decode_q4_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t max_context_len);

/*
 * ---- Rotary positions ----
 *
 * The pages rotate q and k by their positions before the attention block
 * (get_rope in layers/rotary_embedding.py, theta 1e6). These calls do that step,
 * alone or together with store_kvcache of the same rows.
 *
 * pkv_rope_frequencies -- host-side, once per model: the angle that each of the
 * rotary_dim/2 pairs of a head turns per position, f_i = theta^(-2i/rotary_dim)
 * radians and what a scaling makes of it for longer contexts:
 *   PKV_ROPE_NONE    f_i
 *   PKV_ROPE_LINEAR  f_i / factor
 *   PKV_ROPE_NTK     theta * factor^(r/(r-2)) in theta's place (r = rotary_dim; r = 2: as PKV_ROPE_NONE)
 *   PKV_ROPE_BANDS   g f_i + (1 - g) f_i / factor, with g = (turns over
 *                    original_max_position - a) / (b - a) clamped to 0..1
 *                    (a, b: the low and high frequency factors, 1 and 4 for instance)
 *   PKV_ROPE_YARN    (1 - g) f_i + g f_i / factor, g rising from 0 to 1 between the pairs that turn a and b times over
 *                    original_max_position (a = 32, b = 1 for instance; the pairs' numbers rounded down and up and
 *                    clamped to 0..r-1), and *h_magnitude = 0.1 ln(factor) + 1
 * h_freqs: [rotary_dim/2] int64 on the host, f_i in units of 2^-64 full turns per
 * position (rounded towards zero): position * f_i modulo 2^64 is the exact
 * fraction of a turn. *h_magnitude: what turned values are multiplied by (1 but for
 * PKV_ROPE_YARN). Arguments that a scaling does not use are ignored. Returns PKV_OK, PKV_ERR_NULL_POINTER,
 * PKV_ERR_UNSUPPORTED (rotary_dim odd, below 2 or above 1024; no such scaling) or
 * PKV_ERR_BAD_SIZE (theta <= 1, factor < 1, original_max_position < 1, a >= b (BANDS) or a <= b or b <= 0 (YARN), or
 * values that are not finite).
 */
#define PKV_ROPE_NONE 0
#define PKV_ROPE_LINEAR 1
#define PKV_ROPE_NTK 2
#define PKV_ROPE_BANDS 3
#define PKV_ROPE_YARN 4
int pkv_rope_frequencies(int32_t rotary_dim, double theta, int32_t scaling, double factor,
                         double original_max_position, double a, double b, int64_t* h_freqs, float* h_magnitude);

/*
 * pkv_rope -- turns the first rotary_dim elements of every head of q and k by the
 * row's position; the others are copied. Pair i is elements i and i + rotary_dim/2,
 * or, interleaved, 2i and 2i + 1:
 *   a' = (a cos - b sin) * magnitude,  b' = (b cos + a sin) * magnitude
 * in fp32, rounded once.
 *   q, k          [num_tokens, num_heads | num_kv_heads, head_dim], heads and dims
 *                 contiguous, rows *_row_stride elements apart (views of a fused qkv
 *                 are fine). One of the two head counts may be 0.
 *   positions     [num_tokens] int64, any values (negative ones turn backwards).
 *   freqs         [rotary_dim/2] int64 on the device (pkv_rope_frequencies).
 *   q_out, k_out  as q and k; may be the same rows (in place), else must not overlap them.
 * head_dim up to 1024, rotary_dim even and at most head_dim. 16-byte vectors where
 * pointers are 16-byte aligned and strides and head_dim multiples of 8 (fastest with
 * head_dim and rotary_dim multiples of 16); any 2-byte alignment otherwise.
 */
int pkv_rope(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const int64_t* positions,
             const int64_t* freqs, int32_t rotary_dim, float magnitude, int32_t interleaved, int32_t num_tokens,
             int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_row_stride,
             void* k_out, int64_t k_out_row_stride, cudaStream_t stream);
int pkv_rope_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const int64_t* positions,
                 const int64_t* freqs, int32_t rotary_dim, float magnitude, int32_t interleaved, int32_t num_tokens,
                 int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, void* q_out, int64_t q_out_row_stride,
                 void* k_out, int64_t k_out_row_stride, cudaStream_t stream);

/*
 * pkv_rope_store_kvcache -- pkv_rope of q and k, then pkv_store_kvcache of the
 * turned k and of v, in one launch and with the same results: k is turned on its
 * way to its slot and not written anywhere else. Slots, caches and their errors
 * are as for pkv_store_kvcache (a row with slot -1 only has its q turned).
 *   v  [num_tokens, num_kv_heads, head_dim], rows v_row_stride elements apart.
 */
int pkv_rope_store_kvcache(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                           int64_t v_row_stride, const int64_t* positions, const int64_t* freqs, int32_t rotary_dim,
                           float magnitude, int32_t interleaved, const int32_t* slot_mapping, int32_t num_tokens,
                           int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int64_t num_slots, void* q_out,
                           int64_t q_out_row_stride, void* k_cache, void* v_cache, cudaStream_t stream);
int pkv_rope_store_kvcache_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                               int64_t v_row_stride, const int64_t* positions, const int64_t* freqs,
                               int32_t rotary_dim, float magnitude, int32_t interleaved, const int32_t* slot_mapping,
                               int32_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                               int64_t num_slots, void* q_out, int64_t q_out_row_stride, void* k_cache, void* v_cache,
                               cudaStream_t stream);

/*
 * ---- Attention with modified scores and masks ----
 *
 * The attention calls above take softmax(scale * q.k) over all keys up to the
 * query's position. These take other scores and other sets of visible keys, for
 * models that need them, over the same cache, for any head counts (num_heads a
 * multiple of num_kv_heads, at most 8192). For a query at position p and a key at
 * position t, in this order:
 *   x = softmax_scale * q . k
 *   x = softcap * tanh(x / softcap)          where softcap > 0 (0: no cap)
 *   x = x - slopes[head] * |p - t|           where slopes != NULL ([num_heads] fp32, any finite values)
 * and the key takes part where all of these hold:
 *   t <= p, or t < prefix_lens[sequence]     (prefill, where prefix_lens != NULL: keys that every row sees)
 *   t < length of the sequence
 *   t >= key_starts[row]                     where key_starts != NULL (the first position of the row's document, say)
 *   p - t < window                           where window > 0
 * A key's position t is its place in the sequence: the place in its blocks, over the cache. After pkv_evict_kvcache,
 * which moves tokens up, each head for itself, that is no longer the token's position in the text: window, slopes,
 * key_starts and prefix_lens then count places in the cache, and a model that means positions cannot use them there. Scale
 * and cap take no positions, and rotary ones stay in the rows.
 *
 * A row that sees no key gets zeros. Values at keys that take no part, infinities and NaN among them, reach no result
 * (but for the choice between two forms of tanh in the prefill, see there); in V of keys that take part they come out as
 * the sums have them. Products take the 16-bit rows as they are and add up in fp32; scores, maxima and sums are fp32. For
 * the product with V shares are rounded to the rows' 16 bits, in the decode with what that lost as a second 16-bit number;
 * of fp16 rows shares below 2^-32 of the row's largest are lost.
 */

/*
 * pkv_decode_mod -- pkv_decode with the scores and masks above: one query row per
 * sequence, at position context_lens[b] - 1. Arguments and errors as for pkv_decode but for
 *   num_blocks  at most 2^23 - 1 (and not 0)
 *   key_starts  [num_seqs] int32, or NULL
 *   weights     NULL, or fp32 [num_blocks, num_kv_heads, 256], 16-byte aligned: each token's attention added up over the
 *         calls, beside the cache. For every key that takes part, weights[slot / 256][kv head][slot % 256] += the sum over the kv
 *         head's query heads of its softmax probability; the newest token's (position context_lens[b] - 1) starts
 *         from 0 in this call, whatever was there. What a prompt's tokens start from is the caller's to fill in.
 *         Sequences of one call must not share blocks then (their additions would race).
 *   workspace  >= pkv_decode_mod_workspace_bytes(...) bytes, 16-byte aligned. It holds nothing between calls and needs
 *         no initialisation; calls that share it must not overlap in time.
 * How sequences are split over the GPU follows from the call's lengths alone, and partial results are joined in order,
 * so equal calls give equal bits.
 */
int pkv_decode_mod(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache, int32_t num_blocks,
                   const int32_t* block_tables, int32_t block_table_stride, const int32_t* context_lens,
                   int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   int32_t max_context_len, float softmax_scale, float softcap, const float* slopes, int32_t window,
                   const int32_t* key_starts, float* weights, void* out, void* workspace, size_t workspace_bytes,
                   cudaStream_t stream);
int pkv_decode_mod_f16(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                       int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                       const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                       float softcap, const float* slopes, int32_t window, const int32_t* key_starts, float* weights,
                       void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Workspace bytes pkv_decode_mod(_f16) needs for these sizes, with weights (1) or without (0); 0 for sizes it refuses. */
size_t pkv_decode_mod_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                      int32_t max_context_len, int32_t weights);

/*
 * pkv_prefill_varlen_mod -- pkv_prefill_varlen with the scores and masks above, for any head counts. Query row i of
 * sequence b sits at position Lk_b - Lq_b + i, as there; keys come from contiguous k/v (block_tables == NULL) or from
 * the paged cache. Arguments and errors as for pkv_prefill_varlen but for
 *   num_blocks   at most 2^23 - 1
 *   key_starts   [total_q] int32, one per query row, or NULL: with documents packed into a sequence, the position at
 *                which the row's document starts
 *   prefix_lens  [num_seqs] int32, or NULL: keys at positions below are seen by every row, also by rows before them
 * There is no tile plan. Rows of q and out that belong to no sequence are left as they were. A NaN or an infinity in V
 * reaches the rows that its key takes part in, and no others; rows of a tile beside it that do not see it are computed
 * one by one, at some 0.1 us for each key that they see.
 * tanh is a polynomial off by at most 7e-6 of a score for bf16 rows and 6e-7 for fp16, or, where a tile holds scores
 * beyond the cap, taken from the exponential: keys of the tile that take no part have a say in that, so they may change a
 * result by as much.
 */
int pkv_prefill_varlen_mod(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                           int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                           int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                           int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                           int32_t block_table_stride, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                           int32_t head_dim, int32_t block_size, float softmax_scale, float softcap,
                           const float* slopes, int32_t window, const int32_t* key_starts, const int32_t* prefix_lens,
                           void* out, cudaStream_t stream);
int pkv_prefill_varlen_mod_f16(const void* q, int64_t q_row_stride, int32_t total_q, const void* k, const void* v,
                               int64_t kv_row_stride, int32_t total_k, const void* k_cache, const void* v_cache,
                               int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k,
                               int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                               int32_t block_table_stride, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                               int32_t head_dim, int32_t block_size, float softmax_scale, float softcap,
                               const float* slopes, int32_t window, const int32_t* key_starts,
                               const int32_t* prefix_lens, void* out, cudaStream_t stream);

/*
 * pkv_evict_kvcache -- cuts every sequence of more than `budget` tokens down to
 * `budget`: of each kv head the tokens at the first `first` positions, the newest
 * `recent` ones, and of the others those with the largest weights (as pkv_decode_mod
 * adds them up beside the cache), equal weights in order of position. The pages keep
 * every token of a sequence; this call has no counterpart there. Kept tokens keep
 * their order and move up: token kept[b][h][j] of head h becomes token j, its K and V
 * rows and its weight with it. Each head chooses for itself, so a slot may then hold
 * different tokens of different heads, and what counts positions in the attention calls above counts places from then
 * on. Shorter sequences keep all their tokens.
 *   k_cache, v_cache  [num_blocks, 256, num_kv_heads, 128], 16-bit elements of either type, 16-byte aligned
 *   weights           fp32 [num_blocks, num_kv_heads, 256]; a NaN counts as larger than any number
 *   max_context_len   upper bound on context_lens[b] (<= 2^24)
 *   new_block_tables  [num_seqs, new_block_table_stride] int32: the blocks that the kept tokens are copied to (of
 *                     shorter sequences all tokens), none of them in a block_tables row of the call; the old blocks
 *                     are only read, so sequences may share them. Its rows have room for min(budget, max_context_len)
 *                     tokens. NULL: in place, within the sequence's own blocks, which no other sequence may share then.
 *                     Blocks behind the new length are free afterwards.
 *   kept              int32 [num_seqs, num_kv_heads, budget] out: old positions in rising order, -1 behind the last
 *   new_context_lens  int32 [num_seqs] out, min(context_lens[b], budget); must not overlap context_lens (PKV_ERR_BAD_SIZE)
 * 1 <= budget <= 2^24, first + recent <= budget. Slots behind the new length are left as they were. Bad lengths
 * (taken as 0) and blocks (their tokens are not moved) set PKV_DEVERR_BAD_SEQLEN and PKV_DEVERR_BAD_BLOCK.
 */
int pkv_evict_kvcache(void* k_cache, void* v_cache, float* weights, int32_t num_blocks, const int32_t* block_tables,
                      int32_t block_table_stride, const int32_t* context_lens, int32_t num_seqs, int32_t num_kv_heads,
                      int32_t head_dim, int32_t block_size, int32_t max_context_len, int32_t budget, int32_t first,
                      int32_t recent, const int32_t* new_block_tables, int32_t new_block_table_stride, int32_t* kept,
                      int32_t* new_context_lens, cudaStream_t stream);

/*
 * pkv_build_prefill_metadata / pkv_build_decode_metadata -- the per-step index
 * preparation of engine/model_runner.py (prepare_prefill, prepare_decode in
 * "vLLM 学习笔记 02：nano-vllm 源码逐段精读"; worked example in
 * "Nano-vLLM代码手撕笔记", section "请求执行 – 输入序列预处理与context构建"),
 * computed on the GPU from what the scheduler has per sequence, so no
 * per-token host loop and no per-token host-to-device copy is needed.
 * Bit-identical to the host definition. A token whose block-table entry is
 * outside [0, num_blocks) gets slot -1 and sets PKV_DEVERR_BAD_BLOCK.
 *
 * Prefill: sequence b computes positions [num_cached_tokens[b],
 * num_cached_tokens[b] + num_scheduled_tokens[b]).
 *   cu_seqlens_q[num_seqs+1]  prefix sums of num_scheduled_tokens
 *   cu_seqlens_k[num_seqs+1]  prefix sums of num_cached + num_scheduled
 *   max_seqlens[2]            {max_seqlen_q, max_seqlen_k} (device; the
 *                             attention calls accept any upper bounds instead)
 *   slot_mapping[capacity], positions[capacity] (int64)  one entry per new
 *                             token, sequence by sequence; tokens beyond
 *                             `capacity` are not written (PKV_DEVERR_BAD_SEQLEN).
 * Decode: num_tokens[b] = len(seq) including the token being stored;
 *   slot_mapping[b] = slot of position len-1, context_lens[b] = len,
 *   positions[b] = len-1; rows with len 0 are padding (slot -1, context 0).
 * All arrays are int32 device arrays except positions (int64, as the pages'
 * torch.int64 positions). block_tables is [num_seqs, block_table_stride], -1 padded.
 */
int pkv_build_prefill_metadata(const int32_t* num_cached_tokens, const int32_t* num_scheduled_tokens,
                               const int32_t* block_tables, int32_t block_table_stride, int32_t num_blocks,
                               int32_t num_seqs, int32_t capacity, int32_t* cu_seqlens_q, int32_t* cu_seqlens_k,
                               int32_t* max_seqlens, int32_t* slot_mapping, int64_t* positions, cudaStream_t stream);
int pkv_build_decode_metadata(const int32_t* num_tokens, const int32_t* block_tables, int32_t block_table_stride,
                              int32_t num_blocks, int32_t num_seqs, int32_t* slot_mapping, int32_t* context_lens,
                              int64_t* positions, cudaStream_t stream);

/*
 * pkv_device_error -- read (and optionally clear) the current device's
 * error word (PKV_DEVERR_* bits OR-ed by every kernel of this library since
 * the last clear). Synchronises `stream`, so do not call it inside a graph
 * capture. bits may be NULL when only clearing.
 */
int pkv_device_error(uint32_t* bits, int clear, cudaStream_t stream);

/*
 * pkv_selftest_wait_timeout -- failure-detection self test: launches one
 * block that waits on a barrier nothing will ever complete, with the given
 * bound in nanoseconds (clamped to [1000, 100000000]). The wait must give
 * up, set PKV_DEVERR_TIMEOUT and return; the GPU stays usable.
 */
int pkv_selftest_wait_timeout(uint64_t limit_ns, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H_ */
