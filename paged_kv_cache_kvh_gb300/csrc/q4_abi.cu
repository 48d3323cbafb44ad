// q4_abi.cu -- extern "C" entry points of the 4-bit paged cache (declared in include/pkv.h).
//
// Arguments are checked on the host before anything is launched, like those of
// the 16-bit entry points. These kernels take any number of kv heads, with one or
// an even number of query heads to each.
#include "pkv_common.cuh"

namespace pkv {
struct FusedStore {
  const void* k;
  int64_t k_row_stride;
  const void* v;
  int64_t v_row_stride;
  const int32_t* slot_mapping;
};
cudaError_t launch_store_q4(const void* k, int64_t k_stride, const void* v, int64_t v_stride, void* k_cache,
                            void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t hkv,
                            int64_t num_slots, unsigned int* err, cudaStream_t stream, Elem elem);
cudaError_t launch_load_q4(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                           int32_t hkv, int64_t num_slots, void* k, void* v, unsigned int* err, cudaStream_t stream,
                           Elem elem);
size_t decode_q4_workspace_bytes(int32_t num_seqs, int32_t hkv, int32_t group, int32_t max_ctx);
cudaError_t launch_decode_q4(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                             int32_t num_blocks, const int32_t* block_tables, int32_t bt_stride,
                             const int32_t* context_lens, int32_t num_seqs, int32_t hkv, int32_t group,
                             int32_t max_ctx, float scale, void* out, void* workspace, size_t workspace_bytes,
                             unsigned int* err, cudaStream_t stream, const FusedStore* fused, Elem elem);
cudaError_t launch_prefill_q4(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache,
                              const void* v_cache, int32_t num_blocks, const int32_t* cu_q, const int32_t* cu_k,
                              int32_t max_seqlen_q, int32_t max_seqlen_k, const int32_t* block_tables,
                              int32_t bt_stride, int32_t num_seqs, int32_t hq, int32_t hkv, float scale,
                              const int32_t* items, int32_t num_items, void* out, unsigned int* err,
                              cudaStream_t stream, Elem elem);
}  // namespace pkv

namespace {

constexpr int32_t kMaxHeads = 8192;  // as pkv_store_kvcache: rows of at most 2^20 elements

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int launched(cudaError_t e) {
  if (e == cudaSuccess) return PKV_OK;
  (void)cudaGetLastError();
  return PKV_ERR_CUDA;
}

int check_cache_shape(int32_t num_kv_heads, int32_t head_dim, int32_t block_size) {
  if (head_dim != pkv::kHeadDim || block_size != pkv::kBlockSize || num_kv_heads <= 0 || num_kv_heads > kMaxHeads)
    return PKV_ERR_UNSUPPORTED;
  return PKV_OK;
}

// Query heads come one to a kv head, or in pairs that share one.
int check_heads(int32_t num_heads, int32_t num_kv_heads) {
  if (num_kv_heads <= 0 || num_heads <= 0 || num_heads > kMaxHeads || num_heads % num_kv_heads != 0)
    return PKV_ERR_UNSUPPORTED;
  const int32_t g = num_heads / num_kv_heads;
  return g == 1 || g % 2 == 0 ? PKV_OK : PKV_ERR_UNSUPPORTED;
}

int store_common(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, void* k_cache,
                 void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                 int32_t head_dim, int32_t block_size, int32_t num_blocks, cudaStream_t stream, pkv::Elem elem) {
  int st = check_cache_shape(num_kv_heads, head_dim, block_size);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_blocks < 0) return PKV_ERR_BAD_SIZE;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PKV_ERR_NULL_POINTER;
  const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
  if (k_row_stride < row || v_row_stride < row) return PKV_ERR_BAD_STRIDE;
  if (!aligned(k, 2) || !aligned(v, 2) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return PKV_ERR_ALIGNMENT;
  unsigned int* err = nullptr;
  st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  return launched(pkv::launch_store_q4(k, k_row_stride, v, v_row_stride, k_cache, v_cache, slot_mapping, num_tokens,
                                       num_kv_heads, static_cast<int64_t>(num_blocks) * block_size, err, stream, elem));
}

int load_common(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, void* k, void* v,
                cudaStream_t stream, pkv::Elem elem) {
  int st = check_cache_shape(num_kv_heads, head_dim, block_size);
  if (st != PKV_OK) return st;
  if (num_tokens < 0 || num_blocks < 0) return PKV_ERR_BAD_SIZE;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !k_cache || !v_cache || !slot_mapping) return PKV_ERR_NULL_POINTER;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16)) return PKV_ERR_ALIGNMENT;
  unsigned int* err = nullptr;
  st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  return launched(pkv::launch_load_q4(k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads,
                                      static_cast<int64_t>(num_blocks) * block_size, k, v, err, stream, elem));
}

int decode_common(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache, int32_t num_blocks,
                  const int32_t* block_tables, int32_t block_table_stride, const int32_t* context_lens,
                  int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  int32_t max_context_len, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream, const pkv::FusedStore* fused, pkv::Elem elem) {
  int st = check_cache_shape(num_kv_heads, head_dim, block_size);
  if (st == PKV_OK) st = check_heads(num_heads, num_kv_heads);
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || num_blocks < 0 || block_table_stride < 0 || max_context_len < 0 ||
      max_context_len > (1 << 24))
    return PKV_ERR_BAD_SIZE;
  if (num_seqs == 0) return PKV_OK;
  if (!(softmax_scale > 0.f)) return PKV_ERR_BAD_SIZE;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out) return PKV_ERR_NULL_POINTER;
  if (q_row_stride < static_cast<int64_t>(num_heads) * head_dim) return PKV_ERR_BAD_STRIDE;
  if (!aligned(q, 16) || q_row_stride % 8 != 0 || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(out, 16))
    return PKV_ERR_ALIGNMENT;
  const int32_t group = num_heads / num_kv_heads;
  if (!workspace || workspace_bytes < pkv::decode_q4_workspace_bytes(num_seqs, num_kv_heads, group, max_context_len))
    return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return PKV_ERR_ALIGNMENT;
  unsigned int* err = nullptr;
  st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  return launched(pkv::launch_decode_q4(q, q_row_stride, k_cache, v_cache, num_blocks, block_tables,
                                        block_table_stride, context_lens, num_seqs, num_kv_heads, group,
                                        max_context_len, softmax_scale, out, workspace, workspace_bytes, err, stream, fused,
                                        elem));
}

int store_decode_common(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                        int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                        int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                        const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream, pkv::Elem elem) {
  if (num_seqs > 0) {
    if (!k || !v || !slot_mapping) return PKV_ERR_NULL_POINTER;
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (k_row_stride < row || v_row_stride < row) return PKV_ERR_BAD_STRIDE;
    if (!aligned(k, 16) || !aligned(v, 16) || k_row_stride % 8 != 0 || v_row_stride % 8 != 0) return PKV_ERR_ALIGNMENT;
  }
  const pkv::FusedStore fused{k, k_row_stride, v, v_row_stride, slot_mapping};
  return decode_common(q, q_row_stride, k_cache, v_cache, num_blocks, block_tables, block_table_stride, context_lens,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, softmax_scale, out,
                       workspace, workspace_bytes, stream, &fused, elem);
}

int prefill_common(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache, const void* v_cache,
                   int32_t num_blocks, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int32_t max_seqlen_q,
                   int32_t max_seqlen_k, const int32_t* block_tables, int32_t block_table_stride, int32_t num_seqs,
                   int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                   float softmax_scale, void* out, const void* workspace, size_t workspace_bytes,
                   cudaStream_t stream, pkv::Elem elem) {
  int st = check_cache_shape(num_kv_heads, head_dim, block_size);
  if (st == PKV_OK) st = check_heads(num_heads, num_kv_heads);
  if (st == PKV_OK && num_heads == num_kv_heads) st = PKV_ERR_UNSUPPORTED;  // a CTA takes two heads of one kv head
  if (st != PKV_OK) return st;
  if (num_seqs < 0 || num_seqs > 65535 || total_q < 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || num_blocks < 0 ||
      block_table_stride < 0)
    return PKV_ERR_BAD_SIZE;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return PKV_OK;
  if (!(softmax_scale > 0.f)) return PKV_ERR_BAD_SIZE;
  if (!q || !out || !cu_seqlens_q || !cu_seqlens_k || !k_cache || !v_cache || !block_tables)
    return PKV_ERR_NULL_POINTER;
  if (num_blocks == 0 || block_table_stride == 0) return PKV_ERR_BAD_SIZE;
  if (q_row_stride < static_cast<int64_t>(num_heads) * head_dim) return PKV_ERR_BAD_STRIDE;
  if (!aligned(q, 16) || q_row_stride % 8 != 0 || !aligned(out, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return PKV_ERR_ALIGNMENT;
  const int32_t* items = nullptr;
  int32_t num_items = 0;
  if (workspace && workspace_bytes > 0) {  // a tile plan (pkv_prefill_plan)
    if (workspace_bytes % 4 != 0 || workspace_bytes / 4 > (size_t{1} << 28)) return PKV_ERR_BAD_SIZE;
    if (!aligned(workspace, 4)) return PKV_ERR_ALIGNMENT;
    items = static_cast<const int32_t*>(workspace);
    num_items = static_cast<int32_t>(workspace_bytes / 4);
  }
  unsigned int* err = nullptr;
  st = pkv::device_error_word(&err);
  if (st != PKV_OK) return st;
  return launched(pkv::launch_prefill_q4(q, q_row_stride, total_q, k_cache, v_cache, num_blocks, cu_seqlens_q,
                                         cu_seqlens_k, max_seqlen_q, max_seqlen_k, block_tables, block_table_stride,
                                         num_seqs, num_heads, num_kv_heads, softmax_scale, items, num_items, out, err,
                                         stream, elem));
}

}  // namespace

extern "C" {

// The bf16 and fp16 entry points share one body each; only the rows' element type differs.

int pkv_store_kvcache_q4(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, void* k_cache,
                         void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                         int32_t head_dim, int32_t block_size, int32_t num_blocks, cudaStream_t stream) {
  return store_common(k, k_row_stride, v, v_row_stride, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads,
                      head_dim, block_size, num_blocks, stream, pkv::Elem::kBF16);
}

int pkv_store_kvcache_q4_f16(const void* k, int64_t k_row_stride, const void* v, int64_t v_row_stride, void* k_cache,
                             void* v_cache, const int32_t* slot_mapping, int32_t num_tokens, int32_t num_kv_heads,
                             int32_t head_dim, int32_t block_size, int32_t num_blocks, cudaStream_t stream) {
  return store_common(k, k_row_stride, v, v_row_stride, k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads,
                      head_dim, block_size, num_blocks, stream, pkv::Elem::kF16);
}

int pkv_load_kvcache_q4(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                        int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, void* k,
                        void* v, cudaStream_t stream) {
  return load_common(k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim, block_size, num_blocks, k, v,
                     stream, pkv::Elem::kBF16);
}

int pkv_load_kvcache_q4_f16(const void* k_cache, const void* v_cache, const int32_t* slot_mapping, int32_t num_tokens,
                            int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int32_t num_blocks, void* k,
                            void* v, cudaStream_t stream) {
  return load_common(k_cache, v_cache, slot_mapping, num_tokens, num_kv_heads, head_dim, block_size, num_blocks, k, v,
                     stream, pkv::Elem::kF16);
}

size_t pkv_decode_q4_workspace_bytes(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                     int32_t max_context_len) {
  if (num_seqs <= 0 || num_seqs > 65535 || max_context_len < 0 || max_context_len > (1 << 24) ||
      num_kv_heads > kMaxHeads || check_heads(num_heads, num_kv_heads) != PKV_OK)
    return 0;
  return pkv::decode_q4_workspace_bytes(num_seqs, num_kv_heads, num_heads / num_kv_heads, max_context_len);
}

int pkv_decode_q4(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache, int32_t num_blocks,
                  const int32_t* block_tables, int32_t block_table_stride, const int32_t* context_lens,
                  int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                  int32_t max_context_len, float softmax_scale, void* out, void* workspace, size_t workspace_bytes,
                  cudaStream_t stream) {
  return decode_common(q, q_row_stride, k_cache, v_cache, num_blocks, block_tables, block_table_stride, context_lens,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, softmax_scale, out,
                       workspace, workspace_bytes, stream, nullptr, pkv::Elem::kBF16);
}

int pkv_decode_q4_f16(const void* q, int64_t q_row_stride, const void* k_cache, const void* v_cache,
                      int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                      const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                      int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                      void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return decode_common(q, q_row_stride, k_cache, v_cache, num_blocks, block_tables, block_table_stride, context_lens,
                       num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, softmax_scale, out,
                       workspace, workspace_bytes, stream, nullptr, pkv::Elem::kF16);
}

int pkv_store_decode_q4(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                        int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                        int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                        const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                        int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale, void* out,
                        void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return store_decode_common(q, q_row_stride, k, k_row_stride, v, v_row_stride, slot_mapping, k_cache, v_cache,
                             num_blocks, block_tables, block_table_stride, context_lens, num_seqs, num_heads,
                             num_kv_heads, head_dim, block_size, max_context_len, softmax_scale, out, workspace,
                             workspace_bytes, stream, pkv::Elem::kBF16);
}

int pkv_store_decode_q4_f16(const void* q, int64_t q_row_stride, const void* k, int64_t k_row_stride, const void* v,
                            int64_t v_row_stride, const int32_t* slot_mapping, void* k_cache, void* v_cache,
                            int32_t num_blocks, const int32_t* block_tables, int32_t block_table_stride,
                            const int32_t* context_lens, int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                            int32_t head_dim, int32_t block_size, int32_t max_context_len, float softmax_scale,
                            void* out, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return store_decode_common(q, q_row_stride, k, k_row_stride, v, v_row_stride, slot_mapping, k_cache, v_cache,
                             num_blocks, block_tables, block_table_stride, context_lens, num_seqs, num_heads,
                             num_kv_heads, head_dim, block_size, max_context_len, softmax_scale, out, workspace,
                             workspace_bytes, stream, pkv::Elem::kF16);
}

int pkv_prefill_varlen_q4(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache,
                          const void* v_cache, int32_t num_blocks, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                          const int32_t* block_tables, int32_t block_table_stride, int32_t num_seqs,
                          int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          float softmax_scale, void* out, const void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  return prefill_common(q, q_row_stride, total_q, k_cache, v_cache, num_blocks, cu_seqlens_q, cu_seqlens_k,
                        max_seqlen_q, max_seqlen_k, block_tables, block_table_stride, num_seqs, num_heads,
                        num_kv_heads, head_dim, block_size, softmax_scale, out, workspace, workspace_bytes, stream,
                        pkv::Elem::kBF16);
}

int pkv_prefill_varlen_q4_f16(const void* q, int64_t q_row_stride, int32_t total_q, const void* k_cache,
                          const void* v_cache, int32_t num_blocks, const int32_t* cu_seqlens_q,
                          const int32_t* cu_seqlens_k, int32_t max_seqlen_q, int32_t max_seqlen_k,
                          const int32_t* block_tables, int32_t block_table_stride, int32_t num_seqs,
                          int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                          float softmax_scale, void* out, const void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
  return prefill_common(q, q_row_stride, total_q, k_cache, v_cache, num_blocks, cu_seqlens_q, cu_seqlens_k,
                        max_seqlen_q, max_seqlen_k, block_tables, block_table_stride, num_seqs, num_heads,
                        num_kv_heads, head_dim, block_size, softmax_scale, out, workspace, workspace_bytes, stream,
                        pkv::Elem::kF16);
}

}  // extern "C"
