// C ABI of the speculative decoding step: argument checks and dispatch.  The
// operations are described in include/fused_ce_tvd.h.
#include "fct_internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

constexpr int64_t kMaxSpan = int64_t(1) << 62;

// Adds (n - 1) * stride to *span; false if a size or stride is negative or
// the sum passes 2^62 (so that every offset computed from them is exact).
bool extend(int64_t* span, int64_t n, int64_t stride) {
  if (n < 0 || stride < 0) return false;
  if (n <= 1) return true;
  if (stride > (kMaxSpan - *span) / (n - 1)) return false;
  *span += (n - 1) * stride;
  return true;
}

int check_cache(const fct_kv_cache* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr) return FCT_ERR_INVALID_ARG;
  if (c->dtype != FCT_BF16 && c->dtype != FCT_E4M3) return FCT_ERR_UNSUPPORTED;
  if (c->page_size <= 0 || c->num_pages <= 0 || c->n_heads <= 0 || c->head_dim <= 0)
    return FCT_ERR_INVALID_ARG;
  if (c->head_dim % 8 != 0 || c->head_dim > 256 || c->n_heads > 65536) return FCT_ERR_UNSUPPORTED;
  if (c->num_pages > (int64_t(1) << 40)) return FCT_ERR_UNSUPPORTED;
  int64_t span = c->head_dim;
  if (!extend(&span, c->num_pages, c->page_stride) ||
      !extend(&span, c->page_size, c->slot_stride) || !extend(&span, c->n_heads, c->head_stride))
    return FCT_ERR_INVALID_ARG;
  const size_t vec = c->dtype == FCT_E4M3 ? 8 : 16;
  if (!aligned(c->k, vec) || !aligned(c->v, vec)) return FCT_ERR_ALIGNMENT;
  if (c->page_stride % 8 != 0 || c->slot_stride % 8 != 0 || c->head_stride % 8 != 0)
    return FCT_ERR_ALIGNMENT;
  if (c->dtype == FCT_E4M3) {
    if (c->k_scale == nullptr || c->v_scale == nullptr) return FCT_ERR_INVALID_ARG;
    int64_t scales = 1;
    if (!extend(&scales, c->num_pages, c->scale_page_stride) ||
        !extend(&scales, c->page_size, c->scale_slot_stride) ||
        !extend(&scales, c->n_heads, c->scale_head_stride))
      return FCT_ERR_INVALID_ARG;
  }
  return FCT_OK;
}

int check_pages(const int32_t* table, int64_t ld, int64_t max_pages, const int32_t* context_len,
                int64_t batch) {
  if (table == nullptr || context_len == nullptr) return FCT_ERR_INVALID_ARG;
  if (max_pages <= 0 || ld < max_pages) return FCT_ERR_INVALID_ARG;
  if (max_pages > INT32_MAX) return FCT_ERR_UNSUPPORTED;
  int64_t span = max_pages;
  if (!extend(&span, batch, ld)) return FCT_ERR_INVALID_ARG;
  if (!aligned(table, 4) || !aligned(context_len, 4)) return FCT_ERR_ALIGNMENT;
  return FCT_OK;
}

int check_status(const int32_t* dev_status) {
  return dev_status && !aligned(dev_status, 4) ? FCT_ERR_ALIGNMENT : FCT_OK;
}

// A launch's result as a status; the CUDA error stays for cudaGetLastError.
int launched(cudaError_t e) {
  if (e == cudaErrorInvalidConfiguration) {
    cudaGetLastError();
    return FCT_ERR_UNSUPPORTED;
  }
  return e == cudaSuccess ? FCT_OK : FCT_ERR_CUDA;
}

constexpr int64_t kMaxBatch = int64_t(1) << 24;

}  // namespace

extern "C" {

int fct_kv_cache_write(const void* k, const void* v, int64_t ld_token, int64_t ld_head,
                       fct_dtype dtype, int64_t n_tokens, const int64_t* slots,
                       const fct_kv_cache* cache, int32_t* dev_status, void* stream) {
  if (n_tokens < 0) return FCT_ERR_INVALID_ARG;
  int rc = check_cache(cache);
  if (rc != FCT_OK) return rc;
  if (dtype != FCT_F32 && dtype != FCT_BF16) return FCT_ERR_UNSUPPORTED;
  if (n_tokens == 0) return FCT_OK;
  if (k == nullptr || v == nullptr || slots == nullptr) return FCT_ERR_INVALID_ARG;
  const size_t e = dtype == FCT_F32 ? 4 : 2;
  int64_t span = cache->head_dim;
  if (!extend(&span, n_tokens, ld_token) || !extend(&span, cache->n_heads, ld_head))
    return FCT_ERR_INVALID_ARG;
  if (!aligned(k, e) || !aligned(v, e) || !aligned(slots, 8)) return FCT_ERR_ALIGNMENT;
  if ((rc = check_status(dev_status)) != FCT_OK) return rc;
  int sms = 0, device = 0;
  if ((rc = fct::current_device_sms(&sms, &device)) != FCT_OK) return rc;
  return launched(fct::launch_kv_write(
      fct::KvWriteArgs{k, v, ld_token, ld_head, dtype, n_tokens, slots, *cache, dev_status},
      sms, static_cast<cudaStream_t>(stream)));
}

int fct_kv_cache_move(const fct_kv_cache* cache, const int32_t* block_table, int64_t ld_table,
                      int64_t max_pages, const int32_t* context_len, int64_t batch,
                      const int32_t* path, int64_t ld_path, int64_t path_len, const int32_t* count,
                      int32_t* dev_status, void* stream) {
  if (batch < 0 || path_len < 0) return FCT_ERR_INVALID_ARG;
  int rc = check_cache(cache);
  if (rc != FCT_OK) return rc;
  if (batch == 0 || path_len == 0) return FCT_OK;
  if (batch > kMaxBatch) return FCT_ERR_UNSUPPORTED;
  if ((rc = check_pages(block_table, ld_table, max_pages, context_len, batch)) != FCT_OK) return rc;
  if (path == nullptr || count == nullptr || ld_path < path_len) return FCT_ERR_INVALID_ARG;
  int64_t span = path_len;
  if (!extend(&span, batch, ld_path)) return FCT_ERR_INVALID_ARG;
  if (!aligned(path, 4) || !aligned(count, 4)) return FCT_ERR_ALIGNMENT;
  if ((rc = check_status(dev_status)) != FCT_OK) return rc;
  int sms = 0, device = 0;
  if ((rc = fct::current_device_sms(&sms, &device)) != FCT_OK) return rc;
  return launched(fct::launch_kv_move(
      fct::KvMoveArgs{*cache, {block_table, ld_table, max_pages, context_len, batch}, path, ld_path,
                      path_len, count, dev_status},
      static_cast<cudaStream_t>(stream)));
}

size_t fct_tree_attention_workspace_size(int64_t n_nodes, int32_t n_q_heads, int32_t n_heads,
                                         int32_t head_dim) {
  if (n_nodes <= 0 || n_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_heads != 0) return 0;
  if (head_dim <= 0 || head_dim % 8 != 0 || head_dim > 256) return 0;
  int sms = 0, device = 0;
  if (fct::current_device_sms(&sms, &device) != FCT_OK) return 0;
  return fct::attn_workspace_bytes(n_nodes, n_q_heads, n_heads, head_dim, sms);
}

int fct_tree_attention(const void* q, int64_t ld_q_node, int64_t ld_q_head, int64_t n_nodes,
                       int32_t n_q_heads, const fct_kv_cache* cache, const int32_t* block_table,
                       int64_t ld_table, int64_t max_pages, const int32_t* context_len,
                       const int32_t* node_start, int64_t batch, const int64_t* tree_mask,
                       int64_t mask_words, float scale, void* out, int64_t ld_out_node,
                       int64_t ld_out_head, float* lse, void* workspace, size_t workspace_bytes,
                       int32_t* dev_status, void* stream) {
  if (n_nodes < 0 || batch < 0 || n_q_heads <= 0) return FCT_ERR_INVALID_ARG;
  int rc = check_cache(cache);
  if (rc != FCT_OK) return rc;
  if (n_q_heads % cache->n_heads != 0) return FCT_ERR_INVALID_ARG;
  if (!(scale == scale)) return FCT_ERR_INVALID_ARG;
  if (n_nodes == 0 || batch == 0) return FCT_OK;
  if (batch > kMaxBatch || n_nodes > INT32_MAX) return FCT_ERR_UNSUPPORTED;
  if ((rc = check_pages(block_table, ld_table, max_pages, context_len, batch)) != FCT_OK) return rc;
  // positions are 32-bit in the kernels, with room for a tile past the last
  if (max_pages > ((int64_t(1) << 31) - 1024) / cache->page_size) return FCT_ERR_UNSUPPORTED;
  if (n_nodes * (n_q_heads / cache->n_heads) > INT32_MAX) return FCT_ERR_UNSUPPORTED;
  if (q == nullptr || out == nullptr || node_start == nullptr) return FCT_ERR_INVALID_ARG;
  if (mask_words < 0 || (tree_mask == nullptr) != (mask_words == 0)) return FCT_ERR_INVALID_ARG;
  if (mask_words > (int64_t(1) << 24)) return FCT_ERR_UNSUPPORTED;
  int64_t span_q = cache->head_dim, span_o = cache->head_dim;
  if (!extend(&span_q, n_nodes, ld_q_node) || !extend(&span_q, n_q_heads, ld_q_head) ||
      !extend(&span_o, n_nodes, ld_out_node) || !extend(&span_o, n_q_heads, ld_out_head))
    return FCT_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(out, 2) || !aligned(node_start, 4) || !aligned(tree_mask, 8) ||
      !aligned(lse, 4))
    return FCT_ERR_ALIGNMENT;
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
  if (q0 < o0 + 2 * uintptr_t(span_o) && o0 < q0 + 2 * uintptr_t(span_q)) return FCT_ERR_INVALID_ARG;
  if ((rc = check_status(dev_status)) != FCT_OK) return rc;
  int sms = 0, device = 0;
  if ((rc = fct::current_device_sms(&sms, &device)) != FCT_OK) return rc;
  const size_t need = fct::attn_workspace_bytes(n_nodes, n_q_heads, cache->n_heads, cache->head_dim, sms);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return FCT_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return FCT_ERR_ALIGNMENT;
  return launched(fct::launch_attention(
      fct::AttnArgs{q, ld_q_node, ld_q_head, n_nodes, n_q_heads, *cache,
                    {block_table, ld_table, max_pages, context_len, batch}, node_start, tree_mask,
                    mask_words, scale, out, ld_out_node, ld_out_head, lse, workspace, dev_status},
      sms, device, static_cast<cudaStream_t>(stream)));
}

int fct_spec_verify(const void* target, int64_t ld_target, const void* draft, int64_t ld_draft,
                    fct_dtype dtype, int64_t n_nodes, int64_t V, const int64_t* tokens,
                    const int32_t* parent, const int32_t* node_start, int64_t batch,
                    const float* uniform, const float* noise, int64_t ld_noise,
                    const float* temperature, int64_t max_depth, int64_t* out_tokens,
                    int32_t* path, int32_t* count, int32_t* dev_status, void* stream) {
  if (n_nodes < 0 || batch < 0 || V <= 0 || max_depth < 0) return FCT_ERR_INVALID_ARG;
  if (dtype != FCT_F32 && dtype != FCT_BF16) return FCT_ERR_UNSUPPORTED;
  if (batch == 0) return FCT_OK;
  if (batch > kMaxBatch || V > (int64_t(1) << 30) || max_depth > INT32_MAX)
    return FCT_ERR_UNSUPPORTED;
  if (node_start == nullptr || noise == nullptr || out_tokens == nullptr || count == nullptr ||
      (path == nullptr && max_depth > 0))
    return FCT_ERR_INVALID_ARG;
  if (n_nodes > 0 && (target == nullptr || tokens == nullptr || parent == nullptr ||
                      uniform == nullptr))
    return FCT_ERR_INVALID_ARG;
  if (ld_target < V || ld_noise < V || (draft != nullptr && ld_draft < V)) return FCT_ERR_INVALID_ARG;
  int64_t span = V, span_n = V, span_d = V;
  if (!extend(&span, n_nodes, ld_target) || !extend(&span_n, batch, ld_noise) ||
      (draft != nullptr && !extend(&span_d, n_nodes, ld_draft)))
    return FCT_ERR_INVALID_ARG;
  const size_t e = dtype == FCT_F32 ? 4 : 2;
  if (!aligned(target, e) || !aligned(draft, e) || !aligned(tokens, 8) || !aligned(parent, 4) ||
      !aligned(node_start, 4) || !aligned(uniform, 4) || !aligned(noise, 4) ||
      !aligned(temperature, 4) || !aligned(out_tokens, 8) || !aligned(path, 4) ||
      !aligned(count, 4))
    return FCT_ERR_ALIGNMENT;
  int rc = check_status(dev_status);
  if (rc != FCT_OK) return rc;
  int sms = 0, device = 0;
  if ((rc = fct::current_device_sms(&sms, &device)) != FCT_OK) return rc;
  return launched(fct::launch_verify(
      fct::VerifyArgs{target, draft, ld_target, ld_draft, dtype, n_nodes, V, tokens, parent,
                      node_start, batch, uniform, noise, ld_noise, temperature, max_depth,
                      out_tokens, path, count, dev_status},
      sms, device, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
