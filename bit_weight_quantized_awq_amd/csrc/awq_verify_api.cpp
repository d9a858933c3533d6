// C-ABI entry points of the serving-pass operators (include/awq.h): host
// validation, then one launch call each.
#include <hip/hip_runtime.h>

#include "awq.h"
#include "awq_device.h"
#include "awq_lock.h"
#include "awq_plan.h"
#include "awq_verify.h"

namespace {
int status_of(hipError_t e) { return e == hipSuccess ? AWQ_SUCCESS : AWQ_ERROR_HIP; }
}  // namespace

extern "C" {

int awq_batch_layout(const void* cached_lens, const void* new_counts, const void* blocks_held,
                     const void* free_blocks, const void* free_start, const void* parents,
                     void* block_table, void* q_start, void* slots, void* positions,
                     void* requests, void* tree_mask, void* blocks_held_out, void* status,
                     int64_t B, int64_t T, int64_t num_free, int64_t table_width,
                     int64_t block_size, int64_t num_blocks, int64_t mask_words, void* stream) {
  awq::LayoutArgs a{};
  a.cached_lens = static_cast<const int32_t*>(cached_lens);
  a.new_counts = static_cast<const int32_t*>(new_counts);
  a.blocks_held = static_cast<const int32_t*>(blocks_held);
  a.free_blocks = static_cast<const int32_t*>(free_blocks);
  a.free_start = static_cast<const int32_t*>(free_start);
  a.parents = static_cast<const int32_t*>(parents);
  a.block_table = static_cast<int32_t*>(block_table);
  a.q_start = static_cast<int32_t*>(q_start);
  a.slots = static_cast<int32_t*>(slots);
  a.positions = static_cast<int32_t*>(positions);
  a.requests = static_cast<int32_t*>(requests);
  a.tree_mask = static_cast<uint64_t*>(tree_mask);
  a.blocks_held_out = static_cast<int32_t*>(blocks_held_out);
  a.status = static_cast<int32_t*>(status);
  const int st = awq::validate_layout(a, B, T, num_free, table_width, block_size, num_blocks,
                                      mask_words);
  if (st != AWQ_SUCCESS) return st;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.num_free = static_cast<int>(num_free);
  a.table_width = static_cast<int>(table_width);
  a.block_size = static_cast<int>(block_size);
  a.num_blocks = static_cast<int>(num_blocks);
  a.mask_words = static_cast<int>(mask_words);
  return status_of(awq::launch_layout(a, static_cast<hipStream_t>(stream)));
}

int awq_kv_write(const void* k, const void* v, const void* slots, const awq_kv_cache* cache,
                 int64_t T, int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                 int64_t v_head_stride, int dtype, void* stream) {
  awq::KvWriteArgs a{};
  a.k = k;
  a.v = v;
  a.slots = static_cast<const int32_t*>(slots);
  a.T = T;
  a.k_token_stride = k_token_stride;
  a.k_head_stride = k_head_stride;
  a.v_token_stride = v_token_stride;
  a.v_head_stride = v_head_stride;
  a.dtype = dtype;
  const int st = awq::validate_kv_write(a, cache);
  if (st != AWQ_SUCCESS) return st;
  if (T == 0) return AWQ_SUCCESS;
  a.cache = *cache;
  return status_of(awq::launch_kv_write(a, static_cast<hipStream_t>(stream)));
}

size_t awq_tree_attention_workspace_size(int64_t B, int64_t T, int64_t heads, int64_t kv_heads,
                                         int64_t head_dim) {
  return awq::attention_workspace_size(B, T, heads, kv_heads, head_dim);
}

int awq_tree_attention(const void* q, const awq_kv_cache* cache, const void* block_table,
                       const void* cached_lens, const void* q_start, const void* tree_mask,
                       void* out, int64_t B, int64_t T, int64_t heads, int64_t table_width,
                       int64_t table_stride, int64_t mask_words, int64_t q_token_stride,
                       int64_t q_head_stride, double scale, int dtype, void* workspace,
                       size_t workspace_bytes, void* stream) {
  awq::AttentionArgs a{};
  a.q = q;
  a.block_table = static_cast<const int32_t*>(block_table);
  a.cached_lens = static_cast<const int32_t*>(cached_lens);
  a.q_start = static_cast<const int32_t*>(q_start);
  a.tree_mask = static_cast<const uint64_t*>(tree_mask);
  a.out = out;
  a.table_stride = table_stride;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.scale = static_cast<float>(scale);
  a.dtype = dtype;
  const int st = awq::validate_attention(a, cache, B, T, heads, table_width, mask_words, scale);
  if (st != AWQ_SUCCESS) return st;
  if (T == 0) return AWQ_SUCCESS;
  a.cache = *cache;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.heads = static_cast<int>(heads);
  a.table_width = static_cast<int>(table_width);
  a.mask_words = static_cast<int>(mask_words);
  const size_t need = awq::attention_workspace_size(B, T, heads, cache->heads, cache->head_dim);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return AWQ_ERROR_WORKSPACE;
    if (!awq::aligned(workspace, 256)) return AWQ_ERROR_MISALIGNED;
  }
  const awq::WorkspaceLock lock(workspace);
  return status_of(awq::launch_attention(a, workspace, static_cast<hipStream_t>(stream)));
}

int awq_process_logits(const awq_logits* args, void* stream) {
  const int st = awq::validate_logits(args);
  if (st != AWQ_SUCCESS) return st;
  if (args->rows == 0) return AWQ_SUCCESS;
  return status_of(awq::launch_logits(*args, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
