// Host-side validation of the serving-pass operators (HIP-free).
#include "awq_verify.h"

#include <float.h>

#include "awq_plan.h"

namespace awq {

namespace {

// a * b <= lim for non-negative a, b, without overflow.
bool product_fits(int64_t a, int64_t b, int64_t lim) { return b == 0 || a <= lim / b; }

bool activation_dtype(int d) { return d == AWQ_F16 || d == AWQ_BF16; }

}  // namespace

int validate_layout(const LayoutArgs& a, int64_t B, int64_t T, int64_t num_free,
                    int64_t table_width, int64_t block_size, int64_t num_blocks,
                    int64_t mask_words) {
  if (B <= 0 || T < 0 || num_free < 0 || table_width <= 0 || block_size <= 0 || num_blocks <= 0 ||
      mask_words < 0)
    return AWQ_ERROR_INVALID_VALUE;
  if (!a.cached_lens || !a.new_counts || !a.blocks_held || !a.block_table || !a.q_start ||
      !a.blocks_held_out || !a.status || (num_free > 0 && !a.free_blocks))
    return AWQ_ERROR_INVALID_VALUE;
  if (T > 0 && (!a.slots || !a.positions || !a.requests)) return AWQ_ERROR_INVALID_VALUE;
  if (a.tree_mask && mask_words == 0) return AWQ_ERROR_INVALID_VALUE;
  if (B > kLayoutMaxRequests || T > kInt32Max || num_free > kInt32Max || mask_words > kInt32Max ||
      block_size > kInt32Max || num_blocks > kInt32Max)
    return AWQ_ERROR_SHAPE;
  if (!product_fits(num_blocks, block_size, kInt32Max) || !product_fits(B, table_width, kInt32Max))
    return AWQ_ERROR_SHAPE;
  const void* words[] = {a.cached_lens, a.new_counts, a.blocks_held, a.free_blocks,
                         a.free_start,  a.parents,    a.block_table, a.q_start,
                         a.slots,       a.positions,  a.requests,    a.blocks_held_out,
                         a.status};
  for (const void* p : words)
    if (!aligned(p, 4)) return AWQ_ERROR_MISALIGNED;
  if (!aligned(a.tree_mask, 8)) return AWQ_ERROR_MISALIGNED;
  return AWQ_SUCCESS;
}

int validate_cache(const awq_kv_cache* c) {
  if (!c || !c->k || !c->v) return AWQ_ERROR_INVALID_VALUE;
  if (c->num_blocks <= 0 || c->block_size <= 0 || c->heads <= 0 || c->head_dim <= 0)
    return AWQ_ERROR_INVALID_VALUE;
  if (c->dtype != AWQ_F16 && c->dtype != AWQ_BF16 && c->dtype != AWQ_E4M3)
    return AWQ_ERROR_INVALID_VALUE;
  if (c->dtype != AWQ_E4M3 && (c->k_scale || c->v_scale)) return AWQ_ERROR_INVALID_VALUE;
  const int64_t strides[] = {c->k_block_stride, c->k_slot_stride, c->k_head_stride,
                             c->v_block_stride, c->v_slot_stride, c->v_head_stride};
  for (int64_t s : strides)
    if (s < 0) return AWQ_ERROR_INVALID_VALUE;
  if (!product_fits(c->num_blocks, c->block_size, kInt32Max) || c->heads > 65535)
    return AWQ_ERROR_SHAPE;
  const int64_t unit = c->dtype == AWQ_E4M3 ? 16 : 8;  // elements in 16 bytes
  for (int64_t s : strides)
    if (s % unit != 0) return AWQ_ERROR_MISALIGNED;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) ||
      !aligned(c->v_scale, 4))
    return AWQ_ERROR_MISALIGNED;
  return AWQ_SUCCESS;
}

int validate_kv_write(const KvWriteArgs& a, const awq_kv_cache* cache) {
  if (a.T < 0 || !activation_dtype(a.dtype)) return AWQ_ERROR_INVALID_VALUE;
  const int st = validate_cache(cache);
  if (st != AWQ_SUCCESS) return st;
  if (cache->dtype != AWQ_E4M3 && cache->dtype != a.dtype) return AWQ_ERROR_INVALID_VALUE;
  if (a.T > 0 && (!a.k || !a.v || !a.slots)) return AWQ_ERROR_INVALID_VALUE;
  const int64_t strides[] = {a.k_token_stride, a.k_head_stride, a.v_token_stride, a.v_head_stride};
  for (int64_t s : strides)
    if (s < 0) return AWQ_ERROR_INVALID_VALUE;
  if (cache->head_dim % 16 != 0) return AWQ_ERROR_SHAPE;
  if (a.T > kInt32Max || cache->head_dim > 65536 ||
      !product_fits(a.T, cache->heads * (cache->head_dim / 8), kInt32Max))
    return AWQ_ERROR_SHAPE;
  for (int64_t s : strides)
    if (s % 8 != 0) return AWQ_ERROR_MISALIGNED;
  if (!aligned(a.k, 16) || !aligned(a.v, 16) || !aligned(a.slots, 4)) return AWQ_ERROR_MISALIGNED;
  return AWQ_SUCCESS;
}

int validate_attention(const AttentionArgs& a, const awq_kv_cache* cache, int64_t B, int64_t T,
                       int64_t heads, int64_t table_width, int64_t mask_words, double scale) {
  if (B <= 0 || T < 0 || heads <= 0 || table_width <= 0 || mask_words < 0 || a.table_stride < 0 ||
      a.q_token_stride < 0 || a.q_head_stride < 0 || !activation_dtype(a.dtype))
    return AWQ_ERROR_INVALID_VALUE;
  if (!(scale >= -FLT_MAX && scale <= FLT_MAX)) return AWQ_ERROR_INVALID_VALUE;
  const int st = validate_cache(cache);
  if (st != AWQ_SUCCESS) return st;
  if (cache->dtype != AWQ_E4M3 && cache->dtype != a.dtype) return AWQ_ERROR_INVALID_VALUE;
  if (T > 0 && (!a.q || !a.out)) return AWQ_ERROR_INVALID_VALUE;
  if (!a.block_table || !a.cached_lens || !a.q_start || (a.tree_mask && mask_words == 0))
    return AWQ_ERROR_INVALID_VALUE;
  const int64_t D = cache->head_dim;
  if ((D != 64 && D != 128 && D != 256) || heads % cache->heads != 0) return AWQ_ERROR_SHAPE;
  if (B > kInt32Max || T > kInt32Max || heads > 65535 || mask_words > kInt32Max / 64 ||
      !product_fits(B, table_width, kInt32Max) ||
      !product_fits(table_width, cache->block_size, kInt32Max) ||
      !product_fits(T, heads, kInt32Max))
    return AWQ_ERROR_SHAPE;
  if (a.q_token_stride % 8 != 0 || a.q_head_stride % 8 != 0 || !aligned(a.q, 16) ||
      !aligned(a.out, 16) || !aligned(a.block_table, 4) || !aligned(a.cached_lens, 4) ||
      !aligned(a.q_start, 4) || !aligned(a.tree_mask, 8))
    return AWQ_ERROR_MISALIGNED;
  return AWQ_SUCCESS;
}

int attention_block_rows(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim) {
  const int64_t mean = (T * (heads / kv_heads) + B - 1) / B;
  if (mean <= 16) return 16;
  if (head_dim > 128) return 64;
  return mean <= 32 ? 32 : 128;
}

namespace {
constexpr int64_t kOwnerBytes = (int64_t{kAttentionGroups} + 8) * kOwnerWords * 4;
// Blocks of more than 32 rows run one work-group per CU.
int64_t slot_rows(int64_t rows) { return 2 * (rows > 32 ? kAttentionGroups / 2 : kAttentionGroups) * rows; }
}  // namespace

size_t attention_workspace_size(int64_t B, int64_t T, int64_t heads, int64_t kv_heads,
                                int64_t head_dim) {
  if (B <= 0 || T <= 0 || heads <= 0 || kv_heads <= 0 || heads % kv_heads != 0 ||
      (head_dim != 64 && head_dim != 128 && head_dim != 256) || B > kInt32Max ||
      !product_fits(T, heads, kInt32Max))
    return 0;
  const int64_t rows = slot_rows(attention_block_rows(B, T, heads, kv_heads, head_dim));
  return kAtomicRegionBytes + static_cast<size_t>(kOwnerBytes + rows * (8 + 4 * head_dim));
}

AttentionLaunch plan_attention(const AttentionArgs& a, void* workspace) {
  AttentionLaunch p{};
  p.a = a;
  p.group = a.heads / static_cast<int>(a.cache.heads);
  // shift = 31 + ceil(log2 d): the multiplier exceeds 2^shift / d by less
  // than one part in 2^31, too little for a dividend below 2^31 to notice.
  const uint64_t d = static_cast<uint64_t>(a.cache.block_size);
  int log = 0;
  while ((uint64_t{1} << log) < d) ++log;
  p.block_shift = 31 + log;
  p.block_mul = static_cast<uint32_t>((uint64_t{1} << p.block_shift) / d + 1);
  const int64_t furthest = a.cache.k_slot_stride > a.cache.v_slot_stride ? a.cache.k_slot_stride
                                                                         : a.cache.v_slot_stride;
  p.near_slots = furthest <= kInt32Max / 128;   // elements of up to 2 bytes
  // The units of a key head are no more than the row blocks of every request
  // times the units of the longest row that the table can name.
  const int rows_of_block =
      attention_block_rows(a.B, a.T, a.heads, a.cache.heads, a.cache.head_dim);
  const int64_t blocks = static_cast<int64_t>(a.T) * p.group / rows_of_block + a.B;
  const int64_t keys = static_cast<int64_t>(a.table_width) * a.cache.block_size;
  const int64_t units = (keys + kAttentionUnit - 1) / kAttentionUnit;
  p.most = product_fits(blocks, units, kAttentionGroups) ? blocks * units : kAttentionGroups;
  // The accumulators at the start belong to awq_gemm, which needs them zero.
  char* ws = static_cast<char*>(workspace) + kAtomicRegionBytes;
  const int64_t rows = slot_rows(rows_of_block);
  p.owners = reinterpret_cast<int32_t*>(ws);
  p.stats = reinterpret_cast<RowStat*>(ws + kOwnerBytes);
  p.sums = reinterpret_cast<float*>(ws + kOwnerBytes + rows * 8);
  return p;
}

void form_teams(AttentionLaunch& p, int groups, int team_step) {
  const int heads = static_cast<int>(p.a.cache.heads);
  int teams = groups / heads;
  if (teams > p.most) teams = static_cast<int>(p.most);
  p.teams = teams > 1 ? teams : 1;
  p.groups = p.teams * heads;
  p.team_step = team_step;
}

int validate_logits(const awq_logits* a) {
  if (!a) return AWQ_ERROR_INVALID_VALUE;
  if (a->rows < 0 || a->vocab <= 0 || a->batch < 0 || a->history < 0 || a->biases < 0 ||
      a->mask_words < 0 || a->logits_stride < 0 || a->out_stride < 0 || a->tokens_stride < 0 ||
      a->grammar_stride < 0)
    return AWQ_ERROR_INVALID_VALUE;
  if (a->dtype != AWQ_F16 && a->dtype != AWQ_BF16 && a->dtype != AWQ_F32)
    return AWQ_ERROR_INVALID_VALUE;
  if (a->rows > 0 && (!a->logits || !a->out)) return AWQ_ERROR_INVALID_VALUE;
  if (a->tokens && (!a->prompt_lens || !a->lens)) return AWQ_ERROR_INVALID_VALUE;
  if ((a->bias_ids == nullptr) != (a->bias_values == nullptr)) return AWQ_ERROR_INVALID_VALUE;
  const int drafts = (a->draft_tokens != nullptr) + (a->tree_mask != nullptr) +
                     (a->q_start != nullptr);
  if (drafts != 0 && (drafts != 3 || a->mask_words == 0)) return AWQ_ERROR_INVALID_VALUE;
  // The grid is one work-group per row and chunk of at least 1024 entries.
  if (a->rows > kInt32Max || a->vocab > kInt32Max - 65536 ||
      !product_fits(a->rows, a->vocab / 1024 + 1, kInt32Max / 1024) || a->batch > kInt32Max ||
      a->history >= kLogitsMaxHistory || a->biases > kLogitsMaxBiases ||
      a->mask_words >= kLogitsMaxHistory / 64 ||
      a->history + 64 * a->mask_words >= kLogitsMaxHistory)
    return AWQ_ERROR_SHAPE;
  const size_t e = a->dtype == AWQ_F32 ? 4 : 2;
  if (!aligned(a->logits, e) || !aligned(a->out, e)) return AWQ_ERROR_MISALIGNED;
  const void* words[] = {a->requests,  a->tokens,   a->prompt_lens, a->lens,
                         a->repetition, a->frequency, a->presence,   a->bias_ids,
                         a->bias_values, a->grammar_mask, a->draft_tokens, a->q_start};
  for (const void* p : words)
    if (!aligned(p, 4)) return AWQ_ERROR_MISALIGNED;
  if (!aligned(a->tree_mask, 8)) return AWQ_ERROR_MISALIGNED;
  return AWQ_SUCCESS;
}

}  // namespace awq
