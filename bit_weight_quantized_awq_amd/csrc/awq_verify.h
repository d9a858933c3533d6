// Host-side validation and planning of the serving-pass operators
// (awq_batch_layout, awq_kv_write, awq_tree_attention, awq_process_logits).
// HIP-free, like awq_plan.h, so that every check can run without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "awq.h"

namespace awq {

constexpr int64_t kInt32Max = (int64_t{1} << 31) - 1;

// awq_batch_layout keeps two int32 prefix sums per request in LDS, and up to
// 1024 requests two of their lengths as well.
constexpr int64_t kLayoutMaxRequests = 16384;

// awq_process_logits packs, per vocabulary entry, the count of the output
// part (19 bits), a prompt flag and the index of a bias entry plus one
// (12 bits) into one LDS word.
constexpr int64_t kLogitsMaxHistory = int64_t{1} << 19;
constexpr int64_t kLogitsMaxBiases = (int64_t{1} << 12) - 1;

struct LayoutArgs {
  const int32_t* cached_lens;
  const int32_t* new_counts;
  const int32_t* blocks_held;
  const int32_t* free_blocks;
  const int32_t* free_start;  // may be null
  const int32_t* parents;     // may be null
  int32_t* block_table;
  int32_t* q_start;
  int32_t* slots;
  int32_t* positions;
  int32_t* requests;
  uint64_t* tree_mask;  // may be null
  int32_t* blocks_held_out;
  int32_t* status;
  int B, T, num_free, table_width, block_size, num_blocks, mask_words;
};

struct KvWriteArgs {
  const void* k;
  const void* v;
  const int32_t* slots;
  awq_kv_cache cache;
  int64_t T, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
  int dtype;
};

struct AttentionArgs {
  const void* q;
  awq_kv_cache cache;
  const int32_t* block_table;
  const int32_t* cached_lens;
  const int32_t* q_start;
  const uint64_t* tree_mask;  // may be null
  void* out;
  int64_t table_stride, q_token_stride, q_head_stride;
  int B, T, heads, table_width, mask_words;
  float scale;
  int dtype;
};

// awq_tree_attention splits its keys over at most kAttentionGroups
// work-groups (two per CU), in units of kAttentionUnit keys.
constexpr int kAttentionGroups = 512;
constexpr int kAttentionUnit = 128;
constexpr int kOwnerWords = 8;  // of a work-group's entry in `owners`

struct RowStat {
  float ref, sum;
};

struct AttentionLaunch {
  AttentionArgs a;
  int group;            // query heads of a key head
  int64_t most;         // units of a key head at most
  int teams, groups;    // teams of one work-group per key head; work-groups
  int team_step;        // from a work-group to the next team's of its head: 1, or
                        // the number of heads
  uint32_t block_mul;   // x / block_size = (x * block_mul) >> block_shift for x < 2^31
  int block_shift;
  bool near_slots;      // 64 slots of a page lie within 2^31 bytes
  // Workspace: what a work-group leaves of its first and its last row block
  // (2 * groups slots of R rows), and which row block it is the first of.
  float* sums;          // [slot][row][channel]
  RowStat* stats;       // [slot][row]: reference, sum of weights
  int32_t* owners;      // [group][kOwnerWords]: parts, start, head, first row, rows, request; then
                        // the number of work-groups that had units; unused
                        // by one team, whose row blocks are whole
};

// Rows of a row block.  A row block's keys are read once for all its rows:
// the smallest block that holds the mean request, since larger ones keep more
// registers and LDS per work-group; the largest one shares keys between waves.
int attention_block_rows(int64_t B, int64_t T, int64_t heads, int64_t kv_heads, int64_t head_dim);
AttentionLaunch plan_attention(const AttentionArgs& a, void* workspace);
// Sets teams and groups for at most `groups` work-groups, or one per key head
// where there are more heads.
void form_teams(AttentionLaunch& p, int groups, int team_step);

int validate_layout(const LayoutArgs& a, int64_t B, int64_t T, int64_t num_free,
                    int64_t table_width, int64_t block_size, int64_t num_blocks,
                    int64_t mask_words);
int validate_cache(const awq_kv_cache* c);
int validate_kv_write(const KvWriteArgs& a, const awq_kv_cache* cache);
int validate_attention(const AttentionArgs& a, const awq_kv_cache* cache, int64_t B, int64_t T,
                       int64_t heads, int64_t table_width, int64_t mask_words, double scale);
size_t attention_workspace_size(int64_t B, int64_t T, int64_t heads, int64_t kv_heads,
                                int64_t head_dim);
int validate_logits(const awq_logits* a);

}  // namespace awq
