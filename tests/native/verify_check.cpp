// Drives the HIP-free validation and planning of the serving-pass operators
// over a grid of arguments, extreme sizes among them, under ASan/UBSan.
// Prints "verify_check ok" and exits 0 when every expectation holds.
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include <initializer_list>

#include "awq.h"
#include "awq_plan.h"
#include "awq_verify.h"

static int failures = 0;
#define EXPECT(cond)                                                                        \
  do {                                                                                      \
    if (!(cond)) {                                                                          \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond);        \
      ++failures;                                                                           \
    }                                                                                       \
  } while (0)

using namespace awq;

static awq_kv_cache cache(int64_t blocks, int64_t size, int64_t heads, int64_t dim, int dtype) {
  static char memory[16] __attribute__((aligned(16)));
  awq_kv_cache c{};
  c.k = c.v = memory;
  c.num_blocks = blocks;
  c.block_size = size;
  c.heads = heads;
  c.head_dim = dim;
  c.k_head_stride = c.v_head_stride = dim;
  c.k_slot_stride = c.v_slot_stride = heads * dim;
  c.k_block_stride = c.v_block_stride = size <= (int64_t{1} << 20) ? size * heads * dim : 0;
  c.dtype = dtype;
  return c;
}

static const int64_t kSizes[] = {-1, 0, 1, 2, 63, 64, 16383, 16384, 16385, (int64_t{1} << 31) - 1,
                                 int64_t{1} << 31, (int64_t{1} << 62) + 8, INT64_MAX};
static const int64_t kFew[] = {-1, 0, 1, 64, (int64_t{1} << 31) - 1, INT64_MAX};

static void check_layout() {
  static int32_t word[4] __attribute__((aligned(16)));
  LayoutArgs a{};
  a.cached_lens = a.new_counts = a.blocks_held = a.free_blocks = word;
  a.block_table = a.q_start = a.slots = a.positions = a.requests = word;
  a.blocks_held_out = a.status = word;
  int accepted = 0;
  for (int64_t B : kSizes)
    for (int64_t T : kFew)
      for (int64_t F : kFew)
        for (int64_t W : kSizes)
          for (int64_t bs : kFew)
            for (int64_t n : kFew)
              for (int64_t words : kFew) {
                const int st = validate_layout(a, B, T, F, W, bs, n, words);
                if (st != AWQ_SUCCESS) continue;
                ++accepted;
                EXPECT(B >= 1 && B <= kLayoutMaxRequests && T >= 0 && T <= kInt32Max);
                EXPECT(W >= 1 && W <= kInt32Max / B && n >= 1 && bs <= kInt32Max / n);
              }
  EXPECT(accepted > 0);
}

static void check_write() {
  static char memory[16] __attribute__((aligned(16)));
  KvWriteArgs a{};
  a.k = a.v = memory;
  a.slots = reinterpret_cast<const int32_t*>(memory);
  const int64_t dims[] = {16, 48, 128, 65536, 65552, INT64_MAX - 15};
  int accepted = 0;
  for (int64_t T : kSizes)
    for (int64_t heads : kSizes)
      for (int64_t dim : dims)
        for (int dtype = -1; dtype <= 4; ++dtype)
          for (int kind = -1; kind <= 4; ++kind) {
            if (heads > 65536 || dim > 65552) {
              awq_kv_cache c = cache(4, 16, 1, 16, kind);
              c.heads = heads;
              c.head_dim = dim;
              a.T = T;
              a.dtype = dtype;
              EXPECT(validate_kv_write(a, &c) != AWQ_SUCCESS);
              continue;
            }
            const awq_kv_cache c = cache(4, 16, heads, dim, kind);
            a.T = T;
            a.dtype = dtype;
            if (validate_kv_write(a, &c) != AWQ_SUCCESS) continue;
            ++accepted;
            // Threads of a launch, 16 channels each.
            EXPECT(T <= kInt32Max / (heads * (dim / 16)));
            EXPECT(dtype == AWQ_F16 || dtype == AWQ_BF16);
            EXPECT(kind == dtype || kind == AWQ_E4M3);
          }
  EXPECT(accepted > 0);
  EXPECT(validate_kv_write(a, nullptr) == AWQ_ERROR_INVALID_VALUE);
}

// The plan of an accepted call: what it writes lies in the workspace that
// was asked for, and its quotients are right.
static void check_plan(const AttentionArgs& given, const awq_kv_cache& c, int64_t B, int64_t T,
                       int64_t heads, int64_t W) {
  AttentionArgs a = given;
  a.cache = c;
  a.B = static_cast<int>(B);
  a.T = static_cast<int>(T);
  a.heads = static_cast<int>(heads);
  a.table_width = static_cast<int>(W);
  const size_t bytes = attention_workspace_size(B, T, heads, c.heads, c.head_dim);
  EXPECT(bytes > kAtomicRegionBytes && bytes < (size_t{1} << 30));
  char* const base = reinterpret_cast<char*>(uintptr_t{1} << 40);
  const int64_t R = attention_block_rows(B, T, heads, c.heads, c.head_dim);
  EXPECT(R == 16 || R == 32 || R == 64 || R == 128);
  for (int per_cu = 1; per_cu <= 2; ++per_cu) {
    if (per_cu == 2 && R > 32) continue;   // one work-group a CU
    for (int spread = 0; spread < 2; ++spread) {
      AttentionLaunch p = plan_attention(a, base);
      form_teams(p, 256 * per_cu, spread ? static_cast<int>(c.heads) : 1);
      EXPECT(p.group * c.heads == heads && p.teams >= 1 && p.groups == p.teams * c.heads);
      EXPECT(p.teams == 1 || p.groups <= 256 * per_cu);
      EXPECT(p.most >= 1);
      if (p.teams > 1) {   // otherwise nothing is left for another kernel
        const int64_t slots = 2 * static_cast<int64_t>(p.groups);
        EXPECT(reinterpret_cast<char*>(p.owners) == base + kAtomicRegionBytes);
        EXPECT(reinterpret_cast<char*>(p.owners + kOwnerWords * (kAttentionGroups + 1)) <=
               reinterpret_cast<char*>(p.stats));
        EXPECT(reinterpret_cast<char*>(p.stats + slots * R) <= reinterpret_cast<char*>(p.sums));
        EXPECT(reinterpret_cast<char*>(p.sums + slots * R * c.head_dim) <= base + bytes);
        EXPECT(reinterpret_cast<uintptr_t>(p.sums) % 16 == 0 && reinterpret_cast<uintptr_t>(p.stats) % 8 == 0);
      }
      const uint64_t d = static_cast<uint64_t>(c.block_size);
      for (uint64_t x : {uint64_t{0}, d - 1, d, 2 * d - 1, 7 * d, uint64_t{kInt32Max} / d * d - 1,
                         uint64_t{kInt32Max} / d * d, uint64_t{kInt32Max} - 1, uint64_t{kInt32Max}}) {
        if (x > uint64_t{kInt32Max}) continue;
        EXPECT(((x * p.block_mul) >> p.block_shift) == x / d);
      }
    }
  }
}

static void check_attention() {
  static char memory[16] __attribute__((aligned(16)));
  AttentionArgs a{};
  a.q = memory;
  a.out = memory;
  a.block_table = a.cached_lens = a.q_start = reinterpret_cast<const int32_t*>(memory);
  a.q_token_stride = a.q_head_stride = 64;
  const int64_t heads[] = {0, 1, 3, 8, 300, 600, 65535, 65536, INT64_MAX};
  const int64_t kv_heads[] = {1, 3, 8, 300, 65535, 65536};
  const int64_t dims[] = {0, 64, 96, 128, 256, 512};
  const int64_t blocks[] = {1, 3, 16, 24, 1 << 20, kInt32Max};
  int accepted = 0;
  for (int64_t B : kSizes)
    for (int64_t T : kSizes)
      for (int64_t h : heads)
        for (int64_t kh : kv_heads)
          for (int64_t dim : dims)
            for (int64_t bs : blocks)
              for (int64_t W : {int64_t{0}, int64_t{1}, int64_t{7}, int64_t{8192}, kInt32Max, INT64_MAX}) {
                awq_kv_cache c = cache(1, bs, kh, dim, AWQ_F16);
                c.k_block_stride = c.v_block_stride = 0;
                const size_t bytes = attention_workspace_size(B, T, h, kh, dim);
                if (validate_attention(a, &c, B, T, h, W, 0, 0.1) != AWQ_SUCCESS) continue;
                ++accepted;
                EXPECT(B >= 1 && T >= 0 && T <= kInt32Max / h && h % kh == 0);
                EXPECT((bytes == 0) == (T == 0));
                if (T > 0) check_plan(a, c, B, T, h, W);
              }
  EXPECT(accepted > 0);
  for (int64_t d = 1; d <= 5000; ++d) check_plan(a, cache(1, d, 8, 128, AWQ_F16), 3, 9, 32, 400);
  const awq_kv_cache c = cache(10, 16, 8, 128, AWQ_F16);
  const auto scaled = [&](double scale) { return validate_attention(a, &c, 2, 4, 32, 8, 0, scale); };
  for (double s : {0.0, -1.0, 1e-300, 1e38, -static_cast<double>(FLT_MAX)}) EXPECT(scaled(s) == AWQ_SUCCESS);
  // What float32 does not hold would make every score infinite.
  for (double s : {1e39, -1e300, static_cast<double>(INFINITY), static_cast<double>(NAN)})
    EXPECT(scaled(s) == AWQ_ERROR_INVALID_VALUE);
}

static void check_logits() {
  static char memory[16] __attribute__((aligned(16)));
  awq_logits a{};
  a.logits = a.out = memory;
  int accepted = 0;
  for (int64_t rows : kSizes)
    for (int64_t vocab : kSizes)
      for (int64_t batch : kFew)
        for (int64_t history : kSizes)
          for (int64_t biases : {int64_t{0}, int64_t{4095}, int64_t{4096}, INT64_MAX})
            for (int64_t words : kSizes) {
              a.rows = rows;
              a.vocab = vocab;
              a.batch = batch;
              a.history = history;
              a.biases = biases;
              a.mask_words = words;
              a.dtype = AWQ_F16;
              if (validate_logits(&a) != AWQ_SUCCESS) continue;
              ++accepted;
              // Work-groups, and the counts that a word of LDS holds.
              EXPECT(rows <= kInt32Max / (vocab / 1024 + 1));
              EXPECT(history + 64 * words < kLogitsMaxHistory && biases <= kLogitsMaxBiases);
            }
  EXPECT(accepted > 0);
  EXPECT(validate_logits(nullptr) == AWQ_ERROR_INVALID_VALUE);
}

int main() {
  check_layout();
  check_write();
  check_attention();
  check_logits();
  if (failures) return 1;
  printf("verify_check ok\n");
  return 0;
}
