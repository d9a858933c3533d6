// Runs awq_batch_layout's kernel on the CPU over lengths whose sums pass
// 2^31, with every operand in memory of its own size.  Each case: the kernel
// against the definition in 64 bits, where a sum past 2^31 - 1 is held there.
// Prints "layout_check ok" and exits 0 when every expectation holds.
#include <stdio.h>

#include <string>

#include "layout_kernel_source.h"   // csrc/awq_layout.hip

static int failures = 0;
#define EXPECT(cond, ...)                                                        \
  do {                                                                           \
    if (!(cond)) {                                                               \
      fprintf(stderr, "%s:%d: expectation failed: %s ", __FILE__, __LINE__, #cond); \
      fprintf(stderr, __VA_ARGS__);                                              \
      fprintf(stderr, "\n");                                                     \
      ++failures;                                                                \
    }                                                                            \
  } while (0)

typedef std::vector<int32_t> Ints;
static const int64_t kMost = (int64_t{1} << 31) - 1;
static int32_t held(int64_t x) { return static_cast<int32_t>(x < kMost ? x : kMost); }

static void check(const char* name, const Ints& cached, const Ints& counts, const Ints& blocks_held,
                  int T, const Ints& parents, int W, int bs, int num_free, int words) {
  printf("[case] %s B=%zu T=%d\n", name, cached.size(), T);
  fflush(stdout);
  const int B = static_cast<int>(cached.size());
  Ints free(num_free), start{0}, table(static_cast<size_t>(B) * W, -1), q_start(B + 1, -7), slots(T, -7),
      positions(T, -7), requests(T, -7), held_out(B, -7), status(4, -7);
  for (int i = 0; i < num_free; ++i) free[i] = i;
  std::vector<uint64_t> mask(static_cast<size_t>(T) * words, 77);
  awq::LayoutArgs a{};
  a.cached_lens = cached.data();
  a.new_counts = counts.data();
  a.blocks_held = blocks_held.data();
  a.free_blocks = free.data();
  a.free_start = start.data();
  a.parents = parents.empty() ? nullptr : parents.data();
  a.block_table = table.data();
  a.q_start = q_start.data();
  a.slots = slots.data();
  a.positions = positions.data();
  a.requests = requests.data();
  a.tree_mask = words ? mask.data() : nullptr;
  a.blocks_held_out = held_out.data();
  a.status = status.data();
  a.B = B;
  a.T = T;
  a.num_free = num_free;
  a.table_width = W;
  a.block_size = bs;
  a.num_blocks = num_free;
  a.mask_words = words;
  EXPECT(awq::launch_layout(a, nullptr) == hipSuccess, "%s", name);

  int64_t tokens = 0, lack = 0, longest = 0, next = 0;
  for (int b = 0; b < B; ++b) {
    const int64_t c = std::max(0, cached[b]), n = std::max(0, counts[b]), h = std::max(0, blocks_held[b]);
    EXPECT(q_start[b] == held(tokens), "%s request %d: %d", name, b, q_start[b]);
    longest = std::max(longest, c + n);
    const int64_t need = std::max<int64_t>(0, (c + n + bs - 1) / bs - h);
    const int64_t fit = std::min(need, std::max<int64_t>(0, W - h));
    const int64_t gained = std::min<int64_t>(fit, num_free - next);
    lack += need - gained;
    next += gained;
    EXPECT(held_out[b] == held(h + gained), "%s request %d: %d", name, b, held_out[b]);
    std::vector<int> depth;
    for (int64_t i = 0; i < n && tokens + i < T; ++i) {
      const int64_t t = tokens + i;
      const int p = parents.empty() ? static_cast<int>(i) - 1 : parents[t];
      depth.push_back(p >= 0 && p < i ? depth[p] + 1 : 0);
      EXPECT(requests[t] == b, "%s token %ld: %d", name, (long)t, requests[t]);
      EXPECT(positions[t] == held(c + depth[i]), "%s token %ld: %d", name, (long)t, positions[t]);
      const int64_t e = (c + i) / bs;
      const int page = e < W ? table[static_cast<size_t>(b) * W + e] : -1;
      EXPECT(slots[t] == (page < 0 ? -1 : page * bs + (c + i) % bs), "%s token %ld: %d", name, (long)t, slots[t]);
      if (words && i < 64) EXPECT(mask[t * words] >> i & 1, "%s token %ld", name, (long)t);
    }
    tokens += n;
  }
  EXPECT(q_start[B] == held(tokens), "%s: %d", name, q_start[B]);
  for (int64_t t = tokens; t < T; ++t) EXPECT(requests[t] == -1 && slots[t] == -1, "%s token %ld", name, (long)t);
  EXPECT(status[0] == next, "%s: %d", name, status[0]);
  EXPECT(status[1] == held(lack), "%s: %d", name, status[1]);
  EXPECT(status[2] == held(tokens), "%s: %d", name, status[2]);
  EXPECT(status[3] == held(longest), "%s: %d", name, status[3]);
}

int main() {
  const int32_t most = INT32_MAX;
  Ints parents(600);
  for (int t = 0; t < 600; ++t) parents[t] = t % 3 == 0 ? 0 : t - 1;
  // A batch whose sums are small, for the check itself.
  check("small", {5, 0, 33}, {3, 0, 400}, {1, 0, 3}, 420, parents, 40, 16, 60, 1);
  check("chains", {5, 0, 33}, {3, 0, 400}, {1, 0, 3}, 420, {}, 40, 16, 60, 2);
  // int32 prefixes would be 0, 2^31 - 1, -2, ...: token 1 in request 2 at
  // index 3, its root two words before the parents.
  check("three", {0, 0, 0, 0}, {most, most, 100, 0}, {0, 0, 0, 0}, 100, parents, 2, 16, 8, 1);
  check("five", {9, 9, 9, 9, 9}, {most, most, most, most, most}, {1, 1, 1, 1, 1}, 300, parents, 2, 16, 8, 1);
  check("five chains", {9, 9, 9, 9, 9}, {most, most, most, most, most}, {1, 1, 1, 1, 1}, 300, {}, 2, 16, 8, 1);
  check("first small", {0, 0, 0, 0}, {40, most, most, 7}, {0, 0, 0, 0}, 64, parents, 4, 16, 30, 1);
  check("long contexts", {most, most - 3, 7}, {5, 9, most}, {0, most, 2}, 30, parents, 3, 1, 30, 1);
  // Every thread of the sums, four requests each and more.
  check("many", Ints(300, 2), Ints(300, most / 8), Ints(300, 0), 500, parents, 1, 16, 9, 1);
  check("many small first", Ints(1500, 20), [&] {
    Ints n(1500, 1);
    n[400] = n[900] = n[1499] = most - 5;
    return n;
  }(), Ints(1500, 2), 600, parents, 2, 16, 9, 1);
  if (failures) return 1;
  printf("layout_check ok\n");
  return 0;
}
