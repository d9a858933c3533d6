// awq_batch_layout: block tables, slots, positions and ancestor masks of a
// pass, from the requests' lengths.
//
// Two exclusive prefix sums over the requests (new tokens, new blocks) decide
// everything; each output entry then follows from a binary search in them.
// A few KB for a batch: the bound is latency, so it is ONE launch in which
// every work-group repeats the sums over all requests (12 bytes a request,
// from L2) in LDS instead of waiting for a first kernel's.  What such a launch
// takes is its chain of loads and stores that wait for each other: all loads
// that do not depend on the sums are asked for before them, up to 1024
// requests stay in registers and LDS afterwards (PER: requests a thread keeps,
// 0: none), and nothing is stored before the last barrier, which would wait
// for it (16 requests of one token 7.2 -> 3.5 us, 256 trees of up to 32 tokens
// 9.4 -> 6.1).
#include "awq_device.h"
#include "awq_verify.h"

namespace awq {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxWorkGroups = 2048;
// Parents kept in LDS: those of a work-group's own tokens and of the tokens
// before them that one request of up to 768 more tokens reaches back to.  A
// walk that leaves the window reads global memory.
constexpr int kWindowBefore = 768;

// a + b for a, b >= 0, held at 2^31 - 1.  Lengths are whatever the device
// holds, and a sum of tokens that wrapped would place a token before the
// first one of its request.  Held sums do not depend on their order.
__device__ __forceinline__ int held_sum(int a, int b) {
  return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b),
                              static_cast<uint32_t>(kInt32Max)));
}

// Index of the last request whose prefix is <= x, for 0 <= x below the sum.
__device__ __forceinline__ int find_request(const int32_t* prefix, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Request {
  int cached, added, held;
  int fit;    // new blocks that have a table entry
  int lack;   // new blocks past the table's width
};

__device__ __forceinline__ Request load_request(const LayoutArgs& a, int b) {
  Request r;
  r.cached = max(0, a.cached_lens[b]);
  r.added = max(0, a.new_counts[b]);
  r.held = max(0, a.blocks_held[b]);
  const uint32_t end = static_cast<uint32_t>(r.cached) + static_cast<uint32_t>(r.added);
  const int64_t total = end == 0 ? 0 : int64_t{(end - 1) / static_cast<uint32_t>(a.block_size)} + 1;
  const int64_t need = total > r.held ? total - r.held : 0;
  const int64_t room = a.table_width > r.held ? a.table_width - r.held : 0;
  r.fit = static_cast<int>(need < room ? need : room);
  r.lack = static_cast<int>(need - r.fit < kInt32Max ? need - r.fit : kInt32Max);
  return r;
}

template <int PER>
__global__ __launch_bounds__(kThreads) void layout_kernel(LayoutArgs a) {
  extern __shared__ int32_t smem[];
  int32_t* first_token = smem;        // B
  int32_t* first_block = smem + a.B;  // B
  int32_t* cached_of = smem + 2 * a.B;  // B (PER > 0)
  int32_t* held_of = smem + 3 * a.B;    // B (PER > 0)
  __shared__ int32_t sums[4][kThreads / 64];
  constexpr int kWindow = kWindowBefore + kThreads;
  __shared__ int32_t window[kWindow];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool lead = blockIdx.x == 0;  // writes what there is once per batch

  const int first = a.free_start ? max(0, a.free_start[0]) : 0;
  // The window of the tokens from t0 on: it starts at window_start(t0).
  auto window_start = [](int64_t t0) { return static_cast<int>(max(t0 - kWindowBefore, int64_t{0})); };
  int32_t ahead[kWindow / kThreads];
  auto read_window = [&](int64_t t0) {
    const int64_t end = min(t0 + kThreads, static_cast<int64_t>(a.T));
#pragma unroll
    for (int x = 0; x < kWindow / kThreads; ++x) {
      const int64_t t = static_cast<int64_t>(window_start(t0)) + x * kThreads + tid;
      ahead[x] = t < end ? a.parents[t] : -1;
    }
  };
  auto put_window = [&] {
#pragma unroll
    for (int x = 0; x < kWindow / kThreads; ++x) window[x * kThreads + tid] = ahead[x];
  };
  if (a.parents) read_window(static_cast<int64_t>(blockIdx.x) * kThreads);

  // Each thread owns `per` consecutive requests: its own sums, a scan of the
  // threads' sums, then its requests' prefixes.
  const int per = PER ? PER : (a.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int my_tokens = 0, my_blocks = 0, my_lack = 0, my_longest = 0;
  Request kept[PER ? PER : 1];
  auto sum_up = [&](const Request& r) {
    my_tokens = held_sum(my_tokens, r.added);
    my_blocks += r.fit;   // at most the entries of the table
    my_lack = held_sum(my_lack, r.lack);
    my_longest = max(my_longest, held_sum(r.cached, r.added));
  };
  if constexpr (PER) {
#pragma unroll
    for (int x = 0; x < PER; ++x) {
      kept[x] = Request{0, 0, 0, 0, 0};
      if (b0 + x < b1) kept[x] = load_request(a, b0 + x);
    }
#pragma unroll
    for (int x = 0; x < PER; ++x) sum_up(kept[x]);
  } else {
    for (int b = b0; b < b1; ++b) sum_up(load_request(a, b));
  }
  int st = my_tokens, sb = my_blocks;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int ut = __shfl_up(st, d), ub = __shfl_up(sb, d);
    if (lane >= d) {
      st = held_sum(st, ut);
      sb += ub;
    }
  }
  if (lead) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      my_longest = max(my_longest, __shfl_xor(my_longest, d));
      my_lack = held_sum(my_lack, __shfl_xor(my_lack, d));
    }
  }
  if (lane == 63) {
    sums[0][wave] = st;
    sums[1][wave] = sb;
    sums[2][wave] = my_longest;
    sums[3][wave] = my_lack;
  }
  const int lane_before = __shfl_up(st, 1);   // a held sum cannot be taken back from
  __syncthreads();
  int tokens = 0, blocks = 0, pt = lane ? lane_before : 0, pb = sb - my_blocks;
#pragma unroll
  for (int w = 0; w < kThreads / 64; ++w) {
    pt = held_sum(pt, w < wave ? sums[0][w] : 0);
    pb += w < wave ? sums[1][w] : 0;
    tokens = held_sum(tokens, sums[0][w]);
    blocks += sums[1][w];
  }
  const int avail = max(0, a.num_free - first);
  auto put_request = [&](int b, const Request& r) {
    first_token[b] = pt;
    first_block[b] = pb;
    if constexpr (PER) {
      cached_of[b] = r.cached;
      held_of[b] = r.held;
    }
    pt = held_sum(pt, r.added);
    pb += r.fit;
  };
  if constexpr (PER) {
#pragma unroll
    for (int x = 0; x < PER; ++x)
      if (b0 + x < b1) put_request(b0 + x, kept[x]);
  } else {
    for (int b = b0; b < b1; ++b) put_request(b, load_request(a, b));
  }
  if (a.parents) put_window();
  __syncthreads();
  // Nothing is stored to global memory above, since a barrier waits for that.
  if (lead) {
    for (int b = tid; b < a.B; b += kThreads) {
      const int next = b + 1 < a.B ? first_block[b + 1] : blocks;
      const int gained = next - first_block[b], h = PER ? held_of[b] : max(0, a.blocks_held[b]);
      a.q_start[b] = first_token[b];
      a.blocks_held_out[b] = h + min(max(avail - first_block[b], 0), gained);
    }
    if (tid == 0) {
      const int taken = min(blocks, avail);
      int longest = 0, lacking = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 64; ++w) {
        longest = max(longest, sums[2][w]);
        lacking = held_sum(lacking, sums[3][w]);
      }
      a.q_start[a.B] = tokens;
      a.status[0] = first + taken;
      a.status[1] = held_sum(lacking, blocks - taken);
      a.status[2] = tokens;
      a.status[3] = longest;
    }
  }

  auto cached = [&](int b) { return PER ? cached_of[b] : max(0, a.cached_lens[b]); };
  auto held = [&](int b) { return PER ? held_of[b] : max(0, a.blocks_held[b]); };
  const int stride = gridDim.x * kThreads;
  for (uint32_t x = blockIdx.x * kThreads + tid; x < static_cast<uint32_t>(blocks); x += stride) {
    const int j = static_cast<int>(x);
    const int b = find_request(first_block, a.B, j);
    const int e = held(b) + (j - first_block[b]);
    a.block_table[static_cast<int64_t>(b) * a.table_width + e] =
        j < avail ? a.free_blocks[first + j] : -1;
  }

  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kThreads; t0 < a.T; t0 += stride) {
    const int w0 = window_start(t0);
    if (a.parents && t0 >= stride) {
      read_window(t0);
      __syncthreads();  // the window of the round before has been read
      put_window();
      __syncthreads();
    }
    if (t0 + tid >= a.T) continue;
    const int t = static_cast<int>(t0) + tid;
    int b = -1, i = 0, c = 0, slot = -1, depth = 0;
    if (t < tokens) {
      b = find_request(first_token, a.B, t);
      i = t - first_token[b];
      c = cached(b);
      const int h = held(b);
      const uint32_t at = static_cast<uint32_t>(c) + static_cast<uint32_t>(i);
      const uint32_t e = at / static_cast<uint32_t>(a.block_size);
      int page = -1;
      if (e < static_cast<uint32_t>(a.table_width)) {
        // New entries are read from the list: another work-group may still
        // have to write them to the table.
        const int j = first_block[b] + static_cast<int>(e) - h;
        if (static_cast<int>(e) < h)
          page = a.block_table[static_cast<int64_t>(b) * a.table_width + e];
        else if (j < avail)
          page = a.free_blocks[first + j];
      }
      if (page >= 0 && page < a.num_blocks)
        slot = page * a.block_size + static_cast<int>(at - e * static_cast<uint32_t>(a.block_size));
      depth = i;
    }
    uint64_t* mask = a.tree_mask ? a.tree_mask + static_cast<int64_t>(t) * a.mask_words : nullptr;
    if (b < 0) {
      for (int w = 0; mask && w < a.mask_words; ++w) mask[w] = 0;
    } else if (a.parents) {
      // From the token to its root; indices fall, so the walk ends and each
      // mask word is complete when the walk has left it.
      const int base = t - i;
      int word = mask ? a.mask_words : 0;
      depth = 0;
      uint64_t bits = 0;
      for (int at = i;;) {
        if (mask) {
          const int w = at >> 6;
          while (word > w) {
            if (word < a.mask_words) mask[word] = bits;
            bits = 0;
            --word;
          }
          if (w < a.mask_words) bits |= uint64_t{1} << (at & 63);
        }
        const int g = base + at;
        const int p = g >= w0 ? window[g - w0] : a.parents[g];
        if (p < 0 || p >= at) break;
        at = p;
        ++depth;
      }
      while (mask && word >= 0) {
        if (word < a.mask_words) mask[word] = bits;
        bits = 0;
        --word;
      }
    } else if (mask) {
      for (int w = 0; w < a.mask_words; ++w) {
        const int left = i + 1 - 64 * w;
        mask[w] = left <= 0 ? 0 : left >= 64 ? ~uint64_t{0} : (uint64_t{1} << left) - 1;
      }
    }
    a.slots[t] = slot;
    a.positions[t] = held_sum(c, depth);
    a.requests[t] = b;
  }
}

template <int PER>
hipError_t launch(const LayoutArgs& a, int grid, hipStream_t stream) {
  const size_t lds = static_cast<size_t>(a.B) * (PER ? 16 : 8);
  if (lds > 48 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(layout_kernel<PER>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(lds));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((layout_kernel<PER>), dim3(grid), dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_layout(const LayoutArgs& a, hipStream_t stream) {
  const int64_t groups = (static_cast<int64_t>(a.T) + kThreads - 1) / kThreads;
  const int grid = static_cast<int>(groups < 1 ? 1 : groups > kMaxWorkGroups ? kMaxWorkGroups : groups);
  if (a.B <= kThreads) return launch<1>(a, grid, stream);
  if (a.B <= 4 * kThreads) return launch<4>(a, grid, stream);
  return launch<0>(a, grid, stream);
}

}  // namespace awq
