// awq_tree_attention: drafted tokens against a paged cache.
//
// Bound by HBM while a key serves up to a few hundred rows: every key and
// value is read once per row block, and the products are a few percent of
// the matrix cores' rate.  What the layout below is for is keeping tens of
// KB in flight per CU over scattered blocks and giving every work-group the
// same number of keys however ragged the batch is.
//
// * Rows.  The rows that share a key head (tokens x query heads of its
//   group) form row blocks of R = 16 NT rows, so a key read once serves all
//   of them.  NT follows the mean number of rows (attention_block_rows).
// * Split.  A unit is 128 keys of one (request, row block).  The units of the
//   whole batch are numbered in that order, and team t of W takes the units
//   from total * t / W on: equal shares, whatever the lengths.  A team is one
//   work-group per key head, so the heads of a key, neighbours in memory, are
//   read at about the same time.  The lengths are device data, so each
//   work-group sums them itself (12 bytes a request, from L2).  A run of keys
//   that is not the whole row block leaves (max, sum, weighted values) in the
//   workspace for attention_combine_kernel: at most two of them per
//   work-group.
//   Neighbouring work-groups, which one XCD runs, are teams of one head where
//   waves have keys of their own, and heads of one team where they share them
//   (the other way round: 32 requests of 0.5-8K tokens 77.4 -> 80.4 us, e4m3
//   trees 209 -> 217; trees of 13-64 tokens 74.1 -> 75.9, 131K context 131.3
//   -> 134.3).
// * Waves.  Up to 32 rows (attention_kernel), wave x of four takes every
//   fourth tile of 32 keys, for all R rows: no barrier and no sharing inside
//   the loop, which ends with one merge through LDS.  With more rows the
//   waves share the keys (attention_wide_kernel).
// * Loads.  Keys and values go HBM -> LDS in 16-byte pieces without passing
//   registers, into buffers of the wave alone.  The keys of tile i + S are
//   requested when the scores of tile i are done, its values when tile i's
//   values have been used, and both are awaited by counting.  Block numbers
//   come the same way, two tiles ahead.  Pieces of a row are permuted by XOR
//   so that the reads below have no bank conflicts.
// * Products.  S^T = K Q^T leaves in a lane the scores of ONE row and of the
//   keys 4g..4g+3 and 16+4g..16+4g+3 (g = lane / 16), which is the operand
//   that O^T = V^T P^T takes with its 32 keys in that order: the weights
//   never move between lanes.  V^T comes from transposing LDS reads.
// * Softmax.  A row's reference starts 2^7 below its first maximum and moves
//   only when a score passes it by 2^15, so the usual tile has no reduction
//   over lanes and no rescaling of the sums.  A row's largest weight lies in
//   2^7 .. 2^15: the top of float16's range, so the weights that are rounded
//   to it for the matrix cores keep their precision down to 2^-21 of the
//   largest, and a long context of small ones is not lost.  Their sum is of
//   the unrounded ones.  The rounding to 16 bits takes the error against 64
//   bits from that of the rounded output alone, 2.1e-4 of its size in float16
//   and 1.7e-3 in bfloat16, to 2.8e-4 and 2.2e-3; a second product with what
//   it leaves over takes it back, but 131K context then takes 158.7 us and
//   not 134.0, trees of 13-64 tokens 81.8 and not 74.2, e4m3 trees 211 and
//   not 206.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "awq_device.h"
#include "awq_plan.h"
#include "awq_verify.h"

namespace awq {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short short4v __attribute__((ext_vector_type(4)));
typedef int int2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kTile = 32;                       // keys of a wave's step
constexpr int kUnit = kTile * kWaves;           // keys of a unit
static_assert(kUnit == kAttentionUnit, "the planner counts in units");
constexpr float kLift = 7.f, kSlack = 15.f;     // see "Softmax" above

template <bool BF16> struct Act {
  using T = _Float16;
  using V8 = half8_t;
  using V2 = half2_t;
};
template <> struct Act<true> {
  using T = __bf16;
  using V8 = bf16x8_t;
  using V2 = bf16x2_t;
};

__device__ __forceinline__ floatx4 mfma(half8_t a, half8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma(bf16x8_t a, bf16x8_t b, floatx4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Four e4m3 values as the 16-bit type (exact: at most 4 significant bits and
// exponents -9..8).
__device__ __forceinline__ void widen(uint32_t w, half2_t* o) {
  o[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, false);
  o[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, true);
}
__device__ __forceinline__ void widen(uint32_t w, bf16x2_t* o) {
  o[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false);
  o[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true);
}
template <bool BF16>
__device__ __forceinline__ typename Act<BF16>::V8 widen8(uint32_t lo, uint32_t hi) {
  union {
    typename Act<BF16>::V2 p[4];
    typename Act<BF16>::V8 v;
  } u;
  widen(lo, u.p);
  widen(hi, u.p + 2);
  return u.v;
}

// Copies to LDS as inline assembly: the compiler does not track them (it
// would make every LDS read wait for all of them), and the waits below count
// them.  Lane i writes lds + 16 i (4 i).  A copy must not follow a scalar
// write of m0 directly (one wait state), which the compiler sees to for its
// own instructions only.
__device__ __forceinline__ void copy16(uint64_t from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(lds) : "memory");
}
// The same from `base` (one for the wave) + off.  Scalar registers that a
// vector instruction has written (a lane read, or a spilled one read back) may
// be a copy's base only five wait states later.
__device__ __forceinline__ void copy16(uint64_t base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 4\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "{m0}"(lds) : "memory");
}
__device__ __forceinline__ void copy4(uint64_t from, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  static_assert(N < 64, "six-bit counter");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lds_reads() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(p)));
}
// A copy of v that the compiler takes for a new value: what is computed from
// it is computed where it is used, and not kept in registers from further out.
__device__ __forceinline__ int fresh(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
// A pointer into LDS from its address.
template <class T>
__device__ __forceinline__ __attribute__((address_space(3))) T* lds_at(uint32_t addr) {
  return (__attribute__((address_space(3))) T*)(uintptr_t)addr;
}
template <class T>
__device__ __forceinline__ T uniform(T v) {
  static_assert(sizeof(T) == 4, "one register");
  return __builtin_bit_cast(T, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
}

// What keys and values that no row may see are read from.
__device__ __attribute__((aligned(512))) const uint32_t kZeroRow[128] = {};

template <bool E4M3, int D, int NT>
struct Shape {
  static constexpr int ES = E4M3 ? 1 : 2;
  static constexpr int ROW = D * ES;        // bytes of a key
  static constexpr int P = ROW / 16;        // its 16-byte pieces
  static constexpr int PER = P >= 16 ? 1 : 16 / P;   // keys in 256 bytes
  static constexpr int TILE = kTile * ROW;  // bytes of a tile of keys (or values)
  static constexpr int CP = TILE / 1024;    // copies of a tile
  static constexpr int R = 16 * NT;
  // Work-groups per CU: two, unless the sums and the queries of NT row tiles
  // need more than half of the registers or the buffers of half of the LDS.
  static constexpr int OCC = (D * NT >= 512 || 8 * TILE > 65536) ? 1 : 2;
  // Tiles in flight ahead of the one in use.
  static constexpr int STG = 16 * TILE <= 131072 / OCC ? 2 : 1;
  static constexpr int WAVE = 2 * STG * TILE;               // a wave's buffers
  static constexpr int BUF = kWaves * WAVE;
  static constexpr int PASS = kWaves * R * D * 4 <= BUF ? NT : 1;   // row tiles merged at a time
  static constexpr int MERGE = kWaves * 16 * PASS * D * 4;  // overlays the buffers
  static constexpr int DATA = BUF > MERGE ? BUF : MERGE;
  static constexpr int TAB = DATA;                          // block numbers: ring of 2 STG
  static constexpr int TABW = 2 * STG * 256;
  static constexpr int ADR = TAB + kWaves * TABW;           // 64 addresses a wave
  static constexpr int STAT = ADR + kWaves * 512;           // (reference, sum) of each wave and row
  static constexpr int SCAN = STAT + kWaves * R * 8;
  static constexpr int STRD = SCAN + 64;                     // base and strides of keys and values
  static constexpr int LDS = STRD + kWaves * 64;

  // Which 16-byte piece of key `k` a piece is kept as: a fragment read takes
  // one piece of each of 16 keys.
  static constexpr __device__ __forceinline__ int kswz(int k) {
    return P >= 16 ? (k & 15) : (k / PER) & (P - 1);
  }
  // The same for values: a transposing read takes 32 bytes of each of four
  // (16-bit) or 16 bytes of each of eight keys (8-bit).
  static constexpr __device__ __forceinline__ int vswz(int k) {
    if constexpr (E4M3)
      return P >= 16 ? (k & 15) : ((k / PER) ^ (((k >> 4) & 1) << 2)) & (P - 1);
    else
      return P >= 16 ? (k & 7) << 1 : ((k / PER) & (P / 2 - 1)) << 1;
  }
};

// A request's share of the units.
struct Span {
  int start, n, cached, L, blocks, units;   // rows, keys; row blocks; units of a row block
  int64_t all;                              // units of the request
};
template <int R>
__device__ __forceinline__ Span span_of(const AttentionLaunch& p, int b) {
  const AttentionArgs& a = p.a;
  Span s;
  s.start = min(max(a.q_start[b], 0), a.T);
  s.n = max(min(max(a.q_start[b + 1], 0), a.T) - s.start, 0);
  s.cached = max(a.cached_lens[b], 0);
  const int64_t room = static_cast<int64_t>(a.table_width) * a.cache.block_size;
  const int64_t end = static_cast<int64_t>(s.cached) + s.n;
  s.L = static_cast<int>(end < room ? end : room);
  s.blocks = (s.n * p.group + R - 1) / R;
  s.units = (s.L - 1) / kUnit + 1;
  s.all = static_cast<int64_t>(s.blocks) * s.units;
  return s;
}

__device__ __forceinline__ uint32_t divide(uint32_t x, const AttentionLaunch& p) {
  return static_cast<uint32_t>((static_cast<uint64_t>(x) * p.block_mul) >> p.block_shift);
}

// What a wave keeps of its 16 NT rows while it goes over keys.
template <bool BF16, int D, int NT>
struct Rows {
  typename Act<BF16>::V8 q[NT][D / 32];
  floatx4 acc[NT][D / 16];
  float ref[NT], sum[NT];   // sum: over the lane's own keys
  float c;                  // scale of a product, in powers of two
};

// The rows of a wave in their request.
struct Place {
  int start, first, count;   // first token of the request; first row and rows of the wave
  int group;
};

template <bool BF16, bool E4M3, int D, int NT>
__device__ __forceinline__ void load_rows(const AttentionArgs& a, const Place& at, int hk,
                                          Rows<BF16, D, NT>& o) {
  using T = typename Act<BF16>::T;
  const int lane = fresh(threadIdx.x & 63), col = lane & 15, g = lane >> 4;
  // A negative scale turns the queries' signs, so that the largest product is
  // the largest score.  A zero scale, which would make NaN of a hidden key's
  // -infinity, becomes the smallest one: it leaves every finite product, of
  // 2^128 at most, within 2^-21 of zero.
  float c = a.scale * 1.44269504088896340736f;
  if (a.cache.k_scale) c *= static_cast<const float*>(a.cache.k_scale)[hk];
  const uint32_t flip = c < 0.f ? 0x80008000u : 0u;
  o.c = fmaxf(fabsf(c), 0x1p-149f);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = at.first + 16 * nt + col;
    const int i = r / at.group, h = hk * at.group + (r - i * at.group);
    const bool ok = 16 * nt + col < at.count;
    const T* from = static_cast<const T*>(a.q) +
                    (ok ? (at.start + i) * a.q_token_stride + h * a.q_head_stride : 0);
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) {
      // The channels that the keys' fragment holds (see tile_step).
      const int ch = E4M3 ? 64 * (ks >> 1) + 16 * g + 8 * (ks & 1) : 32 * ks + 8 * g;
      u32x4 x = *reinterpret_cast<const u32x4*>(from + ch);
#pragma unroll
      for (int w = 0; w < 4; ++w) x[w] = ok ? x[w] ^ flip : 0u;
      o.q[nt][ks] = __builtin_bit_cast(typename Act<BF16>::V8, x);
    }
    o.ref[nt] = -FLT_MAX;
    o.sum[nt] = 0.f;
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o.acc[nt][d] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
}

// 32 keys and values in LDS against the wave's rows.  `there` tells which of
// the keys there are; `spare`: 1 KB.  DRAFTED: some of the keys may be drafted
// ones, the first of them with index `idx` (negative: in the context), and be
// hidden from some rows.  `scored` is called when the keys have been read,
// `need_values` before the values are, `used` when they have been.
//
// With two waves on a SIMD the vector instructions' issue is what bounds a
// step that HBM does not, so addresses are one register and an XOR each
// (swizzles are linear in the bits of key and piece), and all fragments of a
// product are read before its first one.
template <bool DRAFTED, bool BF16, bool E4M3, int D, int NT, class B, class F, class H, class U>
__device__ __forceinline__ void tile_step(const AttentionArgs& a, const Place& at,
                                          Rows<BF16, D, NT>& o, const char* keys,
                                          const char* vals, char* spare, B there, int idx,
                                          F scored, H need_values, U used) {
  using C = Shape<E4M3, D, NT>;
  using T = typename Act<BF16>::T;
  using V8 = typename Act<BF16>::V8;
  constexpr int DT = D / 16;   // channel tiles
  constexpr int KS = D / 32;   // steps of a score
  const int lane = fresh(threadIdx.x & 63), col = lane & 15, g = lane >> 4;
  floatx4 s[2][NT];
  using KFrag = typename std::conditional<E4M3, u32x4, V8>::type;
  constexpr int KF = E4M3 ? KS / 2 : KS;          // 16-byte fragments of a key
  constexpr int KB = 2 * KF <= 8 ? 2 : 1;         // key tiles whose fragments are read together
  const uint32_t kaddr = lds_addr(keys) + (C::ROW * col + 16 * (g ^ C::kswz(col)));
  uint32_t here = 0;
#pragma unroll
  for (int k0 = 0; k0 < 2; k0 += KB) {
    KFrag x[KB][KF];
#pragma unroll
    for (int b = 0; b < KB; ++b)
#pragma unroll
      for (int cc = 0; cc < KF; ++cc)
        x[b][cc] = *lds_at<const KFrag>((kaddr ^ (64 * cc)) + 16 * C::ROW * (k0 + b));
    if (k0 == 0) here = there();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < KB; ++b) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[k0 + b][nt] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        V8 f;
        if constexpr (E4M3) f = widen8<BF16>(x[b][ks >> 1][2 * (ks & 1)], x[b][ks >> 1][2 * (ks & 1) + 1]);
        else f = x[b][ks];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[k0 + b][nt] = mfma(f, o.q[nt][ks], s[k0 + b][nt]);
      }
    }
  }
  scored();

  // The keys of the tile that the lane's row sees.
  auto seen_by = [&](int nt) -> uint32_t {
    uint32_t bits = here;
    if constexpr (DRAFTED) {
      const int r = 16 * nt + col;
      const int token = (at.first + r) / at.group;   // in its request
      if (r >= at.count) {
        bits = 0;
      } else if (a.tree_mask) {
        const uint64_t* words = a.tree_mask + (static_cast<int64_t>(at.start) + token) * a.mask_words;
        const int w = idx < 0 ? 0 : idx >> 6;
        uint64_t m = w < a.mask_words ? words[w] : 0;
        if (idx < 0) {
          m = (m << -idx) | ((uint64_t{1} << -idx) - 1);
        } else {
          const int sh = idx & 63;
          m >>= sh;
          if (sh > 32 && w + 1 < a.mask_words) m |= words[w + 1] << (64 - sh);
        }
        bits &= static_cast<uint32_t>(m);
      } else {
        const int vis = token - idx + 1;   // keys of the tile up to the token
        bits &= vis >= 32 ? 0xFFFFFFFFu : vis <= 0 ? 0u : (1u << vis) - 1;
      }
    }
    return bits;
  };
  // Unseen keys score -infinity.
  if (DRAFTED || here != 0xFFFFFFFFu) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t bits = seen_by(nt);
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((bits >> (16 * kt + 4 * g + e)) & 1)) s[kt][nt][e] = -INFINITY;
    }
  }

  // Scores are rounded after the scale, and a weight's exponent is the rounded
  // score minus the reference.  With a fused multiply-add (131K context 136.2
  // us, this 137.4; trees of 13-64 tokens 74.9, this 75.1) the score would not
  // be the one that the reference was taken from: beyond 2^27 they differ by
  // more than the lift and the slack, and the weight of a row's largest score
  // would be infinite or zero.
  bool raise = false;
  float top[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    s[0][nt] *= o.c;
    s[1][nt] *= o.c;
    float m = fmaxf(s[0][nt][0], s[1][nt][0]);
#pragma unroll
    for (int e = 1; e < 4; ++e) m = fmaxf(m, fmaxf(s[0][nt][e], s[1][nt][e]));
    top[nt] = m;
    raise |= m > o.ref[nt] + kSlack;
  }
  if (__any(raise)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float m = top[nt];
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      m = fmaxf(m - kLift, o.ref[nt]);
      const float r = __builtin_amdgcn_exp2f(o.ref[nt] - m);
      o.ref[nt] = m;
      o.sum[nt] *= r;
#pragma unroll
      for (int d = 0; d < DT; ++d) o.acc[nt][d] *= r;
    }
  }
  need_values();
  bool odd = false;
  if constexpr (DRAFTED) {
    // A value that overflowed may be one that some rows must not see, and
    // 0 * infinity would reach them through the product below.
    uint32_t bad = 0;
#pragma unroll
    for (int x = 0; x < C::CP; ++x) {
      const u32x4 y = *reinterpret_cast<const u32x4*>(vals + 1024 * x + 16 * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (E4M3) {
          const uint32_t n = ~(y[e] | 0x80808080u);   // a zero byte for a NaN
          bad |= (n - 0x01010101u) & ~n & 0x80808080u;
        } else {
          constexpr uint32_t E = BF16 ? 0x7F80u : 0x7C00u;
          bad |= (y[e] & E) == E || ((y[e] >> 16) & E) == E;
        }
      }
    }
    odd = __any(bad != 0);
  }
  // Half of the values are read before the weights are worked out and half
  // before the first half's products, so that the reads hide behind those.
  constexpr int HT = DT / 2;
  using Frag = typename std::conditional<E4M3, int2v, V8>::type;
  // 8-bit: lanes 2r, 2r + 1 of a group point at key r of its eight; 16-bit:
  // lanes 4r .. 4r + 3 at key r of its four.
  const int vk = E4M3 ? (col & 8 ? 16 : 0) + 4 * g + (col >> 1 & 3) : 4 * g + (col >> 2);
  const uint32_t vaddr = lds_addr(vals) + (C::ROW * vk + 8 * (col & 1) +
                                           16 * ((E4M3 ? 0 : col >> 1 & 1) ^ C::vswz(vk)));
  auto read_values = [&](int d) -> Frag {
    if constexpr (E4M3) {
      return __builtin_amdgcn_ds_read_tr8_b64_v2i32(lds_at<int2v>(vaddr ^ (16 * d)));
    } else {
      union {
        short4v p[2];
        V8 v;
      } x;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        x.p[h] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            lds_at<short4v>((vaddr ^ (32 * d)) + 16 * h * C::ROW));
      return x.v;
    }
  };
  Frag f[HT];
#pragma unroll
  for (int d = 0; d < HT; ++d) f[d] = read_values(d);
  __builtin_amdgcn_sched_barrier(0);
  V8 w[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int kt = 0; kt < 2; ++kt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma clang fp contract(off)
        const float x = __builtin_amdgcn_exp2f(s[kt][nt][e] - o.ref[nt]);
        o.sum[nt] += x;
        w[nt][4 * kt + e] = static_cast<T>(x);
      }
  }
  if (!DRAFTED || !odd) {
    auto product = [&](Frag y, int d) {
      V8 x;
      if constexpr (E4M3) x = widen8<BF16>(y[0], y[1]);
      else x = y;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) o.acc[nt][d] = mfma(x, w[nt], o.acc[nt][d]);
    };
    Frag f2[HT];
#pragma unroll
    for (int d = 0; d < HT; ++d) f2[d] = read_values(HT + d);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int d = 0; d < HT; ++d) product(f[d], d);
    used();
#pragma unroll
    for (int d = 0; d < HT; ++d) product(f2[d], HT + d);
  } else {
    // Key by key, for the rows that see it; the weights of 16 rows at a
    // time (-1: not seen) go through LDS.
    T* ws = reinterpret_cast<T*>(spare);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      wait_lds_reads();
      const uint32_t bits = seen_by(nt);   // a key that is seen may score -infinity, too
#pragma unroll
      for (int kt = 0; kt < 2; ++kt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          ws[16 * (16 * kt + 4 * g + e) + col] =
              bits >> (16 * kt + 4 * g + e) & 1 ? w[nt][4 * kt + e] : static_cast<T>(-1.f);
#pragma unroll 1
      for (int k = 0; k < kTile; ++k) {
        const float x = static_cast<float>(ws[16 * k + col]);
        if (x < 0.f) continue;   // false for NaN
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          // Channels 16 d + 4 g .. + 3 of key k.
          const int byte = (16 * d + 4 * g) * C::ES;
          const char* from = vals + C::ROW * k + 16 * ((byte >> 4) ^ C::vswz(k)) + (byte & 15);
          float v[4];
          if constexpr (E4M3) {
            const uint32_t y = *reinterpret_cast<const uint32_t*>(from);
            v[0] = __builtin_amdgcn_cvt_f32_fp8(y, 0);
            v[1] = __builtin_amdgcn_cvt_f32_fp8(y, 1);
            v[2] = __builtin_amdgcn_cvt_f32_fp8(y, 2);
            v[3] = __builtin_amdgcn_cvt_f32_fp8(y, 3);
          } else {
            const T* y = reinterpret_cast<const T*>(from);
#pragma unroll
            for (int z = 0; z < 4; ++z) v[z] = static_cast<float>(y[z]);
          }
#pragma unroll
          for (int z = 0; z < 4; ++z) o.acc[nt][d][z] = __builtin_fmaf(x, v[z], o.acc[nt][d][z]);
        }
      }
    }
    used();
  }
}

// A team's units: [u0, u1) of `total`, the first in request b, whose units
// start at `base`; `team` is its number among the `active` ones, -1 for none.
// `self` is the work-group's number among those of all teams, `hk` its key
// head.  `scan`: LDS, THREADS / 64 + 2 words.
struct Share {
  int64_t u0, u1, base, total;
  int b, team, active, self, hk;
};
template <int R, int THREADS>
__device__ __forceinline__ Share find_share(const AttentionLaunch& p, int64_t* scan) {
  const AttentionArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Share o{};
  const int per = (a.B + THREADS - 1) / THREADS;
  const int b0 = min(tid * per, a.B), b1 = min(b0 + per, a.B);
  int64_t mine = 0;
  for (int i = b0; i < b1; ++i) mine += span_of<R>(p, i).all;
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  if (lane == 63) scan[wave] = sum;
  __syncthreads();
  int64_t before = sum - mine;
#pragma unroll
  for (int w = 0; w < THREADS / 64; ++w) {
    before += w < wave ? scan[w] : 0;
    o.total += scan[w];
  }
  // Neighbouring shares go to one XCD: row blocks of the same keys lie next
  // to each other and meet in its L2.
  o.active = static_cast<int>(o.total < p.teams ? o.total : p.teams);
  const int heads = static_cast<int>(a.cache.heads), groups = o.active * heads;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int even = groups >> 3, odd = groups & 7;
  o.team = -1;
  if (slot < even + (xcd < odd)) {
    o.self = xcd * even + min(xcd, odd) + slot;
    if (p.team_step == 1) {
      o.hk = o.self / o.active;
      o.team = o.self - o.hk * o.active;
    } else {
      o.team = o.self / heads;
      o.hk = o.self - o.team * heads;
    }
    o.u0 = o.total * o.team / o.active;
    o.u1 = o.total * (o.team + 1) / o.active;
    if (o.u0 >= before && o.u0 < before + mine) {
      int i = b0;
      for (;;) {
        const int64_t all = span_of<R>(p, i).all;
        if (o.u0 < before + all) break;
        before += all;
        ++i;
      }
      scan[THREADS / 64] = i;
      scan[THREADS / 64 + 1] = before;
    }
  }
  __syncthreads();
  o.b = static_cast<int>(scan[THREADS / 64]);
  o.base = scan[THREADS / 64 + 1];
  if (blockIdx.x == 0 && tid == 0) p.owners[kOwnerWords * kAttentionGroups] = p.teams > 1 ? groups : 0;
  return o;
}

// Zeros for the rows of no request.
__device__ __forceinline__ void clear_foreign_rows(const AttentionArgs& a, int head_dim) {
  const int first = min(max(a.q_start[0], 0), a.T), last = min(max(a.q_start[a.B], 0), a.T);
  const int64_t row = static_cast<int64_t>(a.heads) * head_dim / 8;
  u32x4* out = static_cast<u32x4*>(a.out);
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (int64_t i = i0; i < first * row; i += step) out[i] = u32x4{0u, 0u, 0u, 0u};
  for (int64_t i = last * row + i0; i < a.T * row; i += step) out[i] = u32x4{0u, 0u, 0u, 0u};
}

// The run of units from u on that lies in one row block.
struct Segment {
  int first, rows;             // first row and rows of the row block
  int kbeg, kend, units;       // keys; units of the run
  bool starts, ends;           // whether it holds the row block's first and last unit
};
template <int R>
__device__ __forceinline__ Segment segment_at(const AttentionLaunch& p, const Share& w, const Span& sp,
                                              int64_t u) {
  Segment o;
  const int64_t at = u - w.base, left = w.u1 - u;
  const int seg = static_cast<int>(at / sp.units);
  const int ku = static_cast<int>(at - static_cast<int64_t>(seg) * sp.units);
  o.first = seg * R;
  o.rows = min(R, sp.n * p.group - o.first);
  o.units = static_cast<int>(left < sp.units - ku ? left : sp.units - ku);
  o.starts = ku == 0;
  o.ends = ku + o.units == sp.units;
  o.kbeg = ku * kUnit;
  o.kend = o.ends ? sp.L : (ku + o.units) * kUnit;
  return o;
}

// How many work-groups hold units of the row block that starts at u in this
// one's last run; leaves for attention_combine_kernel where its rows are.
__device__ __forceinline__ int own_row_block(const AttentionLaunch& p, const Share& w, const Span& sp,
                                             const Segment& sg, int64_t u) {
  // The one that holds its last unit: the largest x with total * x / active
  // <= last.
  const int64_t last = u + sp.units - 1;
  const int x = static_cast<int>(((last + 1) * w.active - 1) / w.total);   // a team
  if (threadIdx.x == 0) {
    int32_t* o = p.owners + kOwnerWords * w.self;
    o[1] = sp.start;
    o[2] = w.hk;
    o[3] = sg.first;
    o[4] = sg.rows;
    o[5] = w.b;
  }
  return x - w.team + 1;
}

// What a row's weighted values are multiplied by: the values' scale over the
// sum of the weights.  The sum is 0 (otherwise 1 or more) where token i of
// request b sees no key, and the row then is 0, or where every key that it
// sees scores -infinity, whose softmax is NaN: which of the two is looked up
// for such a row alone, since keeping it through the tiles costs (trees of
// 13-64 tokens 74.9 -> 76.4 us).
__device__ __forceinline__ float quotient(const AttentionLaunch& p, int b, int i, int hk, float sum) {
  const AttentionArgs& a = p.a;
  if (sum == 0.f) {
    const Span sp = span_of<16>(p, b);
    const int32_t* table = a.block_table + b * a.table_stride;
    auto there = [&](uint32_t j) {
      const int page = table[divide(j, p)];
      return page >= 0 && page < static_cast<int>(a.cache.num_blocks);
    };
    const int context = min(sp.cached, sp.L), block = static_cast<int>(a.cache.block_size);
    bool seen = false;
#pragma unroll 8
    for (int64_t j = 0; j < context; j += block) seen |= there(static_cast<uint32_t>(j));
    const uint64_t* words = a.tree_mask ? a.tree_mask + (int64_t{sp.start} + i) * a.mask_words : nullptr;
    for (int x = 0; x < sp.L - context && !seen; ++x) {
      const bool bit = words ? (x >> 6) < a.mask_words && (words[x >> 6] >> (x & 63) & 1) : x <= i;
      seen = bit && there(static_cast<uint32_t>(context + x));
    }
    return seen ? NAN : 0.f;
  }
  return (a.cache.v_scale ? static_cast<const float*>(a.cache.v_scale)[hk] : 1.f) / sum;
}

// Four channels of a row whose sums over the run's keys are `o`, its
// reference and weight `st`: the output, or a part of it.
template <bool BF16, int D, int R>
__device__ __forceinline__ void put_row(const AttentionLaunch& p, const Share& w, const Span& sp,
                                        const Segment& sg, int row, int ch, floatx4 o, RowStat st) {
  using T = typename Act<BF16>::T;
  if (sg.starts && sg.ends) {
    const int r = sg.first + row, i = r / p.group, h = w.hk * p.group + (r - i * p.group);
    const float inv = quotient(p, w.b, i, w.hk, st.sum);
    T* to = static_cast<T*>(p.a.out) + (static_cast<int64_t>(sp.start + i) * p.a.heads + h) * D + ch;
    union {
      T t[4];
      u32x2 v;
    } y;
#pragma unroll
    for (int z = 0; z < 4; ++z) y.t[z] = static_cast<T>(o[z] * inv);
    *reinterpret_cast<u32x2*>(to) = y.v;
  } else {
    const int64_t slot = static_cast<int64_t>(sg.starts ? 2 * w.self + 1 : 2 * w.self) * R + row;
    *reinterpret_cast<floatx4*>(p.sums + slot * D + ch) = o;
    if (ch == 0) p.stats[slot] = st;
  }
}

// Joins the sums of WAVES waves, each over its own keys: wave x has the rows
// 16 NT (x % split) .. of the row block, the waves x, x + split, ... the same
// rows.  PASS row tiles of every wave at a time, through `red` (WAVES * 16
// PASS * D floats); `stat`: WAVES * 16 NT entries.
template <bool BF16, int D, int NT, int WAVES, int R, int PASS>
__device__ __forceinline__ void merge_waves(const AttentionLaunch& p, const Share& w, const Span& sp,
                                            const Segment& sg, Rows<BF16, D, NT>& o, int split,
                                            float* red, RowStat* stat) {
  constexpr int W = 16 * NT, PR = D / 4, H = 16 * PASS;   // rows of a wave; pieces of a row; rows at a time
  const int tid = fresh(threadIdx.x), col = tid & 15, g = (tid & 63) >> 4;
  const int wave = uniform(tid >> 6), mine = wave % split;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    o.sum[nt] += __shfl_xor(o.sum[nt], 16);
    o.sum[nt] += __shfl_xor(o.sum[nt], 32);
    if (g == 0) stat[wave * W + 16 * nt + col] = RowStat{o.ref[nt], o.sum[nt]};
  }
  __syncthreads();   // every wave is done with the buffers that `red` overlays
#pragma unroll
  for (int n0 = 0; n0 < NT; n0 += PASS) {
#pragma unroll
    for (int q = 0; q < PASS; ++q) {
      float m = -FLT_MAX;
      for (int x = mine; x < WAVES; x += split) m = fmaxf(m, stat[x * W + 16 * (n0 + q) + col].ref);
      const float r = __builtin_amdgcn_exp2f(o.ref[n0 + q] - m);
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
        *reinterpret_cast<floatx4*>(red + (wave * H + 16 * q + col) * D + 4 * ((4 * d + g) ^ col)) =
            o.acc[n0 + q][d] * r;
    }
    __syncthreads();
    for (int x = tid; x < split * H * PR; x += 64 * WAVES) {
      const int rw = x / (H * PR), rr = x / PR & (H - 1), pc = x & (PR - 1);
      const int row = W * rw + 16 * n0 + rr;
      if (row >= sg.rows) continue;
      const float* from = red + (rw * H + rr) * D + 4 * (pc ^ (rr & 15));
      floatx4 y = *reinterpret_cast<const floatx4*>(from);
      const RowStat* st = stat + rw * W + 16 * n0 + rr;
      RowStat t{st->ref, 0.f};
      for (int z = split; z < WAVES; z += split) {
        y += *reinterpret_cast<const floatx4*>(from + z * H * D);
        t.ref = fmaxf(t.ref, st[z * W].ref);
      }
      for (int z = 0; z < WAVES; z += split)
        t.sum += st[z * W].sum * __builtin_amdgcn_exp2f(st[z * W].ref - t.ref);
      put_row<BF16, D, R>(p, w, sp, sg, row, 4 * pc, y, t);
    }
    __syncthreads();
  }
}

// The addresses of keys, in LDS: base and strides, in bytes, of keys (0-2) and
// values (3-5) of a head.  (Registers would hold them for every lane.)
__device__ __forceinline__ void put_strides(const awq_kv_cache& c, int hk, int es, int64_t* to) {
  const int lane = fresh(threadIdx.x & 63);
  if (lane < 2) {
    to[3 * lane] = reinterpret_cast<int64_t>(lane ? c.v : c.k) +
                   static_cast<int64_t>(es) * hk * (lane ? c.v_head_stride : c.k_head_stride);
    to[3 * lane + 1] = es * (lane ? c.v_block_stride : c.k_block_stride);
    to[3 * lane + 2] = es * (lane ? c.v_slot_stride : c.k_slot_stride);
  }
}

// Groups of GROUP consecutive keys that never cross a page's end: 64 of them
// are looked up at once, one by each lane, and a group's copies then need an
// address of the wave and one instruction per lane.  (Looking up every key in
// its tile took a quarter of the instructions of a step.)
template <int GROUP>
struct Groups {
  uint32_t klo, khi, vlo, vhi;   // of the lane's group: its first key and value
  uint64_t some, full;           // groups with a page; with GROUP keys below L
  __device__ __forceinline__ void look_up(const AttentionLaunch& p, const int32_t* table, int hk, int es,
                                          uint32_t key, int L) {
    const awq_kv_cache& c = p.a.cache;
    const uint32_t e = divide(min(key, static_cast<uint32_t>(L - 1)), p);
    const int page = table[e];
    const bool ok = key < static_cast<uint32_t>(L) && page >= 0 && page < static_cast<int>(c.num_blocks);
    some = __ballot(ok);
    full = __ballot(ok && key + GROUP <= static_cast<uint32_t>(L));
    const int64_t n = ok ? page : 0, off = ok ? key - e * static_cast<uint32_t>(c.block_size) : 0;
    const uint64_t k = reinterpret_cast<uint64_t>(c.k) +
                       es * (hk * c.k_head_stride + n * c.k_block_stride + off * c.k_slot_stride);
    const uint64_t v = reinterpret_cast<uint64_t>(c.v) +
                       es * (hk * c.v_head_stride + n * c.v_block_stride + off * c.v_slot_stride);
    klo = static_cast<uint32_t>(k);
    khi = static_cast<uint32_t>(k >> 32);
    vlo = static_cast<uint32_t>(v);
    vhi = static_cast<uint32_t>(v >> 32);
  }
  __device__ __forceinline__ uint64_t keys(int l) const {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(klo, l)) |
           static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(khi, l))) << 32;
  }
  __device__ __forceinline__ uint64_t values(int l) const {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(vlo, l)) |
           static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(vhi, l))) << 32;
  }
  // How many of the keys of group l, whose first is `key`, there are.
  __device__ __forceinline__ int count(int l, int key, int L) const {
    return full >> l & 1 ? GROUP : some >> l & 1 ? min(L - key, GROUP) : 0;
  }
};

// ------------------------------------------------ up to 32 rows: a wave has keys of its own
template <bool BF16, bool E4M3, int D, int NT>
__global__ __launch_bounds__(kThreads, (Shape<E4M3, D, NT>::OCC)) void attention_kernel(
    AttentionLaunch p) {
  using C = Shape<E4M3, D, NT>;
  constexpr int S = C::STG;
  const AttentionArgs& a = p.a;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int wave = uniform(static_cast<int>(threadIdx.x >> 6));
  Share w = find_share<C::R, kThreads>(p, reinterpret_cast<int64_t*>(smem + C::SCAN));
  clear_foreign_rows(a, D);
  if (w.team < 0) return;
  w.b = uniform(w.b);

  char* kbuf = smem + wave * C::WAVE;
  char* vbuf = kbuf + S * C::TILE;
  const uint32_t klds = uniform(lds_addr(kbuf)), vlds = uniform(lds_addr(vbuf));
  const uint32_t tlds = uniform(lds_addr(smem + C::TAB + wave * C::TABW));
  const int* tab = reinterpret_cast<const int*>(smem + C::TAB + wave * C::TABW);
  uint64_t* adr = reinterpret_cast<uint64_t*>(smem + C::ADR + wave * 512);
  int64_t* strides = reinterpret_cast<int64_t*>(smem + C::STRD + wave * 64);
  int owner_parts = 0;

  for (int64_t u = w.u0; u < w.u1;) {
    Span sp = span_of<C::R>(p, w.b);
    while (u - w.base >= sp.all) {   // requests without rows have no units
      w.base += sp.all;
      sp = span_of<C::R>(p, ++w.b);
    }
    const Segment sg = segment_at<C::R>(p, w, sp, u);
    const int L = sp.L;
    // Tiles of this wave: keys kbeg + 32 (wave + 4 i).
    const int span32 = sg.kend - sg.kbeg - kTile * wave;
    const int tiles = span32 > 0 ? (span32 - 1) / kUnit + 1 : 0;

    const int32_t* table = a.block_table + w.b * a.table_stride;
    auto key_of = [&](int i) {
      return static_cast<uint32_t>(sg.kbeg + kTile * (wave + kWaves * i)) + fresh(threadIdx.x & 31);
    };
    auto fetch_blocks = [&](int i) {
      const uint32_t j = min(key_of(i), static_cast<uint32_t>(L - 1));
      copy4(reinterpret_cast<uint64_t>(table + divide(j, p)), tlds + 256 * (i & (2 * S - 1)));
    };
    // Addresses of a tile's keys (lanes 0-31) and values (lanes 32-63), or
    // of the zero row; returns which of its keys there are.
    put_strides(a.cache, w.hk, C::ES, strides);
    auto make_addresses = [&](int i) -> uint32_t {
      const int lane = fresh(threadIdx.x & 63);
      const int page = tab[64 * (i & (2 * S - 1)) + lane];
      const int64_t* from = strides + 3 * (lane >> 5);
      const uint32_t j = key_of(i);
      const bool ok = j < static_cast<uint32_t>(L) && page >= 0 && page < static_cast<int>(a.cache.num_blocks);
      const uint32_t off = j - divide(j, p) * static_cast<uint32_t>(a.cache.block_size);
      const uint64_t to = from[0] + page * from[1] + off * from[2];
      adr[lane] = ok ? to : reinterpret_cast<uint64_t>(kZeroRow);
      return static_cast<uint32_t>(__ballot(ok));
    };
    auto copy_keys = [&](int i) {
      const int lane = fresh(threadIdx.x & 63);
      const uint32_t to = klds + C::TILE * (i & (S - 1));
      uint64_t from[C::CP];
#pragma unroll
      for (int c = 0; c < C::CP; ++c) {
        const int k = c * (64 / C::P) + lane / C::P;
        from[c] = adr[k] + 16 * ((lane & (C::P - 1)) ^ C::kswz(k));
      }
#pragma unroll
      for (int c = 0; c < C::CP; ++c) copy16(from[c], to + 1024 * c);
    };
    auto copy_values = [&](int i) {
      const int lane = fresh(threadIdx.x & 63);
      const uint32_t to = vlds + C::TILE * (i & (S - 1));
      uint64_t from[C::CP];
#pragma unroll
      for (int c = 0; c < C::CP; ++c) {
        const int k = c * (64 / C::P) + lane / C::P;
        from[c] = adr[32 + k] + 16 * ((lane & (C::P - 1)) ^ C::vswz(k));
      }
#pragma unroll
      for (int c = 0; c < C::CP; ++c) copy16(from[c], to + 1024 * c);
    };

#pragma unroll
    for (int s = 0; s < S; ++s) fetch_blocks(s);
    const Place at{sp.start, sg.first, sg.rows, p.group};
    Rows<BF16, D, NT> rows;
    load_rows<BF16, E4M3, D, NT>(a, at, w.hk, rows);
    uint32_t there[S];   // keys there are, of the tiles in flight
    wait_copies<0>();
#pragma unroll
    for (int s = 0; s < S; ++s) {
      there[s] = 0;
      if (s < tiles) {
        fetch_blocks(s + S);
        there[s] = make_addresses(s);
        copy_keys(s);
        copy_values(s);
      }
    }

    auto step = [&](auto drafted, int i) {
      constexpr bool DRAFTED = decltype(drafted)::value;
      const bool more = i + S < tiles;
      const uint32_t here = there[0];
#pragma unroll
      for (int s = 0; s + 1 < S; ++s) there[s] = there[s + 1];
      if (more) wait_copies<C::CP + (S - 1) * (2 * C::CP + 1)>();
      else wait_copies<0>();
      auto next_keys = [&] {
        wait_lds_reads();
        fetch_blocks(i + 2 * S);
        there[S - 1] = make_addresses(i + S);
        copy_keys(i + S);
      };
      // A tile with drafted keys may need the keys' buffer until its end.
      char* keys = kbuf + C::TILE * (i & (S - 1));
      tile_step<DRAFTED, BF16, E4M3, D, NT>(
          a, at, rows, keys, vbuf + C::TILE * (i & (S - 1)), keys, [&] { return here; },
          sg.kbeg + kTile * (wave + kWaves * i) - sp.cached,
          [&] {
            if (!DRAFTED && more) next_keys();
          },
          [&] {
            if (!DRAFTED && more) wait_copies<(S - 1) * (2 * C::CP + 1) + 1 + C::CP>();
            else wait_copies<0>();
          },
          [&] {
            if (!more) return;
            if (DRAFTED) next_keys();
            wait_lds_reads();
            copy_values(i + S);
          });
    };
    // Tiles of the context alone come first.
    const int context = sp.cached - sg.kbeg - kTile * wave;
    const int plain = min(tiles, context >= kTile ? (context - kTile) / kUnit + 1 : 0);
    int i = 0;
    for (; i < plain; ++i) step(std::false_type{}, i);
    for (; i < tiles; ++i) step(std::true_type{}, i);
    merge_waves<BF16, D, NT, kWaves, C::R, C::PASS>(p, w, sp, sg, rows, 1, reinterpret_cast<float*>(smem),
                                           reinterpret_cast<RowStat*>(smem + C::STAT));
    if (sg.starts && !sg.ends) owner_parts = own_row_block(p, w, sp, sg, u);
    u += sg.units;
  }
  if (threadIdx.x == 0 && p.teams > 1) p.owners[kOwnerWords * w.self] = owner_parts;
}

// ------------------------------------------------ more rows: the waves share the keys
// Eight waves, one work-group per CU.  A step is `STEP` keys, copied by all
// waves and used by all: wave x takes the rows W (x % split) .. and of the
// tiles every (8 / split)th, split = 4 (2 when the row block has at most 2 W
// rows).  One barrier a step: behind it the copies of a later step go into
// the buffer that the last step has left.  The waves of a SIMD are x and
// x + 4; the upper ones ask for their copies after their tile, so that one of
// the two is computing while the other works out addresses.
template <bool E4M3, int D>
struct Wide {
  static constexpr int NT = D > 128 ? 1 : 2;       // row tiles of a wave
  static constexpr int W = 16 * NT, R = 4 * W;
  using C = Shape<E4M3, D, NT>;
  static constexpr int STEP = C::ROW >= 128 ? 64 : 128;
  static constexpr int KEYS = STEP / 8;            // that a wave copies
  static constexpr int CP = KEYS * C::ROW / 1024;  // copies, of its keys as of its values
  static constexpr int HALF = STEP * C::ROW;       // bytes of the keys (values) of a step
  static constexpr int STAGES = 8 * HALF <= 131072 ? 4 : 2;
  static constexpr int AHEAD = STAGES - 1;         // steps in flight behind the one in use
  static constexpr int BUF = 2 * STAGES * HALF;
  static constexpr int MERGE = 8 * W * D * 4;
  static constexpr int SPARE = BUF > MERGE ? BUF : MERGE;
  static constexpr int TAB = SPARE + 8 * 1024;     // block numbers: a ring of STAGES a wave
  static constexpr int TABW = STAGES * 256;
  static constexpr int ADR = TAB + 8 * TABW;
  static constexpr int STAT = ADR + 8 * 256;
  static constexpr int STRD = STAT + 8 * W * 8;
  static constexpr int HERE = STRD + 8 * 64;       // keys there are, of each stage
  static constexpr int SCAN = HERE + STAGES * 16;
  static constexpr int LDS = SCAN + 128;
  static_assert(CP >= 1 && LDS <= 163840, "copies of 1 KB; LDS of a CU");
  static_assert((AHEAD - 1) * (2 * CP + 1) < 64, "six-bit counter");
};
constexpr int kWideThreads = 512;

template <bool BF16, bool E4M3, int D>
__global__ __launch_bounds__(kWideThreads, 2) void attention_wide_kernel(AttentionLaunch p) {
  using Z = Wide<E4M3, D>;
  using C = typename Z::C;
  constexpr int NT = Z::NT;
  const AttentionArgs& a = p.a;
  extern __shared__ __attribute__((aligned(16))) char smem[];
  const int wave = uniform(static_cast<int>(threadIdx.x >> 6));
  Share w = find_share<Z::R, kWideThreads>(p, reinterpret_cast<int64_t*>(smem + Z::SCAN));
  clear_foreign_rows(a, D);
  if (w.team < 0) return;
  w.b = uniform(w.b);

  const uint32_t lds = uniform(lds_addr(smem));
  const bool whole = p.near_slots && a.cache.block_size % Z::KEYS == 0;
  const uint32_t tlds = lds + Z::TAB + wave * Z::TABW;
  const int* tab = reinterpret_cast<const int*>(smem + Z::TAB + wave * Z::TABW);
  uint64_t* adr = reinterpret_cast<uint64_t*>(smem + Z::ADR + wave * 256);
  int64_t* strides = reinterpret_cast<int64_t*>(smem + Z::STRD + wave * 64);
  int owner_parts = 0;

  for (int64_t u = w.u0; u < w.u1;) {
    Span sp = span_of<Z::R>(p, w.b);
    while (u - w.base >= sp.all) {
      w.base += sp.all;
      sp = span_of<Z::R>(p, ++w.b);
    }
    const Segment sg = segment_at<Z::R>(p, w, sp, u);
    const int L = sp.L;
    const int steps = (sg.kend - sg.kbeg - 1) / Z::STEP + 1;
    const int split = sg.rows <= 2 * Z::W ? 2 : 4;
    const int rw = wave % split, kw = wave / split;

    // This wave's keys of step i: kbeg + STEP i + KEYS wave + 0 ..
    const int32_t* table = a.block_table + w.b * a.table_stride;
    auto key_of = [&](int i) {
      return static_cast<uint32_t>(sg.kbeg + Z::STEP * i + Z::KEYS * wave) + fresh(threadIdx.x & (Z::KEYS - 1));
    };
    auto fetch_blocks = [&](int i) {
      const uint32_t j = min(key_of(i), static_cast<uint32_t>(L - 1));
      copy4(reinterpret_cast<uint64_t>(table + divide(j, p)), tlds + 256 * (i & (Z::STAGES - 1)));
    };
    put_strides(a.cache, w.hk, C::ES, strides);
    Groups<Z::KEYS> groups;
    auto copy_group = [&](int i) {
      const int lane = fresh(threadIdx.x & 63), stage = i & (Z::STAGES - 1), l = i & 63;
      const int first = sg.kbeg + Z::STEP * i + Z::KEYS * wave;
      if (l == 0)
        groups.look_up(p, table, w.hk, C::ES, static_cast<uint32_t>(first) + Z::STEP * lane, L);
      const uint64_t ka = groups.keys(l), va = groups.values(l);
      const int there = groups.count(l, first, L);
      const uint32_t kto = lds + 2 * Z::HALF * stage + wave * Z::KEYS * C::ROW;
      const int k = lane / C::P, piece = lane & (C::P - 1);   // of the first copy
      const uint32_t kstep = C::ES * static_cast<uint32_t>(a.cache.k_slot_stride);
      const uint32_t vstep = C::ES * static_cast<uint32_t>(a.cache.v_slot_stride);
      uint32_t koff[Z::CP], voff[Z::CP];
#pragma unroll
      for (int c = 0; c < Z::CP; ++c) {
        const int kc = (Z::KEYS * wave & 31) + c * (64 / C::P);   // swizzles are linear
        koff[c] = (16 * (piece ^ C::kswz(k)) ^ 16 * C::kswz(kc)) + k * kstep;
        voff[c] = (16 * (piece ^ C::vswz(k)) ^ 16 * C::vswz(kc)) + k * vstep;
      }
      if (there == Z::KEYS) {
#pragma unroll
        for (int c = 0; c < Z::CP; ++c)
          copy16(ka + c * (64 / C::P) * static_cast<uint64_t>(kstep), koff[c], kto + 1024 * c);
#pragma unroll
        for (int c = 0; c < Z::CP; ++c)
          copy16(va + c * (64 / C::P) * static_cast<uint64_t>(vstep), voff[c], kto + Z::HALF + 1024 * c);
      } else {
        uint64_t kfrom[Z::CP], vfrom[Z::CP];
#pragma unroll
        for (int c = 0; c < Z::CP; ++c) {
          const bool ok = c * (64 / C::P) + k < there;
          const uint64_t none = reinterpret_cast<uint64_t>(kZeroRow) + 16 * piece;
          kfrom[c] = ok ? ka + c * (64 / C::P) * static_cast<uint64_t>(kstep) + koff[c] : none;
          vfrom[c] = ok ? va + c * (64 / C::P) * static_cast<uint64_t>(vstep) + voff[c] : none;
        }
#pragma unroll
        for (int c = 0; c < Z::CP; ++c) copy16(kfrom[c], kto + 1024 * c);
#pragma unroll
        for (int c = 0; c < Z::CP; ++c) copy16(vfrom[c], kto + Z::HALF + 1024 * c);
      }
      if (lane == 0) {
        char* h = smem + Z::HERE + 16 * stage;
        const uint32_t bits = (1u << there) - 1;
        if constexpr (Z::KEYS == 16) reinterpret_cast<uint16_t*>(h)[wave] = bits;
        else reinterpret_cast<uint8_t*>(h)[wave] = bits;
      }
    };
    // The same for pages that may end inside a wave's keys: key by key.
    auto copy_step = [&](int i) {
      if (whole) {
        copy_group(i);
        return;
      }
      const int lane = fresh(threadIdx.x & 63), stage = i & (Z::STAGES - 1);
      // Addresses: lanes 0 .. KEYS - 1 of the keys, the next KEYS of the values.
      const int page = tab[64 * stage + lane];
      const int64_t* from = strides + 3 * (lane / Z::KEYS & 1);
      const uint32_t j = key_of(i);
      const bool ok = j < static_cast<uint32_t>(L) && page >= 0 && page < static_cast<int>(a.cache.num_blocks);
      const uint32_t off = j - divide(j, p) * static_cast<uint32_t>(a.cache.block_size);
      const uint64_t to = from[0] + page * from[1] + off * from[2];
      if (lane < 2 * Z::KEYS) adr[lane] = ok ? to : reinterpret_cast<uint64_t>(kZeroRow);
      const uint64_t here = __ballot(ok);
      if (lane == 0) {
        char* h = smem + Z::HERE + 16 * stage;
        if constexpr (Z::KEYS == 16) reinterpret_cast<uint16_t*>(h)[wave] = here;
        else reinterpret_cast<uint8_t*>(h)[wave] = here;
      }
      fetch_blocks(i + Z::AHEAD);
      const uint32_t kto = lds + 2 * Z::HALF * stage + wave * Z::KEYS * C::ROW;
      uint64_t kfrom[Z::CP], vfrom[Z::CP];
#pragma unroll
      for (int c = 0; c < Z::CP; ++c) {
        const int k = c * (64 / C::P) + lane / C::P, kk = (Z::KEYS * wave & 31) + k;
        kfrom[c] = adr[k] + 16 * ((lane & (C::P - 1)) ^ C::kswz(kk));
        vfrom[c] = adr[Z::KEYS + k] + 16 * ((lane & (C::P - 1)) ^ C::vswz(kk));
      }
#pragma unroll
      for (int c = 0; c < Z::CP; ++c) copy16(kfrom[c], kto + 1024 * c);
#pragma unroll
      for (int c = 0; c < Z::CP; ++c) copy16(vfrom[c], kto + Z::HALF + 1024 * c);
    };

    if (!whole) {
#pragma unroll
      for (int i = 0; i < Z::AHEAD; ++i) fetch_blocks(i);
    }
    if (!whole) wait_copies<0>();
    for (int i = 0; i < Z::AHEAD && i < steps; ++i) copy_step(i);
    const Place at{sp.start, sg.first + Z::W * rw, sg.rows - Z::W * rw, p.group};
    Rows<BF16, D, NT> rows;
    load_rows<BF16, E4M3, D, NT>(a, at, w.hk, rows);
    for (int i = 0; i < steps; ++i) {
      if (i + Z::AHEAD > steps) wait_copies<0>();
      else if (whole) wait_copies<(Z::AHEAD - 1) * 2 * Z::CP>();
      else wait_copies<(Z::AHEAD - 1) * (2 * Z::CP + 1)>();
      wait_lds_reads();
      __builtin_amdgcn_s_barrier();
      __builtin_amdgcn_sched_barrier(0);
      const bool more = i + Z::AHEAD < steps;
      if (more && wave < 4) copy_step(i + Z::AHEAD);
      const char* keys = smem + 2 * Z::HALF * (i & (Z::STAGES - 1));
      const int tile0 = i * (Z::STEP / kTile);   // the wave's: those with tile % (8 / split) == kw
      for (int t = (kw - tile0) & (8 / split - 1); t < Z::STEP / kTile; t += 8 / split) {
        const int k0 = sg.kbeg + Z::STEP * i + kTile * t;
        if (k0 >= sg.kend || at.count <= 0) break;
        const auto* h = reinterpret_cast<const uint32_t*>(smem + Z::HERE + 16 * (i & (Z::STAGES - 1))) + t;
        auto step = [&](auto drafted) {
          tile_step<decltype(drafted)::value, BF16, E4M3, D, NT>(
              a, at, rows, keys + C::TILE * t, keys + Z::HALF + C::TILE * t,
              smem + Z::SPARE + 1024 * wave, [&] { return uniform(*h); }, k0 - sp.cached, [] {},
              [] {}, [] {});
        };
        if (k0 + kTile <= sp.cached) step(std::false_type{});
        else step(std::true_type{});
      }
      if (more && wave >= 4) copy_step(i + Z::AHEAD);
    }
    merge_waves<BF16, D, NT, 8, Z::R, NT>(p, w, sp, sg, rows, split, reinterpret_cast<float*>(smem),
                                      reinterpret_cast<RowStat*>(smem + Z::STAT));
    if (sg.starts && !sg.ends) owner_parts = own_row_block(p, w, sp, sg, u);
    u += sg.units;
  }
  if (threadIdx.x == 0 && p.teams > 1) p.owners[kOwnerWords * w.self] = owner_parts;
}

// D / 4 lanes per row of a row block that was split: joins the parts that the
// work-groups from its first on left, in their order, four channels a lane.
// The rows of a row block are neighbouring work-groups, so they spread over
// the XCDs: owners are often every 32nd work-group, and with those numbered
// fastest all of the work fell to one XCD (104 rows of 32 parts over 131K
// keys: 25.2 us).  A row is three loads that wait for each other, so what
// counts is how many rows are in flight; a wave per row, its halves taking
// every other part, is slower where row blocks have two or three parts (trees
// of 13-64 tokens: 10.5 us, this 7.2) and level where they have 32.
template <bool BF16, int D>
__global__ __launch_bounds__(kThreads) void attention_combine_kernel(AttentionLaunch p, int R) {
  using T = typename Act<BF16>::T;
  constexpr int LANES = D / 4, ROWS = kThreads / LANES;
  const AttentionArgs& a = p.a;
  const int w = blockIdx.y, lane = threadIdx.x % LANES, ch = 4 * lane;
  const int row = blockIdx.x * ROWS + threadIdx.x / LANES;
  const int32_t* o = p.owners + kOwnerWords * w;
  const int parts = o[0];
  // Entries past the work-groups that had units are another call's.
  if (w >= p.owners[kOwnerWords * kAttentionGroups] || parts == 0 || row >= o[4]) return;
  const int hk = o[2], r = o[3] + row, G = p.group;
  auto slot = [&](int x) {
    return static_cast<int64_t>(x == 0 ? 2 * w + 1 : 2 * (w + x * p.team_step)) * R + row;
  };
  float m = -FLT_MAX;
  for (int x = lane; x < parts; x += LANES) m = fmaxf(m, p.stats[slot(x)].ref);
#pragma unroll
  for (int d = 1; d < LANES; d <<= 1) m = fmaxf(m, __shfl_xor(m, d, LANES));
  float l = 0.f;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int x0 = 0; x0 < parts; x0 += LANES) {
    const int n = min(LANES, parts - x0);
    float f = 0.f, mine = 0.f;
    if (lane < n) {
      const RowStat st = p.stats[slot(x0 + lane)];
      f = __builtin_amdgcn_exp2f(st.ref - m);
      mine = st.sum * f;
    }
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) mine += __shfl_xor(mine, d, LANES);
    l += mine;
    auto add = [&](int x, auto deep) {   // `deep` parts in flight
      constexpr int N = decltype(deep)::value;
      floatx4 v[N];
#pragma unroll
      for (int j = 0; j < N; ++j)
        v[j] = *reinterpret_cast<const floatx4*>(p.sums + slot(x0 + min(x + j, n - 1)) * D + ch);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float fj = __shfl(f, x + j, LANES);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += x + j < n ? v[j][i] * fj : 0.f;
      }
    };
    if (n <= 4) add(0, std::integral_constant<int, 4>{});
    else
      for (int x = 0; x < n; x += 16) add(x, std::integral_constant<int, 16>{});
  }
  const int i = r / G, h = hk * G + (r - i * G);
  const float inv = quotient(p, o[5], i, hk, l);
  T* out = static_cast<T*>(a.out) + (static_cast<int64_t>(o[1] + i) * a.heads + h) * D + ch;
  union {
    T t[4];
    u32x2 v;
  } y;
#pragma unroll
  for (int x = 0; x < 4; ++x) y.t[x] = static_cast<T>(acc[x] * inv);
  *reinterpret_cast<u32x2*>(out) = y.v;
}

template <bool BF16, int D>
hipError_t launch_combine(const AttentionLaunch& p, int R, hipStream_t stream) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.teams == 1) return e;   // one team: every row block is whole
  const int64_t most = static_cast<int64_t>(p.a.T) * p.group;   // rows of any row block
  const int rows = static_cast<int>(most < R ? most : R);
  constexpr int per = kThreads * 4 / D;   // rows of a work-group
  hipLaunchKernelGGL((attention_combine_kernel<BF16, D>), dim3((rows + per - 1) / per, p.groups),
                     dim3(kThreads), 0, stream, p, R);
  return hipGetLastError();
}

template <bool BF16, bool E4M3, int D, int NT>
hipError_t launch_narrow(AttentionLaunch& p, hipStream_t stream) {
  using C = Shape<E4M3, D, NT>;
  static_assert(C::LDS * C::OCC <= 163840, "LDS of a CU");
  form_teams(p, 256 * C::OCC, 1);
  hipLaunchKernelGGL((attention_kernel<BF16, E4M3, D, NT>), dim3(p.groups), dim3(kThreads), C::LDS,
                     stream, p);
  return launch_combine<BF16, D>(p, C::R, stream);
}

template <bool BF16, bool E4M3, int D>
hipError_t launch_shape(AttentionLaunch& p, int rows, hipStream_t stream) {
  if (rows == 16) return launch_narrow<BF16, E4M3, D, 1>(p, stream);
  if constexpr (D <= 128)
    if (rows == 32) return launch_narrow<BF16, E4M3, D, 2>(p, stream);
  using Z = Wide<E4M3, D>;
  form_teams(p, 256, static_cast<int>(p.a.cache.heads));
  hipLaunchKernelGGL((attention_wide_kernel<BF16, E4M3, D>), dim3(p.groups), dim3(kWideThreads),
                     Z::LDS, stream, p);
  return launch_combine<BF16, D>(p, Z::R, stream);
}

template <bool BF16, bool E4M3>
hipError_t launch_dim(AttentionLaunch& p, int rows, hipStream_t stream) {
  switch (p.a.cache.head_dim) {
    case 64: return launch_shape<BF16, E4M3, 64>(p, rows, stream);
    case 128: return launch_shape<BF16, E4M3, 128>(p, rows, stream);
    default: return launch_shape<BF16, E4M3, 256>(p, rows, stream);
  }
}

}  // namespace

hipError_t launch_attention(const AttentionArgs& a, void* workspace, hipStream_t stream) {
  AttentionLaunch p = plan_attention(a, workspace);
  const int rows = attention_block_rows(a.B, a.T, a.heads, a.cache.heads, a.cache.head_dim);
  const bool e4m3 = a.cache.dtype == AWQ_E4M3;
  if (a.dtype == AWQ_BF16)
    return e4m3 ? launch_dim<true, true>(p, rows, stream) : launch_dim<true, false>(p, rows, stream);
  return e4m3 ? launch_dim<false, true>(p, rows, stream) : launch_dim<false, false>(p, rows, stream);
}

}  // namespace awq
