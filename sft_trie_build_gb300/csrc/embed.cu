// Token vectors from a table, and the table's gradient.
//
//   out[n] = scale E[tok[n]],   dE[v] = scale sum_{n : tok[n] = v} d_out[n]
//
// The forward moves bytes only: a few threads take a token, 16 bytes each.
//
// The gradient adds up rows of d_out that lie anywhere, some tokens once, some
// thousands of times, in an order that does not depend on timing:
//   embed_sort_kernel   every block takes a range of tokens out of all positions, in a
//                 fixed order, and sorts (token, position) by token, stable, in one or two
//                 passes over 9 bits or less; no block waits for another one.  It also
//                 writes zeros over the rows of its tokens that do not occur
//   embed_sum_kernel    pieces of 32 sorted entries each: a thread adds its 16 bytes of
//                 channels entry by entry.  A token that occurs 64 times at most is added up
//                 where it begins, also beyond the piece; what a piece holds of
//                 another one goes to the workspace
//   embed_join_kernel   those tokens: the sums of their pieces, in order
// Every row of d_out is read once and every row of dE written once.  Sums are float32.
//
// Ranges are of equal length, so the call waits for the one with the most
// entries.  Measured, frequent tokens all over the vocabulary and at its
// beginning: 16384 x 4096 bf16 over 32000 tokens 127 / 130 us (the zeros hide it),
// 65531 x 1000 float32 over 32003 95 / 148 us.  Tokens that are none are entries
// of the last range: with 9 of 10 of them none, 191 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "follow.cuh"
#include "internal.h"
#include "layout.h"
#include "logit_rows.cuh"
#include "per_device.h"

namespace stp {
namespace {

using rows::Piece;

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;
constexpr int kHeld = 8;            // entries of a lane in registers
constexpr int kMaxWords = 4128;     // of 32 tokens in a block's range: 2^24 tokens over 128 blocks or more
constexpr int kScan = 64;           // positions of a lane in a walk over them
constexpr int kPiece = 32;          // sorted entries of a piece
constexpr int kShort = 64;          // entries of a token that one block adds up, at most
constexpr int kJoinAlong = 32, kJoinRows = kThreads / kJoinAlong;

struct EmbedParams {
  int N, V, C;
  int64_t stride;
  float scale;
  bool check, add;
  const void* table;
  const int32_t* tok;
  void* out;
  uint32_t* err;
  // backward
  int blocks;              // of the sort; each takes whole groups of 32 tokens
  int bits, passes;        // of a sort pass; the last pass writes to `sorted`
  const void* d_out;
  uint64_t* sorted;        // token << 32 | position, ascending; token V: none
  uint64_t* other;
  float* part;             // [pieces][2][C]: what a piece holds of tokens that occur often
  uint32_t* n_long;        // such tokens, and the pieces that they begin in, in any order
  uint32_t* long_at;
  float* d_table;
};

// ---------------------------------------------------------------- forward

// 2^shift threads take a token.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const EmbedParams p, int shift) {
  constexpr int E = Piece<T>::E;
  if (p.check && blockIdx.x == 0) {
    // all tokens, 16 of a thread at a time
    bool bad = false;
    for (int i0 = threadIdx.x; i0 < p.N; i0 += 16 * kThreads)
#pragma unroll
      for (int k = 0; k < 16; ++k) bad |= p.tok[min(i0 + k * kThreads, p.N - 1)] >= p.V;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.err = bad ? kErrBadList : 0;
    return;
  }
  const int64_t n = ((int64_t)(blockIdx.x - p.check) * kThreads + threadIdx.x) >> shift;
  if (n >= p.N) return;
  const int lane = threadIdx.x & ((1 << shift) - 1), step = 1 << shift, pieces = p.C / E;
  const int tok = p.tok[n];
  const bool there = tok >= 0 && tok < p.V;
  if (!p.check && tok >= p.V && lane == 0) atomicOr(p.err, kErrBadList);
  const uint4* from = reinterpret_cast<const uint4*>(static_cast<const T*>(p.table) + (int64_t)(there ? tok : 0) * p.C);
  uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + n * p.stride);
  constexpr int kAhead = 4;
  for (int i = lane; i < pieces; i += kAhead * step) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      v[k] = there && i + k * step < pieces ? __ldg(from + i + k * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * step < pieces) {
        float z[E];
        Piece<T>::get(v[k], z);
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] *= p.scale;
        __stcs(to + i + k * step, Piece<T>::put(z));
      }
  }
}

// ------------------------------------------------------------------- sort

struct SortShared {
  uint32_t hist[kSortWarps][kMaxBins];       // entries of a warp before it, then where the next goes
  uint32_t base[kMaxBins];
  uint32_t seen[kMaxWords];
  uint32_t warp_sum[kSortWarps];
};

// The sum of the warps' numbers before this one, and of all; every thread of the block calls it.
__device__ __forceinline__ uint32_t before_warp(SortShared& sh, uint32_t mine, uint32_t& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) sh.warp_sum[warp] = mine;
  __syncthreads();
  const uint32_t x = sh.warp_sum[lane];
  all = __reduce_add_sync(0xffffffffu, x);
  return __reduce_add_sync(0xffffffffu, lane < warp ? x : 0);
}

__global__ void __launch_bounds__(kSortThreads, 1) embed_sort_kernel(const EmbedParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  SortShared& sh = *reinterpret_cast<SortShared*>(smem);
  const int k = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const unsigned below_me = (1u << lane) - 1;
  // the block's tokens, in groups of 32; V stands for no token
  const int words = (p.V >> 5) + 1;
  const int w0 = (int)((int64_t)words * k / p.blocks), w1 = (int)((int64_t)words * (k + 1) / p.blocks);
  if (w0 == w1) return;   // never the last block
  const uint32_t v0 = (uint32_t)w0 * 32, v1 = (uint32_t)w1 * 32;
  for (int i = t; i < w1 - w0; i += kSortThreads) sh.seen[i] = 0;

  // ---- the block's entries, in a fixed order: kScan positions of a lane
  // at a time, a warp's next to one another.  As unsigned numbers, tokens that
  // are none lie behind all others, in the last block's range.
  constexpr int kRound = kSortThreads * kScan;
  const uint32_t span = k == p.blocks - 1 ? ~v0 : v1 - 1 - v0;
  uint32_t below = 0, first = 0;   // entries of smaller tokens: the block's place among the sorted ones
  if (p.N > kRound) {
    for (int i0 = t; i0 < p.N; i0 += 16 * kSortThreads) {
      uint32_t x[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = i0 + j * kSortThreads < p.N ? (uint32_t)p.tok[i0 + j * kSortThreads] : ~0u;
#pragma unroll
      for (int j = 0; j < 16; ++j) below += x[j] < v0;
    }
    before_warp(sh, __reduce_add_sync(0xffffffffu, below), first);
  }
  uint64_t *even = p.sorted, *odd = p.other;
  uint32_t n = 0;   // the block's entries so far
  for (int r0 = 0; r0 < p.N; r0 += kRound) {
    // a lane's positions: at + 32 j, those below the end
    const int each = min(kScan, ((p.N - r0 + kSortThreads - 1) / kSortThreads + 15) / 16 * 16);
    const int at = r0 + warp * each * 32 + lane;
    const int there = max(0, min(each, (p.N - at + 31) / 32));
    uint64_t in = 0, less = 0;   // bit j: position at + 32 j is the block's, or one of a smaller token
#pragma unroll 1
    for (int j0 = 0; j0 < each; j0 += 16) {
      uint32_t x[16], a = 0, b = 0;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = (uint32_t)p.tok[min(at + (j0 + j) * 32, p.N - 1)];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        a |= x[j] - v0 <= span ? 1u << j : 0;
        b |= x[j] < v0 ? 1u << j : 0;
      }
      in |= (uint64_t)a << j0;
      less |= (uint64_t)b << j0;
    }
    const uint64_t keep = there == 64 ? ~0ull : (1ull << there) - 1;
    in &= keep;
    below = __popcll(less & keep);
    uint32_t all, place = before_warp(sh, __reduce_add_sync(0xffffffffu, (uint32_t)__popcll(in)), all);
    if (p.N <= kRound) before_warp(sh, __reduce_add_sync(0xffffffffu, below), first);
    if (r0 == 0) {
      even += first;
      odd += first;
    }
    place += n;
    n += all;
    uint64_t* to = p.passes & 1 ? odd : even;
    // lane by lane, so that a lane walks its own positions only
    const uint32_t each_in = (uint32_t)__popcll(in);
    uint32_t up = each_in;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    to += place + up - each_in;
    for (; in; in &= in - 1) *to++ = (uint32_t)(at + (__ffsll(in) - 1) * 32);
  }
  __syncthreads();   // the positions are in place
  // their tokens, which a walk position by position would wait for one by one
  bool bad = false;
  for (uint32_t i0 = t; i0 < n; i0 += 8 * kSortThreads) {
    uint64_t* e = (p.passes & 1 ? odd : even) + i0;
    uint32_t at[8];
    int x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) at[j] = i0 + j * kSortThreads < n ? (uint32_t)e[j * kSortThreads] : ~0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = at[j] != ~0u ? p.tok[at[j]] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (at[j] != ~0u) {
        bad |= x[j] >= p.V;
        const uint32_t token = x[j] < 0 || x[j] >= p.V ? (uint32_t)p.V : (uint32_t)x[j];
        e[j * kSortThreads] = (uint64_t)token << 32 | at[j];
        // a word that holds the bit already is not written: many atomics on one word would come one by one
        uint32_t* word = &sh.seen[(token - v0) >> 5];
        if (!(*reinterpret_cast<volatile uint32_t*>(word) >> (token & 31) & 1)) atomicOr(word, 1u << (token & 31));
      }
  }
  bad = __syncthreads_or(bad);   // all of them are the last block's
  if (k == p.blocks - 1 && t == 0) {
    *p.err = bad ? kErrBadList : 0;
    *p.n_long = 0;
  }
  // zeros over the rows of the block's tokens that do not occur, a warp a row:
  // on their way while the entries are sorted
  if (!p.add)
    for (uint32_t v = v0 + warp; v < min(v1, (uint32_t)p.V); v += kSortWarps) {
      if (sh.seen[(v - v0) >> 5] >> (v & 31) & 1) continue;
      float4* row = reinterpret_cast<float4*>(p.d_table + (int64_t)v * p.C);
      for (int i = lane; i < p.C / 4; i += 32) __stcs(row + i, make_float4(0.f, 0.f, 0.f, 0.f));
    }

  // ---- their order by token
  const int bins = 1 << p.bits, groups = (n + 31) / 32;
  const int lo = groups * warp / kSortWarps * 32, hi = min((int)n, groups * (warp + 1) / kSortWarps * 32);
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint64_t* from = (p.passes - pass) & 1 ? odd : even;
    uint64_t* to = (p.passes - pass) & 1 ? even : odd;
    auto bin = [&](uint64_t x) { return ((uint32_t)(x >> 32) - v0) >> (pass * p.bits) & (bins - 1); };
    for (int i = t; i < kSortWarps * bins; i += kSortThreads) sh.hist[i >> p.bits][i & (bins - 1)] = 0;
    __syncthreads();
    // one group of 32 entries: how many of the warp's are before a lane's in its
    // bin, and the counter behind them; the bin's first lane returns its lanes in `group`
    auto rank = [&](int i, uint64_t x, uint32_t& group) {
      const bool on = i < hi;
      const uint32_t b = on ? bin(x) : bins;
      unsigned same = 0xffffffffu;   // the lanes with the same bin
      for (int j = 0; j <= p.bits; ++j) {
        const unsigned ones = __ballot_sync(0xffffffffu, b >> j & 1);
        same &= b >> j & 1 ? ones : ~ones;
      }
      const int mine = __popc(same & below_me);
      const uint32_t before = on ? sh.hist[warp][b] + mine : 0;
      __syncwarp();
      group = on && mine == 0 ? __popc(same) : 0;
      if (group) sh.hist[warp][b] += group;
      __syncwarp();
      return before;
    };
    // the first entries stay in registers, and so do their ranks
    uint64_t held[kHeld];
    uint32_t ranks[kHeld], group[kHeld], other;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) held[h] = lo + h * 32 + lane < hi ? from[lo + h * 32 + lane] : 0;
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (lo + h * 32 < hi) ranks[h] = rank(lo + h * 32 + lane, held[h], group[h]);
    for (int i0 = lo + kHeld * 32; i0 < hi; i0 += 32) rank(i0 + lane, i0 + lane < hi ? from[i0 + lane] : 0, other);
    __syncthreads();
    uint32_t sum = 0;
    if (t < bins)
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sh.hist[w][t];
        sh.hist[w][t] = sum;
        sum += c;
      }
    // where a bin begins
    uint32_t up = sum, all;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    const uint32_t before = before_warp(sh, __shfl_sync(0xffffffffu, up, 31), all);
    if (t < bins) sh.base[t] = before + up - sum;
    __syncthreads();
    const bool more = lo + kHeld * 32 < hi;   // then the counters go on behind the first entries
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (lo + h * 32 + lane < hi) to[sh.base[bin(held[h])] + sh.hist[warp][bin(held[h])] + ranks[h]] = held[h];
    __syncwarp();
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (more && group[h]) atomicAdd(&sh.hist[warp][bin(held[h])], group[h]);
    __syncwarp();
    for (int i0 = lo + kHeld * 32; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const uint64_t x = i < hi ? from[i] : 0;
      const uint32_t before = rank(i, x, other);
      if (i < hi) to[sh.base[bin(x)] + before] = x;
    }
    __syncthreads();
  }
}

// -------------------------------------------------------------------- sum

// A row of dE, or of a part.
template <int E>
__device__ __forceinline__ void put_row(float* to, const float* a, float scale) {
#pragma unroll
  for (int e = 0; e < E; e += 4)
    __stcs(reinterpret_cast<float4*>(to + e),
           make_float4(a[e] * scale, a[e + 1] * scale, a[e + 2] * scale, a[e + 3] * scale));
}

// A row of dE that is added to; each is one thread's.  An addition in memory would
// take numbers below the smallest normal one for 0.
template <int E>
__device__ __forceinline__ void add_row(float* row, const float* a, float scale) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    float4* at = reinterpret_cast<float4*>(row + e);
    const float4 o = __ldcs(at);
    __stcs(at, make_float4(__fadd_rn(o.x, __fmul_rn(a[e], scale)), __fadd_rn(o.y, __fmul_rn(a[e + 1], scale)),
                           __fadd_rn(o.z, __fmul_rn(a[e + 2], scale)), __fadd_rn(o.w, __fmul_rn(a[e + 3], scale))));
  }
}

__device__ __forceinline__ uint32_t token_at(const EmbedParams& p, int64_t i) {
  return (uint32_t)(p.sorted[i] >> 32);
}

// How many of a warp's values, from lane 0 on (from lane 31 down), satisfy a condition without a break.
__device__ __forceinline__ int leading(bool on) { return __clz(__brev(~__ballot_sync(0xffffffffu, on))); }
__device__ __forceinline__ int trailing(bool on) { return __clz(~__ballot_sync(0xffffffffu, on)); }

// blockDim.x threads (whole warps) lie along the channels, blockDim.y pieces are side by side.
// ADD: dE is added to.  Rows of tokens that begin are brought to L2 as far ahead as d_out is read, and
// read from there when their sum is complete: in us, so, with rows read ahead into registers, and with additions in
// memory, 77 / 87 / 77 (16384 x 4096 bf16), 99 / 104 / 93 (65531 x 1000 float32).
template <typename T, bool ADD>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const EmbedParams p) {
  constexpr int E = Piece<T>::E, kAhead = 8;
  const int piece = blockIdx.x * blockDim.y + threadIdx.y, i0 = piece * kPiece;
  if (i0 >= p.N) return;
  const int lane = threadIdx.x & 31, c = (blockIdx.y * blockDim.x + threadIdx.x) * E;
  const bool on = c < p.C;
  const uint32_t none = (uint32_t)p.V;
  wait_for_previous();
  // entries from kShort before the piece to kShort behind it; what is outside is no token
  uint64_t near[kPiece / 32 + 2 * kShort / 32];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    const int i = i0 - kShort + k * 32 + lane;
    near[k] = i >= 0 && i < p.N ? p.sorted[i] : (uint64_t)(i < 0 ? 0xffffffffu : none) << 32;
  }
  auto token = [&](int k) { return (uint32_t)(near[k] >> 32); };
  const uint32_t first = __shfl_sync(0xffffffffu, token(2), 0), last = __shfl_sync(0xffffffffu, token(2), 31);
  // the first token: how far it reaches back and forward
  int back = trailing(token(1) == first), ahead = leading(token(2) == first);
  if (back == 32) back += trailing(token(0) == first);
  if (ahead == 32) ahead += leading(token(3) == first);
  if (ahead == 64) ahead += leading(token(4) == first);
  const bool often = back + ahead > kShort;   // more than kShort entries, so that each of its pieces sees it
  int begin = 0, end = kPiece;
  if (back > 0 && !often) begin = ahead;      // added up where it began
  // the last token, where it begins in this piece and goes on
  bool last_often = often && last == first;
  if (last != first || back == 0) {
    const int in = trailing(token(2) == last);
    int over = leading(token(3) == last);
    if (over == 32) over += leading(token(4) == last);
    if (over > 0) {
      last_often = in + over > kShort;
      if (!last_often) end += over;
      else if (blockIdx.y == 0 && threadIdx.x == 0 && last != none) p.long_at[atomicAdd(p.n_long, 1u)] = piece;
    }
  }
  const T* d = static_cast<const T*>(p.d_out) + c;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  uint32_t now = none;
  auto is_part = [&](uint32_t key) { return (key == first && often) || (key == last && last_often); };
  auto flush = [&] {
    if (on && now != none) {
      float* row = p.d_table + (int64_t)now * p.C + c;
      if (is_part(now))
        put_row<E>(p.part + ((int64_t)piece * 2 + (now == first ? 0 : 1)) * p.C + c, acc, 1.f);
      else if (ADD)
        add_row<E>(row, acc, p.scale);
      else
        put_row<E>(row, acc, p.scale);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
  };
  for (int j0 = begin & ~(kAhead - 1); j0 < end; j0 += kAhead) {
    const uint64_t from = j0 < 32 ? near[2] : j0 < 64 ? near[3] : near[4];
    uint4 v[kAhead];
    uint32_t key[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint64_t x = __shfl_sync(0xffffffffu, from, (j0 + k) & 31);
      key[k] = j0 + k >= begin && j0 + k < end ? (uint32_t)(x >> 32) : none;
      v[k] = on && key[k] != none ? __ldcs(reinterpret_cast<const uint4*>(d + (int64_t)(uint32_t)x * p.stride))
                                  : make_uint4(0, 0, 0, 0);
      if constexpr (ADD)
        if (on && key[k] != none && key[k] != (k ? key[k - 1] : now) && !is_part(key[k]))
          asm volatile("prefetch.global.L2 [%0];" ::"l"(p.d_table + (int64_t)key[k] * p.C + c));
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (key[k] != now) {
        flush();
        now = key[k];
      }
      float z[E];
      Piece<T>::get(v[k], z);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += z[e];
    }
  }
  flush();
}

// Tokens that occur often, one after another for a block: row y of its threads
// takes every kJoinRows-th piece, in order, then the rows' sums are added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const EmbedParams p) {
  constexpr int E = Piece<T>::E, kRead = 8;
  __shared__ float sums[kJoinRows][kJoinAlong][E];
  const int pieces = (p.N + kPiece - 1) / kPiece, lane = threadIdx.x, y = threadIdx.y;
  const int c = (blockIdx.y * kJoinAlong + lane) * E;
  wait_for_previous();
  const uint32_t n = *p.n_long;
  for (uint32_t at = blockIdx.x; at < n; at += gridDim.x) {
    const int piece = p.long_at[at];
    const uint32_t key = token_at(p, (int64_t)piece * kPiece + kPiece - 1), first = token_at(p, (int64_t)piece * kPiece);
    // one past the last piece that holds it: by strides of 32 pieces, then one by one
    int end = piece + 1;
    for (int step = 32; step > 0; step = step == 32 ? 1 : 0)
      while (true) {
        const int q = end + (step == 32 ? lane * 32 + 31 : lane);
        const unsigned more = __ballot_sync(0xffffffffu, q < pieces && token_at(p, (int64_t)q * kPiece) == key);
        end += step * __popc(more);
        if (more != 0xffffffffu) break;
      }
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (c < p.C)
      for (int q0 = piece + y; q0 < end; q0 += kRead * kJoinRows) {
        float4 v[kRead][E / 4];
#pragma unroll
        for (int k = 0; k < kRead; ++k) {
          const int q = q0 + k * kJoinRows;
          const float4* from =
              reinterpret_cast<const float4*>(p.part + ((int64_t)q * 2 + (q == piece && first != key ? 1 : 0)) * p.C + c);
#pragma unroll
          for (int e = 0; e < E / 4; ++e) v[k][e] = q < end ? __ldcs(from + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kRead; ++k)
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            acc[e] += v[k][e / 4].x;
            acc[e + 1] += v[k][e / 4].y;
            acc[e + 2] += v[k][e / 4].z;
            acc[e + 3] += v[k][e / 4].w;
          }
      }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[y][lane][e] = acc[e];
    __syncthreads();
    if (y == 0 && c < p.C) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        for (int r = 1; r < kJoinRows; ++r) acc[e] += sums[r][lane][e];
      float* row = p.d_table + (int64_t)key * p.C + c;
      if (p.add)
        add_row<E>(row, acc, p.scale);
      else
        put_row<E>(row, acc, p.scale);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------- host

stp_status check_embed(const stp_embed_desc* d) {
  if (!d) return fail(STP_EINVAL, "embed descriptor is NULL");
  if (d->dtype != STP_BF16 && d->dtype != STP_FP32) return fail(STP_EUNSUPPORTED, "dtype %d not supported", d->dtype);
  if (d->n_tokens < 0) return fail(STP_EINVAL, "n_tokens < 0");
  if (d->n_tokens > (1 << 28)) return fail(STP_EUNSUPPORTED, "more than 2^28 tokens");
  if (d->vocab < 1 || d->vocab > (1 << 24)) return fail(STP_EUNSUPPORTED, "vocab must lie in [1, 2^24]");
  const int each = d->dtype == STP_BF16 ? 8 : 4;
  if (d->dim < each || d->dim > 65536 || d->dim % each)
    return fail(STP_EUNSUPPORTED, "dim must be a multiple of %d (16 bytes) in [%d, 65536]", each, each);
  if (d->stride < d->dim || d->stride % each)
    return fail(STP_EINVAL, "stride must be at least dim and a multiple of 16 bytes");
  if (!(d->scale >= -1e6f && d->scale <= 1e6f)) return fail(STP_EINVAL, "scale must lie in [-1e6, 1e6]");
  return STP_OK;
}

struct EmbedWs {
  size_t sorted, other, part, long_at, total;
};
EmbedWs embed_ws(const stp_embed_desc* d) {
  EmbedWs w;
  const size_t n = d->n_tokens, pieces = (n + kPiece - 1) / kPiece;
  w.sorted = 256;
  w.other = w.sorted + align256(n * 8);
  w.part = w.other + align256(n * 8);
  w.long_at = w.part + align256(pieces * 2 * d->dim * 4);
  w.total = w.long_at + align256(pieces * 4);
  return w;
}

EmbedParams embed_params(const stp_embed_desc* d, const int32_t* tok, void* ws) {
  EmbedParams p{};
  p.N = d->n_tokens;
  p.V = d->vocab;
  p.C = d->dim;
  p.stride = d->stride;
  p.scale = d->scale;
  p.tok = tok;
  p.err = static_cast<uint32_t*>(ws);
  return p;
}

template <typename T>
cudaError_t run_bwd(EmbedParams p, cudaStream_t s) {
  constexpr int E = Piece<T>::E;
  static PerDevice limit;
  constexpr int smem = sizeof(SortShared);
  cudaError_t e = limit([] {
    return cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  embed_sort_kernel<<<p.blocks, kSortThreads, smem, s>>>(p);
  const int pieces = (p.N + kPiece - 1) / kPiece, along = (p.C / E + 31) / 32 * 32;
  const dim3 block(along < kThreads ? along : kThreads, along < kThreads ? kThreads / along : 1);
  e = cudaGetLastError();
  if (e == cudaSuccess && pieces > 0)
    e = launch_after(p.add ? embed_sum_kernel<T, true> : embed_sum_kernel<T, false>,
                     dim3((pieces + block.y - 1) / block.y, (p.C / E + block.x - 1) / block.x), block, s, p);
  const int often = p.N / (kShort + 1);   // tokens that occur more than kShort times, at most
  if (e == cudaSuccess && often > 0)
    e = launch_after(embed_join_kernel<T>, dim3(often < 128 ? often : 128, (p.C / E + kJoinAlong - 1) / kJoinAlong),
                     dim3(kJoinAlong, kJoinRows), s, p);
  return e;
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_embed_workspace_size(const stp_embed_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_embed(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_embed_workspace_size: NULL output");
  *ws_bytes = embed_ws(desc).total;
  return STP_OK;
}

extern "C" stp_status stp_embed_fwd(const stp_embed_desc* desc, const void* table, const int32_t* d_token_ids,
                                    void* out, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_embed(desc);
  if (st) return st;
  if (!d_ws || reinterpret_cast<uintptr_t>(d_ws) & 255)
    return fail(STP_EINVAL, "stp_embed_fwd: the workspace must be 256-byte aligned");
  if (desc->n_tokens > 0 && (!table || !d_token_ids || !out))
    return fail(STP_EINVAL, "stp_embed_fwd: NULL device pointer");
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(out)) & 15)
    return fail(STP_EINVAL, "stp_embed_fwd: table and out must be 16-byte aligned");
  EmbedParams p = embed_params(desc, d_token_ids, d_ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // One block checks all tokens, 4096 of them a round trip to memory, and saves the
  // word's clearing (16384 x 4096 bf16: 36.2 -> 34.6 us); from rows of 1 KB on it ends before the others do.
  p.check = p.N > 0 && (p.N <= 4096 || p.C * (desc->dtype == STP_BF16 ? 2 : 4) >= 1024);
  p.table = table;
  p.out = out;
  cudaError_t e = p.check ? cudaSuccess : cudaMemsetAsync(d_ws, 0, 4, s);
  if (e == cudaSuccess && p.N > 0) {
    const int pieces = p.C / (desc->dtype == STP_BF16 ? 8 : 4);
    int shift = 0;
    while (shift < 5 && (1 << shift) < pieces) ++shift;
    const unsigned grid = (unsigned)((((int64_t)p.N << shift) + kThreads - 1) / kThreads) + p.check;
    if (desc->dtype == STP_BF16)
      embed_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, shift);
    else
      embed_fwd_kernel<float><<<grid, kThreads, 0, s>>>(p, shift);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_embed_fwd: %s", cudaGetErrorString(e));
  return STP_OK;
}

extern "C" stp_status stp_embed_bwd(const stp_embed_desc* desc, const void* d_out, const int32_t* d_token_ids,
                                    int32_t accumulate, float* d_table, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_embed(desc);
  if (st) return st;
  if (!d_ws || reinterpret_cast<uintptr_t>(d_ws) & 255)
    return fail(STP_EINVAL, "stp_embed_bwd: the workspace must be 256-byte aligned");
  if (!d_table || (desc->n_tokens > 0 && (!d_out || !d_token_ids)))
    return fail(STP_EINVAL, "stp_embed_bwd: NULL device pointer");
  if ((reinterpret_cast<uintptr_t>(d_table) | reinterpret_cast<uintptr_t>(d_out)) & 15)
    return fail(STP_EINVAL, "stp_embed_bwd: d_out and d_table must be 16-byte aligned");
  EmbedParams p = embed_params(desc, d_token_ids, d_ws);
  const EmbedWs w = embed_ws(desc);
  char* ws = static_cast<char*>(d_ws);
  p.add = accumulate != 0;
  p.d_out = d_out;
  p.d_table = d_table;
  p.sorted = reinterpret_cast<uint64_t*>(ws + w.sorted);
  p.other = reinterpret_cast<uint64_t*>(ws + w.other);
  p.part = reinterpret_cast<float*>(ws + w.part);
  p.n_long = reinterpret_cast<uint32_t*>(ws + 16);   // in the error word's 256 bytes
  p.long_at = reinterpret_cast<uint32_t*>(ws + w.long_at);
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  p.blocks = n_sm > 128 ? n_sm : 128;
  const int most = ((p.V >> 5) / p.blocks + 1) * 32;   // tokens of a block
  int width = 1;
  while (((most - 1) >> width) != 0) ++width;
  p.passes = (width + 8) / 9;
  p.bits = (width + p.passes - 1) / p.passes;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess)
    e = desc->dtype == STP_BF16 ? run_bwd<__nv_bfloat16>(p, s) : run_bwd<float>(p, s);
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_embed_bwd: %s", cudaGetErrorString(e));
  return STP_OK;
}
