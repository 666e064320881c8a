// Rows of logits: log-probability of a given token with entropy and the most
// likely tokens, distillation from a teacher's top logits, and the gradients.
//
// With z = scale * logits of a row over V tokens, everything follows from one
// pass that keeps, per thread, a running maximum m, s = sum 2^d and
// t = sum 2^d d for d = (z - m) log2 e (a new maximum rescales both:
// s' = s 2^delta, t' = 2^delta (t + delta s)):
//   lse = scale m + ln s,   entropy = ln s - ln 2 t / s.
// The gradients are a second pass, p = exp(z - lse), written as it goes.
//
// Bound by memory: forward one read of the logits, backward one read and one
// write, the step of both one read and one write too, its second pass out of
// L2.  C blocks share a row (C = 1 when there are rows enough for every SM):
// they are a thread-block cluster and send their sums into each other's shared
// memory, so one launch does a row whatever C is.  A thread streams
// 16-byte pieces through its own ring of slots in shared memory (asynchronous
// copies, no barrier), which keeps 192 KB on the way per SM while other blocks
// of the SM are at their row's end.  A row may start at any address of its
// type: up to one piece's elements at either end of the row are taken one by
// one.
//
// Top tokens without a second pass over the row: a thread remembers the
// maximum of its own strip of pieces.  The K-th largest over groups of four
// threads is a bound that K tokens reach, so only the strips whose maximum
// reaches it can hold one of the K largest; those (about K of 256) are read
// again, out of L2.  Tokens are ordered by one 64-bit key, the value's bits
// and then the id, so ties go to the smaller id whatever the split.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "layout.h"
#include "per_device.h"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace stp {
namespace {

using tc::ex2;

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kMaxTeacher = 256;
constexpr int kMaxSplit = 8;        // blocks of a row: the portable cluster size
constexpr int kFlight = 4;          // pieces of a round per thread
// Rounds on their way per thread, and blocks per SM: forward and backward 3
// and 4 (48 KB in flight per block), the step of both passes 4 and 3, where
// fewer rows in work keep more of them in L2.  Of 2..12 rounds and 1..8 blocks,
// these measured best on rows of 151936 bf16 logits: 8192 rows' statistics 415 us,
// 6.0 TB/s (462 without the ring), 4096 rows' step 411 us, 5.8 TB/s.
constexpr int kPassRounds = 3, kPassBlocks = 4;
constexpr int kStepRounds = 4, kStepBlocks = 3;
constexpr int ring_bytes(int rounds) { return rounds * kFlight * kRowThreads * 16; }
constexpr int kGroups = 64;         // groups of threads whose maxima bound the top tokens
constexpr float kLog2eT = 1.4426950408889634f;
constexpr float kLn2T = 0.6931471805599453f;
// 2^d is 0 below this, so that d = -inf adds 0 to sum 2^d d, not NaN
constexpr float kLowest = -256.f;

// 16 bytes of a row: E elements.
template <typename T>
struct Piece;
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void get(uint4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // the one rounding to bf16, of a finished gradient
  static __device__ __forceinline__ uint4 put(const float* f) {
    return make_uint4(tc::pack_bf16x2(f[0], f[1]), tc::pack_bf16x2(f[2], f[3]), tc::pack_bf16x2(f[4], f[5]),
                      tc::pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ uint4 lowest() {   // -inf in every element
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
};
template <>
struct Piece<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(uint4 v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ uint4 lowest() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// The part of a row that block `rank` of C works on: pieces [b0, b1) from
// element `head` on, and per thread at most one element outside the pieces
// (`extra`, -1 for none): the row's first `head` and last `tail` elements.
struct Part {
  int head, b0, b1, extra;
  int lo, hi;   // elements [lo, hi) of the row: what the block owns
};

template <typename T>
__device__ __forceinline__ Part part_of(const T* row, int V, int rank, int C) {
  constexpr int E = Piece<T>::E;
  const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  Part p;
  p.head = off ? min(V, E - off) : 0;
  const int n = (V - p.head) / E;
  const int tail = V - p.head - n * E;
  p.b0 = (int)((int64_t)n * rank / C);
  p.b1 = (int)((int64_t)n * (rank + 1) / C);
  p.extra = -1;
  const int t = threadIdx.x;
  if (rank == 0 && t < p.head) p.extra = t;
  if (rank == C - 1 && t >= 32 && t - 32 < tail) p.extra = V - tail + t - 32;
  p.lo = rank == 0 ? 0 : p.head + p.b0 * E;
  p.hi = rank == C - 1 ? V : p.head + p.b1 * E;
  return p;
}

// ------------------------------------------------------------------ sums

// m: largest raw logit; s, t: sums of 2^d and 2^d d, d = (logit - m) sl2.  The
// difference comes first: it is near exact where 2^d counts.  Beside a large
// negative mask value (the type's lowest) d is huge or -inf and 2^d is 0; the
// factor d of a sum is then held at kLowest, so that 0 times it is 0.
struct Acc {
  float m, s, t;
};

// Brings the sums of `a` to the reference of a larger maximum.
__device__ __forceinline__ void rebase(Acc& a, float m, float sl2) {
  if (a.m != -INFINITY) {
    const float dl = fmaxf((a.m - m) * sl2, kLowest), f = ex2(dl);
    a.t = f * fmaf(dl, a.s, a.t);
    a.s *= f;
  }
  a.m = m;
}

// Adds N logits, `most` and `least` their extremes; pairs go through the packed
// two-lane operations, which halve the instructions of a pass that issues
// more than it may.
template <int N, bool ENT>
__device__ __forceinline__ void add(Acc& a, const float* z, float most, float least, float sl2) {
  if (most > a.m) rebase(a, most, sl2);
  const float m = a.m == -INFINITY ? 0.f : a.m;
  if (N % 2 || (ENT && !((least - m) * sl2 > -1e30f))) {
    // one by one: d = -inf has to add 0 to t
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float d = (z[e] - m) * sl2, p = ex2(d);
      a.s += p;
      if (ENT) a.t = fmaf(p, fmaxf(d, kLowest), a.t);
    }
  } else {
    const float2 m2 = make_float2(-m, -m), l2 = make_float2(sl2, sl2);
    float2 s = make_float2(0.f, 0.f), t = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e + 1 < N; e += 2) {
      const float2 d = __fmul2_rn(__fadd2_rn(make_float2(z[e], z[e + 1]), m2), l2);
      const float2 p = make_float2(ex2(d.x), ex2(d.y));
      s = __fadd2_rn(s, p);
      if (ENT) t = __ffma2_rn(p, d, t);
    }
    a.s += s.x + s.y;
    if (ENT) a.t += t.x + t.y;
  }
}

template <int N>
__device__ __forceinline__ void extremes(const float* z, float& most, float& least) {
  most = least = z[0];
  if (N % 2) {
#pragma unroll
    for (int e = 1; e + 1 < N; e += 2) {
      most = tc::max3(most, z[e], z[e + 1]);
      asm("min.f32 %0, %0, %1, %2;" : "+f"(least) : "f"(z[e]), "f"(z[e + 1]));
    }
  } else {
    // two chains, then their ends
    float m1 = z[1], l1 = z[1];
#pragma unroll
    for (int e = 2; e + 3 < N; e += 4) {
      most = tc::max3(most, z[e], z[e + 1]);
      m1 = tc::max3(m1, z[e + 2], z[e + 3]);
      asm("min.f32 %0, %0, %1, %2;" : "+f"(least) : "f"(z[e]), "f"(z[e + 1]));
      asm("min.f32 %0, %0, %1, %2;" : "+f"(l1) : "f"(z[e + 2]), "f"(z[e + 3]));
    }
    most = tc::max3(most, m1, z[N - 2]);
    most = fmaxf(most, z[N - 1]);
    least = fminf(fminf(least, l1), fminf(z[N - 2], z[N - 1]));
  }
}

__device__ __forceinline__ Acc merge(Acc a, Acc b, float sl2) {
  if (b.m > a.m) rebase(a, b.m, sl2);
  else if (a.m > b.m) rebase(b, a.m, sl2);
  a.s += b.s;
  a.t += b.t;
  return a;
}

// All threads get the block's sums, added up in a fixed order.
__device__ __forceinline__ Acc block_sum(Acc a, Acc* red, float sl2) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Acc b;
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
    a = merge(a, b, sl2);
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = a;
  __syncthreads();
  a = red[0];
  for (int w = 1; w < kRowWarps; ++w) a = merge(a, red[w], sl2);
  return a;
}

// The row's sums, from those that its blocks have sent (the same in each).
__device__ __forceinline__ Acc merge_all(const Acc* sums, int C, float sl2) {
  Acc a = sums[0];
  for (int r = 1; r < C; ++r) a = merge(a, sums[r], sl2);
  return a;
}

// ln sum exp(z) - scale m.
__device__ __forceinline__ float log_sum(const Acc& a) { return kLn2T * log2f(a.s); }

// A thread's pieces on their way: R rounds of kFlight pieces each, in
// shared memory that no other thread touches, so the copies need no barrier.
template <int R>
struct Ring {
  uint4* slot;        // of this thread; pieces kRowThreads apart
  const uint4* body;
  int b1;

  __device__ __forceinline__ void fetch(int round, int b) const {
    const uint4* s = slot + round * kFlight * kRowThreads;
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      if (b + f * kRowThreads < b1)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(tc::smem_u32(s + f * kRowThreads)),
                     "l"(body + b + f * kRowThreads)
                     : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void start(int b) const {
#pragma unroll
    for (int r = 0; r < R; ++r) fetch(r, b + r * kFlight * kRowThreads);
  }
  // the oldest round has landed
  static __device__ __forceinline__ void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(R - 1) : "memory"); }
  __device__ __forceinline__ uint4 piece(int round, int f) const { return slot[(round * kFlight + f) * kRowThreads]; }
};

template <int R, typename T>
__device__ __forceinline__ Ring<R> ring_of(uint4* buffer, const T* row, const Part& p) {
  return {buffer + threadIdx.x, reinterpret_cast<const uint4*>(row + p.head), p.b1};
}

// One pass over the block's part of a row, whose first rounds are on their
// way.  With TOP, the thread's largest value and the round in which it came
// are kept in (best, round).
template <typename T, bool ENT, bool TOP, int R>
__device__ __forceinline__ Acc pass(const T* row, const Part& p, const Ring<R>& ring, float sl2, float& best,
                                    int& round) {
  constexpr int E = Piece<T>::E;
  Acc a = {-INFINITY, 0.f, 0.f};
  const float extra = p.extra >= 0 ? to_f(row[p.extra]) : 0.f;
  int s = 0;
  for (int b = p.b0 + (int)threadIdx.x, k = 0; b < p.b1; b += kFlight * kRowThreads, ++k) {
    ring.wait();
    float z[kFlight * E];
#pragma unroll
    for (int f = 0; f < kFlight; ++f)
      Piece<T>::get(b + f * kRowThreads < p.b1 ? ring.piece(s, f) : Piece<T>::lowest(), z + f * E);
    float most, least;
    extremes<kFlight * E>(z, most, least);
    if (TOP && most > best) {
      best = most;
      round = k;
    }
    add<kFlight * E, ENT>(a, z, most, least, sl2);
    ring.fetch(s, b + R * kFlight * kRowThreads);
    s = s + 1 == R ? 0 : s + 1;
  }
  if (p.extra >= 0) add<1, ENT>(a, &extra, extra, extra, sl2);
  return a;
}

// ------------------------------------------------------------- top tokens

// Larger value, then smaller id: a larger key.  0 is no token.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t id) {
  const uint32_t b = __float_as_uint(v + 0.f);   // -0 and 0 tie
  return ((uint64_t)(b ^ ((int32_t)b < 0 ? 0xffffffffu : 0x80000000u)) << 32) | (uint32_t)~id;
}
__device__ __forceinline__ float value_of(uint64_t key) {
  const uint32_t u = (uint32_t)(key >> 32);
  return __uint_as_float(u ^ ((int32_t)u < 0 ? 0x80000000u : 0xffffffffu));
}

constexpr int kCand = 512;

struct TopShared {
  __align__(16) uint64_t group[kGroups];
  __align__(16) uint64_t cand[kCand];   // first the threads' maxima, then the candidates
  uint64_t top[kMaxTop];
  __align__(16) uint64_t lists[kMaxSplit * kMaxTop];   // first block: every block's K largest
  uint64_t bound;
  int n_strips, n_cand;
  uint16_t strip[kRowThreads];
};

// Entry of `key` into the warp's list (one key per lane < K, `least` its
// smallest); all lanes call it.
__device__ __forceinline__ void enter(uint64_t& held, uint64_t& least, bool want, uint64_t key) {
  unsigned mask = __ballot_sync(0xffffffffu, want);
  while (mask) {
    const int src = __ffs(mask) - 1;
    mask &= mask - 1;
    const uint64_t k = __shfl_sync(0xffffffffu, key, src);
    if (k <= least) continue;
    const unsigned at = __ballot_sync(0xffffffffu, held == least);
    if ((int)(threadIdx.x & 31) == __ffs(at) - 1) held = k;
    const uint32_t hi = __reduce_min_sync(0xffffffffu, (uint32_t)(held >> 32));
    const uint32_t lo = __reduce_min_sync(0xffffffffu, (uint32_t)(held >> 32) == hi ? (uint32_t)held : 0xffffffffu);
    least = ((uint64_t)hi << 32) | lo;
  }
}

// How many of keys[0..n) come before `mine`, which is keys[at] (equal keys,
// which stand for no token, in order).
__device__ __forceinline__ int rank_of(const uint64_t* keys, int n, uint64_t mine, int at) {
  int rank = 0;
#pragma unroll 8
  for (int j = 0; j < n / 2; ++j) {
    const ulonglong2 o = reinterpret_cast<const ulonglong2*>(keys)[j];
    rank += o.x > mine || (o.x == mine && 2 * j < at);
    rank += o.y > mine || (o.y == mine && 2 * j + 1 < at);
  }
  if (n & 1) rank += keys[n - 1] > mine;
  return rank;
}

// f(key of the token, or 0) on every piece of the chosen strips, one lane a
// piece; all lanes of a warp call f together.  Strips of a warp's width or more
// go to a warp each; the pieces of shorter ones are dealt out over the block,
// which reads them all at once (strips of 10 pieces, 20 tokens: 12.4 us for eight
// rows of eight blocks against 13.3; of 75 pieces it costs, 8192 rows 440 against 418).
// `kept`: the ring of the pass, where it still holds every piece of the block.
template <typename T, typename F>
__device__ __forceinline__ void each_candidate(const T* row, const Part& p, const uint4* kept, const TopShared& sh,
                                               float floor_v, F f) {
  constexpr int E = Piece<T>::E;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint4* body = reinterpret_cast<const uint4*>(row + p.head);
  auto look = [&](int at, const uint4* src) {
    float z[E];
    Piece<T>::get(at < p.b1 ? *src : Piece<T>::lowest(), z);
    bool any = false;
#pragma unroll
    for (int e = 0; e < E; ++e) any = any || (z[e] >= floor_v && z[e] > -INFINITY);
    if (!__any_sync(0xffffffffu, any)) return;
#pragma unroll
    for (int e = 0; e < E; ++e)
      f(z[e] >= floor_v && z[e] > -INFINITY ? key_of(z[e], (uint32_t)(p.head + at * E + e)) : 0);
  };
  const int len = (p.b1 - p.b0 + kRowThreads - 1) / kRowThreads;   // pieces of a strip, the last one perhaps outside
  if (len >= 32) {
    for (int i = warp; i < sh.n_strips; i += kRowWarps)
      for (int j = 0; j < len; j += 32) {
        const int at = p.b0 + sh.strip[i] + (j + lane) * kRowThreads;
        look(at, body + at);
      }
  } else {
    const int total = sh.n_strips * len;
    for (int i0 = warp * 32; i0 < total; i0 += kRowThreads) {
      const int i = i0 + lane;
      const int in = i < total ? sh.strip[i / len] + (i % len) * kRowThreads : p.b1 - p.b0;   // piece of the block
      look(p.b0 + in, kept ? kept + in : body + p.b0 + in);
    }
  }
  if (__any_sync(0xffffffffu, p.extra >= 0)) {
    const float z = p.extra >= 0 ? to_f(row[p.extra]) : -INFINITY;
    f(z >= floor_v && z > -INFINITY ? key_of(z, (uint32_t)p.extra) : 0);
  }
}

// The block's K largest tokens into sh.top, descending, 0 where none is left.
template <typename T>
__device__ void block_top(const T* row, const Part& p, const uint4* kept, float best, int round, int K, TopShared& sh) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint64_t mine = best > -INFINITY ? key_of(best, (uint32_t)round) : 0;
  // groups of threads kGroups apart, so that a short row still fills them
  sh.cand[t] = mine;
  if (t == 0) sh.n_strips = sh.n_cand = 0;
  if (t < K) sh.top[t] = 0;
  __syncthreads();
  if (t < kGroups) {
    uint64_t g = mine;
#pragma unroll
    for (int o = kGroups; o < kRowThreads; o += kGroups) g = sh.cand[t + o] > g ? sh.cand[t + o] : g;
    sh.group[t] = g;
  }
  __syncthreads();
  if (t < kGroups && rank_of(sh.group, kGroups, sh.group[t], t) == K - 1) sh.bound = sh.group[t];
  __syncthreads();
  const uint64_t bound = sh.bound;
  const bool in = mine != 0 && mine >= bound;
  const unsigned who = __ballot_sync(0xffffffffu, in);
  int at = 0;
  if (lane == 0 && who) at = atomicAdd(&sh.n_strips, __popc(who));
  at = __shfl_sync(0xffffffffu, at, 0);
  if (in) sh.strip[at + __popc(who & ((1u << lane) - 1))] = (uint16_t)t;
  __syncthreads();
  const float floor_v = bound ? value_of(bound) : -INFINITY;
  each_candidate(row, p, kept, sh, floor_v, [&](uint64_t key) {
    if (key) {
      const int i = atomicAdd(&sh.n_cand, 1);
      if (i < kCand) sh.cand[i] = key;
    }
  });
  __syncthreads();
  int n = sh.n_cand;
  if (n > kCand) {
    // many values that tie or lie in few strips: a list of K per warp instead
    __syncthreads();
    uint64_t held = lane < K ? 0 : ~0ull, least = 0;
    each_candidate(row, p, kept, sh, floor_v, [&](uint64_t key) { enter(held, least, key > least, key); });
    if (lane < K) sh.cand[warp * K + lane] = held;
    n = kRowWarps * K;
    __syncthreads();
  }
  for (int i = t; i < n; i += kRowThreads) {
    const uint64_t x = sh.cand[i];
    const int rank = rank_of(sh.cand, n, x, i);
    if (rank < K) sh.top[rank] = x;
  }
  __syncthreads();
}

// The K largest of the C blocks' lists, each descending, into sh.top: a key's
// place is its place in its own list and, by halving, those in the others.
__device__ __forceinline__ void merge_top(TopShared& sh, int C, int K) {
  const int t = threadIdx.x, mine = t / K, at = t % K;
  const uint64_t key = t < C * K ? sh.lists[t] : 0;
  if (t < K) sh.top[t] = 0;
  __syncthreads();
  if (key) {
    // how many keys of each list are larger: the lists in step, so that the
    // reads of a step are on their way together
    int lo[kMaxSplit] = {}, rank = 0;
    for (int step = kMaxTop; step > 0; step >>= 1)
#pragma unroll
      for (int l = 0; l < kMaxSplit; ++l)
        if (l < C && lo[l] + step <= K && sh.lists[l * K + lo[l] + step - 1] > key) lo[l] += step;
#pragma unroll
    for (int l = 0; l < kMaxSplit; ++l) rank += l == mine ? at : lo[l];
    if (rank < K) sh.top[rank] = key;
  }
  __syncthreads();
}

// ------------------------------------------------------------------ stats

struct StatsParams {
  int N, V, C, K;
  int64_t stride;
  float scale, sl2;
  const void* z;
  const int32_t* target;
  float* logprob;
  float* entropy;
  float* lse;
  int32_t* top_id;
  float* top_lp;
  uint32_t* err;
  bool check;   // a block past the rows checks all targets
  // backward
  const float* lse_in;
  const float* ent_in;
  const float* g_lp;
  const float* g_ent;
  void* dz;
};

// The device error word, by a block of its own past the rows' (so that no row
// waits for it, and no launch clears the word): whether any of `n` whole
// numbers that are read lies at or above V.
template <typename F>
__device__ __forceinline__ void check_below(int64_t n, int V, uint32_t* err, F value) {
  bool bad = false;
  for (int64_t i = threadIdx.x; i < n; i += kRowThreads) bad = bad || value(i) >= V;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *err = bad ? kErrBadList : 0;
}

// MANY: several blocks per row (C > 1).
template <typename T, bool TOP, bool MANY>
__global__ void __launch_bounds__(kRowThreads, kPassBlocks) stats_fwd_kernel(const StatsParams p) {
  __shared__ Acc red[kRowWarps];
  __shared__ Acc sums[kMaxSplit];   // of the row's blocks
  __shared__ TopShared sh;
  extern __shared__ uint4 buffer[];
  const int C = MANY ? p.C : 1, n = (int)(blockIdx.x / C), rank = MANY ? (int)(blockIdx.x % C) : 0, t = threadIdx.x;
  if (n == p.N) {
    if (rank == 0) check_below(p.N, p.V, p.err, [&](int64_t i) { return p.target[i]; });
    return;
  }
  const int target = p.target[n];
  if (target < 0) {   // the same for every block of the row
    if (rank == 0) {
      if (t == 0) p.logprob[n] = p.entropy[n] = p.lse[n] = 0.f;
      if (TOP && t < p.K) {
        p.top_id[(int64_t)n * p.K + t] = -1;
        p.top_lp[(int64_t)n * p.K + t] = -INFINITY;
      }
    }
    return;
  }
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  const Part part = part_of(row, p.V, rank, C);
  const auto ring = ring_of<kPassRounds>(buffer, row, part);
  ring.start(part.b0 + t);
  if (MANY) cg::this_cluster().barrier_arrive();   // this block runs: others may write to it
  float zt = 0.f;
  if (rank == 0 && t == 0) {
    zt = target < p.V ? to_f(row[target]) : NAN;
    if (!p.check && target >= p.V) atomicOr(p.err, kErrBadList);
  }
  float best = -INFINITY;
  int round = 0;
  Acc a = block_sum(pass<T, true, TOP>(row, part, ring, p.sl2, best, round), red, p.sl2);
  if (TOP) {
    // piece j of a thread's strip lies in slot j of its ring until the ring comes round
    const bool all = part.b1 - part.b0 <= kPassRounds * kFlight * kRowThreads;
    block_top(row, part, all ? buffer : nullptr, best, round, p.K, sh);
  }
  if (MANY) {
    // everything goes to the first block, which then reads its own memory
    cg::cluster_group cl = cg::this_cluster();
    cl.barrier_wait();
    if (t == 0) *cl.map_shared_rank(sums + rank, 0) = a;
    if (TOP && t < p.K) *cl.map_shared_rank(sh.lists + rank * p.K + t, 0) = sh.top[t];
    cl.sync();
    if (rank > 0) return;
    a = merge_all(sums, C, p.sl2);
    if (TOP) merge_top(sh, C, p.K);
  }
  if (rank == 0) {
    const float ls = log_sum(a);
    const bool none = a.m == -INFINITY && a.s == 0.f;   // nothing but -inf
    if (t == 0) {
      p.lse[n] = none ? -INFINITY : fmaf(a.m, p.scale, ls);
      p.logprob[n] = none && !isnan(zt) ? -INFINITY : fmaf(zt - a.m, p.scale, -ls);
      p.entropy[n] = none ? 0.f : kLn2T * (log2f(a.s) - a.t / a.s);
    }
    if (TOP && t < p.K) {
      const uint64_t key = sh.top[t];
      p.top_id[(int64_t)n * p.K + t] = key ? (int32_t)~(uint32_t)key : -1;
      p.top_lp[(int64_t)n * p.K + t] = key ? fmaf(value_of(key) - a.m, p.scale, -ls) : -INFINITY;
    }
  }
}

// Writes f(z, id) over the block's part of a row, whose first rounds are on
// their way: 16-byte pieces where the output row has the input row's
// alignment, else element by element.
template <typename T, int R, typename F>
__device__ __forceinline__ void map_row(const T* row, T* out, const Part& p, const Ring<R>& ring, F f) {
  constexpr int E = Piece<T>::E;
  if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0) {
    uint4* to = reinterpret_cast<uint4*>(out + p.head);
    int s = 0;
    for (int b = p.b0 + (int)threadIdx.x; b < p.b1; b += kFlight * kRowThreads) {
      ring.wait();
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int at = b + k * kRowThreads;
        if (at < p.b1) {
          float z[E];
          Piece<T>::get(ring.piece(s, k), z);
          f(z, p.head + at * E, std::integral_constant<int, E>());
          __stcs(to + at, Piece<T>::put(z));
        }
      }
      ring.fetch(s, b + R * kFlight * kRowThreads);
      s = s + 1 == R ? 0 : s + 1;
    }
    if (p.extra >= 0) {
      float z = to_f(row[p.extra]);
      f(&z, p.extra, std::integral_constant<int, 1>());
      put(out + p.extra, z);
    }
  } else {
    asm volatile("cp.async.wait_all;" ::: "memory");   // the ring is not used
    for (int i = p.lo + (int)threadIdx.x; i < p.hi; i += kRowThreads) {
      float z = to_f(row[i]);
      f(&z, i, std::integral_constant<int, 1>());
      put(out + i, z);
    }
  }
}

// Zeros over the block's part of a row.
template <typename T>
__device__ __forceinline__ void zero_row(T* out, int V, int rank, int C) {
  const Part p = part_of(out, V, rank, C);
  uint4* to = reinterpret_cast<uint4*>(out + p.head);
  for (int b = p.b0 + (int)threadIdx.x; b < p.b1; b += kRowThreads) __stcs(to + b, make_uint4(0, 0, 0, 0));
  if (p.extra >= 0) put(out + p.extra, 0.f);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, kPassBlocks) stats_bwd_kernel(const StatsParams p) {
  const int C = p.C, n = (int)(blockIdx.x / C), rank = (int)(blockIdx.x % C);
  const int target = p.target[n];
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  T* out = static_cast<T*>(p.dz) + (int64_t)n * p.stride;
  const float lse = p.lse_in[n];
  if (target < 0 || target >= p.V || lse == -INFINITY) {   // not wanted, or nothing but -inf
    zero_row(out, p.V, rank, C);
    return;
  }
  const Part part = part_of(row, p.V, rank, C);
  const float scale = p.scale, g = p.g_lp[n] * scale, h = p.g_ent ? p.g_ent[n] * scale : 0.f;
  const float c = p.g_ent ? fmaf(h, p.ent_in[n], g) : g;
  extern __shared__ uint4 buffer[];
  const auto ring = ring_of<kPassRounds>(buffer, row, part);
  ring.start(part.b0 + threadIdx.x);
  map_row(row, out, part, ring, [=](float* z, int id, auto N) {
    float zt = 0.f;
#pragma unroll
    for (int e = 0; e < N(); ++e) {
      const float lp = fmaf(z[e], scale, -lse);
      zt = -ex2(lp * kLog2eT) * fmaf(h, fmaxf(lp, -1e30f), c);
      z[e] = id + e == target ? zt + g : zt;
    }
  });
}

// ---------------------------------------------------------------- distill

struct DistillParams {
  int N, V, C, K;
  int64_t stride;
  float scale, sl2;
  const void* z;
  const int32_t* ids;
  const float* tl;
  const uint8_t* mask;
  float* loss;
  float* lse;
  const float* lse_in;
  const float* g;
  void* dz;
  uint32_t* err;
  bool check;   // a block past the rows checks all ids
};

struct TeacherShared {
  float red[kRowWarps];
  __align__(16) int id[kMaxTeacher];     // -1 when absent
  __align__(16) float q[kMaxTeacher];
};

__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kRowWarps; ++w) v = fmaxf(v, red[w]);
  return v;
}
__device__ __forceinline__ float block_add(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < kRowWarps; ++w) v += red[w];
  return v;
}

// Forward (LSE), backward (GRAD) or both.  Thread k < K holds the teacher's
// k-th entry.  With both, the second pass finds the row in L2.
template <typename T, bool LSE, bool GRAD, bool MANY>
__global__ void __launch_bounds__(kRowThreads, LSE && GRAD ? kStepBlocks : kPassBlocks)
    distill_kernel(const DistillParams p) {
  __shared__ Acc red[kRowWarps];
  __shared__ Acc sums[kMaxSplit];   // of the row's blocks
  __shared__ TeacherShared ts;
  const int C = MANY ? p.C : 1, n = (int)(blockIdx.x / C), rank = MANY ? (int)(blockIdx.x % C) : 0, t = threadIdx.x;
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  T* out = GRAD ? static_cast<T*>(p.dz) + (int64_t)n * p.stride : nullptr;
  extern __shared__ uint4 buffer[];
  if (LSE && n == p.N) {
    if (rank == 0)
      check_below((int64_t)p.N * p.K, p.V, p.err,
                  [&](int64_t i) { return p.mask && !p.mask[i / p.K] ? -1 : p.ids[i]; });
    return;
  }
  const bool wanted = !p.mask || p.mask[n];
  int id = -1;
  float a = -INFINITY;
  if (wanted && t < p.K) {
    id = p.ids[(int64_t)n * p.K + t];
    if (id >= p.V) {
      if (LSE && rank == 0 && !p.check) atomicOr(p.err, kErrBadList);
      id = -1;
    }
    if (id >= 0) a = p.tl[(int64_t)n * p.K + t];
    if (a == -INFINITY) id = -1;
  }
  if (!__syncthreads_or(id >= 0)) {   // the same for every block of the row
    if (LSE && rank == 0 && t == 0) p.loss[n] = p.lse[n] = 0.f;
    if (GRAD) zero_row(out, p.V, rank, C);
    return;
  }
  const Part part = part_of(row, p.V, rank, C);
  const auto ring = ring_of<LSE && GRAD ? kStepRounds : kPassRounds>(buffer, row, part);
  ring.start(part.b0 + t);
  if (LSE && MANY) cg::this_cluster().barrier_arrive();   // this block runs: others may write to it
  const float zk = id >= 0 ? to_f(row[id]) : 0.f;
  const float top = block_max(a, ts.red);
  const float ek = id >= 0 ? ex2((a - top) * p.sl2) : 0.f;   // the difference first, as in the sums
  const float sum = block_add(ek, ts.red);
  const float q = ek / sum;
  if (GRAD && t < kMaxTeacher) {
    ts.id[t] = id;
    ts.q[t] = q;
  }
  // p = exp(x - ref) with x = scale z and ref = lse; with both passes at hand
  // x = scale (z - m) and ref = ln s, which hold for logits of any size: lse
  // itself carries p to |lse| 2^-24 only
  float m = 0.f, ref;
  bool none;   // nothing but -inf
  if (LSE) {
    float best;
    int round;
    Acc s = pass<T, false, false>(row, part, ring, p.sl2, best, round);
    if (GRAD) ring.start(part.b0 + t);   // again, now out of L2
    s = block_sum(s, red, p.sl2);
    if (MANY) {
      cg::cluster_group cl = cg::this_cluster();
      cl.barrier_wait();
      if (t < C) *cl.map_shared_rank(sums + rank, t) = s;
      cl.sync();
      s = merge_all(sums, C, p.sl2);
    }
    const float ls = log_sum(s);
    m = s.m;
    ref = ls;
    none = s.s == 0.f;
    if (rank == 0) {
      const float lnq = fmaf(a - top, p.scale, -kLn2T * log2f(sum));
      const float lnp = none ? -INFINITY : fmaf(zk - m, p.scale, -ls);
      const float term = q != 0.f ? q * (lnq - lnp) : 0.f;
      const float loss = block_add(term, ts.red);
      if (t == 0) {
        p.loss[n] = loss;
        p.lse[n] = fmaf(m, p.scale, ls);
      }
    }
  } else {
    ref = p.lse_in[n];
    none = ref == -INFINITY;
  }
  if (GRAD) {
    const float scale = p.scale, g = p.g[n] * scale;
    __syncthreads();   // every zk is read before a logit may be overwritten
    if (none) {
      asm volatile("cp.async.wait_all;" ::: "memory");
      zero_row(out, p.V, rank, C);
      return;
    }
    const auto prob = [=](float x) {
      return LSE ? ex2(fmaf(x - m, p.sl2, -ref * kLog2eT)) : ex2(fmaf(x, scale, -ref) * kLog2eT);
    };
    map_row(row, out, part, ring, [=](float* z, int, auto N) {
#pragma unroll
      for (int e = 0; e < N(); ++e) z[e] = g * prob(z[e]);
    });
    __syncthreads();   // the block's stores before those of the listed ids
    const bool own = id >= part.lo && id < part.hi;
    if (__any_sync(0xffffffffu, own)) {
      float qs = 0.f;
      bool first = true;
      for (int j = 0; j < p.K; ++j)
        if (ts.id[j] == id) {
          qs += ts.q[j];
          first = first && j >= t;
        }
      if (own && first) put(out + id, g * (prob(zk) - qs));
    }
  }
}

// ------------------------------------------------------------------- host

stp_status check_rows(int n_rows, int vocab, int64_t stride, int dtype, float scale) {
  if (n_rows < 0) return fail(STP_EINVAL, "n_rows < 0");
  if (vocab < 1 || vocab > (1 << 24)) return fail(STP_EUNSUPPORTED, "vocab must lie in [1, 2^24]");
  if (stride < vocab) return fail(STP_EINVAL, "stride must be at least vocab");
  if (dtype != STP_BF16 && dtype != STP_FP32) return fail(STP_EUNSUPPORTED, "dtype %d not supported", dtype);
  if (!(scale > 0.f) || scale > 1e4f) return fail(STP_EINVAL, "scale must be positive");
  return STP_OK;
}

stp_status check_stats(const stp_stats_desc* d) {
  if (!d) return fail(STP_EINVAL, "stats descriptor is NULL");
  if (d->top_k < 0 || d->top_k > kMaxTop) return fail(STP_EUNSUPPORTED, "top_k must lie in [0, %d]", kMaxTop);
  return check_rows(d->n_rows, d->vocab, d->stride, d->dtype, d->scale);
}

stp_status check_distill(const stp_distill_desc* d) {
  if (!d) return fail(STP_EINVAL, "distill descriptor is NULL");
  if (d->n_teacher < 1 || d->n_teacher > kMaxTeacher)
    return fail(STP_EUNSUPPORTED, "n_teacher must lie in [1, %d]", kMaxTeacher);
  return check_rows(d->n_rows, d->vocab, d->stride, d->dtype, d->scale);
}

bool off_type(const void* x, int dtype) {
  return reinterpret_cast<uintptr_t>(x) & (dtype == STP_BF16 ? 1 : 3);
}

// Blocks of a row: more than one where the rows alone do not fill the GPU, while
// a block keeps 16 KB; a cluster's meeting costs more than that of a block
// (2048 rows: 98 us with one block each, 111 with two).
int split_of(int64_t rows, int64_t row_bytes) {
  int c = 1;
  while (c < kMaxSplit && rows * c < 608 && row_bytes / (2 * c) >= 16384) c *= 2;
  return c;
}

// For the step of both passes: the rows in work, kStepBlocks of 152 SMs over C,
// have to stay in L2 from one pass to the next; beyond about 72 MB of its
// 129 they do not (4096 rows of 304 KB: 507 us with one block, 410 with two, 551
// with four, which meet too often).
int step_split_of(int64_t rows, int64_t row_bytes) {
  int c = split_of(rows, row_bytes);
  while (c < kMaxSplit && 152 * kStepBlocks * row_bytes / c > (72 << 20)) c *= 2;
  return c;
}

// The most whole numbers that one block checks: above, the error word is
// cleared first and every row checks its own.  The block saves the clearing's
// launch, about 1 us, but it is the last to start and walks its numbers 256 at a
// time.  Distillation forward in us, one block against every row: 4096 ids of 64 rows
// x 32000 8.3 / 9.3; 8192 of 128 rows 10.3 / 10.3, with a mask 14.4 / 10.3; 65536 of
// 1024 rows x 151936 154 / 55.  Statistics: 1024 rows x 32000 18.7 / 20.7, 4096
// 56.6 / 56.5, 8192 112 / 105.
constexpr int64_t kCheckMost = 4096;

template <typename T, bool LSE, bool GRAD>
const void* distill_by(bool many) {
  return many ? (const void*)distill_kernel<T, LSE, GRAD, true> : (const void*)distill_kernel<T, LSE, GRAD, false>;
}
template <typename T>
const void* distill_of(bool lse, bool grad, bool many) {
  if (!lse) return distill_by<T, false, true>(many);
  return grad ? distill_by<T, true, true>(many) : distill_by<T, true, false>(many);
}

template <typename T>
const void* stats_fwd(bool top, bool many) {
  return top ? (many ? (const void*)stats_fwd_kernel<T, true, true> : (const void*)stats_fwd_kernel<T, true, false>)
             : (many ? (const void*)stats_fwd_kernel<T, false, true> : (const void*)stats_fwd_kernel<T, false, false>);
}

template <typename T>
cudaError_t allow_rings_of() {
  const void* pass[] = {(const void*)stats_bwd_kernel<T>,
                        stats_fwd<T>(false, false), stats_fwd<T>(false, true),
                        stats_fwd<T>(true, false), stats_fwd<T>(true, true),
                        distill_of<T>(true, false, false), distill_of<T>(true, false, true),
                        distill_of<T>(false, true, false), distill_of<T>(false, true, true)};
  cudaError_t e = cudaSuccess;
  for (const bool many : {false, true})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(distill_of<T>(true, true, many), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               ring_bytes(kStepRounds));
  for (const void* k : pass)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(kPassRounds));
  return e;
}

// The kernels' dynamic shared memory, above the default limit.
cudaError_t allow_rings() {
  static PerDevice limits;
  return limits([] {
    const cudaError_t e = allow_rings_of<__nv_bfloat16>();
    return e == cudaSuccess ? allow_rings_of<float>() : e;
  });
}

cudaError_t launch(const void* kernel, int rounds, int64_t rows, int C, void* params, bool cluster, cudaStream_t s) {
  const cudaError_t e = allow_rings();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kRowThreads);
  cfg.dynamicSmemBytes = ring_bytes(rounds);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = C;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = cluster && C > 1 ? 1 : 0;
  void* args[] = {params};
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

DistillParams distill_params(const stp_distill_desc* d, const void* logits, const int32_t* ids, const float* tl,
                             const uint8_t* mask) {
  DistillParams p{};
  p.N = d->n_rows;
  p.V = d->vocab;
  p.K = d->n_teacher;
  p.stride = d->stride;
  p.scale = d->scale;
  p.sl2 = d->scale * kLog2eT;
  p.z = logits;
  p.ids = ids;
  p.tl = tl;
  p.mask = mask;
  return p;
}

int64_t row_bytes(int vocab, int dtype) { return (int64_t)vocab * (dtype == STP_BF16 ? 2 : 4); }

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_token_stats_workspace_size(const stp_stats_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_stats(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_token_stats_workspace_size: NULL output");
  *ws_bytes = 256;
  return STP_OK;
}

extern "C" stp_status stp_token_stats_fwd(const stp_stats_desc* desc, const void* logits, const int32_t* d_targets,
                                          float* logprob, float* entropy, float* lse, int32_t* top_id,
                                          float* top_logprob, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_stats(desc);
  if (st) return st;
  if (!d_ws || reinterpret_cast<uintptr_t>(d_ws) & 255)
    return fail(STP_EINVAL, "stp_token_stats_fwd: the workspace must be 256-byte aligned");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (desc->n_rows > 0 && (!logits || !d_targets || !logprob || !entropy || !lse ||
                           (desc->top_k > 0 && (!top_id || !top_logprob))))
    return fail(STP_EINVAL, "stp_token_stats_fwd: NULL device pointer");
  if (off_type(logits, desc->dtype)) return fail(STP_EINVAL, "stp_token_stats_fwd: logits misaligned for their type");
  const bool check = desc->n_rows > 0 && desc->n_rows <= kCheckMost;
  cudaError_t e = check ? cudaSuccess : cudaMemsetAsync(d_ws, 0, 4, s);
  if (e == cudaSuccess && desc->n_rows > 0) {
    StatsParams p{};
    p.check = check;
    p.N = desc->n_rows;
    p.V = desc->vocab;
    p.K = desc->top_k;
    p.stride = desc->stride;
    p.scale = desc->scale;
    p.sl2 = desc->scale * kLog2eT;
    p.z = logits;
    p.target = d_targets;
    p.logprob = logprob;
    p.entropy = entropy;
    p.lse = lse;
    p.top_id = top_id;
    p.top_lp = top_logprob;
    p.err = static_cast<uint32_t*>(d_ws);
    p.C = split_of(p.N, row_bytes(p.V, desc->dtype));
    const bool top = p.K > 0, many = p.C > 1;
    const void* k = desc->dtype == STP_BF16 ? stats_fwd<__nv_bfloat16>(top, many) : stats_fwd<float>(top, many);
    e = launch(k, kPassRounds, p.N + p.check, p.C, &p, true, s);
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_token_stats_fwd: %s", cudaGetErrorString(e));
  return STP_OK;
}

extern "C" stp_status stp_token_stats_bwd(const stp_stats_desc* desc, const void* logits, const int32_t* d_targets,
                                          const float* lse, const float* entropy, const float* d_logprob,
                                          const float* d_entropy, void* d_logits, void* stream) {
  clear_error();
  stp_status st = check_stats(desc);
  if (st) return st;
  if (desc->n_rows == 0) return STP_OK;
  if (!logits || !d_targets || !lse || !d_logprob || !d_logits || (d_entropy && !entropy))
    return fail(STP_EINVAL, "stp_token_stats_bwd: NULL device pointer");
  if (off_type(logits, desc->dtype) || off_type(d_logits, desc->dtype))
    return fail(STP_EINVAL, "stp_token_stats_bwd: logits misaligned for their type");
  StatsParams p{};
  p.N = desc->n_rows;
  p.V = desc->vocab;
  p.stride = desc->stride;
  p.scale = desc->scale;
  p.z = logits;
  p.target = d_targets;
  p.lse_in = lse;
  p.ent_in = entropy;
  p.g_lp = d_logprob;
  p.g_ent = d_entropy;
  p.dz = d_logits;
  p.C = split_of(p.N, row_bytes(p.V, desc->dtype));
  const cudaError_t e = launch(desc->dtype == STP_BF16 ? (const void*)stats_bwd_kernel<__nv_bfloat16>
                                                       : (const void*)stats_bwd_kernel<float>,
                               kPassRounds, p.N, p.C, &p, false, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_token_stats_bwd: %s", cudaGetErrorString(e));
  return STP_OK;
}

extern "C" stp_status stp_distill_workspace_size(const stp_distill_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_distill(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_distill_workspace_size: NULL output");
  *ws_bytes = 256;
  return STP_OK;
}

static stp_status distill(const char* name, const stp_distill_desc* desc, const void* logits, const int32_t* ids,
                          const float* tl, const uint8_t* mask, const float* lse_in, const float* g, float* loss,
                          float* lse, void* dz, void* ws, bool fwd, bool grad, void* stream) {
  clear_error();
  stp_status st = check_distill(desc);
  if (st) return st;
  if (fwd && (!ws || reinterpret_cast<uintptr_t>(ws) & 255))
    return fail(STP_EINVAL, "%s: the workspace must be 256-byte aligned", name);
  if (desc->n_rows > 0 && (!logits || !ids || !tl || (fwd && (!loss || !lse)) || (grad && (!g || !dz)) ||
                           (!fwd && !lse_in)))
    return fail(STP_EINVAL, "%s: NULL device pointer", name);
  if (off_type(logits, desc->dtype) || off_type(dz, desc->dtype))
    return fail(STP_EINVAL, "%s: logits misaligned for their type", name);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool check = fwd && desc->n_rows > 0 && (int64_t)desc->n_rows * desc->n_teacher <= kCheckMost;
  cudaError_t e = fwd && !check ? cudaMemsetAsync(ws, 0, 4, s) : cudaSuccess;
  if (e == cudaSuccess && desc->n_rows > 0) {
    DistillParams p = distill_params(desc, logits, ids, tl, mask);
    p.loss = loss;
    p.lse = lse;
    p.lse_in = lse_in;
    p.g = g;
    p.dz = dz;
    p.err = static_cast<uint32_t*>(ws);
    p.check = check;
    const int64_t bytes = row_bytes(p.V, desc->dtype);
    const bool both = fwd && grad;
    p.C = both ? step_split_of(p.N, bytes) : split_of(p.N, bytes);
    const void* k = desc->dtype == STP_BF16 ? distill_of<__nv_bfloat16>(fwd, grad, p.C > 1)
                                            : distill_of<float>(fwd, grad, p.C > 1);
    e = launch(k, both ? kStepRounds : kPassRounds, p.N + p.check, p.C, &p, fwd, s);
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "%s: %s", name, cudaGetErrorString(e));
  return STP_OK;
}

extern "C" stp_status stp_distill_fwd(const stp_distill_desc* desc, const void* logits, const int32_t* teacher_ids,
                                      const float* teacher_logits, const uint8_t* d_loss_mask, float* loss,
                                      float* lse, void* d_ws, void* stream) {
  return distill("stp_distill_fwd", desc, logits, teacher_ids, teacher_logits, d_loss_mask, nullptr, nullptr, loss,
                 lse, nullptr, d_ws, true, false, stream);
}

extern "C" stp_status stp_distill_bwd(const stp_distill_desc* desc, const void* logits, const int32_t* teacher_ids,
                                      const float* teacher_logits, const uint8_t* d_loss_mask, const float* lse,
                                      const float* d_loss, void* d_logits, void* stream) {
  return distill("stp_distill_bwd", desc, logits, teacher_ids, teacher_logits, d_loss_mask, lse, d_loss, nullptr,
                 nullptr, d_logits, nullptr, false, true, stream);
}

extern "C" stp_status stp_distill_step(const stp_distill_desc* desc, const void* logits, const int32_t* teacher_ids,
                                       const float* teacher_logits, const uint8_t* d_loss_mask, const float* d_loss,
                                       float* loss, float* lse, void* d_logits, void* d_ws, void* stream) {
  return distill("stp_distill_step", desc, logits, teacher_ids, teacher_logits, d_loss_mask, nullptr, d_loss, loss,
                 lse, d_logits, d_ws, true, true, stream);
}
