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
// write.  C blocks share a row (C = 1 when there are rows enough for every
// SM): they are a thread-block cluster, and their sums meet in the shared
// memory of its first block, so one launch does a row whatever C is.  A block
// streams 16-byte pieces, four per thread in flight; a row may start at any
// address of its type: up to one piece's elements at either end of the row
// are taken one by one.
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

#include "internal.h"
#include "layout.h"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace stp {
namespace {

using tc::ex2;

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
constexpr int kMaxTop = 32;
constexpr int kMaxTeacher = kRowThreads;
constexpr int kMaxSplit = 8;        // blocks of a row: the portable cluster size
constexpr int kGroups = 64;         // groups of threads whose maxima bound the top tokens
constexpr int kFlight = 4;          // pieces in flight per thread
constexpr float kLog2eT = 1.4426950408889634f;
constexpr float kLn2T = 0.6931471805599453f;
// 2^d is 0 below this, so that d = -inf adds 0 to sum 2^d d, not NaN
constexpr float kLowest = -256.f;

template <typename T>
struct Piece;  // 16 bytes of a row
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int E = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float* f) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = tc::pack_bf16x2(f[2 * i], f[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Piece<float> {
  static constexpr int E = 4;
  static __device__ __forceinline__ void load(const float* p, float* f) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
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
// difference comes first: it is near exact where 2^d counts, and a row of the
// type's lowest value, as masks have it, overflows nowhere.
struct Acc {
  float m, s, t;
};

// Brings the sums of `a` to the reference of a larger maximum.
__device__ __forceinline__ void rebase(Acc& a, float m, float sl2) {
  if (a.m != -INFINITY) {
    const float dl = (a.m - m) * sl2, f = ex2(dl);
    a.t = f * fmaf(dl, a.s, a.t);
    a.s *= f;
  }
  a.m = m;
}

template <int N, bool ENT>
__device__ __forceinline__ void add(Acc& a, const float* z, float most, float sl2) {
  if (most > a.m) rebase(a, most, sl2);
  const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const float d = (z[e] - m) * sl2, p = ex2(d);
    a.s += p;
    if (ENT) a.t = fmaf(p, fmaxf(d, kLowest), a.t);
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

// The row's sums in all threads of its blocks.
__device__ __forceinline__ Acc row_sum(Acc a, Acc* red, Acc* mine, int C, float sl2) {
  a = block_sum(a, red, sl2);
  if (C > 1) {
    cg::cluster_group cl = cg::this_cluster();
    if (threadIdx.x == 0) *mine = a;
    cl.sync();
    a = *cl.map_shared_rank(mine, 0);
    for (int r = 1; r < C; ++r) a = merge(a, *cl.map_shared_rank(mine, r), sl2);
  }
  return a;
}

// ln sum exp(z) - scale m.
__device__ __forceinline__ float log_sum(const Acc& a) { return kLn2T * log2f(a.s); }

// One pass over the block's part of a row.  With TOP, the thread's largest
// value and the round in which it came are kept in (best, round).
template <typename T, bool ENT, bool TOP>
__device__ __forceinline__ Acc pass(const T* row, const Part& p, float sl2, float& best, int& round) {
  constexpr int E = Piece<T>::E;
  Acc a = {-INFINITY, 0.f, 0.f};
  const T* body = row + p.head;
  int k = 0;
  for (int b = p.b0 + (int)threadIdx.x; b < p.b1; b += kFlight * kRowThreads, ++k) {
    float z[kFlight * E];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      const int at = b + f * kRowThreads;
      if (at < p.b1) {
        Piece<T>::load(body + (int64_t)at * E, z + f * E);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) z[f * E + e] = -INFINITY;
      }
    }
    float most = z[0];
#pragma unroll
    for (int e = 1; e < kFlight * E; ++e) most = fmaxf(most, z[e]);
    if (TOP && most > best) {
      best = most;
      round = k;
    }
    add<kFlight * E, ENT>(a, z, most, sl2);
  }
  if (p.extra >= 0) {
    const float z = to_f(row[p.extra]);
    add<1, ENT>(a, &z, z, sl2);
  }
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

struct TopShared {
  uint64_t group[kGroups];
  uint64_t bound;
  int n_strips;
  uint16_t strip[kRowThreads];
  uint64_t cand[kRowThreads];
  uint64_t top[kMaxTop];
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

// sh.top[0..K) = the K largest of sh.cand[0..n), descending; n <= kRowThreads.
__device__ __forceinline__ void rank_top(TopShared& sh, int n, int K) {
  __syncthreads();
  if ((int)threadIdx.x < n) {
    const uint64_t mine = sh.cand[threadIdx.x];
    int rank = 0;
    for (int j = 0; j < n; ++j) {
      const uint64_t o = sh.cand[j];
      rank += o > mine || (o == mine && j < (int)threadIdx.x);
    }
    if (rank < K) sh.top[rank] = mine;
  }
  __syncthreads();
}

// The block's K largest tokens into sh.top.
template <typename T>
__device__ void block_top(const T* row, const Part& p, float best, int round, int K, TopShared& sh) {
  constexpr int E = Piece<T>::E;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint64_t mine = best > -INFINITY ? key_of(best, (uint32_t)round) : 0;
  uint64_t g = mine;
#pragma unroll
  for (int o = 1; o < kRowThreads / kGroups; o <<= 1) {
    const uint64_t x = __shfl_xor_sync(0xffffffffu, g, o);
    g = x > g ? x : g;
  }
  if (t % (kRowThreads / kGroups) == 0) sh.group[t / (kRowThreads / kGroups)] = g;
  if (t == 0) sh.n_strips = 0;
  __syncthreads();
  if (t < kGroups) {
    const uint64_t x = sh.group[t];
    int rank = 0;
    for (int j = 0; j < kGroups; ++j) {
      const uint64_t o = sh.group[j];
      rank += o > x || (o == x && j < t);
    }
    if (rank == K - 1) sh.bound = x;
  }
  __syncthreads();
  const uint64_t bound = sh.bound;
  const bool in = mine != 0 && mine >= bound;
  const unsigned who = __ballot_sync(0xffffffffu, in);
  int at = 0;
  if (lane == 0 && who) at = atomicAdd(&sh.n_strips, __popc(who));
  at = __shfl_sync(0xffffffffu, at, 0);
  if (in) sh.strip[at + __popc(who & ((1u << lane) - 1))] = (uint16_t)t;
  __syncthreads();
  uint64_t held = lane < K ? 0 : ~0ull, least = 0;
  const float floor_v = bound ? value_of(bound) : -INFINITY;
  const int n = sh.n_strips;
  for (int i = warp; i < n; i += kRowWarps) {
    const int first = p.b0 + sh.strip[i];
    for (int b = first; b < p.b1; b += 32 * kRowThreads) {
      const int at_b = b + lane * kRowThreads;
      const bool live = at_b < p.b1;
      float z[E];
      if (live) Piece<T>::load(row + p.head + (int64_t)at_b * E, z);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint64_t key = live ? key_of(z[e], (uint32_t)(p.head + at_b * E + e)) : 0;
        enter(held, least, live && z[e] > -INFINITY && z[e] >= floor_v && key > least, key);
      }
    }
  }
  if (__any_sync(0xffffffffu, p.extra >= 0)) {
    const float z = p.extra >= 0 ? to_f(row[p.extra]) : -INFINITY;
    const uint64_t key = key_of(z, (uint32_t)p.extra);
    enter(held, least, z > -INFINITY && key > least, key);
  }
  if (lane < K) sh.cand[warp * K + lane] = held;
  rank_top(sh, kRowWarps * K, K);
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
  // backward
  const float* lse_in;
  const float* ent_in;
  const float* g_lp;
  const float* g_ent;
  void* dz;
};

template <typename T, bool TOP>
__global__ void __launch_bounds__(kRowThreads) stats_fwd_kernel(const StatsParams p) {
  __shared__ Acc red[kRowWarps];
  __shared__ Acc mine;
  __shared__ TopShared sh;
  const int C = p.C, n = (int)(blockIdx.x / C), rank = (int)(blockIdx.x % C), t = threadIdx.x;
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
  float zt = 0.f;
  if (rank == 0 && t == 0) {
    if (target < p.V) {
      zt = to_f(row[target]);
    } else {
      zt = NAN;
      atomicOr(p.err, kErrBadList);
    }
  }
  float best = -INFINITY;
  int round = 0;
  Acc a = pass<T, true, TOP>(row, part, p.sl2, best, round);
  a = row_sum(a, red, &mine, C, p.sl2);
  if (TOP) {
    block_top(row, part, best, round, p.K, sh);
    if (C > 1) {
      cg::cluster_group cl = cg::this_cluster();
      cl.sync();
      if (rank == 0 && t < C * p.K) sh.cand[t] = cl.map_shared_rank(&sh, t / p.K)->top[t % p.K];
      if (rank == 0) rank_top(sh, C * p.K, p.K);
    }
  }
  const float ls = log_sum(a);
  const bool none = a.m == -INFINITY && a.s == 0.f;   // nothing but -inf
  if (rank == 0) {
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
  if (C > 1) cg::this_cluster().sync();   // the first block reads the others' shared memory
}

// Writes f(z, id) over the block's part of a row; `same`: the output row has
// the input row's alignment (else element by element).
template <typename T, typename F>
__device__ __forceinline__ void map_row(const T* row, T* out, const Part& p, F f) {
  constexpr int E = Piece<T>::E;
  const bool same = ((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  if (same) {
    for (int b = p.b0 + (int)threadIdx.x; b < p.b1; b += kFlight * kRowThreads) {
      float z[kFlight][E];
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (b + k * kRowThreads < p.b1) Piece<T>::load(row + p.head + (int64_t)(b + k * kRowThreads) * E, z[k]);
#pragma unroll
      for (int k = 0; k < kFlight; ++k) {
        const int at = b + k * kRowThreads;
        if (at < p.b1) {
          f(z[k], p.head + at * E, std::integral_constant<int, E>());
          Piece<T>::store(out + p.head + (int64_t)at * E, z[k]);
        }
      }
    }
    if (p.extra >= 0) {
      float z = to_f(row[p.extra]);
      f(&z, p.extra, std::integral_constant<int, 1>());
      put(out + p.extra, z);
    }
  } else {
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
  constexpr int E = Piece<T>::E;
  const Part p = part_of(out, V, rank, C);
  const float z[E] = {};
  for (int b = p.b0 + (int)threadIdx.x; b < p.b1; b += kRowThreads) Piece<T>::store(out + p.head + (int64_t)b * E, z);
  if (p.extra >= 0) put(out + p.extra, 0.f);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads) stats_bwd_kernel(const StatsParams p) {
  const int C = p.C, n = (int)(blockIdx.x / C), rank = (int)(blockIdx.x % C);
  const int target = p.target[n];
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  T* out = static_cast<T*>(p.dz) + (int64_t)n * p.stride;
  if (target < 0 || target >= p.V) {
    zero_row(out, p.V, rank, C);
    return;
  }
  const Part part = part_of(row, p.V, rank, C);
  const float scale = p.scale, lse = p.lse_in[n], g = p.g_lp[n] * scale, h = p.g_ent ? p.g_ent[n] * scale : 0.f;
  const float c = p.g_ent ? fmaf(h, p.ent_in[n], g) : g;
  map_row(row, out, part, [=](float* z, int id, auto N) {
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
// k-th entry.  With both, C is chosen so that the rows in work stay in L2
// between the two passes.
template <typename T, bool LSE, bool GRAD>
__global__ void __launch_bounds__(kRowThreads) distill_kernel(const DistillParams p) {
  __shared__ Acc red[kRowWarps];
  __shared__ Acc mine;
  __shared__ TeacherShared ts;
  const int C = p.C, n = (int)(blockIdx.x / C), rank = (int)(blockIdx.x % C), t = threadIdx.x;
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  T* out = GRAD ? static_cast<T*>(p.dz) + (int64_t)n * p.stride : nullptr;
  const bool wanted = !p.mask || p.mask[n];
  int id = -1;
  float a = -INFINITY;
  if (wanted && t < p.K) {
    id = p.ids[(int64_t)n * p.K + t];
    if (id >= p.V) {
      if (LSE && rank == 0) atomicOr(p.err, kErrBadList);
      id = -1;
    }
    if (id >= 0) a = p.tl[(int64_t)n * p.K + t] * p.sl2;
    if (a == -INFINITY) id = -1;
  }
  if (!__syncthreads_or(id >= 0)) {   // the same for every block of the row
    if (LSE && rank == 0 && t == 0) p.loss[n] = p.lse[n] = 0.f;
    if (GRAD) zero_row(out, p.V, rank, C);
    return;
  }
  const Part part = part_of(row, p.V, rank, C);
  const float zk = id >= 0 ? to_f(row[id]) : 0.f;
  const float top = block_max(a, ts.red);
  const float ek = id >= 0 ? ex2(a - top) : 0.f;
  const float sum = block_add(ek, ts.red);
  const float q = ek / sum;
  if (GRAD) {
    ts.id[t] = id;
    ts.q[t] = q;
  }
  float lse = 0.f;
  if (LSE) {
    float best;
    int round;
    Acc s = pass<T, false, false>(row, part, p.sl2, best, round);
    s = row_sum(s, red, &mine, C, p.sl2);
    const float ls = log_sum(s);
    lse = fmaf(s.m, p.scale, ls);
    if (rank == 0) {
      const float lnq = kLn2T * (a - top - log2f(sum));
      const float term = q != 0.f ? q * (lnq - fmaf(zk - s.m, p.scale, -ls)) : 0.f;
      const float loss = block_add(term, ts.red);
      if (t == 0) {
        p.loss[n] = loss;
        p.lse[n] = lse;
      }
    }
  } else {
    lse = p.lse_in[n];
  }
  if (GRAD) {
    const float scale = p.scale, g = p.g[n] * scale;
    __syncthreads();   // every zk is read before a logit may be overwritten
    map_row(row, out, part, [=](float* z, int, auto N) {
#pragma unroll
      for (int e = 0; e < N(); ++e) z[e] = g * ex2(fmaf(z[e], scale, -lse) * kLog2eT);
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
      if (own && first) put(out + id, g * (ex2(fmaf(zk, scale, -lse) * kLog2eT) - qs));
    }
  }
  if (LSE && C > 1) cg::this_cluster().sync();   // blocks read each other's shared memory
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

// Blocks of a row: enough that the GPU is full, while a block keeps 16 KB.
int split_of(int64_t rows, int64_t row_bytes) {
  int c = 1;
  while (c < kMaxSplit && rows * c < 608 && row_bytes / (2 * c) >= 16384) c *= 2;
  return c;
}

cudaError_t launch(const void* kernel, int64_t rows, int C, void* params, bool cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(rows * C));
  cfg.blockDim = dim3(kRowThreads);
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
  cudaError_t e = cudaMemsetAsync(d_ws, 0, 4, s);
  if (e == cudaSuccess && desc->n_rows > 0) {
    StatsParams p{};
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
    const void* k = desc->dtype == STP_BF16
                        ? (p.K ? (const void*)stats_fwd_kernel<__nv_bfloat16, true>
                               : (const void*)stats_fwd_kernel<__nv_bfloat16, false>)
                        : (p.K ? (const void*)stats_fwd_kernel<float, true> : (const void*)stats_fwd_kernel<float, false>);
    e = launch(k, p.N, p.C, &p, true, s);
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
                               p.N, p.C, &p, false, static_cast<cudaStream_t>(stream));
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
  cudaError_t e = fwd ? cudaMemsetAsync(ws, 0, 4, s) : cudaSuccess;
  if (e == cudaSuccess && desc->n_rows > 0) {
    DistillParams p = distill_params(desc, logits, ids, tl, mask);
    p.loss = loss;
    p.lse = lse;
    p.lse_in = lse_in;
    p.g = g;
    p.dz = dz;
    p.err = static_cast<uint32_t*>(ws);
    const int64_t bytes = row_bytes(p.V, desc->dtype);
    p.C = split_of(p.N, bytes);
    // both passes: the rows in work at one time have to stay in L2
    if (fwd && grad)
      while (p.C < kMaxSplit && bytes / p.C > 40960) p.C *= 2;
    const bool b = desc->dtype == STP_BF16;
    const void* k = fwd && grad ? (b ? (const void*)distill_kernel<__nv_bfloat16, true, true>
                                     : (const void*)distill_kernel<float, true, true>)
                    : fwd       ? (b ? (const void*)distill_kernel<__nv_bfloat16, true, false>
                                     : (const void*)distill_kernel<float, true, false>)
                                : (b ? (const void*)distill_kernel<__nv_bfloat16, false, true>
                                     : (const void*)distill_kernel<float, false, true>);
    e = launch(k, p.N, p.C, &p, fwd, s);
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
