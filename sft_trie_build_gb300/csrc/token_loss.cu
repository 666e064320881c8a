// Rows of logits: log-probability of a given token with entropy and the most
// likely tokens, distillation from a teacher's top logits, and the gradients.
//
// Everything follows from the passes over rows in logit_rows.cuh.  Bound by
// memory: forward one read of the logits, backward one read and one write, the
// step of both one read and one write too, its second pass out of L2.
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
#include "logit_rows.cuh"
#include "per_device.h"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace stp {
namespace {

using namespace rows;
using tc::ex2;

constexpr int kMaxTop = 32;
constexpr int kMaxTeacher = 256;
constexpr int kGroups = 64;         // groups of threads whose maxima bound the top tokens

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
      // below kLowest p is 0, and ln p is held there, so that its product with a large h stays finite
      zt = -ex2(lp * kLog2eT) * fmaf(h, fmaxf(lp, kLowest), c);
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
  return e == cudaSuccess ? launch_rows(kernel, rounds, rows, C, params, cluster, s) : e;
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
