// Passes over rows of logits, shared by the operators that read them
// (token_loss.cu, policy_loss.cu).
//
// With z = scale * logits of a row over V tokens, one pass keeps, per thread, a
// running maximum m, s = sum 2^d and t = sum 2^d d for d = (z - m) log2 e (a new
// maximum rescales both: s' = s 2^delta, t' = 2^delta (t + delta s)):
//   lse = scale m + ln s,   entropy = ln s - ln 2 t / s.
// The gradients are a second pass, p = exp(z - lse), written as it goes.
//
// C blocks share a row (C = 1 when there are rows enough for every SM): they
// are a thread-block cluster and send their sums into each other's shared
// memory, so one launch does a row whatever C is.  A thread streams 16-byte
// pieces through its own ring of slots in shared memory (asynchronous copies,
// no barrier), which keeps 192 KB on the way per SM while other blocks of the
// SM are at their row's end.  A row may start at any address of its type: up
// to one piece's elements at either end of the row are taken one by one.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "internal.h"
#include "layout.h"
#include "tc_ptx.cuh"

namespace stp {
namespace rows {

using tc::ex2;

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;
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

// ------------------------------------------------------------------- host

inline stp_status check_rows(int n_rows, int vocab, int64_t stride, int dtype, float scale) {
  if (n_rows < 0) return fail(STP_EINVAL, "n_rows < 0");
  if (vocab < 1 || vocab > (1 << 24)) return fail(STP_EUNSUPPORTED, "vocab must lie in [1, 2^24]");
  if (stride < vocab) return fail(STP_EINVAL, "stride must be at least vocab");
  if (dtype != STP_BF16 && dtype != STP_FP32) return fail(STP_EUNSUPPORTED, "dtype %d not supported", dtype);
  if (!(scale > 0.f) || scale > 1e4f) return fail(STP_EINVAL, "scale must be positive");
  return STP_OK;
}

inline bool off_type(const void* x, int dtype) {
  return reinterpret_cast<uintptr_t>(x) & (dtype == STP_BF16 ? 1 : 3);
}

// Blocks of a row: more than one where the rows alone do not fill the GPU, while
// a block keeps 16 KB; a cluster's meeting costs more than that of a block
// (2048 rows: 98 us with one block each, 111 with two).
inline int split_of(int64_t rows, int64_t row_bytes) {
  int c = 1;
  while (c < kMaxSplit && rows * c < 608 && row_bytes / (2 * c) >= 16384) c *= 2;
  return c;
}

// For the step of both passes: the rows in work, kStepBlocks of 152 SMs over C,
// have to stay in L2 from one pass to the next; beyond about 72 MB of its
// 129 they do not (4096 rows of 304 KB: 507 us with one block, 410 with two, 551
// with four, which meet too often).
inline int step_split_of(int64_t rows, int64_t row_bytes) {
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

inline int64_t row_bytes(int vocab, int dtype) { return (int64_t)vocab * (dtype == STP_BF16 ? 2 : 4); }

// `rows` rows of C blocks each; their shared-memory limit is already raised.
inline cudaError_t launch_rows(const void* kernel, int rounds, int64_t rows, int C, void* params, bool cluster,
                               cudaStream_t s) {
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

}  // namespace rows
}  // namespace stp
