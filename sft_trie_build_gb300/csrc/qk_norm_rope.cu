// RMS norm of every query and key head and the rotation by position, in one
// pass over the projections, and the way back.
//
// For a head vector x of D channels at position t, with the weight w of its
// kind (queries or keys) and r = 1 / sqrt(mean(x^2) + eps):
//   n = x r w;   (y_a, y_b) = (n_a cos - n_b sin, n_a sin + n_b cos)
// over the rotated pairs (a, b), angle t * inv_freq[pair]; channels past
// rotary_dim pass as they are.  With g = the inverse rotation of dy:
//   dw += g x r,   dx = r (g w - x r^2 mean(g w x)).
//
// Bound by memory: the forward reads x and writes y, the backward reads x and
// dy and writes dx.  So a vector lives in registers from its load to its
// store, and nothing else of that size moves.  A lane holds two runs of eight
// channels (16 bytes each in bf16) that are the two sides of eight rotated
// pairs, so the rotation needs no exchange between lanes: runs u and
// u + rotary_dim / 16 for halves, 2u and 2u + 1 for interleaved pairs.  D / 16
// lanes make a vector (G, the next power of two, with the rest idle), a pass
// of a warp takes 32 / G heads of one token.  The next passes' vectors come by
// asynchronous copies into slots of shared memory of the lane's own, so they
// take no registers and need no barrier.  16384 tokens of 32 + 8 heads of 128
// bf16 channels: forward 57 us, 5.9 TB/s, backward 86 us with the sums of dw, 5.8 TB/s.
//
// The angle in turns is position * (inv_freq / 2 pi) mod 1, kept as 64-bit
// fixed point: the product wraps by itself, so a position of a million is as
// exact as position 1 (a float product would be off by 1e-2 radians there).
// The frequencies travel in the launch's parameters.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "internal.h"
#include "layout.h"
#include "per_device.h"
#include "tc_ptx.cuh"

namespace stp {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 512;
constexpr int kQkFwdBlocks = 4, kQkBwdBlocks = 2;    // per SM
constexpr int kQkBwdGrid = 152 * kQkBwdBlocks;       // partial sums of dw a call writes, at most
// Passes on their way per warp.  More than these cost: the forward of 16384 tokens of
// 40 heads of 128 bf16 channels measured 57 us with 2, 3 and 4, 65 with 6, the
// backward 84 with 2, 94 with 3 and 4.
template <typename T>
constexpr int fwd_depth() { return sizeof(T) == 2 ? 3 : 2; }
constexpr int kQkBwdDepth = 2;
// Shared memory of `runs` runs of eight channels per lane and pass.
template <typename T>
constexpr int ring_bytes(int runs, int depth) { return runs * ((int)sizeof(T) / 2) * depth * kQkThreads * 16; }

struct QkParams {
  int N, Hq, Hkv, D, rot;
  int blocks_q, blocks;  // blocks of the queries (backward), of both
  int64_t qs, ks;       // elements between tokens of q / k (and of dx_q / dx_k)
  float eps;
  const void* q;
  const void* k;
  const float* wq;
  const float* wk;
  const int32_t* pos;
  void* q_out;          // forward: y; backward: dx
  void* k_out;
  const void* dq;
  const void* dk;
  float* part;          // [blocks][D] partial dw
  float* dwq;
  float* dwk;
  uint64_t freq[kQkMaxDim / 2];   // turns per position, 2^-64 units
};

// Eight channels as four pairs: kPieces 16-byte pieces of memory.
template <typename T>
struct Run;
template <>
struct Run<__nv_bfloat16> {
  static constexpr int kPieces = 1;
  static __device__ __forceinline__ void get(const uint4* v, float2* f) {
    const uint32_t w[4] = {v->x, v->y, v->z, v->w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  // the one rounding to bf16, of the finished value
  static __device__ __forceinline__ void put(__nv_bfloat16* p, const float2* f) {
    *reinterpret_cast<uint4*>(p) = make_uint4(tc::pack_bf16x2(f[0].x, f[0].y), tc::pack_bf16x2(f[1].x, f[1].y),
                                              tc::pack_bf16x2(f[2].x, f[2].y), tc::pack_bf16x2(f[3].x, f[3].y));
  }
};
template <>
struct Run<float> {
  static constexpr int kPieces = 2;
  static __device__ __forceinline__ void get(const uint4* v, float2* f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = make_float2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
      f[2 * i + 1] = make_float2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
    }
  }
  static __device__ __forceinline__ void put(float* p, const float2* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  }
};

// A lane's vectors on their way, `depth` of them, in shared memory that no
// other thread touches: P pieces each, kQkThreads apart.
template <int P>
struct Lane {
  uint4* slot;
  __device__ __forceinline__ void fetch(int at, int piece, const void* src) const {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                     tc::smem_u32(slot + (at * P + piece) * kQkThreads)),
                 "l"(src)
                 : "memory");
  }
  template <typename T>
  __device__ __forceinline__ void fetch_run(int at, int piece, const T* src) const {
#pragma unroll
    for (int i = 0; i < Run<T>::kPieces; ++i) fetch(at, piece + i, reinterpret_cast<const uint4*>(src) + i);
  }
  template <typename T>
  __device__ __forceinline__ void get_run(int at, int piece, float2* f) const {
    uint4 v[Run<T>::kPieces];
#pragma unroll
    for (int i = 0; i < Run<T>::kPieces; ++i) v[i] = slot[(at * P + piece + i) * kQkThreads];
    Run<T>::get(v, f);
  }
};

// First channels of the two runs of lane u.
template <bool INTER>
__device__ __forceinline__ void run_at(int u, int rot, int& a, int& b) {
  const int half = rot / 16;   // runs on one side of the rotated pairs
  if (INTER || u >= half) {
    a = 16 * u;                // past the rotated channels the runs go in order
    b = a + 8;
  } else {
    a = 8 * u;
    b = 8 * (u + half);
  }
}

// cos and sin of the eight pairs of lane u at position t, (1, 0) past the
// rotated ones.  The 32 / G lanes of the same u make a share each and exchange
// them.
template <int G>
__device__ __forceinline__ void angles(const uint64_t* freq, int u, int rot, int t, float2* c, float2* s) {
  constexpr int NG = 32 / G < 8 ? 32 / G : 8, EACH = 8 / NG;
  const int grp = ((int)threadIdx.x & 31) / G % NG;
  float ce[EACH], se[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    ce[i] = 1.f;
    se[i] = 0.f;
    if (u < rot / 16) {
      // the top 32 bits as a signed part of a turn, in half turns
      const uint64_t turns = (uint64_t)(int64_t)t * freq[8 * u + i * NG + grp];
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &se[i], &ce[i]);
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float cv = ce[e / NG], sv = se[e / NG];
    if (NG > 1) {
      cv = __shfl_sync(0xffffffffu, cv, (e % NG) * G + u);
      sv = __shfl_sync(0xffffffffu, sv, (e % NG) * G + u);
    }
    (e & 1 ? c[e / 2].y : c[e / 2].x) = cv;
    (e & 1 ? s[e / 2].y : s[e / 2].x) = sv;
  }
}

// (a, b) -> (a cos - b sin, a sin + b cos) over a lane's eight pairs; x holds
// its two runs, c and s the pairs' cosines and sines.
template <bool INTER>
__device__ __forceinline__ void rotate(float2* x, const float2* c, const float2* s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (INTER) {
      const float2 a = x[2 * e], b = x[2 * e + 1];   // pairs 2e and 2e + 1
      x[2 * e] = __ffma2_rn(a, make_float2(c[e].x, c[e].x),
                            __fmul2_rn(make_float2(a.y, a.x), make_float2(-s[e].x, s[e].x)));
      x[2 * e + 1] = __ffma2_rn(b, make_float2(c[e].y, c[e].y),
                                __fmul2_rn(make_float2(b.y, b.x), make_float2(-s[e].y, s[e].y)));
    } else {
      const float2 a = x[e], b = x[e + 4];
      x[e] = __ffma2_rn(a, c[e], __fmul2_rn(b, make_float2(-s[e].x, -s[e].y)));
      x[e + 4] = __ffma2_rn(a, s[e], __fmul2_rn(b, c[e]));
    }
  }
}

template <int G>
__device__ __forceinline__ float sum_group(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's place in its warp's run of passes (32 / G heads of one token each:
// the queries' passes of a token, then the keys', then the next token): a
// pointer that goes on by `step` elements but where the tensor or the token
// changes.
template <typename T>
struct Walk {
  T* base[2];          // of queries and keys, at the lane's first head and channel
  int64_t stride[2];   // between tokens
  int64_t tok;
  T* p;
  int pass, pq, passes, step;
  __device__ __forceinline__ void init(T* q, T* k, int64_t qs, int64_t ks, int offset, int64_t unit, int pq_, int pk,
                                       int step_) {
    base[0] = q + offset;
    base[1] = k + offset;
    stride[0] = qs;
    stride[1] = ks;
    pq = pq_;
    passes = pq_ + pk;
    step = step_;
    tok = unit / passes;
    pass = (int)(unit % passes);
    p = pass < pq ? base[0] + tok * qs + pass * step : base[1] + tok * ks + (pass - pq) * step;
  }
  __device__ __forceinline__ void next() {
    p += step;
    if (++pass == pq) p = base[1] + tok * stride[1];
    if (pass == passes) {
      pass = 0;
      p = base[0] + ++tok * stride[0];
    }
  }
};

// An equal run of `units` passes for this warp of the blocks [b0, b0 + blocks).
struct Share {
  int64_t u0;
  int n;
  __device__ __forceinline__ Share(int64_t units, int b0, int blocks) {
    const int64_t warps = (int64_t)blocks * (kQkThreads / 32);
    const int64_t me = (int64_t)((int)blockIdx.x - b0) * (kQkThreads / 32) + (threadIdx.x >> 5);
    const int64_t each = units / warps, more = units % warps;   // the first `more` warps take one more
    u0 = each * me + (me < more ? me : more);
    n = (int)(each + (me < more));
  }
};

__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_copies() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Loads the frequencies and a weight into shared memory.
__device__ __forceinline__ void load_constants(const QkParams& p, const float* src, uint64_t* freq, float* w) {
  for (int i = threadIdx.x; i < p.rot / 2; i += kQkThreads) freq[i] = p.freq[i];
  for (int i = threadIdx.x; i < p.D; i += kQkThreads) w[i] = src ? src[i] : 1.f;
}

__device__ __forceinline__ void load_weight(const float* w, int ra, int rb, float2* wl) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float4 v = *reinterpret_cast<const float4*>(w + (e < 4 ? ra + 2 * e : rb + 2 * e - 8));
    wl[e] = make_float2(v.x, v.y);
    wl[e + 1] = make_float2(v.z, v.w);
  }
}

// Every warp takes an equal run of passes, several of them on their way; a
// token's angles are made when its first pass comes up.
template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(kQkThreads, kQkFwdBlocks) qk_fwd_kernel(const __grid_constant__ QkParams p) {
  __shared__ uint64_t freq[kQkMaxDim / 2];
  __shared__ __align__(16) float w[2][kQkMaxDim];
  extern __shared__ uint4 ring[];
  constexpr int NG = 32 / G, RP = Run<T>::kPieces, DEPTH = fwd_depth<T>();
  const int lane = threadIdx.x & 31, u = lane % G, grp = lane / G;
  const bool on = u < p.D / 16;
  int ra, rb;
  run_at<INTER>(on ? u : 0, p.rot, ra, rb);
  const int pq = (p.Hq + NG - 1) / NG, pk = (p.Hkv + NG - 1) / NG, passes = pq + pk;
  const Share sh((int64_t)p.N * passes, 0, gridDim.x);
  // whether the lane holds a head of pass k
  auto live = [&](int k) { return on && (k < pq ? k * NG + grp < p.Hq : (k - pq) * NG + grp < p.Hkv); };
  const Lane<2 * RP> in = {ring + threadIdx.x};
  Walk<const T> src;
  src.init(static_cast<const T*>(p.q), static_cast<const T*>(p.k), p.qs, p.ks, grp * p.D + ra, sh.u0, pq, pk, NG * p.D);
  int left = sh.n;   // passes not fetched yet
  auto fetch = [&](int at) {
    if (left > 0) {
      if (live(src.pass)) {
        in.fetch_run(at, 0, src.p);
        in.fetch_run(at, RP, src.p + (rb - ra));
      }
      src.next();
      --left;
    }
    commit_copies();
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(d);
  load_constants(p, p.wq, freq, w[0]);
  load_constants(p, p.wk, freq, w[1]);
  __syncthreads();
  const float inv_d = 1.f / (float)p.D;
  float2 c[4], s[4];
  Walk<T> dst;
  dst.init(static_cast<T*>(p.q_out), static_cast<T*>(p.k_out), (int64_t)p.Hq * p.D, (int64_t)p.Hkv * p.D,
           grp * p.D + ra, sh.u0, pq, pk, NG * p.D);
  const int32_t* pos = p.pos + dst.tok;
  int t = sh.n > 0 ? *pos : 0;
  int slot = 0;
  for (int i = 0; i < sh.n; ++i) {
    if (i == 0 || dst.pass == 0) {
      angles<G>(freq, u, p.rot, t, c, s);
      if (sh.n - i > passes - dst.pass) t = *++pos;   // on its way for the next token
    }
    wait_copies<DEPTH - 1>();
    float2 x[8];   // of lanes that hold no head: anything, and not stored
    in.template get_run<T>(slot, 0, x);
    in.template get_run<T>(slot, RP, x + 4);
    float2 ss2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
    for (int e = 1; e < 8; ++e) ss2 = __ffma2_rn(x[e], x[e], ss2);
    const float ss = sum_group<G>(on ? ss2.x + ss2.y : 0.f);
    fetch(slot);
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
    const float2 r2 = make_float2(r, r);
    float2 wl[8];
    load_weight(w[dst.pass >= pq], ra, rb, wl);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __fmul2_rn(x[e], __fmul2_rn(r2, wl[e]));
    rotate<INTER>(x, c, s);
    if (live(dst.pass)) {
      Run<T>::put(dst.p, x);
      Run<T>::put(dst.p + (rb - ra), x + 4);
    }
    dst.next();
  }
}

// The same walk over x and dy.  A block works on the queries or on the keys
// alone, so that a lane carries the sums of one weight; each block adds up its
// lanes' sums in a fixed order and writes them for qk_dw_kernel.
template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(kQkThreads, kQkBwdBlocks) qk_bwd_kernel(const __grid_constant__ QkParams p) {
  __shared__ uint64_t freq[kQkMaxDim / 2];
  __shared__ __align__(16) float w[kQkMaxDim];
  extern __shared__ uint4 ring[];
  constexpr int NG = 32 / G, RP = Run<T>::kPieces, DEPTH = kQkBwdDepth;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = lane % G, grp = lane / G;
  const bool on = u < p.D / 16;
  int ra, rb;
  run_at<INTER>(on ? u : 0, p.rot, ra, rb);
  const bool is_q = (int)blockIdx.x < p.blocks_q;
  const int H = is_q ? p.Hq : p.Hkv, passes = (H + NG - 1) / NG, step = NG * p.D, first = grp * p.D + ra;
  const Share sh((int64_t)p.N * passes, is_q ? 0 : p.blocks_q, is_q ? p.blocks_q : p.blocks - p.blocks_q);
  const int64_t xs = is_q ? p.qs : p.ks, gs = (int64_t)H * p.D;
  const Lane<4 * RP> in = {ring + threadIdx.x};
  // one tensor: no pass is the first of another
  const T* x0 = static_cast<const T*>(is_q ? p.q : p.k);
  const T* g0 = static_cast<const T*>(is_q ? p.dq : p.dk);
  Walk<const T> src, gsrc;
  src.init(x0, x0, xs, xs, first, sh.u0, passes, 0, step);
  gsrc.init(g0, g0, gs, gs, first, sh.u0, passes, 0, step);
  int left = sh.n;
  auto fetch = [&](int at) {
    if (left > 0) {
      if (on && src.pass * NG + grp < H) {
        in.fetch_run(at, 0, src.p);
        in.fetch_run(at, RP, src.p + (rb - ra));
        in.fetch_run(at, 2 * RP, gsrc.p);
        in.fetch_run(at, 3 * RP, gsrc.p + (rb - ra));
      }
      src.next();
      gsrc.next();
      --left;
    }
    commit_copies();
  };
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) fetch(d);
  load_constants(p, is_q ? p.wq : p.wk, freq, w);
  __syncthreads();
  const float inv_d = 1.f / (float)p.D;
  float2 c[4], s[4], dw[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = make_float2(0.f, 0.f);
  T* d0 = static_cast<T*>(is_q ? p.q_out : p.k_out);
  Walk<T> dst;
  dst.init(d0, d0, xs, xs, first, sh.u0, passes, 0, step);
  const int32_t* pos = p.pos + dst.tok;
  int t = sh.n > 0 ? *pos : 0;
  int slot = 0;
  for (int i = 0; i < sh.n; ++i) {
    if (i == 0 || dst.pass == 0) {
      angles<G>(freq, u, p.rot, t, c, s);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = make_float2(-s[e].x, -s[e].y);
      if (sh.n - i > passes - dst.pass) t = *++pos;
    }
    wait_copies<DEPTH - 1>();
    const bool live = on && dst.pass * NG + grp < H;
    float2 x[8], g[8];
    if (live) {
      in.template get_run<T>(slot, 0, x);
      in.template get_run<T>(slot, RP, x + 4);
      in.template get_run<T>(slot, 2 * RP, g);
      in.template get_run<T>(slot, 3 * RP, g + 4);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = g[e] = make_float2(0.f, 0.f);
    }
    rotate<INTER>(g, c, s);
    float2 ss2 = make_float2(0.f, 0.f), dot2 = make_float2(0.f, 0.f), wl[8];
    load_weight(w, ra, rb, wl);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ss2 = __ffma2_rn(x[e], x[e], ss2);
      dot2 = __ffma2_rn(__fmul2_rn(g[e], wl[e]), x[e], dot2);
    }
    fetch(slot);
    slot = slot + 1 == DEPTH ? 0 : slot + 1;
    const float ss = sum_group<G>(ss2.x + ss2.y);
    const float dot = sum_group<G>(dot2.x + dot2.y);
    // a lane group without a head adds 0 to dw: with eps = 0 its r would be infinite
    const float r = live ? rsqrtf(fmaf(ss, inv_d, p.eps)) : 0.f;
    const float m = -dot * inv_d * r * r * r;   // dx = g w r + x m
    const float2 r2 = make_float2(r, r), m2 = make_float2(m, m);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 gr = __fmul2_rn(g[e], r2);
      dw[e] = __ffma2_rn(gr, x[e], dw[e]);
      g[e] = __ffma2_rn(gr, wl[e], __fmul2_rn(x[e], m2));
    }
    if (live) {
      Run<T>::put(dst.p, g);
      Run<T>::put(dst.p + (rb - ra), g + 4);
    }
    dst.next();
  }
  // the warp's groups, then the block's warps
  // (over the ring, which is done with: eight rows of D <= 512 sums fit)
  float* red = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      dw[e].x += __shfl_xor_sync(0xffffffffu, dw[e].x, o);
      dw[e].y += __shfl_xor_sync(0xffffffffu, dw[e].y, o);
    }
  __syncthreads();
  if (on && grp == 0) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *reinterpret_cast<float2*>(red + warp * p.D + ra + 2 * e) = dw[e];
      *reinterpret_cast<float2*>(red + warp * p.D + rb + 2 * e) = dw[4 + e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.D; i += kQkThreads) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kQkThreads / 32; ++k) t += red[k * p.D + i];
    p.part[(int64_t)blockIdx.x * p.D + i] = t;
  }
}

// Adds up the blocks' partial sums: 32 channels of one weight per block, eight
// rows of threads over the partials, in a fixed order.
__global__ void __launch_bounds__(256) qk_dw_kernel(const float* __restrict__ part, int D, int blocks_q, int blocks,
                                                    float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float red[8][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), row = threadIdx.x >> 5;
  const bool is_q = blockIdx.y == 0;
  const int b0 = is_q ? 0 : blocks_q, b1 = is_q ? blocks_q : blocks;
  float t = 0.f;
  if (col < D)
    for (int b = b0 + row; b < b1; b += 8) t += part[(int64_t)b * D + col];
  red[row][threadIdx.x & 31] = t;
  __syncthreads();
  if (row == 0 && col < D) {
    t = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) t += red[k][threadIdx.x];
    (is_q ? dwq : dwk)[col] = t;
  }
}

stp_status check_qk(const stp_qk_desc* d) {
  if (!d) return fail(STP_EINVAL, "qk descriptor is NULL");
  if (d->n_tokens < 0) return fail(STP_EINVAL, "n_tokens < 0");
  if (d->n_q_heads < 1 || d->n_kv_heads < 1 || d->n_q_heads > 4096 || d->n_kv_heads > 4096)
    return fail(STP_EUNSUPPORTED, "n_q_heads and n_kv_heads must lie in [1, 4096]");
  if (d->dtype != STP_BF16 && d->dtype != STP_FP32) return fail(STP_EUNSUPPORTED, "dtype %d not supported", d->dtype);
  if (d->head_dim < 16 || d->head_dim > kQkMaxDim || d->head_dim % 16)
    return fail(STP_EUNSUPPORTED, "head_dim must be a multiple of 16 in [16, %d] (got %d)", kQkMaxDim, d->head_dim);
  if (d->rotary_dim < 0 || d->rotary_dim > d->head_dim || d->rotary_dim % 16)
    return fail(STP_EUNSUPPORTED, "rotary_dim must be a multiple of 16 in [0, head_dim] (got %d)", d->rotary_dim);
  if (d->interleaved != 0 && d->interleaved != 1) return fail(STP_EINVAL, "interleaved must be 0 or 1");
  if (!(d->eps >= 0.f) || d->eps > 1.f) return fail(STP_EINVAL, "eps must lie in [0, 1]");
  const int64_t unit = d->dtype == STP_BF16 ? 8 : 4;
  if (d->q_stride < (int64_t)d->n_q_heads * d->head_dim || d->k_stride < (int64_t)d->n_kv_heads * d->head_dim ||
      d->q_stride % unit || d->k_stride % unit)
    return fail(STP_EINVAL, "q_stride and k_stride must hold a token's heads and be multiples of 16 bytes");
  return STP_OK;
}

stp_status fill_qk(const stp_qk_desc* d, const double* inv_freq, QkParams& p) {
  p.N = d->n_tokens;
  p.Hq = d->n_q_heads;
  p.Hkv = d->n_kv_heads;
  p.D = d->head_dim;
  p.rot = d->rotary_dim;
  p.qs = d->q_stride;
  p.ks = d->k_stride;
  p.eps = d->eps;
  for (int i = 0; i < d->rotary_dim / 2; ++i) {
    if (!std::isfinite(inv_freq[i])) return fail(STP_EINVAL, "inv_freq[%d] is not finite", i);
    double turns = inv_freq[i] / 6.283185307179586;
    turns -= std::floor(turns);
    // 2^-64 units in two halves, each exact in a double
    const double x = turns * 4294967296.0, hi = std::floor(x);
    p.freq[i] = ((uint64_t)hi << 32) + (uint64_t)((x - hi) * 4294967296.0);
  }
  return STP_OK;
}

bool off16(const void* x) { return reinterpret_cast<uintptr_t>(x) & 15; }

// Launches KERNEL<T, G, INTER> for the descriptor's type, vector width and
// pairs; the dynamic shared memory RING(T) may pass the default limit, which is
// raised once per kernel and device.
#define STP_QK_LAUNCH(KERNEL, GRID, RING)                                                          \
  do {                                                                                             \
    const int units = desc->head_dim / 16;                                                         \
    if (units <= 1) STP_QK_T(KERNEL, 1, GRID, RING);                                               \
    else if (units <= 2) STP_QK_T(KERNEL, 2, GRID, RING);                                          \
    else if (units <= 4) STP_QK_T(KERNEL, 4, GRID, RING);                                          \
    else if (units <= 8) STP_QK_T(KERNEL, 8, GRID, RING);                                          \
    else if (units <= 16) STP_QK_T(KERNEL, 16, GRID, RING);                                        \
    else STP_QK_T(KERNEL, 32, GRID, RING);                                                         \
  } while (0)
#define STP_QK_T(KERNEL, G, GRID, RING)                                                            \
  do {                                                                                             \
    if (desc->dtype == STP_BF16 && desc->interleaved)                                              \
      STP_QK_RUN((KERNEL<__nv_bfloat16, G, true>), GRID, RING(__nv_bfloat16));                     \
    else if (desc->dtype == STP_BF16)                                                              \
      STP_QK_RUN((KERNEL<__nv_bfloat16, G, false>), GRID, RING(__nv_bfloat16));                    \
    else if (desc->interleaved)                                                                    \
      STP_QK_RUN((KERNEL<float, G, true>), GRID, RING(float));                                     \
    else                                                                                           \
      STP_QK_RUN((KERNEL<float, G, false>), GRID, RING(float));                                    \
  } while (0)
#define STP_QK_RUN(K, GRID, SMEM)                                                                  \
  do {                                                                                             \
    static PerDevice limit;                                                                        \
    const cudaError_t allowed = limit([] {                                                         \
      return cudaFuncSetAttribute((const void*)K, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM); \
    });                                                                                            \
    if (allowed != cudaSuccess) return fail(STP_ECUDA, "q/k norm: %s", cudaGetErrorString(allowed)); \
    K<<<GRID, kQkThreads, SMEM, s>>>(p);                                                           \
  } while (0)
#define STP_QK_FWD_RING(T) (ring_bytes<T>(2, fwd_depth<T>()))
#define STP_QK_BWD_RING(T) (ring_bytes<T>(4, kQkBwdDepth))

int heads_per_pass(int head_dim) {
  int g = 1;
  while (g < head_dim / 16) g <<= 1;
  return 32 / g;
}

// Blocks for `units` passes: a pass per warp, up to `most`.
int64_t blocks_of(int64_t units, int64_t most) {
  const int64_t n = (units + kQkThreads / 32 - 1) / (kQkThreads / 32);
  return n < most ? n : most;
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_qk_norm_rope_workspace_size(const stp_qk_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_qk(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_qk_norm_rope_workspace_size: NULL output");
  *ws_bytes = align256((size_t)kQkBwdGrid * desc->head_dim * 4);
  return STP_OK;
}

extern "C" stp_status stp_qk_norm_rope_fwd(const stp_qk_desc* desc, const void* q, const void* k, const float* w_q,
                                           const float* w_k, const double* inv_freq,
                                           const int32_t* d_position_ids, void* q_out, void* k_out, void* stream) {
  clear_error();
  stp_status st = check_qk(desc);
  if (st) return st;
  if (desc->rotary_dim > 0 && !inv_freq) return fail(STP_EINVAL, "stp_qk_norm_rope_fwd: inv_freq is NULL");
  if (desc->n_tokens == 0) return STP_OK;
  if (!q || !k || !d_position_ids || !q_out || !k_out)
    return fail(STP_EINVAL, "stp_qk_norm_rope_fwd: NULL device pointer");
  if (off16(q) || off16(k) || off16(q_out) || off16(k_out))
    return fail(STP_EINVAL, "stp_qk_norm_rope_fwd: tensors must be 16-byte aligned");
  QkParams p{};
  st = fill_qk(desc, inv_freq, p);
  if (st) return st;
  p.q = q;
  p.k = k;
  p.wq = w_q;
  p.wk = w_k;
  p.pos = d_position_ids;
  p.q_out = q_out;
  p.k_out = k_out;
  const int per = heads_per_pass(p.D);
  const int64_t units = (int64_t)p.N * ((p.Hq + per - 1) / per + (p.Hkv + per - 1) / per);
  // With tokens enough, one per warp, so that the blocks in work read and write
  // one moving stretch of memory (57 us of 16384 tokens; equal shares of the whole for
  // as many warps as are resident 65); with fewer, equal shares.
  const int64_t token_per_warp = ((int64_t)p.N + kQkThreads / 32 - 1) / (kQkThreads / 32);
  p.blocks = (int)blocks_of(units, token_per_warp > 152 * kQkFwdBlocks ? token_per_warp : 152 * kQkFwdBlocks);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  STP_QK_LAUNCH(qk_fwd_kernel, (unsigned)p.blocks, STP_QK_FWD_RING);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_qk_norm_rope_fwd: %s", cudaGetErrorString(e));
  return STP_OK;
}

extern "C" stp_status stp_qk_norm_rope_bwd(const stp_qk_desc* desc, const void* q, const void* k, const float* w_q,
                                           const float* w_k, const double* inv_freq,
                                           const int32_t* d_position_ids, const void* d_q, const void* d_k, void* dx_q,
                                           void* dx_k, float* dw_q, float* dw_k, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_qk(desc);
  if (st) return st;
  if (desc->rotary_dim > 0 && !inv_freq) return fail(STP_EINVAL, "stp_qk_norm_rope_bwd: inv_freq is NULL");
  if (!dw_q || !dw_k) return fail(STP_EINVAL, "stp_qk_norm_rope_bwd: NULL device pointer");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (desc->n_tokens == 0) {
    cudaError_t e = cudaMemsetAsync(dw_q, 0, (size_t)desc->head_dim * 4, s);
    if (e == cudaSuccess) e = cudaMemsetAsync(dw_k, 0, (size_t)desc->head_dim * 4, s);
    if (e != cudaSuccess) return fail(STP_ECUDA, "stp_qk_norm_rope_bwd: %s", cudaGetErrorString(e));
    return STP_OK;
  }
  if (!q || !k || !d_position_ids || !d_q || !d_k || !dx_q || !dx_k || !d_ws)
    return fail(STP_EINVAL, "stp_qk_norm_rope_bwd: NULL device pointer");
  if (off16(q) || off16(k) || off16(d_q) || off16(d_k) || off16(dx_q) || off16(dx_k) ||
      reinterpret_cast<uintptr_t>(d_ws) & 255)
    return fail(STP_EINVAL, "stp_qk_norm_rope_bwd: tensors must be 16-byte and the workspace 256-byte aligned");
  QkParams p{};
  st = fill_qk(desc, inv_freq, p);
  if (st) return st;
  p.q = q;
  p.k = k;
  p.wq = w_q;
  p.wk = w_k;
  p.pos = d_position_ids;
  p.q_out = dx_q;
  p.k_out = dx_k;
  p.dq = d_q;
  p.dk = d_k;
  p.part = static_cast<float*>(d_ws);
  const int per = heads_per_pass(p.D);
  const int64_t nq = (p.Hq + per - 1) / per, nk = (p.Hkv + per - 1) / per;
  // queries and keys get blocks by their passes, half a pass more for the
  // angles of a token, and one at least
  int64_t bq = (kQkBwdGrid * (2 * nq + 1) + nq + nk + 1) / (2 * (nq + nk + 1));
  bq = bq < 1 ? 1 : bq > kQkBwdGrid - 1 ? kQkBwdGrid - 1 : bq;
  p.blocks_q = (int)blocks_of(p.N * nq, bq);
  p.blocks = p.blocks_q + (int)blocks_of(p.N * nk, kQkBwdGrid - bq);
  STP_QK_LAUNCH(qk_bwd_kernel, (unsigned)p.blocks, STP_QK_BWD_RING);
  qk_dw_kernel<<<dim3((unsigned)((p.D + 31) / 32), 2), 256, 0, s>>>(p.part, p.D, p.blocks_q, p.blocks, dw_q, dw_k);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_qk_norm_rope_bwd: %s", cudaGetErrorString(e));
  return STP_OK;
}
