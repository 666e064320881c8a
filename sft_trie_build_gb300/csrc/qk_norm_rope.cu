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
// lanes make a vector (G, the next power of two, with the rest idle), a warp
// takes 32 / G heads of one token at a time.
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

namespace stp {
namespace {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 512;
constexpr int kQkBwdBlocks = 608;   // partial sums of dw a call writes, at most

struct QkParams {
  int N, Hq, Hkv, D, rot;
  int hp, parts;        // forward: heads of a work item, items of a token
  int blocks_q, blocks;  // backward: blocks of the queries, of both
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

// Eight channels: 16 bytes of bf16 or 32 of float.
template <typename T>
struct Run;
template <>
struct Run<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* f) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // the one rounding to bf16, of the finished value
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Run<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* f) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
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

// cos and sin of the eight pairs of lane u at position t; (1, 0) past them.
__device__ __forceinline__ void angles(const uint64_t* freq, int u, int rot, int t, float* c, float* s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c[e] = 1.f;
    s[e] = 0.f;
  }
  if (u < rot / 16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint64_t turns = (uint64_t)(int64_t)t * freq[8 * u + e];
      // the top 32 bits as a signed part of a turn, in half turns
      sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s[e], &c[e]);
    }
  }
}

// (a, b) -> (a cos - b sin, a sin + b cos) over the lane's eight pairs.
template <bool INTER>
__device__ __forceinline__ void rotate(float* x, const float* c, const float* s) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float& a = x[INTER ? 2 * e : e];
    float& b = x[INTER ? 2 * e + 1 : e + 8];
    const float a0 = a, b0 = b;
    a = fmaf(a0, c[e], -b0 * s[e]);
    b = fmaf(a0, s[e], b0 * c[e]);
  }
}

template <int G>
__device__ __forceinline__ float sum_group(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One work item: `hp` heads (queries first, then keys) of one token, by one
// warp; two vectors per lane are in flight.
template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(kQkThreads) qk_fwd_kernel(const __grid_constant__ QkParams p) {
  __shared__ uint64_t freq[kQkMaxDim / 2];
  __shared__ __align__(16) float w[2][kQkMaxDim];
  for (int i = threadIdx.x; i < p.rot / 2; i += kQkThreads) freq[i] = p.freq[i];
  for (int i = threadIdx.x; i < p.D; i += kQkThreads) {
    w[0][i] = p.wq ? p.wq[i] : 1.f;
    w[1][i] = p.wk ? p.wk[i] : 1.f;
  }
  __syncthreads();
  constexpr int NG = 32 / G, R = 2;
  const int lane = threadIdx.x & 31, u = lane % G, grp = lane / G;
  const bool on = u < p.D / 16;
  int ra, rb;
  run_at<INTER>(on ? u : 0, p.rot, ra, rb);
  const float inv_d = 1.f / (float)p.D;
  const int H = p.Hq + p.Hkv;
  const int64_t items = (int64_t)p.N * p.parts;
  const int64_t step = (int64_t)gridDim.x * (kQkThreads / 32);
  for (int64_t it = (int64_t)blockIdx.x * (kQkThreads / 32) + (threadIdx.x >> 5); it < items; it += step) {
    const int64_t tok = it / p.parts;
    const int h0 = (int)(it - tok * p.parts) * p.hp, h1 = min(H, h0 + p.hp);
    float c[8], s[8];
    angles(freq, u, p.rot, p.pos[tok], c, s);
    for (int hb = h0; hb < h1; hb += NG * R) {
      Run<T> xa[R], xb[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int h = hb + k * NG + grp;
        xa[k].zero();
        xb[k].zero();
        if (on && h < h1) {
          const T* src = h < p.Hq ? static_cast<const T*>(p.q) + tok * p.qs + (int64_t)h * p.D
                                  : static_cast<const T*>(p.k) + tok * p.ks + (int64_t)(h - p.Hq) * p.D;
          xa[k].load(src + ra);
          xb[k].load(src + rb);
        }
      }
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const int h = hb + k * NG + grp;
        float x[16];
        xa[k].get(x);
        xb[k].get(x + 8);
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
        ss = sum_group<G>(ss);
        const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
        const bool is_q = h < p.Hq;
        const float* wv = w[is_q ? 0 : 1];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const float4 wa = *reinterpret_cast<const float4*>(wv + ra + e);
          const float4 wb = *reinterpret_cast<const float4*>(wv + rb + e);
          x[e] *= r * wa.x; x[e + 1] *= r * wa.y; x[e + 2] *= r * wa.z; x[e + 3] *= r * wa.w;
          x[8 + e] *= r * wb.x; x[9 + e] *= r * wb.y; x[10 + e] *= r * wb.z; x[11 + e] *= r * wb.w;
        }
        rotate<INTER>(x, c, s);
        if (on && h < h1) {
          T* dst = is_q ? static_cast<T*>(p.q_out) + (tok * p.Hq + h) * p.D
                        : static_cast<T*>(p.k_out) + (tok * p.Hkv + (h - p.Hq)) * p.D;
          Run<T>::store(dst + ra, x);
          Run<T>::store(dst + rb, x + 8);
        }
      }
    }
  }
}

// A block works on the queries or on the keys alone, so that a lane carries
// the sums of one weight; each block adds up its lanes' sums in a fixed order
// and writes them for qk_dw_kernel.
template <typename T, int G, bool INTER>
__global__ void __launch_bounds__(kQkThreads) qk_bwd_kernel(const __grid_constant__ QkParams p) {
  __shared__ uint64_t freq[kQkMaxDim / 2];
  __shared__ __align__(16) float w[kQkMaxDim];
  __shared__ __align__(16) float red[kQkThreads / 32][kQkMaxDim];
  const bool is_q = (int)blockIdx.x < p.blocks_q;
  const float* wsrc = is_q ? p.wq : p.wk;
  for (int i = threadIdx.x; i < p.rot / 2; i += kQkThreads) freq[i] = p.freq[i];
  for (int i = threadIdx.x; i < p.D; i += kQkThreads) w[i] = wsrc ? wsrc[i] : 1.f;
  __syncthreads();
  constexpr int NG = 32 / G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, u = lane % G, grp = lane / G;
  const bool on = u < p.D / 16;
  int ra, rb;
  run_at<INTER>(on ? u : 0, p.rot, ra, rb);
  const float inv_d = 1.f / (float)p.D;
  const int H = is_q ? p.Hq : p.Hkv;
  const int64_t xs = is_q ? p.qs : p.ks;
  const T* xin = static_cast<const T*>(is_q ? p.q : p.k);
  const T* dy = static_cast<const T*>(is_q ? p.dq : p.dk);
  T* dx = static_cast<T*>(is_q ? p.q_out : p.k_out);
  const int block = is_q ? blockIdx.x : blockIdx.x - p.blocks_q;
  const int64_t step = (int64_t)(is_q ? p.blocks_q : p.blocks - p.blocks_q) * (kQkThreads / 32);
  float dw[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) dw[e] = 0.f;
  const int parts = (H + p.hp - 1) / p.hp;
  const int64_t items = (int64_t)p.N * parts;
  for (int64_t it = (int64_t)block * (kQkThreads / 32) + warp; it < items; it += step) {
    const int64_t tok = it / parts;
    const int h0 = (int)(it - tok * parts) * p.hp, h1 = min(H, h0 + p.hp);
    float c[8], s[8];
    angles(freq, u, p.rot, p.pos[tok], c, s);
#pragma unroll
    for (int e = 0; e < 8; ++e) s[e] = -s[e];
    for (int hb = h0; hb < h1; hb += NG) {
      const int h = hb + grp;
      const bool live = on && h < h1;
      Run<T> xa, xb, ga, gb;
      xa.zero();
      xb.zero();
      ga.zero();
      gb.zero();
      if (live) {
        const T* src = xin + tok * xs + (int64_t)h * p.D;
        const T* gsrc = dy + (tok * H + h) * p.D;
        xa.load(src + ra);
        xb.load(src + rb);
        ga.load(gsrc + ra);
        gb.load(gsrc + rb);
      }
      float x[16], g[16];
      xa.get(x);
      xb.get(x + 8);
      ga.get(g);
      gb.get(g + 8);
      rotate<INTER>(g, c, s);
      float ss = 0.f, dot = 0.f;
      float wl[16];
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        *reinterpret_cast<float4*>(wl + e) = *reinterpret_cast<const float4*>(w + ra + e);
        *reinterpret_cast<float4*>(wl + 8 + e) = *reinterpret_cast<const float4*>(w + rb + e);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        ss = fmaf(x[e], x[e], ss);
        dot = fmaf(g[e] * wl[e], x[e], dot);
      }
      ss = sum_group<G>(ss);
      dot = sum_group<G>(dot);
      const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
      const float m = dot * inv_d * r * r;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        dw[e] = fmaf(g[e], x[e] * r, dw[e]);
        g[e] = r * fmaf(g[e], wl[e], -x[e] * m);
      }
      if (live) {
        T* dst = dx + tok * xs + (int64_t)h * p.D;
        Run<T>::store(dst + ra, g);
        Run<T>::store(dst + rb, g + 8);
      }
    }
  }
  // the warp's groups, then the block's warps
#pragma unroll
  for (int e = 0; e < 16; ++e)
#pragma unroll
    for (int o = G; o < 32; o <<= 1) dw[e] += __shfl_xor_sync(0xffffffffu, dw[e], o);
  if (on && grp == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[warp][ra + e] = dw[e];
      red[warp][rb + e] = dw[8 + e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.D; i += kQkThreads) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kQkThreads / 32; ++k) t += red[k][i];
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

// Launches `K<T, G, INTER>` for the descriptor's type, vector width and pairs.
#define STP_QK_LAUNCH(KERNEL, GRID)                                                                    \
  do {                                                                                                 \
    const int units = desc->head_dim / 16;                                                             \
    const int g = units <= 1 ? 1 : units <= 2 ? 2 : units <= 4 ? 4 : units <= 8 ? 8 : units <= 16 ? 16 : 32; \
    if (desc->dtype == STP_BF16) {                                                                     \
      STP_QK_G(KERNEL, __nv_bfloat16, GRID);                                                           \
    } else {                                                                                           \
      STP_QK_G(KERNEL, float, GRID);                                                                   \
    }                                                                                                  \
  } while (0)
#define STP_QK_G(KERNEL, T, GRID)                      \
  switch (g) {                                         \
    case 1: STP_QK_I(KERNEL, T, 1, GRID); break;       \
    case 2: STP_QK_I(KERNEL, T, 2, GRID); break;       \
    case 4: STP_QK_I(KERNEL, T, 4, GRID); break;       \
    case 8: STP_QK_I(KERNEL, T, 8, GRID); break;       \
    case 16: STP_QK_I(KERNEL, T, 16, GRID); break;     \
    default: STP_QK_I(KERNEL, T, 32, GRID); break;     \
  }
#define STP_QK_I(KERNEL, T, G, GRID)                           \
  do {                                                         \
    if (desc->interleaved)                                     \
      KERNEL<T, G, true><<<GRID, kQkThreads, 0, s>>>(p);       \
    else                                                       \
      KERNEL<T, G, false><<<GRID, kQkThreads, 0, s>>>(p);      \
  } while (0)

int heads_per_pass(int head_dim) {
  int g = 1;
  while (g < head_dim / 16) g <<= 1;
  return 32 / g;
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_qk_norm_rope_workspace_size(const stp_qk_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_qk(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_qk_norm_rope_workspace_size: NULL output");
  *ws_bytes = align256((size_t)kQkBwdBlocks * desc->head_dim * 4);
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
  const int H = p.Hq + p.Hkv, pass = heads_per_pass(p.D) * 2;
  const int64_t passes = (H + pass - 1) / pass;
  // A token's angles are computed once per work item: one item for all heads
  // of a token, unless that leaves most of the GPU's warps without work.
  int64_t parts = p.N >= 4096 ? 1 : (4096 + p.N - 1) / p.N;
  parts = parts < passes ? parts : passes;
  p.hp = (int)((passes + parts - 1) / parts) * pass;
  p.parts = (H + p.hp - 1) / p.hp;
  const int64_t blocks = ((int64_t)p.N * p.parts + kQkThreads / 32 - 1) / (kQkThreads / 32);
  const unsigned grid = (unsigned)(blocks < 152 * 8 ? blocks : 152 * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  STP_QK_LAUNCH(qk_fwd_kernel, grid);
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
  const int H = p.Hq + p.Hkv, pass = heads_per_pass(p.D);
  int64_t parts = p.N >= 4096 ? 1 : (4096 + p.N - 1) / p.N;
  p.hp = (int)((((H + pass - 1) / pass) + parts - 1) / parts) * pass;
  const int64_t pq = (p.Hq + p.hp - 1) / p.hp, pk = (p.Hkv + p.hp - 1) / p.hp;
  const int64_t need_q = (p.N * pq + kQkThreads / 32 - 1) / (kQkThreads / 32);
  const int64_t need_k = (p.N * pk + kQkThreads / 32 - 1) / (kQkThreads / 32);
  // blocks in proportion to the heads, at most kQkBwdBlocks and one at least
  int64_t bq = (int64_t)kQkBwdBlocks * p.Hq / H;
  bq = bq < 1 ? 1 : bq > kQkBwdBlocks - 1 ? kQkBwdBlocks - 1 : bq;
  int64_t bk = kQkBwdBlocks - bq;
  p.blocks_q = (int)(bq < need_q ? bq : need_q);
  p.blocks = p.blocks_q + (int)(bk < need_k ? bk : need_k);
  STP_QK_LAUNCH(qk_bwd_kernel, (unsigned)p.blocks);
  qk_dw_kernel<<<dim3((unsigned)((p.D + 31) / 32), 2), 256, 0, s>>>(p.part, p.D, p.blocks_q, p.blocks, dw_q, dw_k);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_qk_norm_rope_bwd: %s", cudaGetErrorString(e));
  return STP_OK;
}
