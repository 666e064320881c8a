// Clipped policy loss on rows of logits, with a KL term towards a reference
// policy and an entropy term: loss, gradient, and both in one launch.
//
// Per row, from one pass (logit_rows.cuh): lp = z_t - lse and the entropy H;
//   r = exp(lp - old),  k = exp(ref - lp) - (ref - lp) - 1,
//   loss = -min(r A, clip(r, 1 - lo, 1 + hi) A) + beta k - gamma H.
// Its derivatives by lp and H are two numbers of the row,
//   g = -A r [r not clipped] + beta (1 - exp(ref - lp))  and  -gamma,
// so the gradient by a logit is
//   dz_v = w scale (g ([v = t] - p_v) + gamma p_v (ln p_v + H)).
//
// Bound by memory, as token_loss.cu: forward one read, backward one read and
// one write, the step one read and one write, its second pass out of L2.  The
// token's own logit is put right by one store after the pass, so that the pass
// compares no ids.  Short rows are a warp's, whose sums take no meeting of a
// block.
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

struct PolicyParams {
  int N, V, C;
  int64_t stride;
  float scale, sl2, low, high, beta, gamma;   // low = 1 - clip_low, high = 1 + clip_high
  const void* z;
  const int32_t* target;
  const float* old_lp;
  const float* ref_lp;   // may be null
  const float* adv;
  const float* w;
  float* loss;
  float* logprob;
  float* entropy;
  float* lse;
  float* kl;             // may be null
  // backward
  const float* lp_in;
  const float* ent_in;
  const float* lse_in;
  void* dz;
  uint32_t* err;
  bool check;   // a block past the rows checks all targets
};

// exp(x) - x - 1 without the cancellation near 0: its series to x^9 / 9!, which
// is within 2^-24 of it on [-1/2, 1/2].  Far up the rest is below exp(x)'s last
// bit (and infinity stays one).
__device__ __forceinline__ float exp_rest(float x) {
  if (x > 40.f) return expm1f(x);
  if (fabsf(x) > 0.5f) return expm1f(x) - x;
  float s = 1.f / 362880;
  s = fmaf(s, x, 1.f / 40320);
  s = fmaf(s, x, 1.f / 5040);
  s = fmaf(s, x, 1.f / 720);
  s = fmaf(s, x, 1.f / 120);
  s = fmaf(s, x, 1.f / 24);
  s = fmaf(s, x, 1.f / 6);
  s = fmaf(s, x, 0.5f);
  return s * x * x;
}

// The terms of a row and their derivative by lp.
struct Terms {
  float loss, kl, g;   // loss without the entropy term
};

__device__ __forceinline__ Terms terms_of(const PolicyParams& p, int n, float lp) {
  const float a = p.adv[n], r = expf(lp - p.old_lp[n]);
  const float bound = a >= 0.f ? p.high : p.low;
  const bool out = a >= 0.f ? r > bound : r < bound;
  Terms t;
  t.loss = -a * (out ? bound : r);
  t.g = out ? 0.f : -a * r;
  t.kl = 0.f;
  if (p.ref_lp) {
    const float x = p.ref_lp[n] - lp;
    t.kl = exp_rest(x);
    if (p.beta != 0.f) {   // 0 times an infinite term is no term
      t.loss = fmaf(p.beta, t.kl, t.loss);
      t.g = fmaf(-p.beta, expm1f(x), t.g);
    }
  }
  return t;
}

// ln s in two numbers, of which the first is exact: s = 2^e f with f near 1, and
// ln 2 is split so that e times its first part has no rounding (Cody and Waite's
// reduction).  The log-probability of a likely token is the difference of two
// numbers near 10, whose own roundings would be all its error.
__device__ __forceinline__ float2 log_parts(float s) {
  if (!(s > 0.f && s < INFINITY)) return make_float2(logf(s), 0.f);
  const int bits = __float_as_int(s), up = (bits & 0x7fffff) > 0x3504f3;   // f above the root of 2 is halved
  const float e = (float)((bits >> 23) - 127 + up);
  const float f = __int_as_float((bits & 0x7fffff) | ((127 - up) << 23));
  return make_float2(e * 0.693359375f, fmaf(e, -2.12194440e-4f, logf(f)));
}

// What a row has besides its gradient, from its sums.
// p = exp(scale (x - m)) / s and ln p = scale (x - m) - ref, which hold for
// logits of any size; from lse alone ref = lse, m = 0.
struct Row {
  float m, ref, ent, lp, inv;   // inv = 1 / s
};
__device__ __forceinline__ Row row_of(const PolicyParams& p, const Acc& s, float zt) {
  const bool none = s.m == -INFINITY && s.s == 0.f;   // nothing but -inf
  const float2 ln = log_parts(s.s);
  Row r;
  r.m = s.m;
  r.ref = ln.x + ln.y;
  r.lp = none && !isnan(zt) ? -INFINITY : fmaf(zt - r.m, p.scale, -ln.x) - ln.y;
  r.inv = 1.f / s.s;
  r.ent = none ? 0.f : fmaf(-kLn2T, s.t * r.inv, ln.x) + ln.y;
  return r;
}
__device__ __forceinline__ void put_outputs(const PolicyParams& p, int n, const Row& r, const Terms& term) {
  p.lse[n] = r.m == -INFINITY && r.lp == -INFINITY ? -INFINITY : fmaf(r.m, p.scale, r.ref);
  p.logprob[n] = r.lp;
  p.entropy[n] = r.ent;
  p.loss[n] = p.gamma != 0.f ? fmaf(-p.gamma, r.ent, term.loss) : term.loss;
  if (p.kl) p.kl[n] = term.kl;
}
__device__ __forceinline__ void put_unread(const PolicyParams& p, int n, int target) {
  const float x = target < 0 ? 0.f : NAN;
  p.loss[n] = p.logprob[n] = p.entropy[n] = p.lse[n] = x;
  if (p.kl) p.kl[n] = x;
  if (!p.check && target >= p.V) atomicOr(p.err, kErrBadList);
}

// An infinite factor of a gradient (a ratio beyond float32's range) is held at
// the largest number that bf16 has, too, so that 0 times it is 0.
__device__ __forceinline__ float held(float x) { return isinf(x) ? copysignf(0x1.fep127f, x) : x; }

// dz = p (h ln p + c), and g more for the token itself.  LSE: from the row's
// maximum and sum (whose inverse is in h2 and c), else from lse alone.  Where ln p
// lies below kLowest p is 0 already, and ln p is held there, so that its product
// with a large weight stays finite.
template <bool LSE>
struct RowGrad {
  float scale, sl2, sub, up, shift, h2, c, g;
  __device__ __forceinline__ RowGrad(const PolicyParams& p, int n, const Row& r, const Terms& term) {
    const float w = p.w[n] * p.scale, h = held(w * p.gamma), inv = LSE ? r.inv : 1.f;
    g = held(w * term.g);
    c = held((p.gamma != 0.f ? fmaf(h, r.ent, -g) : -g) * inv);
    h2 = h * kLn2T * inv;
    scale = p.scale;
    sl2 = p.sl2;
    shift = -r.ref * kLog2eT;
    up = -r.ref;
    sub = -r.m;
  }
  __device__ __forceinline__ float operator()(float x) const {
    const float d = LSE ? (x + sub) * sl2 : fmaf(x, scale, up) * kLog2eT;
    const float l2 = LSE ? d + shift : d;   // ln p in units of ln 2
    return ex2(d) * fmaf(h2, fmaxf(l2, kLowest), c);
  }
  // Two by two, as the pass issues more than it may; without an entropy term p times one number.
  template <bool ENT, int N>
  __device__ __forceinline__ void apply(float* z) const {
    if constexpr (N % 2) {
#pragma unroll
      for (int e = 0; e < N; ++e) z[e] = (*this)(z[e]);
    } else {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float2 x = make_float2(z[e], z[e + 1]);
        const float2 d =
            LSE ? __fmul2_rn(__fadd2_rn(x, make_float2(sub, sub)), make_float2(sl2, sl2))
                : __fmul2_rn(__ffma2_rn(x, make_float2(scale, scale), make_float2(up, up)), make_float2(kLog2eT, kLog2eT));
        float2 term = make_float2(c, c);
        if constexpr (ENT) {
          const float2 l = LSE ? __fadd2_rn(d, make_float2(shift, shift)) : d;
          term = __ffma2_rn(make_float2(h2, h2), make_float2(fmaxf(l.x, kLowest), fmaxf(l.y, kLowest)), term);
        }
        const float2 p2 = __fmul2_rn(make_float2(ex2(d.x), ex2(d.y)), term);
        z[e] = p2.x;
        z[e + 1] = p2.y;
      }
    }
  }
};

constexpr int kShortFlight = 8;   // logits of a lane at a time, in a warp's row

// Whether rows are a warp's: short ones, and many of them or very short ones.
// Measured in us, a block's and a warp's, of 20000 bf16 rows: step of 1000 logits 157 / 41,
// of 4096 193 / 120, of 8000 206 / 243; forward of 1000 108 / 22, of 8000 141 / 98;
// step of 200 rows of 2048 8.6 / 13.5.
bool short_rows(int n, int vocab, bool grad) {
  return vocab <= (grad ? 4096 : 8192) && (n >= 1216 || vocab <= 512);
}

template <typename T, bool LSE, bool GRAD>
__global__ void __launch_bounds__(kRowThreads) policy_short_kernel(const PolicyParams p) {
  if (LSE && p.check && blockIdx.x == gridDim.x - 1) {
    check_below(p.N, p.V, p.err, [&](int64_t i) { return p.target[i]; });
    return;
  }
  const int n = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (n >= p.N) return;
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  T* out = GRAD ? static_cast<T*>(p.dz) + (int64_t)n * p.stride : nullptr;
  const int target = p.target[n];
  if (target < 0 || target >= p.V) {
    if (LSE && lane == 0) put_unread(p, n, target);
    if (GRAD)
      for (int i = lane; i < p.V; i += 32) put(out + i, 0.f);
    return;
  }
  const auto load = [&](int i0, float* z) {
#pragma unroll
    for (int k = 0; k < kShortFlight; ++k) z[k] = i0 + k * 32 < p.V ? to_f(row[i0 + k * 32]) : -INFINITY;
  };
  const float zt = to_f(row[target]);
  Row r{};
  if (LSE) {
    Acc a = {-INFINITY, 0.f, 0.f};
    for (int i0 = lane; i0 - lane < p.V; i0 += 32 * kShortFlight) {
      float z[kShortFlight], most, least;
      load(i0, z);
      extremes<kShortFlight>(z, most, least);
      add<kShortFlight, true>(a, z, most, least, p.sl2);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      Acc b;
      b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
      b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
      b.t = __shfl_xor_sync(0xffffffffu, a.t, o);
      a = merge(a, b, p.sl2);
    }
    r = row_of(p, a, zt);
  } else {
    r = {0.f, p.lse_in[n], p.ent_in[n], p.lp_in[n], 1.f};
  }
  const Terms term = terms_of(p, n, r.lp);
  if (LSE && lane == 0) put_outputs(p, n, r, term);
  if (GRAD) {
    __syncwarp();   // every lane has zt before a logit may be overwritten
    const RowGrad<LSE> grad(p, n, r, term);
    const bool zero = r.lp == -INFINITY;   // no step can raise it
    for (int i0 = lane; i0 - lane < p.V; i0 += 32 * kShortFlight) {
      float z[kShortFlight];
      load(i0, z);
      grad.template apply<true, kShortFlight>(z);
#pragma unroll
      for (int k = 0; k < kShortFlight; ++k) {
        const int i = i0 + k * 32;
        if (i < p.V) put(out + i, zero ? 0.f : i == target ? grad(zt) + grad.g : z[k]);
      }
    }
  }
}

// Forward (LSE), backward (GRAD) or both.  MANY: several blocks per row.  FOUR: a
// step's rows are small enough for as many blocks on an SM as a pass has.
template <typename T, bool LSE, bool GRAD, bool MANY, bool FOUR = false>
__global__ void __launch_bounds__(kRowThreads, LSE && GRAD && !FOUR ? kStepBlocks : kPassBlocks)
    policy_kernel(const PolicyParams p) {
  __shared__ Acc red[kRowWarps];
  __shared__ Acc sums[kMaxSplit];   // of the row's blocks
  extern __shared__ uint4 buffer[];
  const int C = MANY ? p.C : 1, n = (int)(blockIdx.x / C), rank = MANY ? (int)(blockIdx.x % C) : 0, t = threadIdx.x;
  if (LSE && n == p.N) {
    if (rank == 0) check_below(p.N, p.V, p.err, [&](int64_t i) { return p.target[i]; });
    return;
  }
  const T* row = static_cast<const T*>(p.z) + (int64_t)n * p.stride;
  T* out = GRAD ? static_cast<T*>(p.dz) + (int64_t)n * p.stride : nullptr;
  const int target = p.target[n];
  if (target < 0 || target >= p.V) {   // the same for every block of the row
    if (LSE && rank == 0 && t == 0) put_unread(p, n, target);
    if (GRAD) zero_row(out, p.V, rank, C);
    return;
  }
  const Part part = part_of(row, p.V, rank, C);
  const auto ring = ring_of<LSE && GRAD && !FOUR ? kStepRounds : kPassRounds>(buffer, row, part);
  ring.start(part.b0 + t);
  if (LSE && MANY) cg::this_cluster().barrier_arrive();   // this block runs: others may write to it
  const bool mine = target >= part.lo && target < part.hi;
  // backward alone: other blocks may write over what is not their part already
  const float zt = LSE || mine ? to_f(row[target]) : 0.f;
  Row r;
  if (LSE) {
    float best;
    int round;
    Acc s = pass<T, true, false>(row, part, ring, p.sl2, best, round);
    if (GRAD) ring.start(part.b0 + t);   // again, now out of L2
    s = block_sum(s, red, p.sl2);
    if (MANY) {
      cg::cluster_group cl = cg::this_cluster();
      cl.barrier_wait();
      if (t < C) *cl.map_shared_rank(sums + rank, t) = s;
      cl.sync();
      s = merge_all(sums, C, p.sl2);
    }
    r = row_of(p, s, zt);
  } else {
    r = {0.f, p.lse_in[n], p.ent_in[n], p.lp_in[n], 1.f};
  }
  const Terms term = terms_of(p, n, r.lp);
  if (LSE && rank == 0 && t == 0) put_outputs(p, n, r, term);
  if (GRAD) {
    __syncthreads();   // every zt is read before a logit may be overwritten
    if (r.lp == -INFINITY) {   // no step can raise it
      asm volatile("cp.async.wait_all;" ::: "memory");
      zero_row(out, p.V, rank, C);
      return;
    }
    const RowGrad<LSE> grad(p, n, r, term);
    if (grad.h2 == 0.f)
      map_row(row, out, part, ring, [=](float* z, int, auto N) { grad.template apply<false, decltype(N)::value>(z); });
    else
      map_row(row, out, part, ring, [=](float* z, int, auto N) { grad.template apply<true, decltype(N)::value>(z); });
    __syncthreads();   // the block's stores before that of the token
    if (mine && t == 0) put(out + target, grad(zt) + grad.g);
  }
}

// ------------------------------------------------------------------- host

stp_status check_policy(const stp_policy_desc* d) {
  if (!d) return fail(STP_EINVAL, "policy descriptor is NULL");
  if (!(d->clip_low >= 0.f && d->clip_low <= 1.f) || !(d->clip_high >= 0.f && d->clip_high <= 1e4f))
    return fail(STP_EINVAL, "clip_low must lie in [0, 1] and clip_high in [0, 1e4]");
  if (!(d->kl_coef >= 0.f && d->kl_coef <= 1e4f) || !(d->entropy_coef >= -1e4f && d->entropy_coef <= 1e4f))
    return fail(STP_EINVAL, "kl_coef must lie in [0, 1e4] and entropy_coef in [-1e4, 1e4]");
  return check_rows(d->n_rows, d->vocab, d->stride, d->dtype, d->scale);
}

// How the rows of a call are taken.
enum Form { kWarp, kBlock, kFour, kMany };

// A step's rows of up to 100 KB: four blocks on an SM.  Measured in us, three and four: rows of 64 KB
// (16000) 380 / 341, of 100 KB (8000) 270 / 258, of 120 KB (8000) 317 / 348.
constexpr int64_t kFourBytes = 100 << 10;

template <typename T, bool LSE, bool GRAD>
const void* policy_as(Form f) {
  if (f == kWarp) return (const void*)policy_short_kernel<T, LSE, GRAD>;
  if constexpr (!LSE) return (const void*)policy_kernel<T, false, true, true>;
  if constexpr (LSE && GRAD)
    if (f == kFour) return (const void*)policy_kernel<T, true, true, false, true>;
  return f == kMany ? (const void*)policy_kernel<T, LSE, GRAD, true> : (const void*)policy_kernel<T, LSE, GRAD, false>;
}
template <typename T>
const void* policy_of(bool lse, bool grad, Form f) {
  if (!lse) return policy_as<T, false, true>(f);
  return grad ? policy_as<T, true, true>(f) : policy_as<T, true, false>(f);
}
int rounds_of(bool lse, bool grad, Form f) { return lse && grad && f != kFour ? kStepRounds : kPassRounds; }

// The kernels' dynamic shared memory, above the default limit.
cudaError_t allow_policy() {
  static PerDevice limits;
  return limits([] {
    cudaError_t e = cudaSuccess;
    for (const bool lse : {false, true})
      for (const bool grad : {false, true})
        for (const Form f : {kBlock, kFour, kMany})
          for (const void* k : {policy_of<__nv_bfloat16>(lse, grad, f), policy_of<float>(lse, grad, f)})
            if (e == cudaSuccess)
              e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes(rounds_of(lse, grad, f)));
    return e;
  });
}

// What the three calls share; p holds the pointers.
stp_status policy(const char* name, const stp_policy_desc* d, PolicyParams p, void* ws, bool fwd, bool grad,
                  void* stream) {
  clear_error();
  stp_status st = check_policy(d);
  if (st) return st;
  if (fwd && (!ws || reinterpret_cast<uintptr_t>(ws) & 255))
    return fail(STP_EINVAL, "%s: the workspace must be 256-byte aligned", name);
  if (d->n_rows > 0 &&
      (!p.z || !p.target || !p.old_lp || !p.adv || (fwd && (!p.loss || !p.logprob || !p.entropy || !p.lse)) ||
       (grad && (!p.w || !p.dz)) || (!fwd && (!p.lp_in || !p.ent_in || !p.lse_in))))
    return fail(STP_EINVAL, "%s: NULL device pointer", name);
  if (d->kl_coef != 0.f && d->n_rows > 0 && !p.ref_lp)
    return fail(STP_EINVAL, "%s: kl_coef needs ref_logprob", name);
  if (off_type(p.z, d->dtype) || off_type(p.dz, d->dtype))
    return fail(STP_EINVAL, "%s: logits misaligned for their type", name);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.check = fwd && d->n_rows > 0 && d->n_rows <= kCheckMost;
  cudaError_t e = fwd && !p.check ? cudaMemsetAsync(ws, 0, 4, s) : cudaSuccess;
  if (e == cudaSuccess && d->n_rows > 0) {
    p.N = d->n_rows;
    p.V = d->vocab;
    p.stride = d->stride;
    p.scale = d->scale;
    p.sl2 = d->scale * kLog2eT;
    p.low = 1.f - d->clip_low;
    p.high = 1.f + d->clip_high;
    p.beta = d->kl_coef;
    p.gamma = d->entropy_coef;
    p.err = static_cast<uint32_t*>(ws);
    const int64_t bytes = row_bytes(p.V, d->dtype);
    const bool both = fwd && grad;
    p.C = both ? step_split_of(p.N, bytes) : split_of(p.N, bytes);
    const Form f = short_rows(p.N, p.V, grad) ? kWarp : p.C > 1 ? kMany : both && bytes <= kFourBytes ? kFour : kBlock;
    const void* k = d->dtype == STP_BF16 ? policy_of<__nv_bfloat16>(fwd, grad, f) : policy_of<float>(fwd, grad, f);
    if (f == kWarp) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)(((int64_t)p.N + kRowWarps - 1) / kRowWarps + p.check));
      cfg.blockDim = dim3(kRowThreads);
      cfg.stream = s;
      void* args[] = {&p};
      e = cudaLaunchKernelExC(&cfg, k, args);
    } else {
      e = allow_policy();
      if (e == cudaSuccess) e = launch_rows(k, rounds_of(fwd, grad, f), p.N + p.check, p.C, &p, fwd, s);
    }
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "%s: %s", name, cudaGetErrorString(e));
  return STP_OK;
}

PolicyParams given(const void* logits, const int32_t* targets, const float* old_lp, const float* ref_lp,
                   const float* adv) {
  PolicyParams p{};
  p.z = logits;
  p.target = targets;
  p.old_lp = old_lp;
  p.ref_lp = ref_lp;
  p.adv = adv;
  return p;
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_policy_workspace_size(const stp_policy_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_policy(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_policy_workspace_size: NULL output");
  *ws_bytes = 256;
  return STP_OK;
}

extern "C" stp_status stp_policy_fwd(const stp_policy_desc* desc, const void* logits, const int32_t* d_targets,
                                     const float* old_logprob, const float* ref_logprob, const float* advantage,
                                     float* loss, float* logprob, float* entropy, float* lse, float* kl, void* d_ws,
                                     void* stream) {
  PolicyParams p = given(logits, d_targets, old_logprob, ref_logprob, advantage);
  p.loss = loss;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.kl = kl;
  return policy("stp_policy_fwd", desc, p, d_ws, true, false, stream);
}

extern "C" stp_status stp_policy_bwd(const stp_policy_desc* desc, const void* logits, const int32_t* d_targets,
                                     const float* old_logprob, const float* ref_logprob, const float* advantage,
                                     const float* logprob, const float* entropy, const float* lse,
                                     const float* d_loss, void* d_logits, void* stream) {
  PolicyParams p = given(logits, d_targets, old_logprob, ref_logprob, advantage);
  p.lp_in = logprob;
  p.ent_in = entropy;
  p.lse_in = lse;
  p.w = d_loss;
  p.dz = d_logits;
  return policy("stp_policy_bwd", desc, p, nullptr, false, true, stream);
}

extern "C" stp_status stp_policy_step(const stp_policy_desc* desc, const void* logits, const int32_t* d_targets,
                                      const float* old_logprob, const float* ref_logprob, const float* advantage,
                                      const float* d_loss, float* loss, float* logprob, float* entropy, float* lse,
                                      float* kl, void* d_logits, void* d_ws, void* stream) {
  PolicyParams p = given(logits, d_targets, old_logprob, ref_logprob, advantage);
  p.loss = loss;
  p.logprob = logprob;
  p.entropy = entropy;
  p.lse = lse;
  p.kl = kl;
  p.w = d_loss;
  p.dz = d_logits;
  return policy("stp_policy_step", desc, p, d_ws, true, true, stream);
}
