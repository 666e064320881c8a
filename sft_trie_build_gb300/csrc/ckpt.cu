// Activations kept in 8 bits (layout and rounding: ckpt.h), and their return.
//
// Bound by memory: storing reads x and writes 34/32 bytes an element, restoring the
// reverse.  A warp takes 16 tokens x 64 channels and a lane two channels of all
// 16 tokens: rows of x are read 128 bytes (bf16) at a time, the lane's codes
// are two whole 16-byte pieces of the checkpoint, and nothing passes through
// shared memory.  The largest magnitude of 32 channels is found by exchange among 16
// lanes, for two tokens in one register.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ckpt.h"
#include "internal.h"
#include "layout.h"

namespace stp {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 16;   // of a warp
constexpr int kGroups = kCkTokens / kTokens;

struct CkptParams {
  int N, C, CB, along;   // blocks that lie along the channels
  int64_t stride;
  const void* x;
  void* y;
  uint8_t* ck;
};

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// cvt.e4m3x2: `hi` in the upper byte
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

// Exponent field of the scale of a float's magnitude, given by its bits: monotone in it.
__device__ __forceinline__ uint32_t scale_of(uint32_t bits) {
  if (bits >= 0x7f800000u) return kCkNaN;
  return (uint32_t)max((int)((bits + 0x1fffffu) >> 23) - 8, kCkLeast);   // carries above 1.75
}

// Two channels of one token as they lie in memory.
template <typename T>
struct Two;
template <>
struct Two<__nv_bfloat16> {
  uint32_t w;
  __device__ __forceinline__ void get(const __nv_bfloat16* p) { w = __ldcs(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void get1(const __nv_bfloat16* p) { w = *reinterpret_cast<const uint16_t*>(p); }
  __device__ __forceinline__ float lo() const { return __uint_as_float(w << 16); }
  __device__ __forceinline__ float hi() const { return __uint_as_float(w & 0xffff0000u); }
  static __device__ __forceinline__ void put(__nv_bfloat16* p, uint32_t v) { __stcs(reinterpret_cast<uint32_t*>(p), v); }
  static __device__ __forceinline__ void put1(__nv_bfloat16* p, uint32_t v) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)v;
  }
};
template <>
struct Two<float> {
  float2 w;
  __device__ __forceinline__ void get(const float* p) { w = __ldcs(reinterpret_cast<const float2*>(p)); }
  __device__ __forceinline__ void get1(const float* p) { w = make_float2(*p, 0.f); }
  __device__ __forceinline__ float lo() const { return w.x; }
  __device__ __forceinline__ float hi() const { return w.y; }
  static __device__ __forceinline__ void put(float* p, uint32_t v) {
    __stcs(reinterpret_cast<float2*>(p), make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)));
  }
  static __device__ __forceinline__ void put1(float* p, uint32_t v) { *p = __uint_as_float(v << 16); }
};

// WIDE: rows of x start at whole pairs.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) ckpt_save_kernel(const CkptParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = blockIdx.x / p.along;   // of tokens
  const int c = ((blockIdx.x - group * p.along) * (kThreads / 32) + warp) * 64 + lane * 2, n0 = group * kTokens;
  if ((c & ~63) >= p.CB * kCkChannels) return;   // the warp lies past the last block
  const T* x = static_cast<const T*>(p.x) + c;
  Two<T> v[kTokens];
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const bool on = n0 + i < p.N;
    const T* at = x + (int64_t)(n0 + i) * p.stride;
    v[i] = {};
    if (on && WIDE && c + 1 < p.C) v[i].get(at);
    else if (on && c < p.C) {
      v[i].get1(at);
      if (!WIDE && c + 1 < p.C) {
        Two<T> b = {};
        b.get1(at + 1);
        if constexpr (sizeof(T) == 2) v[i].w |= b.w << 16;
        else v[i].w.y = b.w.x;
      }
    }
  }
  uint32_t code[2][4], scale[kTokens / 2];
#pragma unroll
  for (int i = 0; i < kTokens; i += 2) {
    // the larger magnitude of each of two tokens, low and high half
    uint32_t m;
    if constexpr (sizeof(T) == 2) {
      const uint32_t a = v[i].w & 0x7fff7fffu, b = v[i + 1].w & 0x7fff7fffu;
      m = max_u16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    } else {
      const uint32_t a = max(__float_as_uint(v[i].lo()) & 0x7fffffffu, __float_as_uint(v[i].hi()) & 0x7fffffffu);
      const uint32_t b = max(__float_as_uint(v[i + 1].lo()) & 0x7fffffffu, __float_as_uint(v[i + 1].hi()) & 0x7fffffffu);
      m = scale_of(a) | scale_of(b) << 16;
    }
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = max_u16x2(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t s0 = sizeof(T) == 2 ? scale_of(m << 16) : m & 0xffff;
    const uint32_t s1 = sizeof(T) == 2 ? scale_of(m & 0xffff0000u) : m >> 16;
    const float f0 = s0 == kCkNaN ? 0.f : __uint_as_float((254 - s0) << 23);
    const float f1 = s1 == kCkNaN ? 0.f : __uint_as_float((254 - s1) << 23);
    uint32_t lo = to_e4m3x2(v[i].lo() * f0, v[i + 1].lo() * f1);
    uint32_t hi = to_e4m3x2(v[i].hi() * f0, v[i + 1].hi() * f1);
    // infinities and NaN times 0 are no codes
    const uint32_t keep = (s0 == kCkNaN ? 0u : 0xffu) | (s1 == kCkNaN ? 0u : 0xff00u);
    lo &= keep;
    hi &= keep;
    scale[i / 2] = s0 << 7 | s1 << 23;
    if (i & 2) {
      code[0][i / 4] = pack_codes(code[0][i / 4] | lo << 16);
      code[1][i / 4] = pack_codes(code[1][i / 4] | hi << 16);
    } else {
      code[0][i / 4] = lo;
      code[1][i / 4] = hi;
    }
  }
  const int cb = c / kCkChannels, in = c & (kCkChannels - 1), q = group & (kGroups - 1);
  if (cb >= p.CB) return;
  uint8_t* block = p.ck + ((int64_t)(group / kGroups) * p.CB + cb) * kCkBlock;
  uint4* to = reinterpret_cast<uint4*>(block + q * 512 + in * 16);
  to[0] = make_uint4(code[0][0], code[0][1], code[0][2], code[0][3]);
  to[1] = make_uint4(code[1][0], code[1][1], code[1][2], code[1][3]);
  if (in == 0) {
    uint4* scales = reinterpret_cast<uint4*>(block + kCkCodes + q * 32);
    scales[0] = make_uint4(scale[0], scale[1], scale[2], scale[3]);
    scales[1] = make_uint4(scale[4], scale[5], scale[6], scale[7]);
  }
}

template <typename T, bool WIDE>
__global__ void __launch_bounds__(kThreads) ckpt_load_kernel(const CkptParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = blockIdx.x / p.along;   // of tokens
  const int c = ((blockIdx.x - group * p.along) * (kThreads / 32) + warp) * 64 + lane * 2, n0 = group * kTokens;
  if (c >= p.C) return;
  const int cb = c / kCkChannels, in = c & (kCkChannels - 1), q = group & (kGroups - 1);
  const uint8_t* block = p.ck + ((int64_t)(group / kGroups) * p.CB + cb) * kCkBlock;
  const uint4* from = reinterpret_cast<const uint4*>(block + q * 512 + in * 16);
  const uint4* scales = reinterpret_cast<const uint4*>(block + kCkCodes + q * 32);
  const uint4 a4 = __ldcs(from), b4 = __ldcs(from + 1), s4 = scales[0], t4 = scales[1];
  const uint32_t a[4] = {a4.x, a4.y, a4.z, a4.w}, b[4] = {b4.x, b4.y, b4.z, b4.w};
  const uint32_t s[8] = {s4.x, s4.y, s4.z, s4.w, t4.x, t4.y, t4.z, t4.w};
  T* y = static_cast<T*>(p.y) + c;
#pragma unroll
  for (int i = 0; i < kTokens; i += 2) {
    // two tokens of either channel, then two channels of either token
    const uint32_t va = values_bf16x2(i & 2 ? late_codes(a[i / 4]) : early_codes(a[i / 4]), s[i / 2]);
    const uint32_t vb = values_bf16x2(i & 2 ? late_codes(b[i / 4]) : early_codes(b[i / 4]), s[i / 2]);
    const uint32_t v[2] = {__byte_perm(va, vb, 0x5410), __byte_perm(va, vb, 0x7632)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (n0 + i + k >= p.N) return;
      T* at = y + (int64_t)(n0 + i + k) * p.stride;
      if (WIDE && c + 1 < p.C) Two<T>::put(at, v[k]);
      else {
        Two<T>::put1(at, v[k]);
        if (c + 1 < p.C) Two<T>::put1(at + 1, v[k] >> 16);
      }
    }
  }
}

stp_status check_ckpt(const stp_ckpt_desc* d) {
  if (!d) return fail(STP_EINVAL, "checkpoint descriptor is NULL");
  if (d->dtype != STP_BF16 && d->dtype != STP_FP32) return fail(STP_EUNSUPPORTED, "dtype %d not supported", d->dtype);
  if (d->n_tokens < 0) return fail(STP_EINVAL, "n_tokens < 0");
  if (d->n_tokens > (1 << 24)) return fail(STP_EUNSUPPORTED, "more than 2^24 tokens");
  if (d->dim < 1 || d->dim > 65536) return fail(STP_EUNSUPPORTED, "dim must lie in [1, 65536]");
  if (d->stride < d->dim) return fail(STP_EINVAL, "stride must be at least dim");
  return STP_OK;
}

template <typename T>
void launch(const CkptParams& p, bool save, bool wide, cudaStream_t s) {
  // every 16 tokens of the last block are written, so that it ends in zeros
  const int groups = save ? (int)ck_token_blocks(p.N) * kGroups : (p.N + kTokens - 1) / kTokens;
  const unsigned grid = (unsigned)groups * p.along;
  if (save && wide) ckpt_save_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
  else if (save) ckpt_save_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
  else if (wide) ckpt_load_kernel<T, true><<<grid, kThreads, 0, s>>>(p);
  else ckpt_load_kernel<T, false><<<grid, kThreads, 0, s>>>(p);
}

stp_status ckpt(const char* name, const stp_ckpt_desc* d, const void* x, void* y, const void* ck, void* stream) {
  clear_error();
  stp_status st = check_ckpt(d);
  if (st) return st;
  if (d->n_tokens == 0) return STP_OK;
  const void* t = x ? x : y;
  if (!t || !ck) return fail(STP_EINVAL, "%s: NULL device pointer", name);
  if (reinterpret_cast<uintptr_t>(ck) & 255) return fail(STP_EINVAL, "%s: the checkpoint must be 256-byte aligned", name);
  const int size = d->dtype == STP_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(t) & (size - 1)) return fail(STP_EINVAL, "%s: the tensor is misaligned for its type", name);
  CkptParams p{};
  p.N = d->n_tokens;
  p.C = d->dim;
  p.CB = (int)ck_channel_blocks(p.C);
  p.along = (p.CB * kCkChannels + kThreads * 2 - 1) / (kThreads * 2);
  p.stride = d->stride;
  p.x = x;
  p.y = y;
  p.ck = static_cast<uint8_t*>(const_cast<void*>(ck));
  const bool wide = reinterpret_cast<uintptr_t>(t) % (2 * size) == 0 && p.stride % 2 == 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (size == 2) launch<__nv_bfloat16>(p, x != nullptr, wide, s);
  else launch<float>(p, x != nullptr, wide, s);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(STP_ECUDA, "%s: %s", name, cudaGetErrorString(e));
  return STP_OK;
}

}  // namespace

stp_status check_ckpt_desc(const stp_ckpt_desc* d) { return check_ckpt(d); }

}  // namespace stp

using namespace stp;

extern "C" stp_status stp_ckpt_size(const stp_ckpt_desc* desc, size_t* ckpt_bytes) {
  clear_error();
  stp_status st = check_ckpt_desc(desc);
  if (st) return st;
  if (!ckpt_bytes) return fail(STP_EINVAL, "stp_ckpt_size: NULL output");
  *ckpt_bytes = align256((size_t)(ck_token_blocks(desc->n_tokens) * ck_channel_blocks(desc->dim)) * kCkBlock);
  return STP_OK;
}

extern "C" stp_status stp_ckpt_save(const stp_ckpt_desc* desc, const void* x, void* d_ckpt, void* stream) {
  if (!x && desc && desc->n_tokens > 0) return fail(STP_EINVAL, "stp_ckpt_save: NULL device pointer");
  return ckpt("stp_ckpt_save", desc, x, nullptr, d_ckpt, stream);
}

extern "C" stp_status stp_ckpt_load(const stp_ckpt_desc* desc, const void* d_ckpt, void* x, void* stream) {
  return ckpt("stp_ckpt_load", desc, nullptr, x, d_ckpt, stream);
}
