// Activations kept in 8 bits (layout and rounding: ckpt.h), and their return.
//
// Bound by memory: storing reads x and writes 34/32 bytes an element, restoring the
// reverse.  A warp takes 16 tokens x 64 channels and a lane two channels of all
// 16 tokens: rows of x are read 128 bytes (bf16) at a time, the lane's codes
// are two whole 16-byte pieces of the checkpoint, and nothing passes through
// shared memory.  The largest magnitudes of 16 lanes' 32 channels are found by
// halving: a lane gives away the tokens of which it is not to know the maximum, two tokens
// in a register, so that a lane works out the scales of two tokens instead of
// all sixteen (16384 x 4096 bf16: 40 us against 50 with every lane working out
// all; 38 since tokens that are all there are read without tests).
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

// A float's magnitude as 16 bits, monotone in it and exact at the borders
// between scales: its upper half, and a last bit for what lies below.
__device__ __forceinline__ uint32_t key_of(uint32_t bits) {
  bits &= 0x7fffffffu;
  return bits >> 16 | ((bits & 0xffffu) != 0);
}

// The scale of a largest magnitude (its key) as bf16, and one over it: above 1.75 the exponent carries.
__device__ __forceinline__ void scale_of(uint32_t key, uint32_t& scale, uint32_t& inverse) {
  const uint32_t field = max((int)((key + 0x1fu) >> 7) - 8, (int)kCkLeast);
  const bool finite = key < 0x7f80u;
  scale = finite ? field << 7 : kCkNaN;
  inverse = finite ? (254 - field) << 7 : 0;
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
  if (WIDE && n0 + kTokens <= p.N && (c | 63) < p.C) {   // all of it is there
#pragma unroll
    for (int i = 0; i < kTokens; ++i) v[i].get(x + (n0 + i) * p.stride);
  } else {
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const bool on = n0 + i < p.N;
      const T* at = x + (n0 + i) * p.stride;
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
  }
  // the larger magnitude of the lane's two channels, two tokens in a register
  uint32_t m[kTokens / 2];
#pragma unroll
  for (int i = 0; i < kTokens; i += 2) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t a = v[i].w & 0x7fff7fffu, b = v[i + 1].w & 0x7fff7fffu;
      m[i / 2] = max_u16x2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
    } else {
      m[i / 2] = max_u16x2(key_of(__float_as_uint(v[i].lo())) | key_of(__float_as_uint(v[i + 1].lo())) << 16,
                           key_of(__float_as_uint(v[i].hi())) | key_of(__float_as_uint(v[i + 1].hi())) << 16);
    }
  }
  // among 16 lanes: lane 2 j and 2 j + 1 come to hold tokens 2 j and 2 j + 1
#pragma unroll
  for (int o = 8, left = 4; o > 1; o >>= 1, left >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < left; ++i) {
      const uint32_t keep = up ? m[i + left] : m[i], give = up ? m[i] : m[i + left];
      m[i] = max_u16x2(keep, __shfl_xor_sync(0xffffffffu, give, o));
    }
  }
  m[0] = max_u16x2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1));
  uint32_t s0, s1, r0, r1;
  scale_of(m[0] & 0xffffu, s0, r0);
  scale_of(m[0] >> 16, s1, r1);
  const uint32_t scales = s0 | s1 << 16, inverse = r0 | r1 << 16;
  uint32_t code[2][kTokens / 4];
#pragma unroll
  for (int i = 0; i < kTokens; i += 4) {
    uint32_t lo[2], hi[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t f = __shfl_sync(0xffffffffu, inverse, (lane & 16) | (i + 2 * k));
      const float f0 = __uint_as_float(f << 16), f1 = __uint_as_float(f & 0xffff0000u);
      lo[k] = to_e4m3x2(v[i + 2 * k].lo() * f0, v[i + 2 * k + 1].lo() * f1);
      hi[k] = to_e4m3x2(v[i + 2 * k].hi() * f0, v[i + 2 * k + 1].hi() * f1);
    }
    code[0][i / 4] = pack_codes(lo[0], lo[1]);
    code[1][i / 4] = pack_codes(hi[0], hi[1]);
  }
  const int cb = c / kCkChannels, in = c & (kCkChannels - 1), q = group & (kGroups - 1);
  if (cb >= p.CB) return;
  uint8_t* block = p.ck + ((int64_t)(group / kGroups) * p.CB + cb) * kCkBlock;
  uint4* to = reinterpret_cast<uint4*>(block + q * 512 + in * 16);
  to[0] = make_uint4(code[0][0], code[0][1], code[0][2], code[0][3]);
  to[1] = make_uint4(code[1][0], code[1][1], code[1][2], code[1][3]);
  if (!(lane & 1)) reinterpret_cast<uint32_t*>(block + kCkCodes + q * 32)[(lane & 15) / 2] = scales;
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
  const bool full = n0 + kTokens <= p.N;
#pragma unroll
  for (int i = 0; i < kTokens; i += 2) {
    // two tokens of either channel, then two channels of either token
    const uint32_t va = values_bf16x2(i & 2 ? late_codes(a[i / 4]) : early_codes(a[i / 4]), s[i / 2]);
    const uint32_t vb = values_bf16x2(i & 2 ? late_codes(b[i / 4]) : early_codes(b[i / 4]), s[i / 2]);
    const uint32_t v[2] = {__byte_perm(va, vb, 0x5410), __byte_perm(va, vb, 0x7632)};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!full && n0 + i + k >= p.N) return;
      T* at = y + (n0 + i + k) * p.stride;
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
  if (reinterpret_cast<uintptr_t>(t) & (size - 1))
    return fail(STP_EINVAL, "%s: the tensor is misaligned for its type", name);
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
