// Layout of an activation checkpoint in 8 bits, and its exact return to bf16.
//
// A checkpoint of x [N, C] is an array of blocks of 64 tokens x 32 channels,
// channel blocks of the same tokens side by side, 2112 bytes each:
//   codes  uint8 [4][32][16]   e4m3 code of token 16 q + i and channel c at [q][c][i]
//   scale  uint8 [64]          of each token: 2^(scale - 127) times a code is the value
// Tokens lie next to one another, as the weight gradient contracts over them: a
// thread that owns a channel reads 16 tokens at once.  Tokens and channels past
// the end are zeros.  The scale is the smallest power of two, from 2^-117 on, at which the 32
// channels' largest magnitude is at most 448 (e4m3's largest); a block that
// holds an infinity or a NaN has scale 255 and codes 0, which return as NaN.
//
// A code has four significant bits and a power of two leaves them as they are,
// so the values are exact in bf16 (the smallest is 2^-9 2^-117, a normal number).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace stp {

constexpr int kCkTokens = 64, kCkChannels = 32;
constexpr int kCkCodes = kCkTokens * kCkChannels;
constexpr int kCkBlock = kCkCodes + kCkTokens;   // bytes, a multiple of 16
constexpr int kCkLeast = 10;                     // scale of 2^-117
constexpr int kCkNaN = 255;

inline int64_t ck_token_blocks(int64_t n) { return (n + kCkTokens - 1) / kCkTokens; }
inline int64_t ck_channel_blocks(int64_t c) { return (c + kCkChannels - 1) / kCkChannels; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two codes, in bits 8..15 and 24..31 of x, times 2^120 2^-127 each: the code's
// exponent and fraction in bf16's places are the value times 2^-120, below the
// smallest normal for e4m3's subnormals; the product with 2^120 is exact.
__device__ __forceinline__ uint32_t codes_bf16x2(uint32_t x) {
  return mul_bf16x2((x & 0x80008000u) | ((x >> 4) & 0x07f007f0u), 0x7b807b80u);
}

// Factors 2^(scale - 127) as bf16 of two tokens whose scales lie in bytes 0 and 2.
__device__ __forceinline__ uint32_t scales_bf16x2(uint32_t b) { return b << 7; }

}  // namespace stp
