// Layout of an activation checkpoint in 8 bits, and its exact return to bf16.
//
// A checkpoint of x [N, C] is an array of blocks of 128 tokens x 32 channels,
// channel blocks of the same tokens side by side, 4352 bytes each:
//   codes  uint32 [8][32][4]   e4m3 codes of tokens 16 q + 4 i .. 16 q + 4 i + 3, channel c, at [q][c][i]
//   scale  bf16 [128]          of each token: scale times a code is the value
// Tokens lie next to one another, as the weight gradient contracts over them: a
// thread that owns a channel reads 16 tokens at once.  Tokens and channels past
// the end are zeros.  The scale is the smallest power of two, from 2^-117 on, at which the 32
// channels' largest magnitude is at most 448 (e4m3's largest); a block that
// holds an infinity or a NaN has scale NaN and any codes, and returns as NaN.
//
// A code has four significant bits and a power of two leaves them as they are,
// so the values are exact in bf16 (the smallest is 2^-9 2^-117, a normal number).
// Its exponent and fraction, in the places of bf16's lowest exponent bits and
// highest fraction bits, are the value times 2^-120 (below the smallest normal
// number for e4m3's subnormals), and multiplying by 2^120 is exact.
//
// The four codes of a word are laid out so that they come back as two pairs with
// five operations: the later two tokens' bits are in place (sign 15, exponent
// and fraction 10..4 of a half), the earlier two's fill the gaps, four places away
// from theirs (sign in 11, upper exponent bits in 14..12, the rest in 3..0).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace stp {

constexpr int kCkTokens = 128, kCkChannels = 32;
constexpr int kCkCodes = kCkTokens * kCkChannels;
constexpr int kCkBlock = kCkCodes + kCkTokens * 2;   // bytes, a multiple of 16
constexpr uint32_t kCkLeast = 10;                    // exponent field of 2^-117
constexpr uint32_t kCkNaN = 0x7fc0;                  // a bf16 NaN

inline int64_t ck_token_blocks(int64_t n) { return (n + kCkTokens - 1) / kCkTokens; }
inline int64_t ck_channel_blocks(int64_t c) { return (c + kCkChannels - 1) / kCkChannels; }

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two and two codes of successive tokens, each pair in a number's lower bytes,
// to their places in a word, and back; `early` are the first two tokens' values times 2^-120,
// `late` the other two's.
__device__ __forceinline__ uint32_t pack_codes(uint32_t early, uint32_t late) {
  const uint32_t x = __byte_perm(early, 0, 0x1404), y = __byte_perm(late, 0, 0x1404);   // in the halves' upper bytes
  return (x & 0x70007000u) | ((x >> 8) & 0x000f000fu) | ((x >> 4) & 0x08000800u) | (y & 0x80008000u) |
         ((y >> 4) & 0x07f007f0u);
}
__device__ __forceinline__ uint32_t late_codes(uint32_t w) { return w & 0x87f087f0u; }
__device__ __forceinline__ uint32_t early_codes(uint32_t w) {
  return ((w << 4) & 0x80f080f0u) | ((w >> 4) & 0x07000700u);
}

// Codes as above times their scales.
__device__ __forceinline__ uint32_t values_bf16x2(uint32_t codes, uint32_t scales) {
  return mul_bf16x2(mul_bf16x2(codes, 0x7b807b80u), scales);
}

}  // namespace stp
