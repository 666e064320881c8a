// Weight gradient of a projection from its input kept in 8 bits:
//
//   dW[c, m] (+)= sum_n x^[n, c] dY[n, m],   x^ as ckpt.h restores it.
//
// x^ is exact in bf16, so the products are those of the stored values; sums are
// float32 on the tensor cores (tcgen05, M = 128 channels, N <= 256 columns of
// dY, K = tokens).
//
// Two blocks of a cluster multiply a tile of 256 channels x up to 256 columns
// together (cta_group::2): each holds the sums of its 128 channels in TMEM and half of
// dY's columns in shared memory.  Operand A is in TMEM, too: a warp owns 32
// channels, a lane one of them (a TMEM lane), reads the codes of 128 tokens from
// shared memory, turns them to bf16 (ckpt.h) and stores them to TMEM, four stages of 64
// columns behind the 256 columns of sums.  So shared memory carries the codes and half a tile of dY, by
// bulk and tensor copies, and is read for operand B only.  dY lies there as in memory, tokens x columns
// (MN-major, 128-byte swizzle).
//
// The tensor core's accumulator drops bits below its own last one in every step,
// which adds up over thousands of tokens (8e-6 of the result over 16384, where
// float32 sums are at 6e-7).  So the sums are taken out every kChunk stages and
// added in registers: warp group w keeps columns [w W / 2, (w + 1) W / 2) of its
// 128 channels.  The same two warp groups convert, one the even and one the odd
// stages, and are some stages ahead when they turn to the sums, so that the
// tensor core waits for the reading of TMEM alone; results leave for memory
// while it works on.
//
// Measured: 16384 tokens, 4096 x 6144: 506-524 us in a long run, 1573-1630 TFLOP/s, 0.92-0.95 of the
// measured sustained bf16 rate, and 451-464 us in runs of a few calls, up to 1829 TFLOP/s, 0.95 of the
// burst rate; taking the sums out costs about 20.  Adding to dW costs 42 us
// more, and 23 more for 65531 tokens, 1000 x 523.  Tiles narrower than 256
// columns are bound by the conversion, 0.55-0.65 us a stage whatever their width:
// 65531 tokens, 1000 x 523: 66 us.  The warp that multiplies walks its loop as a
// whole, so that descriptors stay in uniform registers (one lane alone took 650
// cycles to issue a stage's eight products: 491 us).
//
// Work: whole tiles first, one per pair of blocks and wave, all pairs at the
// same tokens, so that what they read together stays in L2; the tiles of the
// last, partial wave are cut along the tokens into as many equal parts as there are pairs for
// each, so that the pairs of one part read the same tokens too (with shares of equal size
// across tiles, 65531 tokens of 1000 channels x 523 columns were read three times: 82 us against 73).
// Parts of a tile go to the workspace and wgrad_join_kernel adds them in order.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <mutex>

#include "ckpt.h"
#include "follow.cuh"
#include "internal.h"
#include "layout.h"
#include "per_device.h"
#include "tc_ptx.cuh"

namespace cg = cooperative_groups;

namespace stp {

stp_status check_ckpt_desc(const stp_ckpt_desc* d);

namespace {

using namespace tc;

constexpr int kThreads = 384;       // warps 0-7 convert and add up, 8 loads dY, 9 multiplies, 10 loads codes
// Registers of a thread: 168 at launch (65536 / 384), of which the warps that keep no sums give theirs up:
// 2 x 232 + 40 = 3 x 168.
constexpr int kRegsSums = 232, kRegsRest = 40;
constexpr int kGroups = 2;          // warp groups among them
// A stage is 128 tokens.  With 64 (and twice as many) a stage's waits and arrivals, about 600
// cycles of its converting group, took as long as its conversion: 745 us for the
// 16384-token projection against 549 at the time.
constexpr int kStages = 4;
constexpr int kAhead = 3;           // stages converted ahead when sums are taken: less than kStages
// A group meets each of its stages in every round of the ring: else a wait by
// parity would take the phase two rounds before for the one it wants.
static_assert(kStages % kGroups == 0 && kAhead < kStages, "ring of stages");
constexpr int kChunk = 16;          // stages between two takings
constexpr int kTileC = 256, kHalfC = 128, kTileM = 256;
constexpr int kBoxBytes = kCkTokens * 64 * 2;       // 64 columns of a stage's tokens
constexpr int kYBytes = 2 * kBoxBytes;              // a block's half of the columns
constexpr int kCodeBytes = 4 * kCkBlock;            // 128 channels of them
constexpr int kStageRow = 20;       // floats of a row of results on their way: 16, and 4 so that rows lie in other banks
constexpr int kOffCodes = kStages * kYBytes, kOffStage = kOffCodes + kStages * kCodeBytes,
              kOffBars = kOffStage + 8 * 32 * kStageRow * 4;
constexpr int kSmem = kOffBars + 512 + 1024;
constexpr int kColA = 256;          // first TMEM column of A's stages
constexpr size_t kPartBytes = (size_t)kHalfC * kTileM * 4;   // of a block
constexpr int kLeastBlocks = 3;     // stages of a part at least
constexpr int kLeastM = 32;         // columns of a tile made narrower, at least

struct WgradParams {
  int N, C, M, CB, KB, W;       // W: columns of a tile, a multiple of 16
  int CT, MT;                   // tiles along channels and columns
  int whole, rest, parts;       // waves of whole tiles; tiles of the last wave, and parts that each is cut into
  bool add, vec;                // vec: rows of dW start at whole 16 bytes
  const uint8_t* ck;
  float* dw;
  float* part;                  // [parts][rest][2][64][128][4]: part, tile, block, column / 4, channel, column % 4
  uint32_t* err;
};

struct Segment {
  int tile, kb0, kb1, slot;   // slot: of the workspace, -1 when the tile is whole
};

// Barriers: the codes of a stage have landed and are read (each block's own),
// dY of both blocks has landed and A of both is in place (first block's), the
// stage is multiplied (both); the sums of a chunk are ready (both) and taken by both (first
// block's).  Codes are fetched again as soon as they are read, so that their way from memory
// does not lie between a product and the next conversion for its stage.
enum {
  W_CF = 0,
  W_CE = kStages,
  W_BF = 2 * kStages,
  W_AF = 3 * kStages,
  W_E = 4 * kStages,
  W_DF = 5 * kStages,
  W_DE,
  W_DRAIN,
  W_COUNT
};

// ---- a pair's instructions

__device__ __forceinline__ uint32_t in_block(uint32_t addr, int block) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(block));
  return r;
}

// mbar_wait with the SM's clock, which is near, in place of the global timer:
// a stage's waits lie on the path from one product to the next.
constexpr long long kWaitLimitCycles = 4000000000ll;   // about 2 s
constexpr uint64_t kDrainLimitNs = 20000000000ull;     // of a whole launch
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      *abort = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// Arrives on a barrier of either block.  What the barriers between the blocks
// order lies in TMEM, which tcgen05's own waits and fences order, so no wider
// scope is asked for: a release at cluster scope waits for all memory (1250 us
// against 783 for the 16384-token projection).
__device__ __forceinline__ void arrive_in(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tile load whose bytes count on a barrier of either block of the pair.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tmov.b64 db, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], db, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi));
}

// Arrives on the barrier of both blocks once all products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}

// 16 bytes of shared memory (through a generic address they take longer).
__device__ __forceinline__ uint4 load_shared(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}

// A channel's codes of 64 tokens (the first or the second half of a block's)
// in shared memory to bf16 pairs of successive tokens.
__device__ __forceinline__ void convert(uint32_t block, int lane, int part, uint32_t* r) {
  const uint32_t codes = block + part * 2048 + lane * 16, scales = block + kCkCodes + part * 128;
  uint4 c[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) c[q] = load_shared(codes + q * 512);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 s = load_shared(scales + q * 32), t = load_shared(scales + q * 32 + 16);   // the same for all lanes
    r[q * 8] = values_bf16x2(early_codes(c[q].x), s.x);
    r[q * 8 + 1] = values_bf16x2(late_codes(c[q].x), s.y);
    r[q * 8 + 2] = values_bf16x2(early_codes(c[q].y), s.z);
    r[q * 8 + 3] = values_bf16x2(late_codes(c[q].y), s.w);
    r[q * 8 + 4] = values_bf16x2(early_codes(c[q].z), t.x);
    r[q * 8 + 5] = values_bf16x2(late_codes(c[q].z), t.y);
    r[q * 8 + 6] = values_bf16x2(early_codes(c[q].w), t.z);
    r[q * 8 + 7] = values_bf16x2(late_codes(c[q].w), t.w);
  }
}

// The stages of a pair in order: whole tiles, then its part of one.
struct Walk {
  Segment s;
  int i = 0, kb = 0, n, whole, KB, CT, pairs, ct, mt;   // the tile's place along channels and columns
  Segment last;
  __device__ __forceinline__ Walk(const WgradParams& p, int g, int pairs_)
      : whole(p.whole), KB(p.KB), CT(p.CT), pairs(pairs_) {
    n = whole;
    s.tile = g - pairs;
    if (g < p.rest * p.parts) {
      const int part = g / p.rest;
      last = {whole * pairs + g - part * p.rest, (int)((int64_t)KB * part / p.parts),
              (int)((int64_t)KB * (part + 1) / p.parts), p.parts > 1 ? g : -1};
      ++n;
    }
    enter();
  }
  __device__ __forceinline__ void enter() {
    if (i < whole) s = {s.tile + pairs, 0, KB, -1};
    else if (i < n) s = last;
    kb = s.kb0;
    mt = s.tile / CT;
    ct = s.tile - mt * CT;
  }
  __device__ __forceinline__ bool on() const { return i < n; }
  __device__ __forceinline__ void next() {
    if (++kb == s.kb1) {
      ++i;
      enter();
    }
  }
};

// Four columns of a row of dW; `left` of them exist.
__device__ __forceinline__ void put4(const WgradParams& p, float* at, float4 v, int left) {
  if (p.vec && left >= 4) {
    float4* to = reinterpret_cast<float4*>(at);
    if (p.add) {
      const float4 o = *to;
      v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
    }
    *to = v;
  } else {
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < left) at[k] = x[k] + (p.add ? at[k] : 0.f);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap ty, const WgradParams p) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint8_t* codes = smem + kOffCodes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + W_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = blockIdx.x & 1, g = blockIdx.x >> 1,
            pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int b = 0; b < W_COUNT; ++b)
      mbar_init(&bars[b], b >= W_AF && b < W_AF + kStages ? 8 : b >= W_CE && b < W_CE + kStages ? 4 : b == W_DE ? 16 : 1);
    *abort_flag = 0;
    if (blockIdx.x == 0) *p.err = 0;   // a lost wait sets it seconds later
    fence_mbar_init();
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before_sync();
  cg::this_cluster().sync();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  if (warp >= 8) {
    regs_dec<kRegsRest>();
    if (warp == 8) {
      if (lane == 0) {
        // -------------------------------------------------------------- dY
        tma_prefetch_desc(&ty);
        const int boxes = (p.W / 2 + 63) / 64;
        int it = 0, last[kStages];   // phase of a stage's last load
        for (int st = 0; st < kStages; ++st) last[st] = -1;
        for (Walk w(p, g, pairs); w.on(); w.next(), ++it) {
          const int st = it % kStages, n = it / kStages;
          if (it >= kStages && !wait(&bars[W_E + st], (n - 1) & 1, abort_flag, p.err)) break;
          const int m0 = w.mt * p.W + block * (p.W / 2);
          const uint32_t bar = in_block(smem_u32(&bars[W_BF + st]), 0);
          if (block == 0) mbar_expect_tx(&bars[W_BF + st], 2 * boxes * kBoxBytes);
          for (int b = 0; b < boxes; ++b)
            tma_load_pair(smem + st * kYBytes + b * kBoxBytes, &ty, bar, m0 + b * 64, w.kb * kCkTokens);
          last[st] = n & 1;
        }
        // nothing is on its way to this block's memory or barriers when it ends
        for (int st = 0; st < kStages; ++st) {
          if (block == 0 && last[st] >= 0) mbar_wait_drain(&bars[W_BF + st], last[st]);
          if (last[st] >= 0) wait(&bars[W_E + st], last[st], abort_flag, p.err);
        }
      }
      __syncwarp();
    } else if (warp == 10) {
      if (lane == 0) {
        // ----------------------------------------------------------- codes
        int it = 0, last[kStages];
        for (int st = 0; st < kStages; ++st) last[st] = -1;
        for (Walk w(p, g, pairs); w.on(); w.next(), ++it) {
          const int st = it % kStages, n = it / kStages, cb = w.ct * 8 + block * 4;
          if (it >= kStages && !wait(&bars[W_CE + st], (n - 1) & 1, abort_flag, p.err)) break;
          if (cb < p.CB) {
            const uint32_t bytes = min(4, p.CB - cb) * kCkBlock;
            mbar_expect_tx(&bars[W_CF + st], bytes);
            bulk_load(codes + st * kCodeBytes, p.ck + ((int64_t)w.kb * p.CB + cb) * kCkBlock, bytes, &bars[W_CF + st]);
            last[st] = n & 1;
          } else {
            mbar_arrive(&bars[W_CF + st]);   // channels past the end: nothing comes
          }
        }
        for (int st = 0; st < kStages; ++st)
          if (last[st] >= 0) mbar_wait_drain(&bars[W_CF + st], last[st]);
      }
      __syncwarp();
    } else if (warp == 9) {
      // the whole warp walks, so that addresses stay in uniform registers; one lane issues
      const bool one = elect_one();
      if (block == 0) {
        // --------------------------------------------------------- products
        const uint32_t idesc = idesc_bf16(kTileC, p.W, 0, 1), b0 = desc_lo_mnmajor(smem_u32(smem));
        int it = 0, chunk = 0, in = 0;
        for (Walk w(p, g, pairs); w.on(); ++it) {
          if (in == 0 && chunk > 0 &&
              !__all_sync(0xffffffffu, wait(&bars[W_DE], (chunk - 1) & 1, abort_flag, p.err)))
            break;
          const int st = it % kStages;
          const uint32_t phase = (it / kStages) & 1;
          if (!__all_sync(0xffffffffu, wait(&bars[W_BF + st], phase, abort_flag, p.err) &&
                                           wait(&bars[W_AF + st], phase, abort_flag, p.err)))
            break;
          fence_after_sync();
          if (one) {
            const uint32_t b_lo = b0 + st * (kYBytes >> 4), a = tmem + kColA + st * 64;
#pragma unroll
            for (int kk = 0; kk < kCkTokens / 16; ++kk)
              mma_pair(tmem, a + kk * 8, b_lo + kk * (2048 >> 4), idesc, in > 0 || kk > 0);
            commit_pair(&bars[W_E + st]);
          }
          __syncwarp();
          const int tile = w.i;
          w.next();
          if (++in == kChunk || w.i != tile) {
            if (one) commit_pair(&bars[W_DF]);
            in = 0;
            ++chunk;
          }
        }
        if (one) {
          commit_pair(&bars[W_DRAIN]);
          if (chunk > 0) wait(&bars[W_DE], (chunk - 1) & 1, abort_flag, p.err);   // the other block's last arrivals, too
        }
        __syncwarp();
      }
      // nothing of the pair is in flight behind this; the second block's wait is
      // all it does, so it looks rarely
      if (lane == 0) {
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(&bars[W_DRAIN], 0) && globaltimer() - t0 < kDrainLimitNs) __nanosleep(500);
      }
      __syncwarp();
    }
  } else {
    regs_inc<kRegsSums>();
    const int group = warp >> 2, w4 = warp & 3, half = p.W / 2;
    const uint32_t lane_base = (uint32_t)(w4 * 32) << 16;
    const uint32_t codes_at = smem_u32(codes) + w4 * kCkBlock;
    const uint32_t taken = in_block(smem_u32(&bars[W_DE]), 0);
    float* stage = reinterpret_cast<float*>(smem + kOffStage) + warp * 32 * kStageRow;
    float acc[kTileM / 2];
#pragma unroll
    for (int e = 0; e < kTileM / 2; ++e) acc[e] = 0.f;
    int it = 0, end = 0, chunk = 0;   // stages converted, and at the end of the chunk
    bool ok = true;
    Walk c(p, g, pairs);
    for (Walk d(p, g, pairs); d.on() && ok; ++chunk) {
      // the chunk: up to kChunk stages of one segment
      const int len = min(kChunk, d.s.kb1 - d.kb);
      end += len;
      for (; c.on() && it < end + kAhead; ++it, c.next()) {
        // the tensor core waits: first the sums
        if (it >= end && __any_sync(0xffffffffu, test(&bars[W_DF], chunk & 1))) break;
        if (it % kGroups != group) continue;
        const int st = it % kStages, n = it / kStages;
        // the codes, and TMEM's stage
        if (!__all_sync(0xffffffffu, wait(&bars[W_CF + st], n & 1, abort_flag, p.err) &&
                                         (it < kStages || wait(&bars[W_E + st], (n - 1) & 1, abort_flag, p.err)))) {
          ok = false;
          break;
        }
        __syncwarp();
        fence_after_sync();
        if (c.ct * 8 + block * 4 + w4 < p.CB) {   // channels past the end: sums that nothing reads
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t r[32];
            convert(codes_at + st * kCodeBytes, lane, h, r);
            tmem_st32(tmem + lane_base + kColA + st * 64 + h * 32, r);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[W_CE + st]);   // the codes are read
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) arrive_in(in_block(smem_u32(&bars[W_AF + st]), 0));
      }
      if (!ok || !__all_sync(0xffffffffu, wait(&bars[W_DF], chunk & 1, abort_flag, p.err))) break;
      fence_after_sync();
#pragma unroll
      for (int j = 0; j < kTileM / 2; j += 16)
        if (j < half) {
          uint32_t x[16];
          tmem_ld16(tmem + lane_base + group * half + j, x);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[j + e] += __uint_as_float(x[e]);
        }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_in(taken);
      const int ct = d.ct, mt = d.mt, slot = d.s.slot, segment = d.i;
      d.kb += len - 1;
      d.next();
      if (d.i == segment) continue;
      // the segment's results, 16 columns of 32 channels at a time through
      // shared memory, so that they leave in rows
      const int c0 = ct * kTileC + block * kHalfC + w4 * 32, m0 = mt * p.W + group * half;
      float4* part = reinterpret_cast<float4*>(p.part) + (size_t)(max(slot, 0) * 2 + block) * (kPartBytes / 16) +
                     w4 * 32 + lane + group * half / 4 * kHalfC;
#pragma unroll
      for (int j = 0; j < kTileM / 2; j += 16) {
        if (j >= half) continue;
        if (slot >= 0) {
#pragma unroll
          for (int e = j; e < j + 16; e += 4)
            if (e < half) part[e / 4 * kHalfC] = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        } else {
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(stage + lane * kStageRow + e) =
                make_float4(acc[j + e], acc[j + e + 1], acc[j + e + 2], acc[j + e + 3]);
          __syncwarp();
          const int e = (lane & 3) * 4, left = min(half, p.M - m0) - j - e;
          for (int r = lane >> 2; r < 32 && c0 + r < p.C; r += 8)
            put4(p, p.dw + (int64_t)(c0 + r) * p.M + m0 + j + e,
                 *reinterpret_cast<const float4*>(stage + r * kStageRow + e), left);
        }
      }
#pragma unroll
      for (int e = 0; e < kTileM / 2; ++e) acc[e] = 0.f;
    }
  }

  __syncwarp();
  fence_before_sync();
  cg::this_cluster().sync();
  fence_after_sync();
  if (warp == 9)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Adds up the parts of a tile of the last wave; a block does 4 columns x 256 channels.
__global__ void __launch_bounds__(256) wgrad_join_kernel(const WgradParams p) {
  const int tile = blockIdx.y, c4 = blockIdx.x, block = threadIdx.x >> 7, r = threadIdx.x & 127;
  const size_t slot = 2 * kPartBytes / 16;
  const float4* from = reinterpret_cast<const float4*>(p.part) + tile * slot + (size_t)block * (kPartBytes / 16) +
                       c4 * kHalfC + r;
  wait_for_previous();
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int g = 0; g < p.parts; g += 8) {
    float4 v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      v[k] = g + k < p.parts ? __ldcs(from + (size_t)(g + k) * p.rest * slot) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 8; ++k) sum = make_float4(sum.x + v[k].x, sum.y + v[k].y, sum.z + v[k].z, sum.w + v[k].w);
  }
  const int which = p.CT * p.MT - p.rest + tile, c = which % p.CT * kTileC + threadIdx.x;
  const int m0 = which / p.CT * p.W, m = m0 + c4 * 4, end = min(p.M, m0 + p.W);
  if (c < p.C && m < end) put4(p, p.dw + (int64_t)c * p.M + m, sum, end - m);
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(p);
  });
  return fn;
}

// dY [N, M], rows `stride` elements apart: boxes of 64 columns x 128 tokens; zeros outside.
bool make_map(CUtensorMap* m, const void* base, int N, int M, int64_t stride) {
  EncodeFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)M, (cuuint64_t)N};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {64, kCkTokens};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

stp_status check_wgrad(const stp_ckpt_desc* d, int cols) {
  stp_status st = check_ckpt_desc(d);
  if (st) return st;
  if (cols < 1 || cols > (1 << 20)) return fail(STP_EUNSUPPORTED, "cols must lie in [1, 2^20]");
  return STP_OK;
}

// Tiles and their parts on a GPU of n_sm SMs; returns the launch's pairs.  The
// last wave's tiles are cut where that saves more stages (0.57 us each) than
// joining costs, about 6 and one for every 1500 columns of all parts.  Measured in us, cut
// and whole: 12 tiles of 32 stages 16.5 / 26, of 16 stages 14.4 / 16.1, of 8 13.5 / 11.3.
// Where few tiles stay whole they are made narrower instead, as many as there
// are pairs: 4 tiles of 4 stages 14.3 us, 16 tiles 8.1.
int plan(WgradParams& p, const stp_ckpt_desc* d, int cols, int n_sm) {
  p.N = d->n_tokens;
  p.C = d->dim;
  p.M = cols;
  p.CB = (int)ck_channel_blocks(p.C);
  p.KB = (int)ck_token_blocks(p.N);
  p.CT = (p.C + kTileC - 1) / kTileC;
  p.MT = (p.M + kTileM - 1) / kTileM;
  const int pairs = n_sm / 2;
  const auto tiles = [&] {
    p.W = ((p.M + p.MT - 1) / p.MT + 15) / 16 * 16;   // tiles of one width, not full ones and a narrow last
    p.MT = (p.M + p.W - 1) / p.W;
    p.whole = (int)((int64_t)p.CT * p.MT / pairs);
    p.rest = (int)((int64_t)p.CT * p.MT % pairs);
    p.parts = 1;
  };
  tiles();
  const int parts = p.rest ? std::min(pairs / p.rest, p.KB / kLeastBlocks) : 1;
  if (parts > 1 && p.KB - (p.KB + parts - 1) / parts > 6 + (int64_t)p.rest * parts * p.W / 1500) {
    p.parts = parts;
  } else if (p.whole == 0 && p.CT <= pairs / 2) {
    p.MT = std::max(p.MT, std::min((p.M + kLeastM - 1) / kLeastM, pairs / p.CT));
    tiles();
  }
  return p.whole > 0 ? pairs : p.rest * p.parts;
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_ckpt_wgrad_workspace_size(const stp_ckpt_desc* desc, int32_t cols, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_wgrad(desc, cols);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_ckpt_wgrad_workspace_size: NULL output");
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_ckpt_wgrad_workspace_size: %s", cudaGetErrorString(e));
  WgradParams p{};
  plan(p, desc, cols, n_sm);
  *ws_bytes = 256 + (p.parts > 1 ? 2 * (size_t)p.parts * p.rest * kPartBytes : 0);
  return STP_OK;
}

extern "C" stp_status stp_ckpt_wgrad(const stp_ckpt_desc* desc, int32_t cols, const void* d_ckpt, const void* d_y,
                                     int64_t y_stride, int32_t accumulate, float* d_w, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_wgrad(desc, cols);
  if (st) return st;
  if (!d_w || !d_ws || (desc->n_tokens > 0 && (!d_ckpt || !d_y)))
    return fail(STP_EINVAL, "stp_ckpt_wgrad: NULL device pointer");
  if ((reinterpret_cast<uintptr_t>(d_ckpt) | reinterpret_cast<uintptr_t>(d_ws)) & 255 ||
      reinterpret_cast<uintptr_t>(d_y) & 15 || reinterpret_cast<uintptr_t>(d_w) & 3)
    return fail(STP_EINVAL, "stp_ckpt_wgrad: checkpoint and workspace 256-byte, d_y 16-byte, d_w 4-byte aligned");
  if (y_stride < cols || y_stride % 8)
    return fail(STP_EINVAL, "stp_ckpt_wgrad: y_stride must be at least cols and a multiple of 8");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (desc->n_tokens == 0) {
    e = cudaMemsetAsync(d_ws, 0, 4, s);
    if (e == cudaSuccess && !accumulate) e = cudaMemsetAsync(d_w, 0, (size_t)desc->dim * cols * 4, s);
  } else {
    int dev = 0, n_sm = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
    static PerDevice limit;
    if (e == cudaSuccess)
      e = limit([] { return cudaFuncSetAttribute(wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (e != cudaSuccess) return fail(STP_ECUDA, "stp_ckpt_wgrad: %s", cudaGetErrorString(e));
    WgradParams p{};
    const int pairs = plan(p, desc, cols, n_sm);
    p.add = accumulate != 0;
    p.vec = reinterpret_cast<uintptr_t>(d_w) % 16 == 0 && p.M % 4 == 0;
    p.ck = static_cast<const uint8_t*>(d_ckpt);
    p.dw = d_w;
    p.part = reinterpret_cast<float*>(static_cast<char*>(d_ws) + 256);
    p.err = static_cast<uint32_t*>(d_ws);
    CUtensorMap ty;
    if (!make_map(&ty, d_y, p.N, p.M, y_stride)) return fail(STP_ECUDA, "stp_ckpt_wgrad: tensor map encoding failed");
    wgrad_kernel<<<2 * pairs, kThreads, kSmem, s>>>(ty, p);
    e = cudaGetLastError();
    if (e == cudaSuccess && p.parts > 1) e = launch_after(wgrad_join_kernel, dim3(p.W / 4, p.rest), dim3(256), s, p);
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_ckpt_wgrad: %s", cudaGetErrorString(e));
  return STP_OK;
}
