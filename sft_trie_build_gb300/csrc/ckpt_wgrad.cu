// Weight gradient of a projection from its input kept in 8 bits:
//
//   dW[c, m] (+)= sum_n x^[n, c] dY[n, m],   x^ as ckpt.h restores it.
//
// x^ is exact in bf16, so the products are those of the stored values; sums are
// float32 on the tensor cores (tcgen05, M = 128 channels, N <= 256 columns of
// dY, K = tokens).
//
// Operand A is never in shared memory: a warp owns 32 channels, a lane one of them
// (a TMEM lane, too), reads its codes of 64 tokens straight from the checkpoint, turns them to bf16
// (ckpt.h) and stores them to TMEM.  dY arrives by TMA as it lies, tokens x
// columns (MN-major, 128-byte swizzle).  TMEM: 256 columns of sums, then one
// 32-column stage of A for every stage of dY in shared memory.
//
// Work: whole tiles first, one per block and wave, all blocks at the same
// tokens, so that what they read together stays in L2; the tiles of the last, partial wave
// are cut along the tokens into equal parts for all blocks.  Parts of a tile go
// to the workspace and wgrad_join_kernel adds them in order.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <mutex>

#include "ckpt.h"
#include "internal.h"
#include "layout.h"
#include "per_device.h"
#include "tc_ptx.cuh"

namespace stp {

stp_status check_ckpt_desc(const stp_ckpt_desc* d);

namespace {

using namespace tc;

constexpr int kThreads = 192;       // warps 0-3 convert and store results, 4 loads, 5 multiplies
constexpr int kStages = 6;
constexpr int kTileC = 128, kTileM = 256;
constexpr int kBoxBytes = 64 * 64 * 2;              // 64 tokens x 64 columns
constexpr int kStageBytes = 4 * kBoxBytes;
constexpr int kSmem = kStages * kStageBytes + 1024 + 256;
constexpr int kColA = 256;          // first TMEM column of A's stages
constexpr size_t kPartBytes = (size_t)kTileC * kTileM * 4;
constexpr int kLeastBlocks = 4;     // token blocks of a part at least

struct WgradParams {
  int N, C, M, CB, KB, W;       // W: columns of a tile, a multiple of 16
  int CT, MT;                   // tiles along channels and columns
  int whole, rest, parts;       // waves of whole tiles; tiles of the last wave, and blocks that share them
  bool add, vec;                // vec: rows of dW start at whole 16 bytes
  const uint8_t* ck;
  float* dw;
  float* part;                  // [2 * parts][64][128][4]: column / 4, channel, column % 4
  uint32_t* err;
};

// The share of block g in the last wave: token blocks [at, end) of `rest` tiles of KB each.
__host__ __device__ __forceinline__ int64_t share(const WgradParams& p, int g) {
  return (int64_t)p.rest * p.KB * g / p.parts;
}

struct Segment {
  int tile, kb0, kb1, slot;   // slot: of the workspace, -1 when the tile is whole
};

// Segment i of block g; false when there is none.
__device__ __forceinline__ bool segment(const WgradParams& p, int g, int grid, int i, Segment& s) {
  if (i < p.whole) {
    s = {i * grid + g, 0, p.KB, -1};
    return true;
  }
  if (g >= p.parts) return false;
  const int64_t at = share(p, g), end = share(p, g + 1);
  const int64_t first = at / p.KB, tile = first + (i - p.whole);
  const int64_t a = tile * p.KB > at ? tile * p.KB : at, b = (tile + 1) * p.KB < end ? (tile + 1) * p.KB : end;
  if (a >= b) return false;
  s.tile = p.whole * grid + (int)tile;
  s.kb0 = (int)(a - tile * p.KB);
  s.kb1 = (int)(b - tile * p.KB);
  s.slot = s.kb0 == 0 && s.kb1 == p.KB ? -1 : 2 * g + (tile != first);
  return true;
}

enum { W_BF = 0, W_AF = kStages, W_E = 2 * kStages, W_DF = 3 * kStages, W_DE, W_DRAIN, W_COUNT };

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}

// 64 tokens of a channel and their scales on their way to a lane's registers.
struct Codes {
  uint4 code[4], scale[4];
  __device__ __forceinline__ void get(const WgradParams& p, int tb, int cb, int lane) {
    if (cb < p.CB) {
      const uint4* block = reinterpret_cast<const uint4*>(p.ck + ((int64_t)tb * p.CB + cb) * kCkBlock);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        code[q] = __ldg(block + q * 32 + lane);
        scale[q] = __ldg(block + kCkCodes / 16 + q);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) code[q] = scale[q] = make_uint4(0, 0, 0, 0);
    }
  }
  // bf16 pairs of successive tokens
  __device__ __forceinline__ void put(uint32_t* r) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t c[4] = {code[q].x, code[q].y, code[q].z, code[q].w};
      const uint32_t s[4] = {scale[q].x, scale[q].y, scale[q].z, scale[q].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        r[q * 8 + w * 2] = mul_bf16x2(codes_bf16x2(__byte_perm(c[w], 0, 0x1404)), scales_bf16x2(__byte_perm(s[w], 0, 0x4140)));
        r[q * 8 + w * 2 + 1] =
            mul_bf16x2(codes_bf16x2(__byte_perm(c[w], 0, 0x3424)), scales_bf16x2(__byte_perm(s[w], 0, 0x4342)));
      }
    }
  }
};

// B operand: 64-column boxes kBoxBytes apart (leading dimension), 8-token groups 1024 bytes apart.
__device__ __forceinline__ uint32_t desc_lo_b(uint32_t addr) {
  return ((addr & 0x3FFFFu) >> 4) | ((uint32_t)(kBoxBytes >> 4) << 16);
}

__global__ void __launch_bounds__(kThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap ty, const WgradParams p) {
  extern __shared__ uint8_t smem_dyn[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + W_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = blockIdx.x, grid = gridDim.x;

  if (threadIdx.x == 0) {
    for (int b = 0; b < W_COUNT; ++b)
      mbar_init(&bars[b], (b >= W_AF && b < W_AF + kStages) || b == W_DE ? 4 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tmem = *tmem_slot;
  const int boxes = (p.W + 63) / 64;
  Segment s;

  if (warp == 4) {
    if (lane == 0) {
      tma_prefetch_desc(&ty);
      int it = 0, last_phase[kStages];
      for (int st = 0; st < kStages; ++st) last_phase[st] = -1;
      bool ok = true;
      for (int i = 0; ok && segment(p, g, grid, i, s); ++i) {
        const int m0 = s.tile / p.CT * p.W;
        for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
          const int st = it % kStages, n = it / kStages;
          if (it >= kStages && !mbar_wait(&bars[W_E + st], (n - 1) & 1, abort_flag, p.err)) {
            ok = false;
            break;
          }
          mbar_expect_tx(&bars[W_BF + st], boxes * kBoxBytes);
          for (int b = 0; b < boxes; ++b)
            tma_load_2d(smem + st * kStageBytes + b * kBoxBytes, &ty, &bars[W_BF + st], m0 + b * 64, kb * 64);
          last_phase[st] = n & 1;
        }
      }
      for (int st = 0; st < kStages; ++st)
        if (last_phase[st] >= 0) mbar_wait_drain(&bars[W_BF + st], last_phase[st]);
    }
    __syncwarp();
  } else if (warp == 5) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(kTileC, p.W, 0, 1);
      int it = 0;
      bool ok = true;
      for (int i = 0; ok && segment(p, g, grid, i, s); ++i) {
        if (i > 0 && !mbar_wait(&bars[W_DE], (i - 1) & 1, abort_flag, p.err)) break;
        fence_after_sync();
        for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
          const int st = it % kStages;
          const uint32_t phase = (it / kStages) & 1;
          if (!mbar_wait(&bars[W_BF + st], phase, abort_flag, p.err) ||
              !mbar_wait(&bars[W_AF + st], phase, abort_flag, p.err)) {
            ok = false;
            break;
          }
          fence_after_sync();
          const uint32_t b_lo = desc_lo_b(smem_u32(smem) + st * kStageBytes), a = tmem + kColA + st * 32;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts_lo(tmem, a + kk * 8, b_lo + kk * (2048 >> 4), idesc, kb > s.kb0 || kk > 0);
          mma_commit(&bars[W_E + st]);
        }
        if (ok) mma_commit(&bars[W_DF]);
      }
      mma_commit(&bars[W_DRAIN]);
      mbar_wait_drain(&bars[W_DRAIN], 0);
    }
    __syncwarp();
  } else {
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && segment(p, g, grid, i, s); ++i) {
      const int ct = s.tile % p.CT, cb = ct * 4 + warp;
      Codes next;
      next.get(p, s.kb0, cb, lane);
      for (int kb = s.kb0; kb < s.kb1; ++kb, ++it) {
        const int st = it % kStages;
        const Codes now = next;
        if (kb + 1 < s.kb1) next.get(p, kb + 1, cb, lane);
        uint32_t r[32];
        now.put(r);
        if (it >= kStages &&
            !__all_sync(0xffffffffu, mbar_wait(&bars[W_E + st], (it / kStages - 1) & 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        fence_after_sync();
        tmem_st32(tmem + lane_base + kColA + st * 32, r);
        tmem_st_wait();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars[W_AF + st]);
      }
      if (!ok || !__all_sync(0xffffffffu, mbar_wait(&bars[W_DF], i & 1, abort_flag, p.err))) break;
      fence_after_sync();
      const int c = ct * kTileC + warp * 32 + lane, m0 = s.tile / p.CT * p.W, width = min(p.W, p.M - m0);
      float* row = p.dw + (int64_t)c * p.M + m0;
      float4* part = reinterpret_cast<float4*>(p.part) + (size_t)max(s.slot, 0) * (kPartBytes / 16) + warp * 32 + lane;
      for (int j = 0; j < p.W; j += 32) {
        uint32_t x[32];
        tmem_ld32(tmem + lane_base + j, x);
        tmem_ld_wait();
        if (s.slot >= 0) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            if (j + e < p.W)
              part[(j + e) / 4 * kTileC] = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]),
                                                       __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
        } else if (c < p.C) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if (p.vec && j + e + 3 < width) {
              float4* at = reinterpret_cast<float4*>(row + j + e);
              float4 v = make_float4(__uint_as_float(x[e]), __uint_as_float(x[e + 1]), __uint_as_float(x[e + 2]),
                                     __uint_as_float(x[e + 3]));
              if (p.add) {
                const float4 o = *at;
                v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
              }
              *at = v;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (j + e + k < width) row[j + e + k] = __uint_as_float(x[e + k]) + (p.add ? row[j + e + k] : 0.f);
            }
          }
        }
      }
      fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars[W_DE]);
    }
  }

  __syncwarp();
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp == 5) tmem_dealloc(tmem, 512);
}

// Adds up the parts of a tile of the last wave; a block does 8 columns x 128 channels.
__global__ void __launch_bounds__(256) wgrad_join_kernel(const WgradParams p) {
  const int tile = blockIdx.y;   // of the last wave
  const int64_t a = (int64_t)tile * p.KB, b = a + p.KB, all = (int64_t)p.rest * p.KB;
  int g = (int)(a * p.parts / all);   // the first block whose share reaches past a
  while (g > 0 && share(p, g) > a) --g;
  while (share(p, g + 1) <= a) ++g;
  if (share(p, g) <= a && share(p, g + 1) >= b) return;   // one block did it all
  const int cg4 = blockIdx.x * 2 + (threadIdx.x >> 7), r = threadIdx.x & 127;
  if (cg4 * 4 >= p.W) return;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (; g < p.parts && share(p, g) < b; ++g) {
    const int slot = 2 * g + (share(p, g) / p.KB != tile);
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p.part) + (size_t)slot * (kPartBytes / 16) + cg4 * kTileC + r);
    sum = make_float4(sum.x + v.x, sum.y + v.y, sum.z + v.z, sum.w + v.w);
  }
  const int all_tile = p.CT * p.MT - p.rest + tile, c = all_tile % p.CT * kTileC + r;
  const int m0 = all_tile / p.CT * p.W, m = m0 + cg4 * 4, end = min(p.M, m0 + p.W);
  if (c >= p.C) return;
  float* at = p.dw + (int64_t)c * p.M + m;
  const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (m + k < end) at[k] = v[k] + (p.add ? at[k] : 0.f);
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

// dY [N, M], rows `stride` elements apart: boxes of 64 columns x 64 tokens; zeros outside.
bool make_map(CUtensorMap* m, const void* base, int N, int M, int64_t stride) {
  EncodeFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {(cuuint64_t)M, (cuuint64_t)N};
  cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  cuuint32_t box[2] = {64, 64};
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

// Tiles and the blocks' shares of them on a GPU of n_sm SMs; returns the launch's blocks.
int plan(WgradParams& p, const stp_ckpt_desc* d, int cols, int n_sm) {
  p.N = d->n_tokens;
  p.C = d->dim;
  p.M = cols;
  p.CB = (int)ck_channel_blocks(p.C);
  p.KB = (int)ck_token_blocks(p.N);
  p.CT = (p.C + kTileC - 1) / kTileC;
  p.MT = (p.M + kTileM - 1) / kTileM;
  p.W = ((p.M + p.MT - 1) / p.MT + 15) / 16 * 16;   // tiles of one width, not full ones and a narrow last
  const int64_t tiles = (int64_t)p.CT * p.MT;
  p.whole = (int)(tiles / n_sm);
  p.rest = (int)(tiles % n_sm);
  const int64_t most = (int64_t)p.rest * p.KB / kLeastBlocks;
  p.parts = p.rest == 0 ? 0 : (int)(most < p.rest ? p.rest : most < n_sm ? most : n_sm);
  return p.whole > 0 ? n_sm : p.parts;
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
  *ws_bytes = 256 + (p.parts > p.rest ? 2 * (size_t)p.parts * kPartBytes : 0);
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
  cudaError_t e = cudaMemsetAsync(d_ws, 0, 4, s);
  if (e == cudaSuccess && desc->n_tokens == 0) {
    if (!accumulate) e = cudaMemsetAsync(d_w, 0, (size_t)desc->dim * cols * 4, s);
  } else if (e == cudaSuccess) {
    int dev = 0, n_sm = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
    static PerDevice limit;
    if (e == cudaSuccess)
      e = limit([] { return cudaFuncSetAttribute(wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
    if (e != cudaSuccess) return fail(STP_ECUDA, "stp_ckpt_wgrad: %s", cudaGetErrorString(e));
    WgradParams p{};
    const int grid = plan(p, desc, cols, n_sm);
    p.add = accumulate != 0;
    p.vec = reinterpret_cast<uintptr_t>(d_w) % 16 == 0 && p.M % 4 == 0;
    p.ck = static_cast<const uint8_t*>(d_ckpt);
    p.dw = d_w;
    p.part = reinterpret_cast<float*>(static_cast<char*>(d_ws) + 256);
    p.err = static_cast<uint32_t*>(d_ws);
    CUtensorMap ty;
    if (!make_map(&ty, d_y, p.N, p.M, y_stride)) return fail(STP_ECUDA, "stp_ckpt_wgrad: tensor map encoding failed");
    wgrad_kernel<<<grid, kThreads, kSmem, s>>>(ty, p);
    if (p.parts > p.rest) wgrad_join_kernel<<<dim3((p.W / 4 + 1) / 2, p.rest), 256, 0, s>>>(p);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_ckpt_wgrad: %s", cudaGetErrorString(e));
  return STP_OK;
}
