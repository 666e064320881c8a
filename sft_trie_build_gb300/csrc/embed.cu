// Token vectors from a table, and the table's gradient.
//
//   out[n] = scale E[tok[n]],   dE[v] = scale sum_{n : tok[n] = v} d_out[n]
//
// The forward moves bytes only: a few threads take a token, 16 bytes each.
//
// The gradient adds up rows of d_out that lie anywhere, some tokens once, some
// thousands of times, in an order that does not depend on timing:
//   embed_sort_kernel   one cluster of eight blocks sorts (token, position) by token,
//                 stable, in two or three passes over 9 bits or less; the other
//                 blocks meanwhile write zeros over the rows of tokens that do not occur
//   embed_sum_kernel    pieces of 32 sorted entries each: a thread adds its 16 bytes of
//                 channels entry by entry; a token that lies in one piece is done
//   embed_join_kernel   tokens that reach over pieces: the sums of their pieces, in order
// Every row of d_out is read once and every row of dE written once.  Sums are float32.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "layout.h"
#include "logit_rows.cuh"
#include "per_device.h"

namespace cg = cooperative_groups;

namespace stp {
namespace {

using rows::Piece;

constexpr int kThreads = 256;
constexpr int kSortBlocks = 8;      // the portable cluster size
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxBins = 512;
constexpr int kPiece = 32;          // sorted entries of a piece
constexpr int kJoinWarps = 8;

struct EmbedParams {
  int N, V, C;
  int64_t stride;
  float scale;
  bool check, add;
  const void* table;
  const int32_t* tok;
  void* out;
  uint32_t* err;
  // backward
  int bits, passes;        // of a sort pass; the last pass writes to `sorted`
  const void* d_out;
  uint64_t* sorted;        // token << 32 | position, ascending; token V: none
  uint64_t* other;
  float* part;             // [pieces][2][C]: sums of tokens that reach over pieces
  float* d_table;
};

// ---------------------------------------------------------------- forward

// 2^shift threads take a token.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const EmbedParams p, int shift) {
  constexpr int E = Piece<T>::E;
  if (p.check && blockIdx.x == gridDim.x - 1) {
    rows::check_below(p.N, p.V, p.err, [&](int64_t i) { return p.tok[i]; });
    return;
  }
  const int64_t n = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> shift;
  if (n >= p.N) return;
  const int lane = threadIdx.x & ((1 << shift) - 1), step = 1 << shift, pieces = p.C / E;
  const int tok = p.tok[n];
  const bool there = tok >= 0 && tok < p.V;
  if (!p.check && tok >= p.V && lane == 0) atomicOr(p.err, kErrBadList);
  const uint4* from = reinterpret_cast<const uint4*>(static_cast<const T*>(p.table) + (int64_t)(there ? tok : 0) * p.C);
  uint4* to = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + n * p.stride);
  constexpr int kAhead = 4;
  for (int i = lane; i < pieces; i += kAhead * step) {
    uint4 v[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      v[k] = there && i + k * step < pieces ? __ldg(from + i + k * step) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      if (i + k * step < pieces) {
        float z[E];
        Piece<T>::get(v[k], z);
#pragma unroll
        for (int e = 0; e < E; ++e) z[e] *= p.scale;
        __stcs(to + i + k * step, Piece<T>::put(z));
      }
  }
}

// ------------------------------------------------------------------- sort

struct SortShared {
  uint32_t hist[kSortWarps][kMaxBins];       // entries of a warp before it, then where the next goes
  uint32_t total[kSortBlocks][kMaxBins];     // of each block of the cluster
  uint32_t base[kMaxBins];
  uint32_t warp_sum[kSortWarps];
  uint32_t bad[kSortBlocks];
};

__device__ __forceinline__ uint64_t entry_of(const EmbedParams& p, int i) {
  const int tok = p.tok[i];
  return ((uint64_t)(uint32_t)(tok < 0 || tok >= p.V ? p.V : tok) << 32) | (uint32_t)i;
}

// Writes zeros over the rows of tokens that do not occur, block `at` of `of`.
__device__ void fill_absent(const EmbedParams& p, uint32_t* seen, int at, int of) {
  const int v0 = (int)((int64_t)p.V * at / of), v1 = (int)((int64_t)p.V * (at + 1) / of);
  const int t = threadIdx.x;
  for (int i = t; i < (v1 - v0 + 31) / 32; i += kSortThreads) seen[i] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = t; i < p.N; i += kSortThreads) {
    const int x = p.tok[i] - v0;
    if (x >= 0 && x < v1 - v0) atomicOr(seen + (x >> 5), 1u << (x & 31));
  }
  __syncthreads();
  for (int v = v0 + (t >> 5); v < v1; v += kSortWarps) {
    if (seen[(v - v0) >> 5] >> ((v - v0) & 31) & 1) continue;
    float4* row = reinterpret_cast<float4*>(p.d_table + (int64_t)v * p.C);
    for (int i = t & 31; i < p.C / 4; i += 32) __stcs(row + i, make_float4(0.f, 0.f, 0.f, 0.f));
  }
}

__global__ void __cluster_dims__(kSortBlocks, 1, 1) __launch_bounds__(kSortThreads, 1)
    embed_sort_kernel(const EmbedParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  SortShared& sh = *reinterpret_cast<SortShared*>(smem);
  if (blockIdx.x >= kSortBlocks) {
    fill_absent(p, reinterpret_cast<uint32_t*>(smem), blockIdx.x - kSortBlocks, gridDim.x - kSortBlocks);
    return;
  }
  cg::cluster_group cl = cg::this_cluster();
  const int rank = blockIdx.x, t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int bins = 1 << p.bits;
  // a warp's entries, in order of position over warps and blocks
  const int groups = (p.N + 31) / 32, all = kSortBlocks * kSortWarps, me = rank * kSortWarps + warp;
  const int lo = (int)((int64_t)groups * me / all) * 32, hi = min(p.N, (int)((int64_t)groups * (me + 1) / all) * 32);
  bool bad = false;
  cl.sync();   // every block runs: others may write to it
  for (int pass = 0; pass < p.passes; ++pass) {
    const uint64_t* from = (p.passes - pass) & 1 ? p.other : p.sorted;
    uint64_t* to = (p.passes - pass) & 1 ? p.sorted : p.other;
    const int shift = 32 + pass * p.bits;
    auto get = [&](int i) { return pass == 0 ? entry_of(p, i) : from[i]; };
    auto bin = [&](uint64_t x) { return (uint32_t)(x >> shift) & (bins - 1); };
    for (int i = t; i < kSortWarps * kMaxBins; i += kSortThreads) (&sh.hist[0][0])[i] = 0;
    __syncthreads();
#pragma unroll 4
    for (int i = lo + lane; i < hi; i += 32) {
      if (pass == 0) bad = bad || p.tok[i] >= p.V;
      atomicAdd(&sh.hist[warp][bin(get(i))], 1u);
    }
    bad = __syncthreads_or(bad);
    if (t < bins) {
      uint32_t sum = 0;
#pragma unroll 8
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t c = sh.hist[w][t];
        sh.hist[w][t] = sum;
        sum += c;
      }
      for (int r = 0; r < kSortBlocks; ++r) *cl.map_shared_rank(&sh.total[rank][t], r) = sum;
    }
    if (pass == 0 && t == 0) *cl.map_shared_rank(&sh.bad[rank], 0) = bad;
    cl.sync();
    if (pass == 0 && rank == 0 && t == 0) {
      uint32_t any = 0;
      for (int r = 0; r < kSortBlocks; ++r) any |= sh.bad[r];
      *p.err = any ? kErrBadList : 0;
    }
    // where a bin begins, and this block's entries in it
    uint32_t sum = 0, before = 0;
    if (t < bins)
      for (int r = 0; r < kSortBlocks; ++r) {
        const uint32_t c = sh.total[r][t];
        sum += c;
        before += r < rank ? c : 0;
      }
    uint32_t up = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t x = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += x;
    }
    if (lane == 31) sh.warp_sum[warp] = up;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    if (t < bins) sh.base[t] = before + up - sum;
    __syncthreads();
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const bool on = i < hi;
      const uint64_t x = on ? get(i) : 0;
      const uint32_t b = on ? bin(x) : kMaxBins;
      const unsigned same = __match_any_sync(0xffffffffu, b);
      const int mine = __popc(same & ((1u << lane) - 1));
      if (on) to[sh.base[b] + sh.hist[warp][b] + mine] = x;
      __syncwarp();
      if (on && mine == 0) sh.hist[warp][b] += __popc(same);
      __syncwarp();
    }
    cl.sync();   // the pass's entries are in place, and every block is done with the totals
  }
}

// -------------------------------------------------------------------- sum

template <int E>
__device__ __forceinline__ void put_row(float* to, const float* a, float scale, bool add) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    float4 v = make_float4(a[e] * scale, a[e + 1] * scale, a[e + 2] * scale, a[e + 3] * scale);
    float4* at = reinterpret_cast<float4*>(to + e);
    if (add) {
      const float4 o = *at;
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    __stcs(at, v);
  }
}

__device__ __forceinline__ uint32_t token_at(const EmbedParams& p, int64_t i) {
  return (uint32_t)(p.sorted[i] >> 32);
}

// blockDim.x threads (whole warps) lie along the channels, blockDim.y pieces are side by side.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const EmbedParams p) {
  constexpr int E = Piece<T>::E, kAhead = 8;
  const int64_t piece = (int64_t)blockIdx.x * blockDim.y + threadIdx.y, i0 = piece * kPiece;
  if (i0 >= p.N) return;
  const int n = (int)min((int64_t)kPiece, p.N - i0), lane = threadIdx.x & 31;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * E;
  const bool on = c < p.C;
  const uint64_t mine = lane < n ? p.sorted[i0 + lane] : (uint64_t)p.V << 32;
  const uint32_t after = i0 + n < p.N ? token_at(p, i0 + n) : (uint32_t)p.V;
  const uint32_t before = i0 > 0 ? token_at(p, i0 - 1) : (uint32_t)p.V;
  const uint32_t none = (uint32_t)p.V;
  const T* d = static_cast<const T*>(p.d_out) + c;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  const uint32_t first = (uint32_t)(__shfl_sync(0xffffffffu, mine, 0) >> 32);
  uint32_t now = first;
  auto flush = [&](uint32_t next, bool last) {
    // the token goes on in the next piece, or came from the one before
    const bool over = (last && next == now) || (now == first && before == now);
    if (on) {
      if (over)
        put_row<E>(p.part + (piece * 2 + (now == first ? 0 : 1)) * p.C + c, acc, 1.f, false);
      else
        put_row<E>(p.d_table + (int64_t)now * p.C + c, acc, p.scale, p.add);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
  };
  for (int j0 = 0; j0 < kPiece; j0 += kAhead) {
    uint4 v[kAhead];
    uint32_t key[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint64_t x = __shfl_sync(0xffffffffu, mine, j0 + k);
      key[k] = (uint32_t)(x >> 32);
      v[k] = on && key[k] != none ? __ldcs(reinterpret_cast<const uint4*>(d + (int64_t)(uint32_t)x * p.stride))
                                  : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (key[k] != now) {
        if (now != none) flush(key[k], false);
        now = key[k];
      }
      float z[E];
      Piece<T>::get(v[k], z);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += z[e];
    }
  }
  if (now != none) flush(after, true);
}

// One warp row of 32 E channels per block column; a block whose piece begins a
// token that goes on adds up the token's pieces: warp w takes every eighth, in
// order, then the warps' sums are added in order.
template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32) embed_join_kernel(const EmbedParams p) {
  constexpr int E = Piece<T>::E;
  __shared__ float sums[kJoinWarps][32 * E];
  const int64_t piece = blockIdx.x, i0 = piece * kPiece;
  const int pieces = (p.N + kPiece - 1) / kPiece;
  if (piece + 1 >= pieces) return;
  const uint32_t key = token_at(p, i0 + kPiece - 1), first = token_at(p, i0);
  if (key == (uint32_t)p.V || token_at(p, i0 + kPiece) != key) return;
  if (first == key && i0 > 0 && token_at(p, i0 - 1) == key) return;   // it began before
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.y * 32 * E + lane * E;
  // the last piece that holds it
  int64_t end = piece + 1;   // one past
  while (true) {
    const int64_t q = end + lane;
    const unsigned more = __ballot_sync(0xffffffffu, q < pieces && token_at(p, q * kPiece) == key);
    end += __popc(more);
    if (more != 0xffffffffu) break;
  }
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (c < p.C)
#pragma unroll 4
    for (int64_t q = piece + warp; q < end; q += kJoinWarps) {
      const float4* v =
          reinterpret_cast<const float4*>(p.part + (q * 2 + (q == piece && first != key ? 1 : 0)) * p.C + c);
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 x = __ldcs(v + e / 4);
        acc[e] += x.x;
        acc[e + 1] += x.y;
        acc[e + 2] += x.z;
        acc[e + 3] += x.w;
      }
    }
#pragma unroll
  for (int e = 0; e < E; ++e) sums[warp][lane * E + e] = acc[e];
  __syncthreads();
  if (warp == 0 && c < p.C) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      for (int w = 1; w < kJoinWarps; ++w) acc[e] += sums[w][lane * E + e];
    put_row<E>(p.d_table + (int64_t)key * p.C + c, acc, p.scale, p.add);
  }
}

// ------------------------------------------------------------------- host

stp_status check_embed(const stp_embed_desc* d) {
  if (!d) return fail(STP_EINVAL, "embed descriptor is NULL");
  if (d->dtype != STP_BF16 && d->dtype != STP_FP32) return fail(STP_EUNSUPPORTED, "dtype %d not supported", d->dtype);
  if (d->n_tokens < 0) return fail(STP_EINVAL, "n_tokens < 0");
  if (d->n_tokens > (1 << 28)) return fail(STP_EUNSUPPORTED, "more than 2^28 tokens");
  if (d->vocab < 1 || d->vocab > (1 << 24)) return fail(STP_EUNSUPPORTED, "vocab must lie in [1, 2^24]");
  const int each = d->dtype == STP_BF16 ? 8 : 4;
  if (d->dim < each || d->dim > 65536 || d->dim % each)
    return fail(STP_EUNSUPPORTED, "dim must be a multiple of %d (16 bytes) in [%d, 65536]", each, each);
  if (d->stride < d->dim || d->stride % each)
    return fail(STP_EINVAL, "stride must be at least dim and a multiple of 16 bytes");
  if (!(d->scale >= -1e6f && d->scale <= 1e6f)) return fail(STP_EINVAL, "scale must lie in [-1e6, 1e6]");
  return STP_OK;
}

struct EmbedWs {
  size_t sorted, other, part, total;
};
EmbedWs embed_ws(const stp_embed_desc* d) {
  EmbedWs w;
  const size_t n = d->n_tokens, pieces = (n + kPiece - 1) / kPiece;
  w.sorted = 256;
  w.other = w.sorted + align256(n * 8);
  w.part = w.other + align256(n * 8);
  w.total = w.part + align256(pieces * 2 * d->dim * 4);
  return w;
}

EmbedParams embed_params(const stp_embed_desc* d, const int32_t* tok, void* ws) {
  EmbedParams p{};
  p.N = d->n_tokens;
  p.V = d->vocab;
  p.C = d->dim;
  p.stride = d->stride;
  p.scale = d->scale;
  p.tok = tok;
  p.err = static_cast<uint32_t*>(ws);
  return p;
}

template <typename T>
cudaError_t run_bwd(const EmbedParams& p, int n_sm, cudaStream_t s) {
  constexpr int E = Piece<T>::E;
  static PerDevice limit;
  constexpr int smem = sizeof(SortShared);
  cudaError_t e = limit([] {
    return cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  const int fill = p.add ? 0 : (n_sm / kSortBlocks - 1 > 1 ? n_sm / kSortBlocks - 1 : 1);   // clusters
  embed_sort_kernel<<<kSortBlocks * (1 + fill), kSortThreads, smem, s>>>(p);
  if (p.N > 0) {
    const int pieces = (p.N + kPiece - 1) / kPiece, along = (p.C / E + 31) / 32 * 32;
    const dim3 block(along < kThreads ? along : kThreads, along < kThreads ? kThreads / along : 1);
    embed_sum_kernel<T><<<dim3((pieces + block.y - 1) / block.y, (p.C / E + block.x - 1) / block.x), block, 0, s>>>(p);
    if (pieces > 1)
      embed_join_kernel<T><<<dim3(pieces - 1, (p.C / E + 31) / 32), kJoinWarps * 32, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_embed_workspace_size(const stp_embed_desc* desc, size_t* ws_bytes) {
  clear_error();
  stp_status st = check_embed(desc);
  if (st) return st;
  if (!ws_bytes) return fail(STP_EINVAL, "stp_embed_workspace_size: NULL output");
  *ws_bytes = embed_ws(desc).total;
  return STP_OK;
}

extern "C" stp_status stp_embed_fwd(const stp_embed_desc* desc, const void* table, const int32_t* d_token_ids,
                                    void* out, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_embed(desc);
  if (st) return st;
  if (!d_ws || reinterpret_cast<uintptr_t>(d_ws) & 255)
    return fail(STP_EINVAL, "stp_embed_fwd: the workspace must be 256-byte aligned");
  if (desc->n_tokens > 0 && (!table || !d_token_ids || !out))
    return fail(STP_EINVAL, "stp_embed_fwd: NULL device pointer");
  if ((reinterpret_cast<uintptr_t>(table) | reinterpret_cast<uintptr_t>(out)) & 15)
    return fail(STP_EINVAL, "stp_embed_fwd: table and out must be 16-byte aligned");
  EmbedParams p = embed_params(desc, d_token_ids, d_ws);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.check = p.N > 0 && p.N <= rows::kCheckMost;
  p.table = table;
  p.out = out;
  cudaError_t e = p.check ? cudaSuccess : cudaMemsetAsync(d_ws, 0, 4, s);
  if (e == cudaSuccess && p.N > 0) {
    const int pieces = p.C / (desc->dtype == STP_BF16 ? 8 : 4);
    int shift = 0;
    while (shift < 5 && (1 << shift) < pieces) ++shift;
    const unsigned grid = (unsigned)((((int64_t)p.N << shift) + kThreads - 1) / kThreads) + p.check;
    if (desc->dtype == STP_BF16)
      embed_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(p, shift);
    else
      embed_fwd_kernel<float><<<grid, kThreads, 0, s>>>(p, shift);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_embed_fwd: %s", cudaGetErrorString(e));
  return STP_OK;
}

extern "C" stp_status stp_embed_bwd(const stp_embed_desc* desc, const void* d_out, const int32_t* d_token_ids,
                                    int32_t accumulate, float* d_table, void* d_ws, void* stream) {
  clear_error();
  stp_status st = check_embed(desc);
  if (st) return st;
  if (!d_ws || reinterpret_cast<uintptr_t>(d_ws) & 255)
    return fail(STP_EINVAL, "stp_embed_bwd: the workspace must be 256-byte aligned");
  if (!d_table || (desc->n_tokens > 0 && (!d_out || !d_token_ids)))
    return fail(STP_EINVAL, "stp_embed_bwd: NULL device pointer");
  if ((reinterpret_cast<uintptr_t>(d_table) | reinterpret_cast<uintptr_t>(d_out)) & 15)
    return fail(STP_EINVAL, "stp_embed_bwd: d_out and d_table must be 16-byte aligned");
  EmbedParams p = embed_params(desc, d_token_ids, d_ws);
  const EmbedWs w = embed_ws(desc);
  char* ws = static_cast<char*>(d_ws);
  p.add = accumulate != 0;
  p.d_out = d_out;
  p.d_table = d_table;
  p.sorted = reinterpret_cast<uint64_t*>(ws + w.sorted);
  p.other = reinterpret_cast<uint64_t*>(ws + w.other);
  p.part = reinterpret_cast<float*>(ws + w.part);
  int width = 1;   // bits of a token, V among them
  while ((p.V >> width) != 0) ++width;
  p.passes = (width + 8) / 9;
  p.bits = (width + p.passes - 1) / p.passes;
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess)
    e = desc->dtype == STP_BF16 ? run_bwd<__nv_bfloat16>(p, n_sm, s) : run_bwd<float>(p, n_sm, s);
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_embed_bwd: %s", cudaGetErrorString(e));
  return STP_OK;
}
