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
//                 channels entry by entry.  A token that occurs 64 times at most is added up
//                 where it begins, also beyond the piece; what a piece holds of
//                 another one goes to the workspace
//   embed_join_kernel   those tokens: the sums of their pieces, in order
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
constexpr int kHeld = 8;            // entries of a lane in registers: all of them up to 65536 tokens
constexpr int kPiece = 32;          // sorted entries of a piece
constexpr int kShort = 64;          // entries of a token that one block adds up, at most
constexpr int kJoinAlong = 32, kJoinRows = kThreads / kJoinAlong;

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
  float* part;             // [pieces][2][C]: what a piece holds of tokens that occur often
  uint32_t* n_long;        // such tokens, and the pieces that they begin in, in any order
  uint32_t* long_at;
  float* d_table;
};

// ---------------------------------------------------------------- forward

// 2^shift threads take a token.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_fwd_kernel(const EmbedParams p, int shift) {
  constexpr int E = Piece<T>::E;
  if (p.check && blockIdx.x == 0) {
    // all tokens, 16 of a thread at a time
    bool bad = false;
    for (int i0 = threadIdx.x; i0 < p.N; i0 += 16 * kThreads)
#pragma unroll
      for (int k = 0; k < 16; ++k) bad |= p.tok[min(i0 + k * kThreads, p.N - 1)] >= p.V;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) *p.err = bad ? kErrBadList : 0;
    return;
  }
  const int64_t n = ((int64_t)(blockIdx.x - p.check) * kThreads + threadIdx.x) >> shift;
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
  for (int i0 = t; i0 < p.N; i0 += 16 * kSortThreads) {
    int x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = i0 + k * kSortThreads < p.N ? p.tok[i0 + k * kSortThreads] - v0 : -1;
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (x[k] >= 0 && x[k] < v1 - v0) atomicOr(seen + (x[k] >> 5), 1u << (x[k] & 31));
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
    for (int i = t; i < kSortWarps * bins; i += kSortThreads) sh.hist[i >> p.bits][i & (bins - 1)] = 0;
    // the first entries of the warp stay in registers for both walks
    uint64_t held[kHeld];
#pragma unroll
    for (int k = 0; k < kHeld; ++k) {
      const int i = lo + k * 32 + lane;
      held[k] = i < hi ? get(i) : 0;
      if (pass == 0) bad = bad || (i < hi && p.tok[i] >= p.V);
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (lo + k * 32 + lane < hi) atomicAdd(&sh.hist[warp][bin(held[k])], 1u);
    for (int i = lo + kHeld * 32 + lane; i < hi; i += 32) {
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
      *p.n_long = 0;
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
    before += __reduce_add_sync(0xffffffffu, lane < warp ? sh.warp_sum[lane] : 0);
    if (t < bins) sh.base[t] = before + up - sum;
    __syncthreads();
    auto place = [&](int i, uint64_t x) {
      const bool on = i < hi;
      const uint32_t b = on ? bin(x) : bins;
      // the lanes with the same bin (a match instruction takes the bins one by one, 240 cycles for a warp)
      unsigned same = 0xffffffffu;
      for (int k = 0; k <= p.bits; ++k) {
        const unsigned ones = __ballot_sync(0xffffffffu, b >> k & 1);
        same &= b >> k & 1 ? ones : ~ones;
      }
      const int mine = __popc(same & ((1u << lane) - 1));
      if (on) to[sh.base[b] + sh.hist[warp][b] + mine] = x;
      __syncwarp();
      if (on && mine == 0) sh.hist[warp][b] += __popc(same);
      __syncwarp();
    };
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (lo + k * 32 < hi) place(lo + k * 32 + lane, held[k]);
    for (int i0 = lo + kHeld * 32; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      place(i, i < hi ? get(i) : 0);
    }
    cl.sync();   // the pass's entries are in place, and every block is done with the totals
  }
}

// -------------------------------------------------------------------- sum

// A row of dE, or of a part.  Each is written by one thread, so an addition in
// memory gives the same bits each time, and nothing waits for what was there.
template <int E>
__device__ __forceinline__ void put_row(float* to, const float* a, float scale, bool add) {
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    const float4 v = make_float4(a[e] * scale, a[e + 1] * scale, a[e + 2] * scale, a[e + 3] * scale);
    if (add)
      asm volatile("red.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + e), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                   : "memory");
    else
      __stcs(reinterpret_cast<float4*>(to + e), v);
  }
}

__device__ __forceinline__ uint32_t token_at(const EmbedParams& p, int64_t i) {
  return (uint32_t)(p.sorted[i] >> 32);
}

// How many of a warp's values, from lane 0 on (from lane 31 down), satisfy a condition without a break.
__device__ __forceinline__ int leading(bool on) { return __clz(__brev(~__ballot_sync(0xffffffffu, on))); }
__device__ __forceinline__ int trailing(bool on) { return __clz(~__ballot_sync(0xffffffffu, on)); }

// blockDim.x threads (whole warps) lie along the channels, blockDim.y pieces are side by side.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const EmbedParams p) {
  constexpr int E = Piece<T>::E, kAhead = 8;
  const int piece = blockIdx.x * blockDim.y + threadIdx.y, i0 = piece * kPiece;
  if (i0 >= p.N) return;
  const int lane = threadIdx.x & 31, c = (blockIdx.y * blockDim.x + threadIdx.x) * E;
  const bool on = c < p.C;
  const uint32_t none = (uint32_t)p.V;
  // entries from kShort before the piece to kShort behind it; what is outside is no token
  uint64_t near[kPiece / 32 + 2 * kShort / 32];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    const int i = i0 - kShort + k * 32 + lane;
    near[k] = i >= 0 && i < p.N ? p.sorted[i] : (uint64_t)(i < 0 ? 0xffffffffu : none) << 32;
  }
  auto token = [&](int k) { return (uint32_t)(near[k] >> 32); };
  const uint32_t first = __shfl_sync(0xffffffffu, token(2), 0), last = __shfl_sync(0xffffffffu, token(2), 31);
  // the first token: how far it reaches back and forward
  int back = trailing(token(1) == first), ahead = leading(token(2) == first);
  if (back == 32) back += trailing(token(0) == first);
  if (ahead == 32) ahead += leading(token(3) == first);
  if (ahead == 64) ahead += leading(token(4) == first);
  const bool often = back + ahead > kShort;   // more than kShort entries, so that each of its pieces sees it
  int begin = 0, end = kPiece;
  if (back > 0 && !often) begin = ahead;      // added up where it began
  // the last token, where it begins in this piece and goes on
  bool last_often = often && last == first;
  if (last != first || back == 0) {
    const int in = trailing(token(2) == last);
    int over = leading(token(3) == last);
    if (over == 32) over += leading(token(4) == last);
    if (over > 0) {
      last_often = in + over > kShort;
      if (!last_often) end += over;
      else if (blockIdx.y == 0 && threadIdx.x == 0 && last != none) p.long_at[atomicAdd(p.n_long, 1u)] = piece;
    }
  }
  const T* d = static_cast<const T*>(p.d_out) + c;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  uint32_t now = none;
  auto flush = [&](bool part) {
    if (on && now != none) {
      if (part)
        put_row<E>(p.part + ((int64_t)piece * 2 + (now == first ? 0 : 1)) * p.C + c, acc, 1.f, false);
      else
        put_row<E>(p.d_table + (int64_t)now * p.C + c, acc, p.scale, p.add);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
  };
  for (int j0 = begin & ~(kAhead - 1); j0 < end; j0 += kAhead) {
    const uint64_t from = j0 < 32 ? near[2] : j0 < 64 ? near[3] : near[4];
    uint4 v[kAhead];
    uint32_t key[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const uint64_t x = __shfl_sync(0xffffffffu, from, (j0 + k) & 31);
      key[k] = j0 + k >= begin && j0 + k < end ? (uint32_t)(x >> 32) : none;
      v[k] = on && key[k] != none ? __ldcs(reinterpret_cast<const uint4*>(d + (int64_t)(uint32_t)x * p.stride))
                                  : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (key[k] != now) {
        flush(now == first && often);
        now = key[k];
      }
      float z[E];
      Piece<T>::get(v[k], z);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] += z[e];
    }
  }
  flush((now == first && often) || (now == last && last_often));
}

// Tokens that occur often, one after another for a block: row y of its threads
// takes every kJoinRows-th piece, in order, then the rows' sums are added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) embed_join_kernel(const EmbedParams p) {
  constexpr int E = Piece<T>::E, kRead = 8;
  __shared__ float sums[kJoinRows][kJoinAlong][E];
  const int pieces = (p.N + kPiece - 1) / kPiece, lane = threadIdx.x, y = threadIdx.y;
  const int c = (blockIdx.y * kJoinAlong + lane) * E;
  const uint32_t n = *p.n_long;
  for (uint32_t at = blockIdx.x; at < n; at += gridDim.x) {
    const int piece = p.long_at[at];
    const uint32_t key = token_at(p, (int64_t)piece * kPiece + kPiece - 1), first = token_at(p, (int64_t)piece * kPiece);
    // one past the last piece that holds it: by strides of 32 pieces, then one by one
    int end = piece + 1;
    for (int step = 32; step > 0; step = step == 32 ? 1 : 0)
      while (true) {
        const int q = end + (step == 32 ? lane * 32 + 31 : lane);
        const unsigned more = __ballot_sync(0xffffffffu, q < pieces && token_at(p, (int64_t)q * kPiece) == key);
        end += step * __popc(more);
        if (more != 0xffffffffu) break;
      }
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    if (c < p.C)
      for (int q0 = piece + y; q0 < end; q0 += kRead * kJoinRows) {
        float4 v[kRead][E / 4];
#pragma unroll
        for (int k = 0; k < kRead; ++k) {
          const int q = q0 + k * kJoinRows;
          const float4* from =
              reinterpret_cast<const float4*>(p.part + ((int64_t)q * 2 + (q == piece && first != key ? 1 : 0)) * p.C + c);
#pragma unroll
          for (int e = 0; e < E / 4; ++e) v[k][e] = q < end ? __ldcs(from + e) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int k = 0; k < kRead; ++k)
#pragma unroll
          for (int e = 0; e < E; e += 4) {
            acc[e] += v[k][e / 4].x;
            acc[e + 1] += v[k][e / 4].y;
            acc[e + 2] += v[k][e / 4].z;
            acc[e + 3] += v[k][e / 4].w;
          }
      }
#pragma unroll
    for (int e = 0; e < E; ++e) sums[y][lane][e] = acc[e];
    __syncthreads();
    if (y == 0 && c < p.C) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        for (int r = 1; r < kJoinRows; ++r) acc[e] += sums[r][lane][e];
      put_row<E>(p.d_table + (int64_t)key * p.C + c, acc, p.scale, p.add);
    }
    __syncthreads();
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
  size_t sorted, other, part, long_at, total;
};
EmbedWs embed_ws(const stp_embed_desc* d) {
  EmbedWs w;
  const size_t n = d->n_tokens, pieces = (n + kPiece - 1) / kPiece;
  w.sorted = 256;
  w.other = w.sorted + align256(n * 8);
  w.part = w.other + align256(n * 8);
  w.long_at = w.part + align256(pieces * 2 * d->dim * 4);
  w.total = w.long_at + align256(pieces * 4);
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
  // Clusters that write zeros, all of them resident: of 152 SMs, 16 clusters of eight find a place at a time
  const int fill = p.add ? 0 : n_sm / 10 > 1 ? n_sm / 10 : 1;
  embed_sort_kernel<<<kSortBlocks * (1 + fill), kSortThreads, smem, s>>>(p);
  if (p.N > 0) {
    const int pieces = (p.N + kPiece - 1) / kPiece, along = (p.C / E + 31) / 32 * 32;
    const dim3 block(along < kThreads ? along : kThreads, along < kThreads ? kThreads / along : 1);
    embed_sum_kernel<T>
        <<<dim3((pieces + block.y - 1) / block.y, (p.C / E + block.x - 1) / block.x), block, 0, s>>>(p);
    const int most = p.N / (kShort + 1);   // tokens that occur more often
    if (most > 0)
      embed_join_kernel<T><<<dim3(most < 64 ? most : 64, (p.C / E + kJoinAlong - 1) / kJoinAlong),
                             dim3(kJoinAlong, kJoinRows), 0, s>>>(p);
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
  // One block checks all tokens, 4096 of them a round trip to memory, and saves the
  // word's clearing (5 us beside a forward of 28); from rows of 1 KB on it ends before the others do.
  p.check = p.N > 0 && (p.N <= 4096 || p.C * (desc->dtype == STP_BF16 ? 2 : 4) >= 1024);
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
  p.n_long = reinterpret_cast<uint32_t*>(ws + 16);   // in the error word's 256 bytes
  p.long_at = reinterpret_cast<uint32_t*>(ws + w.long_at);
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
