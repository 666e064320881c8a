// Tile classification of windowed tree attention: query i sees key j iff
//   j <= i, subtree_end[j] >= i, and position[i] < lim[j]
// with lim[j] = position[j] + window, or no limit for the first n_sink
// positions of a path.
//
// Classes are made for blocks of 32 queries x 32 keys, from each block's least
// and largest subtree_end and position, and a tile of 128 x 128 takes its
// class from its sixteen blocks.  A window cuts tiles along both edges of a
// band, and short branches cut many more, so most listed tiles are PARTIAL; of
// a partial tile's blocks the empty ones cost the attention kernels nothing
// and the full ones no mask.  The sixteen classes of a pair are one word.
//
// A block is EMPTY when the keys' subtrees end before it, or when every query
// that they reach (up to their largest subtree_end: qmin) is at or past their
// largest lim.  It is FULL when every subtree reaches its last query and no
// query is past the window of the key at the least position.  Both are exact
// but where a block holds the ends of several branches.
//
// Two launches: the blocks' extremes and lim; then one block per (tile, row)
// for the lists, whose last one to finish in a row numbers the row's pairs.
#include <cuda_runtime.h>

#include <new>
#include <vector>

#include "internal.h"
#include "layout.h"

namespace stp {
namespace {

constexpr int kBlock = 32;                      // tokens of a block
constexpr int kPer = kTile / kBlock;            // blocks of a tile along one side
constexpr int kMaxPosition = 1 << 30;           // positions and windows: two of them add up in an int
constexpr uint32_t kAllFull = 0xaaaaaaaau;      // sixteen times kFull

// A row's arrays (layout.h).
struct RowBlocks {
  const int32_t* smin;
  const int32_t* smax;
  const int32_t* pmin;
  const int32_t* pmax;
  const int32_t* qmin;
  int window, n_sink;
};

// Four neighbouring blocks' values, read at once (16-byte aligned).
struct alignas(16) Four {
  int32_t v[4];
};
__host__ __device__ inline Four four(const int32_t* p) { return *reinterpret_cast<const Four*>(p); }

// The classes of the sixteen blocks of tile (qt, kt).
__host__ __device__ inline uint32_t tile_word(const RowBlocks& b, int qt, int kt) {
  if (kt > qt) return 0;
  const Four smax = four(b.smax + kPer * kt);
  const int q_first = qt * kTile;
  if (kt < qt && smax.v[0] < q_first && smax.v[1] < q_first && smax.v[2] < q_first && smax.v[3] < q_first) return 0;
  const Four smin = four(b.smin + kPer * kt), kmin = four(b.pmin + kPer * kt), kmax = four(b.pmax + kPer * kt);
  const Four qmin = four(b.pmin + kPer * qt), qmax = four(b.pmax + kPer * qt);
  uint32_t word = 0;
#pragma unroll
  for (int q = 0; q < kPer; ++q) {
    const int q0 = q_first + q * kBlock, q1 = q0 + kBlock - 1;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      uint32_t c = kPartial;
      if (kt == qt && k >= q) {
        if (k > q) c = kEmpty;
      } else {
        const int reach = smax.v[k];
        const bool first = kmin.v[k] < b.n_sink;   // some key is a first token
        if (reach < q0) {
          c = kEmpty;
        } else if (!first && (reach < q1 ? b.qmin[reach] : qmin.v[q]) - kmax.v[k] >= b.window) {
          c = kEmpty;
        } else if (smin.v[k] >= q1 && (kmax.v[k] < b.n_sink || qmax.v[q] - kmin.v[k] < b.window)) {
          c = kFull;
        }
      }
      word |= c << (2 * (kPer * q + k));
    }
  }
  return word;
}

struct WindowArgs {
  int T, NT, window, n_sink;
  int64_t cap;
  const int32_t* se;
  const int32_t* pos;
  int32_t *smin, *smax, *pmin, *pmax, *qmin, *lim;
  uint32_t* word;
  int8_t* cls;
  int32_t *csr_cnt, *csr, *csc_cnt, *csc, *crank, *csr_off, *row_base, *pair_count, *ticket, *kind;
  uint32_t* err;
};

__device__ __forceinline__ RowBlocks row_blocks(const WindowArgs& a, int r) {
  const size_t nb = (size_t)r * a.NT * kPer;
  return {a.smin + nb, a.smax + nb, a.pmin + nb, a.pmax + nb, a.qmin + (size_t)r * a.T, a.window, a.n_sink};
}

// One warp per block of 32 tokens.
__global__ void __launch_bounds__(kTile) window_blocks_kernel(const WindowArgs a) {
  const int tile = blockIdx.x, r = blockIdx.y, t = threadIdx.x, lane = t & 31;
  const int j = tile * kTile + t;
  const size_t at = (size_t)r * a.T + j;
  const int se = a.se[at], pos = a.pos[at];
  if (se < j || se >= a.T) atomicOr(a.err, kErrBadSubtreeEnd);
  if (pos < 0 || pos >= kMaxPosition) atomicOr(a.err, kErrBadPosition);
  int low = pos;   // prefix minimum
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, low, o);
    if (lane >= o) low = min(low, y);
  }
  a.qmin[at] = low;
  a.lim[at] = pos < a.n_sink ? 0x7fffffff : pos + a.window;
  const int smin = __reduce_min_sync(0xffffffffu, se), smax = __reduce_max_sync(0xffffffffu, se);
  const int pmax = __reduce_max_sync(0xffffffffu, pos);
  if (lane == 31) {
    const size_t b = ((size_t)r * a.NT + tile) * kPer + (t >> 5);
    a.smin[b] = smin;
    a.smax[b] = smax;
    a.pmin[b] = low;
    a.pmax[b] = pmax;
  }
  if (tile == 0 && t == 0) {
    a.ticket[r] = 0;
    if (r == 0) {
      *a.pair_count = 0;
      a.kind[0] = a.window;
      a.kind[1] = a.n_sink;
    }
  }
}

// Exclusive prefix count of `flag` over the block's 128 threads, and the total.
__device__ __forceinline__ int block_scan(bool flag, int* s_warp, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const unsigned b = __ballot_sync(0xffffffffu, flag);
  if (lane == 0) s_warp[w] = __popc(b);
  __syncthreads();
  int before = 0;
  for (int k = 0; k < w; ++k) before += s_warp[k];
  *total = s_warp[0] + s_warp[1] + s_warp[2] + s_warp[3];
  __syncthreads();
  return before + __popc(b & ((1u << lane) - 1u));
}

// Numbers the row's pairs (query tile major) once all its lists are written:
// csr_off and row_base.  A key tile's entry is then row_base + csr_off + crank,
// which the backward looks up itself (an array of them, made here by the row's
// last block, took 25 us of a 16384-token row).
__device__ void number_pairs(const WindowArgs& a, int r, int* s_warp) {
  const int t = threadIdx.x, lane = t & 31, w = t >> 5;
  const int32_t* cnt = a.csr_cnt + (size_t)r * a.NT;
  int32_t* off = a.csr_off + (size_t)r * a.NT;
  int before = 0;
  for (int q0 = 0; q0 < a.NT; q0 += kTile) {
    const int c = q0 + t < a.NT ? __ldcg(cnt + q0 + t) : 0;
    int x = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[w] = x;
    __syncthreads();
    for (int k = 0; k < w; ++k) x += s_warp[k];
    if (q0 + t < a.NT) off[q0 + t] = before + x - c;
    before += s_warp[0] + s_warp[1] + s_warp[2] + s_warp[3];
    __syncthreads();
  }
  if (t == 0) {
    const int base = atomicAdd(a.pair_count, before);
    if ((int64_t)base + before > a.cap) atomicOr(a.err, kErrCapacity);
    a.row_base[r] = base;
  }
}

__global__ void __launch_bounds__(kTile) window_lists_kernel(const WindowArgs a) {
  __shared__ int s_warp[4];
  __shared__ int s_last;
  const int b = blockIdx.x, r = blockIdx.y, t = threadIdx.x, NT = a.NT;
  const RowBlocks rb = row_blocks(a, r);
  const size_t row = ((size_t)r * NT + b) * NT;
  // query tile b: its classes and its list of key tiles
  int base = 0;
  for (int k0 = 0; k0 < NT; k0 += kTile) {
    const int kt = k0 + t;
    const uint32_t w = kt < NT ? tile_word(rb, b, kt) : 0;
    if (kt < NT) {
      a.word[row + kt] = w;
      a.cls[row + kt] = w == 0 ? kEmpty : w == kAllFull ? kFull : kPartial;
    }
    int tot;
    const int at = base + block_scan(w != 0, s_warp, &tot);
    if (w) {
      a.csr[row + at] = (kt << 1) | (w != kAllFull);
      a.crank[row + kt] = at;
    }
    base += tot;
  }
  if (t == 0) a.csr_cnt[(size_t)r * NT + b] = base;
  // key tile b: its list of query tiles
  base = 0;
  for (int q0 = 0; q0 < NT; q0 += kTile) {
    const int qt = q0 + t;
    const uint32_t w = qt < NT ? tile_word(rb, qt, b) : 0;
    int tot;
    const int at = base + block_scan(w != 0, s_warp, &tot);
    if (w) a.csc[row + at] = (qt << 1) | (w != kAllFull);
    base += tot;
  }
  if (t == 0) a.csc_cnt[(size_t)r * NT + b] = base;
  __threadfence();
  __syncthreads();
  if (t == 0) s_last = atomicAdd(a.ticket + r, 1) == NT - 1;
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  number_pairs(a, r, s_warp);
}

}  // namespace
}  // namespace stp

using namespace stp;

extern "C" stp_status stp_count_window_tile_pairs(const int32_t* subtree_end, const int32_t* position_ids,
                                                  int32_t n_rows, int32_t row_len, int32_t window, int32_t n_sink,
                                                  int64_t* n_pairs) {
  clear_error();
  if (!n_pairs || ((!subtree_end || !position_ids) && n_rows > 0))
    return fail(STP_EINVAL, "stp_count_window_tile_pairs: NULL pointer");
  if (n_rows < 0 || row_len <= 0 || row_len % kTile)
    return fail(STP_EINVAL, "stp_count_window_tile_pairs: need n_rows >= 0 and row_len a positive multiple of 128");
  stp_status st = check_window(window, n_sink);
  if (st) return st;
  const int NB = row_len / kBlock, NT = row_len / kTile;
  int64_t total = 0;
  try {
    std::vector<Four> tiles(4 * (size_t)NT);   // four arrays of NB values
    int32_t *smin = tiles[0].v, *smax = smin + NB, *pmin = smax + NB, *pmax = pmin + NB;
    std::vector<int32_t> qmin(row_len);
    const RowBlocks rb = {smin, smax, pmin, pmax, qmin.data(), clip_window(window), n_sink};
    for (int64_t r = 0; r < n_rows; ++r) {
      const int32_t *se = subtree_end + r * row_len, *pos = position_ids + r * row_len;
      for (int32_t j = 0; j < row_len; ++j) {
        if (se[j] < j || se[j] >= row_len)
          return fail(STP_EINVAL, "stp_count_window_tile_pairs: subtree_end[%lld][%d] = %d outside [j, row_len)",
                      (long long)r, j, se[j]);
        if (pos[j] < 0 || pos[j] >= kMaxPosition)
          return fail(STP_EINVAL, "stp_count_window_tile_pairs: position_ids[%lld][%d] = %d outside [0, 2^30)",
                      (long long)r, j, pos[j]);
        const int b = j / kBlock;
        const bool first = j % kBlock == 0;
        smin[b] = first || se[j] < smin[b] ? se[j] : smin[b];
        smax[b] = first || se[j] > smax[b] ? se[j] : smax[b];
        pmin[b] = first || pos[j] < pmin[b] ? pos[j] : pmin[b];
        pmax[b] = first || pos[j] > pmax[b] ? pos[j] : pmax[b];
        qmin[j] = pmin[b];
      }
      for (int kt = 0; kt < NT; ++kt) {
        int32_t reach = 0;
        for (int k = kt * kPer; k < (kt + 1) * kPer; ++k) reach = smax[k] > reach ? smax[k] : reach;
        for (int qt = kt; qt <= reach / kTile; ++qt) total += tile_word(rb, qt, kt) != 0;
      }
    }
  } catch (const std::bad_alloc&) {
    return fail(STP_ENOMEM, "stp_count_window_tile_pairs: out of memory");
  }
  *n_pairs = total;
  return STP_OK;
}

extern "C" stp_status stp_classify_window(const stp_attn_desc* desc, int32_t window, int32_t n_sink,
                                          const int32_t* d_subtree_end, const int32_t* d_position_ids,
                                          void* d_tile_meta, void* stream) {
  clear_error();
  stp_status st = check_desc(desc);
  if (!st) st = check_window(window, n_sink);
  if (st) return st;
  if (!d_subtree_end || !d_position_ids || !d_tile_meta)
    return fail(STP_EINVAL, "stp_classify_window: NULL device pointer");
  if ((reinterpret_cast<uintptr_t>(d_tile_meta) & 255) ||
      (reinterpret_cast<uintptr_t>(d_subtree_end) | reinterpret_cast<uintptr_t>(d_position_ids)) & 15)
    return fail(STP_EINVAL, "stp_classify_window: tile_meta must be 256-byte, the row arrays 16-byte aligned");
  if ((int64_t)desc->n_rows * desc->row_len > 0x7fffffff)
    return fail(STP_EUNSUPPORTED, "stp_classify_window: more than 2^31 - 1 tokens");
  if (desc->n_rows == 0) return STP_OK;
  const int NT = desc->row_len / kTile;
  const TileMeta m = tile_meta_layout(desc->n_rows, NT);
  char* base = static_cast<char*>(d_tile_meta);
  auto ints = [&](size_t at) { return reinterpret_cast<int32_t*>(base + at); };
  WindowArgs a;
  a.T = desc->row_len;
  a.NT = NT;
  a.window = clip_window(window);
  a.n_sink = n_sink;
  a.cap = pair_capacity(desc->n_rows, NT, desc->max_tile_pairs);
  a.se = d_subtree_end;
  a.pos = d_position_ids;
  a.smin = ints(m.smin);
  a.smax = ints(m.smax);
  a.pmin = ints(m.pmin);
  a.pmax = ints(m.pmax);
  a.qmin = ints(m.qmin);
  a.lim = ints(m.lim);
  a.word = reinterpret_cast<uint32_t*>(base + m.word);
  a.cls = reinterpret_cast<int8_t*>(base + m.cls);
  a.csr_cnt = ints(m.csr_cnt);
  a.csr = ints(m.csr);
  a.csc_cnt = ints(m.csc_cnt);
  a.csc = ints(m.csc);
  a.crank = ints(m.crank);
  a.csr_off = ints(m.csr_off);
  a.row_base = ints(m.row_base);
  a.pair_count = ints(m.pair_count);
  a.ticket = ints(m.ticket);
  a.kind = ints(m.kind);
  a.err = reinterpret_cast<uint32_t*>(base + m.err);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaMemsetAsync(a.err, 0, 4, s);
  if (e == cudaSuccess) {
    const dim3 grid(NT, desc->n_rows);
    window_blocks_kernel<<<grid, kTile, 0, s>>>(a);
    window_lists_kernel<<<grid, kTile, 0, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return fail(STP_ECUDA, "stp_classify_window: %s", cudaGetErrorString(e));
  return STP_OK;
}
