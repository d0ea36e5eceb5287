// Eviction from a cache by accumulated attention weight: which rows stay
// (csa2_evict_select) and the move that closes the rest up (csa2_evict_rows).
#include <cooperative_groups.h>

#include "common.cuh"

namespace csa2 {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Selection.  One cluster of CTAs per (request, head); each CTA holds a
// contiguous slice of the rows between the sink and the recent ones as
// order-preserving 32-bit keys in shared memory (what does not fit is read
// again from L2).  Histograms of 11, 11 and 10 bits, added up over the cluster
// through distributed shared memory, give the key T of the last row kept;
// rows above T stay, and of those equal to T the first in row order.
//
// The masses are read from memory once, and the slice is walked three times
// more, four keys a lane: the first histogram is taken while loading; the keys
// in its chosen bin are listed (they are few, and the other two histograms are
// taken of the list; a list that overflows is replaced by the slice); the rows
// that stay are counted by warp, each warp having a contiguous part; and they
// are written in row order, a warp at a time without further barriers.  With
// the digits taken of whole slices and a block-wide scan every 2048 rows the
// kernel was bound by its instructions (170 to 32 rows, 50 us for 24 x 8 rows
// of 26,000 on average, now 38 us; what is left is each step's fixed cost to a
// warp).
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kHeld = 10240;          // keys of a slice in shared memory (40 KB)
constexpr int kLoads = 8;             // masses in flight a thread
constexpr int kMinSlice = 4096;
constexpr int kSelPlaces = 3 * 152;     // CTAs the GPU holds at a time
constexpr int kBins = 2048;
constexpr int kList = 1024;           // listed keys

struct SelParams {
  int num_req, n_heads;
  const int64_t *kv_start, *kv_len;
  const float *mass;
  int64_t kv_rows;
  int keep, sink, recent;
  int32_t *idx;
  int64_t *new_len;               // null: written behind the selection
  int32_t *d_err;
};

struct SelShared {
  uint32_t hist[kBins];
  uint32_t list[kList];
  uint32_t listed;                // keys offered to the list
  uint32_t scan[kSelWarps];
  uint32_t digit, above;          // a histogram's answer
  uint32_t warp_gt[kSelWarps], warp_eq[kSelWarps];
  uint32_t gt, eq;                // this CTA's rows above T, and equal to it
};

// exclusive prefix sum over the block in thread order
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) tmp[warp] = inc;
  __syncthreads();
  const uint32_t before = lane < warp ? tmp[lane] : 0u;     // warps in front
  return __reduce_add_sync(0xffffffffu, before) + inc - v;
}

// One CTA's slice: `len` candidate rows from src on, `lo` rows behind the
// request's first; kAll: the slices of the cluster fit into shared memory.
template <bool kAll>
__device__ void select_slice(const SelParams &P, SelShared &sh, uint32_t *held,
                             const float *__restrict__ src, int32_t *__restrict__ idx, int lo,
                             uint32_t len, int room, int nc, int rank) {
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // clusters of one CTA need the block's barrier only
  auto sync = [&]() {
    if (nc == 1) __syncthreads(); else cluster.sync();
  };
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.hist[i] = 0;
  if (threadIdx.x == 0) sh.listed = 0;
  __syncthreads();
  for (uint32_t i0 = threadIdx.x; i0 < len; i0 += kLoads * kSelThreads) {
    float m[kLoads];
    if (i0 - threadIdx.x + kLoads * kSelThreads <= len) {     // a whole step
#pragma unroll
      for (int u = 0; u < kLoads; ++u) m[u] = __ldg(src + i0 + u * kSelThreads);
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const uint32_t k = float_key(m[u]);
        if (kAll || i0 + u * kSelThreads < kHeld) held[i0 + u * kSelThreads] = k;
        atomicAdd(&sh.hist[k >> 21], 1u);
      }
    } else {
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        m[u] = i0 + u * kSelThreads < len ? __ldg(src + i0 + u * kSelThreads) : 0.f;
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const uint32_t i = i0 + u * kSelThreads;
        if (i >= len) break;
        const uint32_t k = float_key(m[u]);
        if (kAll || i < kHeld) held[i] = k;
        atomicAdd(&sh.hist[k >> 21], 1u);
      }
    }
  }
  // four keys from i on (a multiple of 4), and how many of them there are
  auto keys_at = [&](uint32_t i, uint32_t (&k)[4]) {
    if (kAll || i < kHeld) {
      const uint4 v = *reinterpret_cast<const uint4 *>(held + i);
      k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) k[e] = i + e < len ? float_key(__ldg(src + i + e)) : 0u;
    }
    return (int)min(4u, len - i);
  };
  // the digit of the histograms' sum whose bin holds the row that is number
  // `room` from above; keys above the digits fixed so far number `above`
  uint32_t fixed = 0, above = 0;
  auto choose = [&](int shift) {
    sync();
    // thread t holds the four bins 2048 - 4t - 4 .., highest first
    const int b0 = kBins - 4 - 4 * threadIdx.x;
    uint4 sum = make_uint4(0, 0, 0, 0);
    for (int c = 0; c < nc; ++c) {
      const uint32_t *hist = nc == 1 ? sh.hist : cluster.map_shared_rank(sh.hist, c);
      const uint4 v = *reinterpret_cast<const uint4 *>(hist + b0);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    uint32_t at = above + block_scan(sum.x + sum.y + sum.z + sum.w, sh.scan);
    const uint32_t v[4] = {sum.w, sum.z, sum.y, sum.x};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (at < (uint32_t)room && at + v[e] >= (uint32_t)room) {
        sh.digit = b0 + 3 - e;
        sh.above = at;
      }
      at += v[e];
    }
    sync();                       // and no histogram is cleared while it is read
    fixed |= sh.digit << shift;
    above = sh.above;
  };
  choose(21);
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.hist[i] = 0;
  for (uint32_t i = 4 * threadIdx.x; i < len; i += 4 * kSelThreads) {
    uint32_t k[4];
    const int c = keys_at(i, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (e < c && ((k[e] ^ fixed) >> 21) == 0) {
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kList) sh.list[at] = k[e];
      }
    }
  }
  __syncthreads();
  const bool whole = sh.listed > kList;
#pragma unroll 1
  for (int pass = 1; pass < 3; ++pass) {
    const int shift = pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 1 ? 2047u : 1023u;
    const int top = pass == 1 ? 21 : 10;
    if (pass == 2) {
      for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.hist[i] = 0;
      __syncthreads();
    }
    auto count = [&](uint32_t k) {
      if (((k ^ fixed) >> top) == 0) atomicAdd(&sh.hist[(k >> shift) & mask], 1u);
    };
    if (whole) {
      for (uint32_t i = 4 * threadIdx.x; i < len; i += 4 * kSelThreads) {
        uint32_t k[4];
        const int c = keys_at(i, k);
        for (int e = 0; e < c; ++e) count(k[e]);
      }
    } else {
      for (uint32_t i = threadIdx.x; i < sh.listed; i += kSelThreads) count(sh.list[i]);
    }
    choose(shift);
  }
  const uint32_t T = fixed, ties = room - above;
  // each warp has a contiguous part of the slice: rows above T and equal to it
  const uint32_t part = ((len + kSelWarps - 1) / kSelWarps + 3) & ~3u;
  const uint32_t p0 = min(len, warp * part), p1 = min(len, p0 + part);
  uint32_t gt = 0, eq = 0;
  for (uint32_t i = p0 + 4 * lane; i < p1; i += 128) {
    uint32_t k[4];
    const int c = keys_at(i, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += e < c && k[e] > T;
      eq += e < c && k[e] == T;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) sh.warp_gt[warp] = gt, sh.warp_eq[warp] = eq;
  __syncthreads();
  // rows in front of this warp's: those of the warps and the CTAs in front
  uint32_t g0 = 0, q0 = 0;
  for (int w = 0; w < kSelWarps; ++w) {
    if (w == warp) gt = g0, eq = q0;
    g0 += sh.warp_gt[w];
    q0 += sh.warp_eq[w];
  }
  if (nc > 1) {
    if (threadIdx.x == 0) sh.gt = g0, sh.eq = q0;
    cluster.sync();
    for (int c = 0; c < rank; ++c) {
      gt += *cluster.map_shared_rank(&sh.gt, c);
      eq += *cluster.map_shared_rank(&sh.eq, c);
    }
  }
  for (uint32_t i0 = p0; i0 < p1; i0 += 128) {
    const uint32_t i = i0 + 4 * lane;
    uint32_t k[4] = {0, 0, 0, 0}, v = 0;
    int c = 0;
    if (i < p1) c = keys_at(i, k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v += e < c && k[e] > T;
      v += (uint32_t)(e < c && k[e] == T) << 16;
    }
    uint32_t inc = v;             // at most 128 in either half
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
    uint32_t g = gt + ((inc - v) & 0xffffu), q = eq + ((inc - v) >> 16);
    if (v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool up = e < c && k[e] > T, tie = e < c && k[e] == T;
        if (up || (tie && q < ties))
          idx[P.sink + g + min(q, ties)] = (int32_t)(P.sink + lo + i + e);
        g += up;
        q += tie;
      }
    }
    gt += all & 0xffffu;
    eq += all >> 16;
  }
  if (nc > 1) cluster.sync();     // no CTA leaves while its counts are read
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(SelParams P) {
  extern __shared__ __align__(16) uint32_t held[];
  __shared__ __align__(16) SelShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t pair = blockIdx.x / nc;
  const int r = (int)(pair / P.n_heads), h = (int)(pair % P.n_heads);
  int64_t start = P.kv_start[r], n = P.kv_len[r];
  if (n < 0 || start < 0 || start > P.kv_rows || n > P.kv_rows - start) {
    if (threadIdx.x == 0 && rank == 0) raise_err(P.d_err, CSA2_DERR_RANGE_ROW);
    start = n = 0;
  }
  int32_t *idx = P.idx + pair * P.keep;
  const int64_t kept = n < P.keep ? n : P.keep;
  if (P.new_len && h == 0 && rank == 0 && threadIdx.x == 0) P.new_len[r] = kept;
  const int gtid = rank * kSelThreads + threadIdx.x, gn = nc * kSelThreads;
  if (n <= P.keep) {              // every row stays (the whole cluster leaves)
    for (int i = gtid; i < P.keep; i += gn) idx[i] = i < n ? i : -1;
    return;
  }
  for (int i = gtid; i < P.sink; i += gn) idx[i] = i;
  for (int i = gtid; i < P.recent; i += gn)
    idx[P.keep - P.recent + i] = (int32_t)(n - P.recent + i);
  const int room = P.keep - P.sink - P.recent;
  if (room == 0) return;
  const int cand = (int)(n - P.sink - P.recent);       // > room
  const int per = (int)(((int64_t)cand + nc - 1) / nc);
  const int lo = (int)min((int64_t)cand, (int64_t)rank * per);
  const uint32_t len = (uint32_t)min((int64_t)cand, (int64_t)lo + per) - lo;
  const float *src = P.mass + (int64_t)h * P.kv_rows + start + P.sink + lo;
  if (per <= kHeld)               // the same for the whole cluster
    select_slice<true>(P, sh, held, src, idx, lo, len, room, nc, rank);
  else
    select_slice<false>(P, sh, held, src, idx, lo, len, room, nc, rank);
}

// The lengths where new_len is kv_len itself: every CTA of the selection reads
// kv_len[r], and threads that disagreed on it would leave others at a barrier,
// so it changes behind the selection only.
__global__ void evict_lengths_kernel(SelParams P, int64_t *new_len) {
  const int r = blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= P.num_req) return;
  const int64_t start = P.kv_start[r], n = P.kv_len[r];
  const bool bad = n < 0 || start < 0 || start > P.kv_rows || n > P.kv_rows - start;
  new_len[r] = bad ? 0 : n < P.keep ? n : P.keep;
}

// ---------------------------------------------------------------------------
// Moving the rows.  Pure data movement: a group of lanes copies one element
// (row, head); a block takes the rows of one (request, head, buffer) in
// ascending batches, loads a whole batch before it stores it, and has a
// barrier between, so that closing up in place is safe: idx ascends, hence
// row i's source is never in front of i, and a later batch's sources lie
// behind every row stored so far.  Where no buffer shares memory with itself,
// several blocks share the rows.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMaxBufs = 8;
constexpr int kUnroll = 8;
constexpr int64_t kMostRows = 1ll << 62;  // no buffer has more; leaves room for a row's offset

struct MoveParams {
  csa2_evict_buf buf[kMaxBufs];
  int vec[kMaxBufs];              // bytes of a lane's piece: 16 or 4
  int shift[kMaxBufs];            // log2 of the pieces of an element, or -1
  int num_req, n_heads, keep;
  const int32_t *idx;
  const int64_t *new_len, *src_start, *dst_start;
  int32_t *d_err;
};

template <typename V, bool kInPlace>
__device__ void move_rows(const MoveParams &P, const csa2_evict_buf &b, int shift, int64_t pair,
                          int64_t s0, int64_t d0, int n, int64_t h, int part, int parts,
                          int &err) {
  const int32_t *idx = P.idx + pair * P.keep;
  const int64_t pieces = b.elem_bytes / (int64_t)sizeof(V);
  const uint8_t *src = static_cast<const uint8_t *>(b.src) + h * b.src_head_stride;
  uint8_t *dst = static_cast<uint8_t *>(b.dst) + h * b.dst_head_stride;
  const int64_t total = n * pieces, batch = (int64_t)kMoveThreads * kUnroll;
  for (int64_t w0 = part * batch; w0 < total; w0 += parts * batch) {
    V v[kUnroll];
    int j[kUnroll];
    int64_t to[kUnroll], p[kUnroll];
    // the rows, then their bytes: each step's loads are all in flight together
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t w = w0 + u * kMoveThreads + threadIdx.x;
      const int64_t i = shift >= 0 ? w >> shift : w / pieces;
      p[u] = (w - i * pieces) * (int64_t)sizeof(V);
      to[u] = d0 + i;
      j[u] = w < total ? __ldg(idx + i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (j[u] >= 0 && (s0 + j[u] >= b.src_rows || to[u] >= b.dst_rows)) {
        err |= CSA2_DERR_RANGE_ROW;
        j[u] = -1;
      }
      to[u] = to[u] * b.dst_row_stride + p[u];
      if (j[u] >= 0)
        v[u] = *reinterpret_cast<const V *>(src + (s0 + j[u]) * b.src_row_stride + p[u]);
    }
    if (kInPlace) __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (j[u] >= 0) *reinterpret_cast<V *>(dst + to[u]) = v[u];
  }
}

// Whether the destination [d0, d0 + n) of request r in a tensor that is its own
// source meets rows between another request's start and last source row, which
// another block may not have read yet, or lies further up over its own (further
// down is safe: the block goes upwards).
__device__ __noinline__ bool meets_sources(const MoveParams &P, const csa2_evict_buf &b, int r, int h, int64_t s0,
                              int64_t d0, int n) {
  bool hit = false;
  for (int q = threadIdx.x; q < P.num_req; q += kMoveThreads) {
    const int64_t len = P.new_len[q], a = min(P.src_start[q], b.src_rows);
    const int m = (int)(len < 0 ? 0 : len < P.keep ? len : P.keep);
    if (m == 0 || a < 0) continue;
    const int64_t behind = a + P.idx[((int64_t)q * P.n_heads + h) * P.keep + m - 1] + 1;
    hit |= d0 < behind && a < d0 + n && (q != r || d0 > s0);
  }
  return __syncthreads_or(hit);
}

template <bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads)
evict_rows_kernel(const __grid_constant__ MoveParams P) {
  const int64_t pair = blockIdx.x;
  const int r = (int)(pair / P.n_heads);
  const csa2_evict_buf &b = P.buf[blockIdx.y];
  // a start behind the buffer counts as its end: near 2^63, start + row would wrap
  // (checked here, since checks of each row against what is left of the buffer cost
  // registers, and with them a CTA to an SM: 46 us instead of 38 for eight prompts
  // of 5,200 rows on average, selection included)
  const int64_t len = P.new_len[r], s0 = min(P.src_start[r], b.src_rows),
                d0 = min(P.dst_start[r], b.dst_rows);
  const int n = (int)(len < 0 ? 0 : len < P.keep ? len : P.keep);
  const int shift = P.shift[blockIdx.y];
  int err = 0;
  if (s0 < 0 || d0 < 0) {
    err = n > 0 ? CSA2_DERR_RANGE_ROW : 0;
  } else if (kInPlace && s0 != d0 && n > 0 && b.src == b.dst &&
             meets_sources(P, b, r, (int)(pair % P.n_heads), s0, d0, n)) {
    err = CSA2_DERR_RANGE_ROW;
  } else if (P.vec[blockIdx.y] == 16) {
    move_rows<uint4, kInPlace>(P, b, shift, pair, s0, d0, n, pair % P.n_heads, blockIdx.z,
                               gridDim.z, err);
  } else {
    move_rows<uint32_t, kInPlace>(P, b, shift, pair, s0, d0, n, pair % P.n_heads, blockIdx.z,
                                  gridDim.z, err);
  }
  if (err) raise_err(P.d_err, err);
}

// Bytes from a buffer's first to behind its last (cut off at 2^62).
uint64_t span(int64_t rows, int64_t row_stride, int64_t heads, int64_t head_stride, int64_t elem) {
  if (rows == 0 || elem == 0) return 0;
  const double most = (double)(rows - 1) * row_stride + (double)(heads - 1) * head_stride + elem;
  return most < 4e18 ? (rows - 1) * row_stride + (heads - 1) * head_stride + elem : 1ull << 62;
}

// Whether a buffer's source and destination may share a byte: their runs of memory
// meet, and they are not columns side by side of the same longer rows.
bool shares_memory(const csa2_evict_buf &b, int64_t heads) {
  const uint64_t one_s = span(1, 0, heads, b.src_head_stride, b.elem_bytes);
  const uint64_t one_d = span(1, 0, heads, b.dst_head_stride, b.elem_bytes);
  const uint64_t step = (uint64_t)b.src_row_stride;
  if (b.src_row_stride == b.dst_row_stride && one_s <= step && one_d <= step && step > 0) {
    const uint64_t s = (uint64_t)(uintptr_t)b.src, d = (uint64_t)(uintptr_t)b.dst;
    const uint64_t off = d >= s ? (d - s) % step : (step - (s - d) % step) % step;
    if (off >= one_s && step - off >= one_d) return false;
  }
  return overlap(
      b.src, span(b.src_rows, b.src_row_stride, heads, b.src_head_stride, b.elem_bytes), b.dst,
      span(b.dst_rows, b.dst_row_stride, heads, b.dst_head_stride, b.elem_bytes));
}

}  // namespace
}  // namespace csa2

extern "C" CSA2_API int csa2_evict_select(int32_t num_req, int32_t n_heads,
                                          const int64_t *kv_start, const int64_t *kv_len,
                                          const float *mass, int64_t kv_rows, int32_t keep,
                                          int32_t sink, int32_t recent, int32_t *idx,
                                          int64_t *new_len, int32_t *d_err,
                                          csa2_stream_t stream) {
  using namespace csa2;
  if (num_req < 0 || n_heads < 1 || kv_rows < 0 || keep < 1 || sink < 0 || recent < 0 ||
      (int64_t)sink + recent > keep)
    return CSA2_ERR_INVALID_ARG;
  if (num_req == 0) return CSA2_OK;
  if (!kv_start || !kv_len || !idx || !new_len || (kv_rows > 0 && !mass))
    return CSA2_ERR_INVALID_ARG;
  if (kv_rows > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  if (!aligned(4, mass, idx, d_err) || !aligned(8, kv_start, kv_len, new_len))
    return CSA2_ERR_UNSUPPORTED;
  const int64_t pairs = (int64_t)num_req * n_heads;
  if (pairs > 0x7fffffffll / 8) return CSA2_ERR_UNSUPPORTED;
  const uint64_t lens = (uint64_t)num_req * 8, ids = (uint64_t)pairs * keep * 4;
  // (cut off at 2^60 cells, which no memory has, so that 64 bits hold the bytes)
  const uint64_t cells = (uint64_t)n_heads * kv_rows;
  const uint64_t weights = (cells < 1ull << 60 ? cells : 1ull << 60) * 4;
  const bool shorten = new_len == kv_len;
  if (overlap(idx, ids, kv_start, lens) || overlap(idx, ids, kv_len, lens) ||
      overlap(idx, ids, mass, weights) || overlap(idx, ids, new_len, lens) ||
      overlap(new_len, lens, kv_start, lens) || overlap(new_len, lens, mass, weights) ||
      (!shorten && overlap(new_len, lens, kv_len, lens)))
    return CSA2_ERR_INVALID_ARG;
  // CTAs to a (request, head): as many as the GPU holds at a time, but no fewer
  // than kMinSlice rows to each on average (8 x 8 rows of 5200: 10.9 us at
  // 4096 a slice, 11.9 at 2048, 16.8 at 1024; 24 x 8 rows of 26,000: 37.6 us
  // with two CTAs, 43 with three, 56 with one).  The lengths are on the device, so
  // this goes by the pool's rows to a request: in a pool far longer than its
  // requests the slices come out shorter than that.
  const int64_t by_rows = kv_rows / num_req / kMinSlice;
  int64_t nc = kSelPlaces / pairs;
  nc = nc < by_rows ? nc : by_rows;
  nc = nc < 1 ? 1 : nc > 8 ? 8 : nc;
  SelParams P{num_req, n_heads, kv_start, kv_len, mass, kv_rows, keep,
              sink,    recent,  idx,      shorten ? nullptr : new_len, d_err};
  constexpr int kSmem = kHeld * 4;
  allow_smem<evict_select_kernel>(kSmem);
  const auto done = [&]() {
    const unsigned blocks = (unsigned)(((int64_t)num_req + 255) / 256);
    if (shorten) evict_lengths_kernel<<<blocks, 256, 0, as_stream(stream)>>>(P, new_len);
    return launch_status();
  };
  if (nc == 1) {                  // a plain launch costs the host less
    evict_select_kernel<<<(unsigned)pairs, kSelThreads, kSmem, as_stream(stream)>>>(P);
    return done();
  }
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)nc, 1, 1};
  cfg.gridDim = dim3((unsigned)(pairs * nc));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = as_stream(stream);
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, evict_select_kernel, P) != cudaSuccess) {
    (void)cudaGetLastError();
    return CSA2_ERR_CUDA;
  }
  return done();
}

extern "C" CSA2_API int csa2_evict_rows(int32_t num_req, int32_t n_heads, const int32_t *idx,
                                        int32_t keep, const int64_t *new_len,
                                        const int64_t *src_start, const int64_t *dst_start,
                                        int32_t n_bufs, const csa2_evict_buf *bufs,
                                        int32_t *d_err, csa2_stream_t stream) {
  using namespace csa2;
  if (num_req < 0 || n_heads < 1 || keep < 1 || n_bufs < 0) return CSA2_ERR_INVALID_ARG;
  if (num_req == 0 || n_bufs == 0) return CSA2_OK;
  if (!idx || !new_len || !src_start || !dst_start || !bufs) return CSA2_ERR_INVALID_ARG;
  if (n_bufs > kMaxBufs) return CSA2_ERR_UNSUPPORTED;
  if (!aligned(4, idx, d_err) || !aligned(8, new_len, src_start, dst_start))
    return CSA2_ERR_UNSUPPORTED;
  MoveParams P{};
  bool in_place = false;
  int64_t most = 0;
  for (int i = 0; i < n_bufs; ++i) {
    const csa2_evict_buf &b = bufs[i];
    if (b.src_rows < 0 || b.dst_rows < 0 || b.elem_bytes < 0 || b.src_row_stride < 0 ||
        b.src_head_stride < 0 || b.dst_row_stride < 0 || b.dst_head_stride < 0)
      return CSA2_ERR_INVALID_ARG;
    if (b.elem_bytes > 0 && b.src_rows > 0 && b.dst_rows > 0 && (!b.src || !b.dst))
      return CSA2_ERR_INVALID_ARG;
    const uint64_t bits = (uint64_t)(uintptr_t)b.src | (uint64_t)(uintptr_t)b.dst |
                          (uint64_t)b.src_row_stride | (uint64_t)b.src_head_stride |
                          (uint64_t)b.dst_row_stride | (uint64_t)b.dst_head_stride |
                          (uint64_t)b.elem_bytes;
    if (bits & 3u) return CSA2_ERR_UNSUPPORTED;
    if (b.elem_bytes > (1 << 24)) return CSA2_ERR_UNSUPPORTED;
    P.buf[i] = b;
    P.buf[i].src_rows = b.src_rows < kMostRows ? b.src_rows : kMostRows;
    P.buf[i].dst_rows = b.dst_rows < kMostRows ? b.dst_rows : kMostRows;
    P.vec[i] = (bits & 15u) ? 4 : 16;
    // sharing memory, the rows are moved in order, whichever views name them
    in_place |= shares_memory(b, n_heads);
    for (int j = 0; j < i; ++j)
      if (b.elem_bytes > 0 && bufs[j].elem_bytes > 0 && bufs[j].dst == b.dst && b.dst)
        return CSA2_ERR_INVALID_ARG;
    const int64_t pieces = b.elem_bytes / P.vec[i];
    if (pieces > most) most = pieces;
    P.shift[i] = -1;
    for (int s = 0; s < 24; ++s)
      if (pieces == (1ll << s)) P.shift[i] = s;
  }
  P.num_req = num_req;
  P.n_heads = n_heads;
  P.keep = keep;
  P.idx = idx;
  P.new_len = new_len;
  P.src_start = src_start;
  P.dst_start = dst_start;
  P.d_err = d_err;
  const int64_t pairs = (int64_t)num_req * n_heads;
  if (pairs > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  int64_t parts = 1;
  if (!in_place) {
    const int64_t batches =
        (most * keep + kMoveThreads * kUnroll - 1) / (kMoveThreads * kUnroll);
    parts = (152 * 8 * 8 + pairs * n_bufs - 1) / (pairs * n_bufs);
    if (parts > batches) parts = batches;
    if (parts < 1) parts = 1;
  }
  const dim3 grid((unsigned)pairs, (unsigned)n_bufs, (unsigned)parts);
  if (in_place)
    evict_rows_kernel<true><<<grid, kMoveThreads, 0, as_stream(stream)>>>(P);
  else
    evict_rows_kernel<false><<<grid, kMoveThreads, 0, as_stream(stream)>>>(P);
  return launch_status();
}
