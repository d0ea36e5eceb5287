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
// again from L2).  Three histogram passes of 11, 11 and 10 bits, added up over
// the cluster through distributed shared memory, give the key T of the last
// row kept; rows above T stay, and of those equal to T the first in row order.
// The masses are read from memory once; the passes and the ordered write run
// on shared memory.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kHeld = 20480;          // keys of a slice in shared memory (80 KB)
constexpr int kBins = 2048;

struct SelParams {
  int num_req, n_heads;
  const int64_t *kv_start, *kv_len;
  const float *mass;
  int64_t kv_rows;
  int keep, sink, recent;
  int32_t *idx;
  int64_t *new_len;
  int32_t *d_err;
};

struct SelShared {
  uint32_t hist[kBins];
  uint32_t scan[kSelThreads / 32];
  uint32_t digit, above;          // the pass's answer
  uint32_t gt, eq;                // this CTA's rows above T, and equal to it
};

// exclusive prefix sum over the block in thread order; `total` gets the sum
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *tmp, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();               // tmp may still be read from the last call
  if (lane == 31) tmp[warp] = inc;
  __syncthreads();
  uint32_t base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const uint32_t t = tmp[w];
    if (w < warp) base += t;
    all += t;
  }
  total = all;
  return base + inc - v;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(SelParams P) {
  extern __shared__ uint32_t held[];
  __shared__ SelShared sh;
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
  if (h == 0 && rank == 0 && threadIdx.x == 0) P.new_len[r] = kept;
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
  const int per = (cand + nc - 1) / nc;
  const int lo = min(cand, rank * per), len = min(cand, lo + per) - lo;
  const float *src = P.mass + (int64_t)h * P.kv_rows + start + P.sink + lo;
  auto key_at = [&](int i) { return i < kHeld ? held[i] : float_key(__ldg(src + i)); };
  for (int i = threadIdx.x; i < len && i < kHeld; i += kSelThreads)
    held[i] = float_key(__ldg(src + i));
  // T, digit by digit: keys above the digits fixed so far are counted in `above`
  uint32_t fixed = 0, above = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    const uint32_t high = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
    for (int i = threadIdx.x; i < kBins; i += kSelThreads) sh.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < len; i += kSelThreads) {
      const uint32_t k = key_at(i);
      if ((k & high) == fixed) atomicAdd(&sh.hist[(k >> shift) & mask], 1u);
    }
    cluster.sync();
    // thread t holds bins 4 t' .. 4 t' + 3 of the cluster's sum, highest first
    const int b0 = kBins - 4 - 4 * threadIdx.x;
    uint4 sum = make_uint4(0, 0, 0, 0);
    for (int c = 0; c < nc; ++c) {
      const uint4 v = *reinterpret_cast<const uint4 *>(cluster.map_shared_rank(sh.hist, c) + b0);
      sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
    }
    uint32_t total;
    uint32_t at = above + block_scan(sum.x + sum.y + sum.z + sum.w, sh.scan, total);
    const uint32_t v[4] = {sum.w, sum.z, sum.y, sum.x};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (at < (uint32_t)room && at + v[e] >= (uint32_t)room) {
        sh.digit = b0 + 3 - e;
        sh.above = at;
      }
      at += v[e];
    }
    cluster.sync();               // and no histogram is cleared while it is read
    fixed |= sh.digit << shift;
    above = sh.above;
  }
  const uint32_t T = fixed, ties = room - above;
  // rows above T and equal to it in the slices in front of this one
  uint32_t gt = 0, eq = 0;
  for (int i = threadIdx.x; i < len; i += kSelThreads) {
    const uint32_t k = key_at(i);
    gt += k > T;
    eq += k == T;
  }
  {
    uint32_t tg, te;
    block_scan(gt, sh.scan, tg);
    block_scan(eq, sh.scan, te);
    if (threadIdx.x == 0) sh.gt = tg, sh.eq = te;
  }
  cluster.sync();
  uint32_t gt0 = 0, eq0 = 0;
  for (int c = 0; c < rank; ++c) {
    gt0 += *cluster.map_shared_rank(&sh.gt, c);
    eq0 += *cluster.map_shared_rank(&sh.eq, c);
  }
  // in row order, 4 rows to a thread
  for (int i0 = 0; i0 < len; i0 += 4 * kSelThreads) {
    uint32_t k[4], g4 = 0, e4 = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 4 * threadIdx.x + e;
      k[e] = i < len ? key_at(i) : 0u;
      g4 += i < len && k[e] > T;
      e4 += i < len && k[e] == T;
    }
    uint32_t tot;
    const uint32_t before = block_scan(g4 | (e4 << 16), sh.scan, tot);   // at most 2048 each
    uint32_t g = gt0 + (before & 0xffffu), q = eq0 + (before >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = i0 + 4 * threadIdx.x + e;
      if (i >= len) break;
      const bool is_eq = k[e] == T;
      if (k[e] > T || (is_eq && q < ties))
        idx[P.sink + g + min(q, ties)] = P.sink + lo + i;
      g += k[e] > T;
      q += is_eq;
    }
    gt0 += tot & 0xffffu;
    eq0 += tot >> 16;
  }
  cluster.sync();                 // no CTA leaves while its counts are read
}

// ---------------------------------------------------------------------------
// Moving the rows.  Pure data movement: a group of lanes copies one element
// (row, head); a block takes the rows of one (request, head, buffer) in
// ascending batches, loads a whole batch before it stores it, and has a
// barrier between, so that closing up in place is safe: idx ascends, hence
// row i's source is never in front of i, and a later batch's sources lie
// behind every row stored so far.  Where nothing moves in place, several
// blocks share the rows.
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMaxBufs = 8;
constexpr int kUnroll = 8;

struct MoveParams {
  csa2_evict_buf buf[kMaxBufs];
  int vec[kMaxBufs];              // bytes of a lane's piece: 16 or 4
  int n_heads, keep;
  const int32_t *idx;
  const int64_t *new_len, *src_start, *dst_start;
  int32_t *d_err;
};

template <typename V>
__device__ void move_rows(const MoveParams &P, const csa2_evict_buf &b, int64_t pair, int64_t s0,
                          int64_t d0, int n, int64_t h, int part, int parts, int &err) {
  const int32_t *idx = P.idx + pair * P.keep;
  const int pieces = (int)(b.elem_bytes / sizeof(V));
  const uint8_t *src = static_cast<const uint8_t *>(b.src) + h * b.src_head_stride;
  uint8_t *dst = static_cast<uint8_t *>(b.dst) + h * b.dst_head_stride;
  const int64_t total = (int64_t)n * pieces, batch = (int64_t)kMoveThreads * kUnroll;
  for (int64_t w0 = part * batch; w0 < total; w0 += parts * batch) {
    V v[kUnroll];
    int64_t to[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t w = w0 + u * kMoveThreads + threadIdx.x;
      to[u] = -1;
      if (w >= total) continue;
      const int64_t i = w / pieces, p = w - i * pieces;
      const int64_t j = idx[i];
      if (j < 0) continue;
      if (s0 + j >= b.src_rows || d0 + i >= b.dst_rows) {
        err |= CSA2_DERR_RANGE_ROW;
        continue;
      }
      v[u] = *reinterpret_cast<const V *>(src + (s0 + j) * b.src_row_stride + p * sizeof(V));
      to[u] = (d0 + i) * b.dst_row_stride + p * sizeof(V);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (to[u] >= 0) *reinterpret_cast<V *>(dst + to[u]) = v[u];
  }
}

__global__ void __launch_bounds__(kMoveThreads)
evict_rows_kernel(MoveParams P) {
  const int64_t pair = blockIdx.x;
  const int r = (int)(pair / P.n_heads);
  const csa2_evict_buf &b = P.buf[blockIdx.y];
  const int64_t len = P.new_len[r], s0 = P.src_start[r], d0 = P.dst_start[r];
  const int n = (int)(len < 0 ? 0 : len < P.keep ? len : P.keep);
  int err = 0;
  if (s0 < 0 || d0 < 0) {
    err = n > 0 ? CSA2_DERR_RANGE_ROW : 0;
  } else if (P.vec[blockIdx.y] == 16) {
    move_rows<uint4>(P, b, pair, s0, d0, n, pair % P.n_heads, blockIdx.z, gridDim.z, err);
  } else {
    move_rows<uint32_t>(P, b, pair, s0, d0, n, pair % P.n_heads, blockIdx.z, gridDim.z, err);
  }
  if (err) raise_err(P.d_err, err);
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
  if ((uintptr_t)mass & 3u) return CSA2_ERR_UNSUPPORTED;
  const int64_t pairs = (int64_t)num_req * n_heads;
  if (pairs > 0x7fffffffll / 8) return CSA2_ERR_UNSUPPORTED;
  // as many CTAs to a row as keep the GPU's places filled
  int nc = 1;
  while (nc < 8 && pairs * nc * 2 <= 2 * 152) nc *= 2;
  SelParams P{num_req, n_heads, kv_start, kv_len, mass, kv_rows, keep,
              sink,    recent,  idx,      new_len, d_err};
  constexpr int kSmem = kHeld * 4;
  allow_smem<evict_select_kernel>(kSmem);
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
  return launch_status();
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
    P.vec[i] = (bits & 15u) ? 4 : 16;
    in_place |= b.src == b.dst;
    const int64_t pieces = b.elem_bytes / P.vec[i];
    if (pieces > most) most = pieces;
  }
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
    parts = (152 * 8 * 4 + pairs * n_bufs - 1) / (pairs * n_bufs);
    if (parts > batches) parts = batches;
    if (parts < 1) parts = 1;
  }
  evict_rows_kernel<<<dim3((unsigned)pairs, (unsigned)n_bufs, (unsigned)parts), kMoveThreads, 0,
                      as_stream(stream)>>>(P);
  return launch_status();
}
