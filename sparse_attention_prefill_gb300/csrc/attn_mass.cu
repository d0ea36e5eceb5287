// Attention weight that queries put on cached rows, added up per row and key
// head (csa2_attn_mass):
//   mass[g, j] (+)= sum_{i sees j, h in group g} exp(c <q[i,h], k[j,g]> - lse[i,h])
//
// Keys are stationary: a work item is up to `span` tiles of 128 keys of one
// request and key head.  Each K tile is an A operand, the packed query tiles
// (dense.cuh) that see it pass as B operands, so S^T[key, query row] has a key
// to a TMEM lane and the sum over queries stays in one thread's register: no
// atomics, a fixed order.  The exponent needs no maximum (lse is given):
// exp2(c' s - lse'), one fused multiply-add and one exponential to a score,
// with -lse' read from shared memory (one value per column, the same for all
// lanes).
//
// Per item the kernel reads its K tiles once and every query tile once (from
// L2, where a request's queries stay).  A decode step is bound by the K rows
// (61 requests of 3,500 rows on average: 72.8 us, 6.2 TB/s).  A window of
// queries takes some 1,200 cycles to a 128 x 128 tile (eight requests of 128
// queries over 2,700 rows on average, 64 heads: 54.8 us), of which the product
// and the exponentials need 512 each on units of their own; no unit is more than
// half busy.  (-lse' as three bf16 channels of the product, instead of reads of
// shared memory, took 56 us; TMEM loads 16 columns ahead of their use 57.6.)  The
// rest is waiting: a warpgroup gives its buffer back once a tile's arithmetic is
// done, and only then can the next product into it be issued, behind those of the
// other three.
// Products and weights rotate over four S^T buffers and four warpgroups:
// product number x of an item (query tile by query tile, the item's key tiles
// within) goes to buffer and warpgroup x % 4.  With four key tiles to an item
// a warpgroup has a key tile to itself; with two or one (few items) 2 or 4
// warpgroups share one and add up at its end.  Different warpgroups are at
// different places of their tiles, which keeps the exponential units busy:
// with all four on quarters of one tile they idled during its barrier and TMEM
// load (63 us for the same window; two warpgroups of twice the registers took
// 75).
//
// Roles (24 warps, one CTA per SM, persistent over items):
//   0-15       weights: warp w reads TMEM sub-partition w % 4 (keys 32(w % 4)
//              .. + 31 of a tile) of buffer w / 4
//   16, 17     issue the products in turn (16: TMEM)
//   18         K and Q tiles by TMA
//   19         looks items up, 32 at a time, and publishes them a few ahead
//   20-23      -lse of the query tiles, a warp to a buffer, so that four tiles'
//              loads are under way
// Every wait is bounded, as in the attention.
#include "dense.cuh"

namespace csa2 {
namespace dense {
namespace {

constexpr int kMaxReq = 8192;
constexpr int kBufs = 4;            // S^T buffers (128 TMEM columns each)
constexpr int kItems = 8;           // items published ahead
constexpr int kMaxK = 6, kMaxQ = 4; // ring stages at most
constexpr int kEpiWarps = 4 * kBufs;    // a warpgroup to a buffer
constexpr int kLseWarps = kBufs;    // a warp to a buffer
constexpr int kIssueWarps = 2;
constexpr int kMassThreads = (kEpiWarps + kIssueWarps + 2 + kLseWarps) * 32;

struct MassParams {
  Seqs seqs;
  int n_heads, n_kv, group, tpt, ncol;   // ncol: tpt * group, rounded up to 32
  int span;                              // key tiles of an item: 1, 2 or 4
  int kst, qst;                          // ring stages
  uint32_t q_stage, off_q, off_cum, off_misc;
  float scale_log2;
  const float *lse;
  const float *mass_in;
  float *mass_out;
  int32_t *d_err;
  uint64_t wait_ns;
};

struct MassItem {
  int q0, n;          // the request's query rows
  int h, keys;        // key head; keys of the item (-1: no more items)
  int qt0, nq;        // first query tile that sees it, and how many
  int64_t row;        // first pool row
  int64_t shift;      // query i sees the item's key x if x <= shift + i
};

struct MassMisc {
  uint64_t k_full[kMaxK], k_empty[kMaxK], q_full[kMaxQ], q_empty[kMaxQ];
  uint64_t s_full[kBufs], s_empty[kBufs], l_full[kBufs];
  uint64_t item_full[kItems], item_empty[kItems], grp, done[kIssueWarps];
  Bound bd;
  uint32_t tmem;
  MassItem item[kItems];
  alignas(16) float nl[kBufs][kTile];    // -lse in log2 units, by query row
  float red[2][kBufs][kTile];            // partial sums by item parity and warpgroup
};

__device__ void schedule_role(const MassParams &P, uint8_t *smem, MassMisc *ms) {
  const int lane = threadIdx.x & 31;
  uint32_t *cum = reinterpret_cast<uint32_t *>(smem + P.off_cum);
  int err = 0;
  uint32_t base = 0;
  for (int i0 = 0; i0 < P.seqs.count; i0 += 32) {
    uint32_t nt = 0;
    if (i0 + lane < P.seqs.count) {
      int64_t start, m;
      seq_keys(P.seqs, i0 + lane, start, m, err);
      nt = (uint32_t)((m + P.span * kTile - 1) / (P.span * kTile));
    }
    uint32_t inc = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (i0 + lane < P.seqs.count) cum[i0 + lane] = base + inc;    // tiles up to this request
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  __syncwarp();
  const int64_t total = (int64_t)base * P.n_kv;
  // a lane to an item: 32 are looked up together, so that their loads overlap
  uint32_t u = 0;
  bool more = true;
  for (int64_t id0 = blockIdx.x; more; id0 += 32 * (int64_t)gridDim.x) {
    const int64_t id = id0 + lane * (int64_t)gridDim.x;
    MassItem it{};
    it.keys = -1;
    if (id < total) {
      const uint32_t tile = (uint32_t)(id / P.n_kv);
      it.h = (int)(id % P.n_kv);
      int lo = 0, hi = P.seqs.count - 1;       // first request with cum > tile
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cum[mid] > tile) hi = mid; else lo = mid + 1;
      }
      // (below 0 only where requests that share rows made the sum wrap)
      const int64_t kt = (int64_t)tile - (lo ? cum[lo - 1] : 0u);
      int64_t start, m;
      seq_rows(P.seqs, lo, it.q0, it.n, err);
      seq_keys(P.seqs, lo, start, m, err);
      const int64_t k0 = kt * P.span * kTile, left = m - k0;
      it.keys = kt < 0 || left < 0 ? 0 : left < P.span * kTile ? (int)left : P.span * kTile;
      it.row = start + k0;
      it.shift = m - it.n - k0;
      const int64_t first = it.shift >= 0 ? 0 : -it.shift;      // first query that sees key 0
      const int tiles = (it.n + P.tpt - 1) / P.tpt;
      it.qt0 = first < it.n ? (int)(first / P.tpt) : tiles;
      it.nq = it.keys > 0 ? tiles - it.qt0 : 0;
    }
    for (int l = 0; l < 32 && more; ++l, ++u) {
      const uint32_t s = u % kItems;
      if (!wait_all(&ms->item_empty[s], ((u / kItems) & 1) ^ 1, &ms->bd)) {
        more = false;
        break;
      }
      if (lane == l) {
        ms->item[s] = it;
        mbar_arrive(&ms->item_full[s]);
      }
      __syncwarp();
      more = __shfl_sync(0xffffffffu, it.keys, l) >= 0;
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane == 0) raise_err(P.d_err, err);
}

// The items of this CTA, one after another, as every role sees them; called by a
// whole warp (kWarp) or by a single thread.
template <bool kWarp, typename F>
__device__ __forceinline__ bool for_items(MassMisc *ms, F f) {
  for (uint32_t u = 0;; ++u) {
    const uint32_t s = u % kItems;
    bool ok = wait_bar(&ms->item_full[s], (u / kItems) & 1, &ms->bd);
    if (kWarp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    MassItem it = ms->item[s];
    if (kWarp) {
      // known to be the same in every lane, or the loop counts as divergent
      it.keys = uniform(it.keys);
      it.nq = uniform(it.nq);
      __syncwarp();
    }
    if (!kWarp || (threadIdx.x & 31) == 0) mbar_arrive(&ms->item_empty[s]);
    if (it.keys < 0) return true;
    if (!f(it)) return false;
  }
}

template <int D>
__device__ void load_role(const MassParams &P, uint8_t *smem, MassMisc *ms,
                          const CUtensorMap *mq, const CUtensorMap *mk) {
  constexpr uint32_t kKStage = (D / 64) * kBlk;
  const uint32_t box = (uint32_t)P.tpt * P.group * 128u * (D / 64);
  uint32_t gk = 0, gq = 0;
  for_items<false>(ms, [&](const MassItem &it) {
    if (it.nq == 0) return true;
    for (int k = 0; k < it.keys; k += kTile, ++gk) {
      const uint32_t sk = gk % P.kst;
      if (!wait_bar(&ms->k_empty[sk], ((gk / P.kst) & 1) ^ 1, &ms->bd)) return false;
      mbar_arrive_expect_tx(&ms->k_full[sk], kKStage);
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(smem + sk * kKStage + c * kBlk, mk, c * 64, it.h, (int)it.row + k,
                    &ms->k_full[sk]);
    }
    for (int t = 0; t < it.nq; ++t, ++gq) {
      const uint32_t sq = gq % P.qst;
      if (!wait_bar(&ms->q_empty[sq], ((gq / P.qst) & 1) ^ 1, &ms->bd)) return false;
      mbar_arrive_expect_tx(&ms->q_full[sq], box);
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(smem + P.off_q + sq * P.q_stage + c * (P.ncol * 128), mq, c * 64,
                    it.h * P.group, it.q0 + (it.qt0 + t) * P.tpt, &ms->q_full[sq]);
    }
    return true;
  });
  // every copy lands before the CTA leaves
  for (uint32_t i = gk > (uint32_t)P.kst ? gk - P.kst : 0; i < gk; ++i)
    drain_bar(&ms->k_full[i % P.kst], (i / P.kst) & 1);
  for (uint32_t i = gq > (uint32_t)P.qst ? gq - P.qst : 0; i < gq; ++i)
    drain_bar(&ms->q_full[i % P.qst], (i / P.qst) & 1);
}

// Two warps issue the products in turn (product x by warp x % 2): what one spends
// between its products, on barriers and commits, the other's cover.  One warp
// alone kept the tensor pipe idle for half of every 1100 cycles.
template <typename T, int D>
__device__ void product_role(const MassParams &P, uint8_t *smem, MassMisc *ms, int which) {
  constexpr uint32_t kKStage = (D / 64) * kBlk;
  const uint32_t idesc = idesc_of<T>(kTile, P.ncol, false);
  const uint32_t tmem = uniform(ms->tmem), qblk = P.ncol * 128;
  const uint64_t kd = make_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t qd = make_desc_sw128(smem_u32(smem + P.off_q), 16, 1024);
  uint32_t sk = 0, pk = 0, sq = 0, pq = 0;     // ring stages and phases
  uint32_t uses = 0;                           // parity of each S^T buffer's uses
  bool ok = true;
  for (uint32_t u = 0; ok; ++u) {
    const uint32_t si = u % kItems;
    if (!(ok = wait_all(&ms->item_full[si], (u / kItems) & 1, &ms->bd))) break;
    const int keys = uniform(ms->item[si].keys), nq = uniform(ms->item[si].nq);
    if (elect_one()) mbar_arrive(&ms->item_empty[si]);
    __syncwarp();
    if (keys < 0) break;
    const int nk = (keys + kTile - 1) / kTile;
    uint32_t ks = sk, kp = pk;                 // the item's K tiles
    for (int t = 0; t < nq && ok; ++t) {
      // once a wait has run out nothing waits any more
      ok = uniform(*(volatile int *)&ms->bd.abort) == 0;
      ks = sk, kp = pk;
      const uint64_t b = desc_add(qd, sq * P.q_stage);
      for (int i = 0; i < nk; ++i) {
        const int x = t * P.span + i;
        const uint32_t sb = x % kBufs;
        const uint64_t a = desc_add(kd, ks * kKStage);
        // The waits by the elected lane itself, between its products.  Both
        // warps wait for every tile, with a product of theirs on it or not:
        // they let it go together, and neither may do so a round early.
        if (elect_one()) {
          if (i == 0) wait_inline(&ms->q_full[sq], pq, &ms->bd);
          if (t == 0) wait_inline(&ms->k_full[ks], kp, &ms->bd);
          if ((x & 1) == which) {
            wait_inline(&ms->s_empty[sb], ((uses >> sb) & 1) ^ 1, &ms->bd);
            fence_after_sync();
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              mma_f16(tmem + sb * kTile, desc_add(a, (k >> 2) * kBlk + (k & 3) * 32),
                      desc_add(b, (k >> 2) * qblk + (k & 3) * 32), idesc, k > 0);
            mma_commit(&ms->s_full[sb]);
          }
          if (t == nq - 1) mma_commit(&ms->k_empty[ks]);
          if (i == nk - 1) mma_commit(&ms->q_empty[sq]);
        }
        __syncwarp();
        uses ^= 1u << sb;
        if (++ks == (uint32_t)P.kst) ks = 0, kp ^= 1;
      }
      if (++sq == (uint32_t)P.qst) sq = 0, pq ^= 1;
    }
    sk = ks, pk = kp;
  }
  if (elect_one()) mma_commit(&ms->done[which]);
  __syncwarp();
  drain_bar(&ms->done[which], 0);
}

// The query tiles of an item that buffer (and warpgroup) `which` gets, t0, t0 +
// step, .. below t1, and the key tile they meet there: product t * span + i
// goes to buffer (t * span + i) % 4.
struct Turns {
  int tile, t0, t1, step;
  __device__ __forceinline__ Turns(const MassParams &P, const MassItem &it, int which) {
    tile = which & (P.span - 1);
    step = kBufs / P.span;
    t0 = which / P.span;
    t1 = tile * kTile < it.keys ? it.nq : 0;
  }
};

// -lse of the query tiles of one S^T buffer
__device__ void lse_role(const MassParams &P, MassMisc *ms, uint32_t which) {
  const int lane = threadIdx.x & 31;
  int tok[4], off[4];              // this lane's rows: token of the tile, head of the group
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    tok[u] = (u * 32 + lane) / P.group;
    off[u] = tok[u] * P.n_heads + (u * 32 + lane) % P.group;
    if (tok[u] >= P.tpt) tok[u] = 0x7fffffff;
  }
  uint32_t uses = 0;
  for_items<true>(ms, [&](const MassItem &it) {
    const Turns w(P, it, which);
    for (int t = w.t0; t < w.t1; t += w.step, ++uses) {
      const int tok0 = (it.qt0 + t) * P.tpt;
      const float *src = P.lse + (int64_t)(it.q0 + tok0) * P.n_heads + it.h * P.group;
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        v[u] = tok[u] < it.n - tok0 ? __ldg(src + off[u]) : -INFINITY;
      if (!wait_all(&ms->s_empty[which], (uses & 1) ^ 1, &ms->bd)) return false;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool none = v[u] == -INFINITY;      // adds nothing
        ms->nl[which][u * 32 + lane] = none ? -INFINITY : -v[u] * 1.4426950408889634f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->l_full[which]);
    }
    return true;
  });
}

// 32 columns from c0 on of a row of S^T: the weights, added to acc
template <bool kEdge>
__device__ __forceinline__ void weigh(uint32_t tmem, const float *nl, uint64_t c2, int lo, int hi,
                                      int c0, uint64_t (&acc)[2]) {
  uint32_t s[32];
  tmem_ld32x32b_x32(tmem + c0, s);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const ulonglong2 n4 = *reinterpret_cast<const ulonglong2 *>(nl + c0 + e);
    const float2 a = unpack2(
        fma2(pack2(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, n4.x));
    const float2 b = unpack2(
        fma2(pack2(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])), c2, n4.y));
    float w[4] = {ex2(a.x), ex2(a.y), ex2(b.x), ex2(b.y)};
    if (kEdge) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (c0 + e + k < lo || c0 + e + k >= hi) w[k] = 0.f;
    }
    acc[0] = add2(acc[0], pack2(w[0], w[1]));
    acc[1] = add2(acc[1], pack2(w[2], w[3]));
  }
}

__device__ void weight_role(const MassParams &P, MassMisc *ms) {
  const int warp = threadIdx.x >> 5, wg = warp >> 2, x = (warp & 3) * 32 + (threadIdx.x & 31);
  const uint32_t tmem = ms->tmem + wg * kTile + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint64_t c2 = pack2(P.scale_log2, P.scale_log2);
  const float *nl = ms->nl[wg];
  uint32_t uses = 0, u = 0;
  for_items<true>(ms, [&](const MassItem &it) {
    const Turns w(P, it, wg);
    const int key = w.tile * kTile + x;            // of the item
    // the first of the key tile's warpgroups stores its masses
    const bool mine = wg < P.span && key < it.keys;
    const int64_t at = (int64_t)it.h * P.seqs.kv_rows + it.row + key;
    float old = 0.f;
    if (mine && P.mass_in) old = P.mass_in[at];
    uint64_t acc[2] = {0, 0};
    for (int t = w.t0; t < w.t1; t += w.step, ++uses) {
      const int tok0 = (it.qt0 + t) * P.tpt;
      const bool ok = wait_bar(&ms->l_full[wg], uses & 1, &ms->bd) &&
                      wait_bar(&ms->s_full[wg], uses & 1, &ms->bd);
      if (!__all_sync(0xffffffffu, ok)) return false;
      fence_after_sync();
      const int64_t shift = it.shift - w.tile * kTile;
      const bool edge = (it.n - tok0) < P.tpt || kTile - 1 - shift - tok0 > 0;
      if (!edge) {
#pragma unroll 1
        for (int c0 = 0; c0 < P.ncol; c0 += 32) weigh<false>(tmem, nl, c2, 0, 0, c0, acc);
      } else {
        // columns [lo, hi) see this key
        const int hi = min(P.tpt, it.n - tok0) * P.group;
        const int64_t first = x - shift - tok0;
        const int lo = first <= 0 ? 0 : first > kTile ? kTile : (int)first * P.group;
#pragma unroll 1
        for (int c0 = 0; c0 < P.ncol; c0 += 32) weigh<true>(tmem, nl, c2, lo, hi, c0, acc);
      }
      fence_before_sync();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->s_empty[wg]);
    }
    const float2 sum2 = unpack2(add2(acc[0], acc[1]));
    float sum = sum2.x + sum2.y;
    if (P.span < kBufs) {          // other warpgroups had query tiles of these keys
      ms->red[u & 1][wg][x] = sum;
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->grp);
      if (!wait_all(&ms->grp, u & 1, &ms->bd)) return false;
      const float(*r)[kTile] = ms->red[u & 1];
      if (mine)
        sum = P.span == 2 ? r[wg][x] + r[wg + 2][x] : (r[0][x] + r[1][x]) + (r[2][x] + r[3][x]);
      ++u;
    }
    if (mine) P.mass_out[at] = old + sum;
    return true;
  });
}

template <typename T, int D>
__global__ void __launch_bounds__(kMassThreads, 1)
attn_mass_kernel(MassParams P, const __grid_constant__ CUtensorMap mq,
                 const __grid_constant__ CUtensorMap mk) {
  extern __shared__ __align__(1024) uint8_t smem[];
  MassMisc *ms = reinterpret_cast<MassMisc *>(smem + P.off_misc);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxK; ++i) mbar_init(&ms->k_full[i], 1), mbar_init(&ms->k_empty[i], kIssueWarps);
    for (int i = 0; i < kMaxQ; ++i) mbar_init(&ms->q_full[i], 1), mbar_init(&ms->q_empty[i], kIssueWarps);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&ms->s_full[i], 1);
      mbar_init(&ms->s_empty[i], 4);
      mbar_init(&ms->l_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ms->item_full[i], 1);
      mbar_init(&ms->item_empty[i], kEpiWarps + kIssueWarps + 1 + kLseWarps);
    }
    mbar_init(&ms->grp, kEpiWarps);
    for (int i = 0; i < kIssueWarps; ++i) mbar_init(&ms->done[i], 1);
    ms->bd.abort = 0;
    ms->bd.wait_ns = P.wait_ns;
    mbar_fence_init();
  }
  // query rows that pad a tile to 32 columns are never fetched: zeros, so that
  // their scores are finite (their -lse is -inf)
  {
    const int pad0 = P.tpt * P.group, pad = (P.ncol - pad0) * 8;   // 16-byte pieces a block
    for (int i = threadIdx.x; i < pad * (D / 64) * P.qst; i += kMassThreads) {
      const int s = i / (pad * (D / 64)), r = i % (pad * (D / 64));
      *reinterpret_cast<uint4 *>(smem + P.off_q + s * P.q_stage + (r / pad) * (P.ncol * 128) +
                                 pad0 * 128 + (r % pad) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
  }
  if (warp == kEpiWarps) {
    tmem_alloc(&ms->tmem, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  constexpr int kLoad = kEpiWarps + kIssueWarps;
  if (warp < kEpiWarps) {
    weight_role(P, ms);
  } else if (warp < kLoad) {
    product_role<T, D>(P, smem, ms, warp - kEpiWarps);
  } else if (warp == kLoad) {
    if ((threadIdx.x & 31) == 0) load_role<D>(P, smem, ms, &mq, &mk);
    __syncwarp();
  } else if (warp == kLoad + 1) {
    schedule_role(P, smem, ms);
  } else {
    lse_role(P, ms, warp - kLoad - 2);
  }
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && ms->bd.abort) raise_err(P.d_err, CSA2_DERR_TIMEOUT);
  if (warp == kEpiWarps) {
    fence_after_sync();
    tmem_dealloc(ms->tmem, 512);
  }
}

template <typename T, int D>
int mass_launch(MassParams &P, int64_t items, const CUtensorMap &mq, const CUtensorMap &mk,
                cudaStream_t st) {
  constexpr uint32_t kKStage = (D / 64) * kBlk;
  constexpr uint32_t kMost = 232448;
  P.q_stage = (uint32_t)P.ncol * 128u * (D / 64);
  P.qst = P.q_stage > 16384 ? 2 : 4;      // query tiles serve several key tiles each
  const uint32_t cum = ((uint32_t)P.seqs.count * 4u + 15u) & ~15u;
  const uint32_t rest = P.qst * P.q_stage + cum + (uint32_t)sizeof(MassMisc);
  const int kst = (int)((kMost - rest) / kKStage);
  P.kst = kst > kMaxK ? kMaxK : kst;
  if (P.kst < 2) return CSA2_ERR_UNSUPPORTED;
  while (P.span > P.kst) P.span /= 2;
  P.off_q = P.kst * kKStage;
  P.off_cum = P.off_q + P.qst * P.q_stage;
  P.off_misc = P.off_cum + cum;
  const int smem = (int)(P.off_misc + sizeof(MassMisc));
  allow_smem<attn_mass_kernel<T, D>>((int)kMost);
  const int grid = (int)(items < sm_count() ? items : sm_count());
  attn_mass_kernel<T, D><<<grid, kMassThreads, smem, st>>>(P, mq, mk);
  return launch_status();
}

}  // namespace
}  // namespace dense
}  // namespace csa2

using namespace csa2::dense;

extern "C" CSA2_API int csa2_attn_mass(const csa2_packed *b, int32_t n_heads, int32_t n_kv_heads,
                                       int32_t dim, int32_t dtype, const void *q, int64_t ldq,
                                       const void *k, int64_t ldk, int64_t kv_rows,
                                       const float *lse, int64_t max_kv, float sm_scale,
                                       const float *mass_in, float *mass_out, int32_t *d_err,
                                       csa2_stream_t stream) {
  Shape s;
  int st = check_packed(b, n_heads, n_kv_heads, dim, dtype, kv_rows, sm_scale, &s);
  if (st != CSA2_OK) return st;
  if (max_kv < 0) return CSA2_ERR_INVALID_ARG;
  if (b->num_req == 0 || kv_rows == 0) return CSA2_OK;
  // without queries the old mass is still carried over
  if (!b->cu_q || !b->kv_start || !b->kv_len || !mass_out) return CSA2_ERR_INVALID_ARG;
  if (b->num_q > 0 && (!q || !lse)) return CSA2_ERR_INVALID_ARG;
  if (b->num_req > kMaxReq) return CSA2_ERR_UNSUPPORTED;
  if ((st = check_rows(k, ldk, s.n_kv, s.dim)) != CSA2_OK) return st;
  if (b->num_q > 0 && (st = check_rows(q, ldq, s.n_heads, s.dim)) != CSA2_OK) return st;
  if (!csa2::aligned(4, mass_in, mass_out, lse, d_err)) return CSA2_ERR_UNSUPPORTED;
  const uint64_t cells = (uint64_t)s.n_kv * kv_rows * 4;
  if (meets_batch(mass_out, cells, b) ||
      meets_rows(mass_out, cells, k, kv_rows, ldk * 2, (int64_t)s.n_kv * s.dim * 2) ||
      meets_rows(mass_out, cells, q, b->num_q, ldq * 2, (int64_t)s.n_heads * s.dim * 2) ||
      (lse && csa2::overlap(mass_out, cells, lse, (uint64_t)b->num_q * s.n_heads * 4)) ||
      (mass_in && mass_in != mass_out && csa2::overlap(mass_out, cells, mass_in, cells)))
    return CSA2_ERR_INVALID_ARG;
  MassParams P{};
  P.seqs = Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, b->kv_start, b->kv_len,
                kv_rows};
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  const int most = kTile / s.group;
  int tpt = 1;      // a tile no longer than the requests' queries on average
  while (tpt < most && (int64_t)tpt * b->num_req < b->num_q) tpt *= 2;
  P.tpt = tpt < most ? tpt : most;
  P.ncol = (P.tpt * P.group + 31) & ~31;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.lse = lse;
  P.mass_in = mass_in;
  P.mass_out = mass_out;
  P.d_err = d_err;
  P.wait_ns = csa2::wait_limit_ns();
  CUtensorMap mq, mk;
  const bool none = b->num_q == 0;
  if (!make_rows_map(&mk, s.bf16, k, kv_rows, s.n_kv, s.dim, ldk, 1, kTile) ||
      !make_rows_map(&mq, s.bf16, none ? k : q, none ? kv_rows : b->num_q,
                     none ? s.n_kv : s.n_heads, s.dim, none ? ldk : ldq, none ? 1 : s.group,
                     P.tpt))
    return CSA2_ERR_UNSUPPORTED;
  // key tiles of an item: as many as leave every SM several items
  const int64_t most_kv = max_kv < kv_rows ? max_kv : kv_rows, all_kv = most_kv * b->num_req;
  const int64_t tiles = ((all_kv < kv_rows ? all_kv : kv_rows) / kTile + b->num_req) * s.n_kv;
  P.span = tiles >= 4 * 6 * kSms ? 4 : tiles >= 2 * 4 * kSms ? 2 : 1;
  const cudaStream_t cs = csa2::as_stream(stream);
  if (s.bf16)
    return s.dim == 128 ? mass_launch<__nv_bfloat16, 128>(P, tiles, mq, mk, cs)
                        : mass_launch<__nv_bfloat16, 64>(P, tiles, mq, mk, cs);
  return s.dim == 128 ? mass_launch<__half, 128>(P, tiles, mq, mk, cs)
                      : mass_launch<__half, 64>(P, tiles, mq, mk, cs);
}
