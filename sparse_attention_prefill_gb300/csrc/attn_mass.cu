// Attention weight that queries put on cached rows, added up per row and key
// head (csa2_attn_mass):
//   mass[g, j] (+)= sum_{i sees j, h in group g} exp(c <q[i,h], k[j,g]> - lse[i,h])
//
// Keys are stationary: a work item is 128 keys of one request and key head.
// Its K tile is the A operand, the packed query tiles (dense.cuh) that see it
// pass as B operands, so S^T[key, query row] has a key to a TMEM lane and the
// sum over queries stays in one thread's register: no atomics, a fixed order.
// The exponent needs no maximum (lse is given): exp2(c' s - lse'), one fused
// multiply-add and one exponential to a score, with -lse' read from shared
// memory (one value per column, the same for all lanes).
//
// Per item the kernel reads the K tile once and every query tile once (from
// L2, where a request's queries stay); a decode step is bound by the K rows,
// a window of queries by the products and exponentials.
//
// Roles (12 warps, one CTA per SM, persistent over items):
//   warps 0-7  weights: warp w reads TMEM sub-partition w % 4 (keys 32(w % 4)
//              .. + 31), the 16-column chunks of parity w / 4
//   warp 8     TMEM; issues the products
//   warp 9     K and Q tiles by TMA
//   warp 10    looks items up a few ahead
//   warp 11    -lse of the query tiles
// S^T has four TMEM buffers, so products run up to four query tiles ahead.
// Every wait is bounded, as in the attention.
#include "dense.cuh"

namespace csa2 {
namespace dense {
namespace {

constexpr int kMaxReq = 8192;
constexpr int kBufs = 4;            // S^T buffers (128 TMEM columns each)
constexpr int kItems = 4;           // items looked up ahead
constexpr int kMaxK = 6, kMaxQ = 4; // ring stages at most
constexpr int kEpiWarps = 8;
constexpr int kMassThreads = 12 * 32;

struct MassParams {
  Seqs seqs;
  int n_heads, n_kv, group, tpt, ncol;   // ncol: tpt * group, rounded up to 16
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
  int h, keys;        // key head; keys of the tile (-1: no more items)
  int qt0, nq;        // first query tile that sees the tile, and how many
  int64_t row;        // first pool row
  int64_t shift;      // query i sees the tile's key x if x <= shift + i
};

struct MassMisc {
  uint64_t k_full[kMaxK], k_empty[kMaxK], q_full[kMaxQ], q_empty[kMaxQ];
  uint64_t s_full[kBufs], s_empty[kBufs], l_full[kBufs];
  uint64_t item_full[kItems], item_empty[kItems], grp, done;
  Bound bd;
  uint32_t tmem;
  MassItem item[kItems];
  alignas(16) float nl[kBufs][kTile];    // -lse in log2 units, by query row
  float red[2][kTile];
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
      nt = (uint32_t)((m + kTile - 1) / kTile);
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
  uint32_t u = 0;
  for (int64_t id = blockIdx.x;; id += gridDim.x, ++u) {
    const uint32_t s = u % kItems;
    if (!wait_all(&ms->item_empty[s], ((u / kItems) & 1) ^ 1, &ms->bd)) break;
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
      const int kt = (int)(tile - (lo ? cum[lo - 1] : 0u));
      int64_t start, m;
      seq_rows(P.seqs, lo, it.q0, it.n, err);
      seq_keys(P.seqs, lo, start, m, err);
      const int64_t left = m - (int64_t)kt * kTile;
      it.keys = left < 0 ? 0 : left < kTile ? (int)left : kTile;
      it.row = start + (int64_t)kt * kTile;
      it.shift = m - it.n - (int64_t)kt * kTile;
      const int64_t first = it.shift >= 0 ? 0 : -it.shift;      // first query that sees key 0
      const int tiles = (it.n + P.tpt - 1) / P.tpt;
      it.qt0 = first < it.n ? (int)(first / P.tpt) : tiles;
      it.nq = it.keys > 0 ? tiles - it.qt0 : 0;
    }
    if (lane == 0) {
      ms->item[s] = it;
      mbar_arrive(&ms->item_full[s]);
    }
    __syncwarp();
    if (it.keys < 0) break;
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane == 0) raise_err(P.d_err, err);
}

// The items of this CTA, one after another, as every role sees them.  `lanes`:
// a single thread (0) or a whole warp (1) calls.
template <bool kWarp, typename F>
__device__ __forceinline__ bool for_items(MassMisc *ms, F f) {
  for (uint32_t u = 0;; ++u) {
    const uint32_t s = u % kItems;
    bool ok = wait_bar(&ms->item_full[s], (u / kItems) & 1, &ms->bd);
    if (kWarp) ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    const MassItem it = ms->item[s];
    if (kWarp) __syncwarp();
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
    const uint32_t sk = gk % P.kst;
    if (!wait_bar(&ms->k_empty[sk], ((gk / P.kst) & 1) ^ 1, &ms->bd)) return false;
    mbar_arrive_expect_tx(&ms->k_full[sk], kKStage);
    for (int c = 0; c < D / 64; ++c)
      tma_load_3d(smem + sk * kKStage + c * kBlk, mk, c * 64, it.h, (int)it.row, &ms->k_full[sk]);
    ++gk;
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

template <typename T, int D>
__device__ void product_role(const MassParams &P, uint8_t *smem, MassMisc *ms) {
  constexpr uint32_t kKStage = (D / 64) * kBlk;
  const uint32_t idesc = idesc_of<T>(kTile, P.ncol, false);
  const uint32_t tmem = uniform(ms->tmem), qblk = P.ncol * 128;
  const uint64_t kd = make_desc_sw128(smem_u32(smem), 16, 1024);
  const uint64_t qd = make_desc_sw128(smem_u32(smem + P.off_q), 16, 1024);
  uint32_t sk = 0, pk = 0, sq = 0, pq = 0, g = 0;     // ring stages and phases
  for_items<true>(ms, [&](const MassItem &it) {
    const int nq = uniform(it.nq);
    if (nq == 0) return true;
    if (!wait_all(&ms->k_full[sk], pk, &ms->bd)) return false;
    const uint64_t a = desc_add(kd, sk * kKStage);
    for (int t = 0; t < nq; ++t, ++g) {
      const uint32_t sb = g % kBufs;
      if (!wait_all(&ms->s_empty[sb], ((g / kBufs) & 1) ^ 1, &ms->bd)) return false;
      if (!wait_all(&ms->q_full[sq], pq, &ms->bd)) return false;
      fence_after_sync();
      const uint64_t b = desc_add(qd, sq * P.q_stage);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16(tmem + sb * kTile, desc_add(a, (k >> 2) * kBlk + (k & 3) * 32),
                  desc_add(b, (k >> 2) * qblk + (k & 3) * 32), idesc, k > 0);
        mma_commit(&ms->s_full[sb]);
        mma_commit(&ms->q_empty[sq]);
      }
      __syncwarp();
      if (++sq == (uint32_t)P.qst) sq = 0, pq ^= 1;
    }
    if (elect_one()) mma_commit(&ms->k_empty[sk]);
    __syncwarp();
    if (++sk == (uint32_t)P.kst) sk = 0, pk ^= 1;
    return true;
  });
  if (elect_one()) mma_commit(&ms->done);
  __syncwarp();
  drain_bar(&ms->done, 0);
}

__device__ void lse_role(const MassParams &P, MassMisc *ms) {
  const int lane = threadIdx.x & 31;
  uint32_t g = 0;
  for_items<true>(ms, [&](const MassItem &it) {
    for (int t = 0; t < it.nq; ++t, ++g) {
      const uint32_t sb = g % kBufs;
      const int tok0 = (it.qt0 + t) * P.tpt;
      float v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int x = u * 32 + lane, tok = tok0 + x / P.group;
        v[u] = -INFINITY;
        if (x < P.tpt * P.group && tok < it.n)
          v[u] = __ldg(P.lse + (int64_t)(it.q0 + tok) * P.n_heads + it.h * P.group + x % P.group);
      }
      if (!wait_all(&ms->s_empty[sb], ((g / kBufs) & 1) ^ 1, &ms->bd)) return false;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool none = v[u] == -INFINITY;      // adds nothing
        ms->nl[sb][u * 32 + lane] = none ? -INFINITY : -v[u] * 1.4426950408889634f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ms->l_full[sb]);
    }
    return true;
  });
}

__device__ void weight_role(const MassParams &P, MassMisc *ms) {
  const int warp = threadIdx.x >> 5, half = warp >> 2, x = (warp & 3) * 32 + (threadIdx.x & 31);
  const uint32_t lane_addr = (uint32_t)(32 * (warp & 3)) << 16;
  const float c = P.scale_log2;
  uint32_t g = 0, u = 0;
  for_items<true>(ms, [&](const MassItem &it) {
    float *out = P.mass_out + (int64_t)it.h * P.seqs.kv_rows + it.row + x;
    const bool mine = half == 0 && x < it.keys;
    float old = 0.f;
    if (mine && P.mass_in) old = P.mass_in[(int64_t)it.h * P.seqs.kv_rows + it.row + x];
    float acc0 = 0.f, acc1 = 0.f;
    for (int t = 0; t < it.nq; ++t, ++g) {
      const uint32_t sb = g % kBufs, ph = (g / kBufs) & 1;
      bool ok = wait_bar(&ms->l_full[sb], ph, &ms->bd) && wait_bar(&ms->s_full[sb], ph, &ms->bd);
      if (!__all_sync(0xffffffffu, ok)) return false;
      fence_after_sync();
      const int tok0 = (it.qt0 + t) * P.tpt;
      // columns [lo, hi) see this key
      const int hi = min(P.tpt, it.n - tok0) * P.group;
      const int64_t first = x - it.shift - tok0;
      const int lo = first <= 0 ? 0 : first > kTile ? kTile : (int)first * P.group;
      const bool edge = hi < P.tpt * P.group || kTile - 1 - it.shift - tok0 > 0;
      for (int c0 = 16 * half; c0 < P.ncol; c0 += 32) {
        uint32_t s[32];
        tmem_ld32x32b_x16(ms->tmem + sb * kTile + c0 + lane_addr, s);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const float4 nl = *reinterpret_cast<const float4 *>(&ms->nl[sb][c0 + e]);
          float w[4] = {ex2(fmaf(__uint_as_float(s[e]), c, nl.x)),
                        ex2(fmaf(__uint_as_float(s[e + 1]), c, nl.y)),
                        ex2(fmaf(__uint_as_float(s[e + 2]), c, nl.z)),
                        ex2(fmaf(__uint_as_float(s[e + 3]), c, nl.w))};
          if (edge) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (c0 + e + k < lo || c0 + e + k >= hi) w[k] = 0.f;
          }
          acc0 += w[0] + w[1];
          acc1 += w[2] + w[3];
        }
      }
      fence_before_sync();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->s_empty[sb]);
    }
    const float acc = acc0 + acc1;
    if (half == 1) ms->red[u & 1][x] = acc;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->grp);
    if (!wait_all(&ms->grp, u & 1, &ms->bd)) return false;
    if (mine) *out = old + (acc + ms->red[u & 1][x]);
    ++u;
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
    for (int i = 0; i < kMaxK; ++i) mbar_init(&ms->k_full[i], 1), mbar_init(&ms->k_empty[i], 1);
    for (int i = 0; i < kMaxQ; ++i) mbar_init(&ms->q_full[i], 1), mbar_init(&ms->q_empty[i], 1);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&ms->s_full[i], 1);
      mbar_init(&ms->s_empty[i], kEpiWarps);
      mbar_init(&ms->l_full[i], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ms->item_full[i], 1);
      mbar_init(&ms->item_empty[i], kEpiWarps + 3);   // weights, products, loads, lse
    }
    mbar_init(&ms->grp, kEpiWarps);
    mbar_init(&ms->done, 1);
    ms->bd.abort = 0;
    ms->bd.wait_ns = P.wait_ns;
    mbar_fence_init();
  }
  // query rows that pad a tile to 16 columns are never fetched: zeros, so that
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
  if (warp == 8) {
    tmem_alloc(&ms->tmem, 512);
    tmem_relinquish();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp < kEpiWarps) {
    weight_role(P, ms);
  } else if (warp == 8) {
    product_role<T, D>(P, smem, ms);
  } else if (warp == 9) {
    if ((threadIdx.x & 31) == 0) load_role<D>(P, smem, ms, &mq, &mk);
    __syncwarp();
  } else if (warp == 10) {
    schedule_role(P, smem, ms);
  } else {
    lse_role(P, ms);
  }
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && ms->bd.abort) raise_err(P.d_err, CSA2_DERR_TIMEOUT);
  if (warp == 8) {
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
  P.qst = P.ncol > 64 ? 3 : 4;
  const uint32_t cum = ((uint32_t)P.seqs.count * 4u + 15u) & ~15u;
  const uint32_t rest = P.qst * P.q_stage + cum + (uint32_t)sizeof(MassMisc);
  int kst = (int)((kMost - rest) / kKStage);
  P.kst = kst > kMaxK ? kMaxK : kst;
  if (P.kst < 2) return CSA2_ERR_UNSUPPORTED;
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
  if (((uintptr_t)mass_in | (uintptr_t)mass_out | (uintptr_t)lse) & 3u) return CSA2_ERR_UNSUPPORTED;
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
  P.ncol = (P.tpt * P.group + 15) & ~15;
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
  const int64_t tiles = (max_kv + kTile - 1) / kTile;
  const int64_t items = (tiles > 0 ? tiles : 1) * b->num_req * s.n_kv;
  const cudaStream_t cs = csa2::as_stream(stream);
  if (s.bf16)
    return s.dim == 128 ? mass_launch<__nv_bfloat16, 128>(P, items, mq, mk, cs)
                        : mass_launch<__nv_bfloat16, 64>(P, items, mq, mk, cs);
  return s.dim == 128 ? mass_launch<__half, 128>(P, items, mq, mk, cs)
                      : mass_launch<__half, 64>(P, items, mq, mk, cs);
}
