// What the tensor-core attention kernels share: items and the warp that hands them
// out, the warp that issues the products, and the end of an item.
#pragma once
#include <type_traits>

#include "dense.cuh"

namespace csa2 {
namespace dense {
namespace {

constexpr int kMmaWarp = 8, kProducerWarp = 9, kItemWarp = 10;
constexpr int kItems = 3;            // items published at a time

struct Item {
  int run, q0, n, tok0;      // run (-1: no work, -2: no more items), its first query row and
                             // rows, first token of the item
  int h, split;
  int64_t start;             // first cache row
  int64_t m;                 // cache rows
  int kt0, nk;               // key tiles
  int steps[2];              // of each stream
  int ntile;                 // query tiles with tokens
  int uncovered;             // a request in no group (own part of a shared-prefix call)
};

// Items of a part's runs, as a warp holds them: lane l has those of an equal
// share of the runs, and the sum up to and with its share.  Unsigned: the runs of
// a malformed batch may lie over one another and sum up to anything.
struct Shares {
  uint32_t own, upto;
};

__device__ __forceinline__ uint32_t lane_scan(uint32_t v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__device__ Shares count_items(const AttnParams &P, int tok, int &err) {
  const int lane = threadIdx.x & 31, per = (P.seqs.count + 31) / 32;
  Shares s{0, 0};
#pragma unroll 4
  for (int i = lane * per; i < min(P.seqs.count, (lane + 1) * per); ++i) {
    int a, c;
    seq_rows(P.seqs, i, a, c, err);
    s.own += ((uint32_t)c + tok - 1) / tok;
  }
  s.upto = lane_scan(s.own);
  return s;
}

// The item of CTA `cta` of the grid, by one warp; run = -1 if it has no work.  kPaged:
// runs have no first row, and at most seqs.kv_rows rows.
template <bool kNarrow, bool kPaged>
__device__ void find_item(const AttnParams &P, uint32_t cta, const Shares &s, Item &it,
                          int &err) {
  const int lane = threadIdx.x & 31;
  const int ns = P.splits > 0 ? P.splits : 1, tok = kNarrow ? P.tpt : 2 * P.tpt;
  const int per = (P.seqs.count + 31) / 32;
  it.split = (int)(cta % ns);
  it.h = (int)(cta / ns % P.n_kv);
  const uint32_t slot = cta / ns / P.n_kv;
  it.run = -1;
  const uint32_t share = __ballot_sync(0xffffffffu, slot < s.upto);
  if (!share) return;
  const int l = __ffs(share) - 1;
  uint32_t base = __shfl_sync(0xffffffffu, s.upto - s.own, l);
  const int end = min(P.seqs.count, (l + 1) * per);
  for (int i0 = l * per; i0 < end && it.run < 0; i0 += 32) {
    // everything of a lane's run at once
    int a = 0, c = 0;
    int64_t start = 0, m = 0;
    if (i0 + lane < end) {
      seq_rows(P.seqs, i0 + lane, a, c, err);
      if (kPaged) {
        m = P.seqs.kv_len[i0 + lane];
        if (m < 0 || m > P.seqs.kv_rows) {
          m = 0;
          if (c) err |= CSA2_DERR_RANGE_ROW;     // (without query rows nobody looks at it)
        }
      } else {
        seq_keys(P.seqs, i0 + lane, start, m, err);
      }
    }
    const uint32_t here = ((uint32_t)c + tok - 1) / tok, inc = lane_scan(here);
    const uint32_t hit = __ballot_sync(0xffffffffu, slot < base + inc);
    if (hit) {
      const int src = __ffs(hit) - 1;
      // the longest key ranges first
      const uint32_t item = __shfl_sync(0xffffffffu, base + inc, src) - 1 - slot;
      if (item >= __shfl_sync(0xffffffffu, here, src)) return;      // sums that wrapped
      it.run = i0 + src;
      it.tok0 = (int)item * tok;
      it.q0 = __shfl_sync(0xffffffffu, a, src);
      it.n = __shfl_sync(0xffffffffu, c, src);
      it.start = __shfl_sync(0xffffffffu, start, src);
      it.m = __shfl_sync(0xffffffffu, m, src);
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (it.run < 0) return;
  it.uncovered = P.cover && !in_groups(P.cover, P.n_cover, it.run, P.seqs);
  it.ntile = min(tok, it.n - it.tok0) > P.tpt ? 2 : 1;
  int nkt[2];                      // key tiles that each query tile needs
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last_tok = min(it.tok0 + (t + 1) * P.tpt, it.n) - 1;
    const int64_t last = P.causal ? it.m - it.n + last_tok : it.m - 1;
    nkt[t] = t < it.ntile && last >= 0 ? (int)(last / kTile) + 1 : 0;
  }
  const int total = max(nkt[0], nkt[1]);
  it.kt0 = 0;
  it.nk = total;
  if (P.splits > 0) {
    const int each = (total + P.splits - 1) / P.splits;
    it.kt0 = min(total, it.split * each);
    it.nk = min(total, it.kt0 + each) - it.kt0;
  }
  if (kNarrow) {
    it.steps[0] = (it.nk + 1) / 2;
    it.steps[1] = it.nk / 2;
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) it.steps[t] = max(0, min(nkt[t] - it.kt0, it.nk));
  }
}

// Publishes items: this CTA's, then those of CTAs of the grid that have not
// started (cluster launch control: the hardware hands out their indices).  The
// next one is asked for once all loads of the last are issued: earlier, and a
// CTA would sit on items that an idle one could take (448 items of 37 steps:
// 194 us with up to four items ahead); later, and the loads would pause.
template <bool kNarrow, bool kPaged, typename M>
__device__ void item_role(const AttnParams &P, M *ms) {
  const int lane = threadIdx.x & 31;
  uint32_t asked = 0, items = 0;
  bool ok = true, more = true, waiting = false;
  int err = 0;
  const Shares shares = count_items(P, kNarrow ? P.tpt : 2 * P.tpt, err);
  uint32_t cta = blockIdx.x;
  Item it;
  while (ok && more) {
    find_item<kNarrow, kPaged>(P, cta, shares, it, err);
    if (it.run >= 0) {
      const uint32_t s = items % kItems;
      ok = wait_all(&ms->item_empty[s], ((items / kItems) & 1) ^ 1, &ms->bd);
      if (ok && lane == 0) {
        ms->item[s] = it;
        mbar_arrive(&ms->item_full[s]);
      }
      __syncwarp();
      ok = ok && wait_all(&ms->loaded, items & 1, &ms->bd);
      ++items;
    }
    if (!ok) break;
    if (lane == 0) {
      mbar_arrive_expect_tx(&ms->clc, 16);
      ask_next(ms->next, &ms->clc);
    }
    waiting = true;
    if (!(ok = wait_all(&ms->clc, asked & 1, &ms->bd))) break;
    waiting = false;
    ++asked;
    more = next_cta(ms->next, cta);
    fence_proxy_async_smem();      // the next answer is written by the async proxy
    __syncwarp();
  }
  if (ok) {
    const uint32_t s = items % kItems;
    ok = wait_all(&ms->item_empty[s], ((items / kItems) & 1) ^ 1, &ms->bd);
    if (ok && lane == 0) {
      ms->item[s].run = -2;
      mbar_arrive(&ms->item_full[s]);
    }
  }
  if (waiting && lane == 0) drain_bar(&ms->clc, asked & 1);
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane == 0) raise_err(P.d_err, err);
}

// One warp issues every product: with Q and the ring's tiles as 16-bit operands, S by
// the instruction kIdS and O by kIdO.  Q is there once q_ready completes.
template <typename C, uint32_t kIdS, uint32_t kIdO, bool kNarrow, typename M>
__device__ void mma_role(uint8_t *smem, M *ms, uint64_t *q_ready) {
  constexpr int D = C::D;
  const uint32_t tmem = uniform(ms->tmem);
  const uint64_t ring_k = make_desc_sw128(smem_u32(smem + C::kOffRing), 16, 1024);
  const uint64_t ring_v = make_desc_sw128(smem_u32(smem + C::kOffRing), kBlk, 1024);
  const uint64_t qd = make_desc_sw128(smem_u32(smem), 16, 1024);
  uint32_t s0 = 0, p0 = 0;          // ring stage and phase of the next tile to take
  uint32_t pq = 0, pp = 0;          // phases of Q, and of P by stream (a bit each)
  // ring stage (low bits) and phase (bit 8) of the tile `n` <= 4 further on
  auto at = [&](uint32_t s, uint32_t p, uint32_t n) {
    s += n;
    if (C::kStages < 4 && s >= 2 * C::kStages) return (s - 2 * C::kStages) | (p << 8);
    return s >= C::kStages ? (s - C::kStages) | ((p ^ 1) << 8) : s | (p << 8);
  };
  for (uint32_t u = 0;; ++u) {
    const uint32_t slot = u % kItems;
    if (!wait_all(&ms->item_full[slot], (u / kItems) & 1, &ms->bd)) break;
    const Item &it = ms->item[slot];
    const int run = uniform(it.run), nk = uniform(it.nk);
    const int steps[2] = {uniform(it.steps[0]), uniform(it.steps[1])};
    if (elect_one()) mbar_arrive(&ms->item_empty[slot]);
    __syncwarp();
    if (run < 0) break;
    if (nk <= 0) continue;
    // products of S[t] with the K tile of a ring stage, by the elected lane
    auto issue_s = [&](int t, uint32_t stage) {
      const uint64_t a = desc_add(qd, kNarrow ? 0 : t * C::kQTile), b = desc_add(ring_k, stage * C::kStage);
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint32_t off = (k >> 2) * kBlk + (k & 3) * 32;
        mma_f16(tmem + t * 128, desc_add(a, off), desc_add(b, off), kIdS, k > 0);
      }
      mma_commit(&ms->s_full[t]);
    };
    const uint32_t second = at(s0, p0, 1);           // a narrow item's second K tile
    const int first = kNarrow && nk > 1 ? 2 : 1;      // K tiles in front of the first V
    if (elect_one()) {
      wait_inline(q_ready, pq, &ms->bd);
      wait_inline(&ms->full[s0], p0, &ms->bd);
      fence_after_sync();
      if (steps[0] > 0) issue_s(0, s0);
      if (steps[1] > 0) {
        if (kNarrow) {
          wait_inline(&ms->full[second & 255], second >> 8, &ms->bd);
          fence_after_sync();
          issue_s(1, second & 255);
          mma_commit(&ms->empty[second & 255]);
        } else {
          issue_s(1, s0);
        }
      }
      mma_commit(&ms->empty[s0]);
      if (nk <= first) mma_commit(&ms->q_empty);
    }
    __syncwarp();
    pq ^= 1;
    const uint32_t v0 = at(s0, p0, first);
    uint32_t sv = v0 & 255, pv = v0 >> 8;            // this step's first V tile
    const int rounds = max(steps[0], steps[1]);
    bool ok = true;
    for (int j = 0; j < rounds && ok; ++j) {
      // once a wait has run out nothing waits any more, and the products of
      // the step at hand read whatever is there
      ok = uniform(*(volatile int *)&ms->bd.abort) == 0;
      // tiles of the ring: V of this step (two of a narrow item, unless its
      // last pair is one tile), then K of the next step
      const int here = kNarrow ? min(2, nk - 2 * j) : 1;
      const int ahead = kNarrow ? max(0, min(2, nk - 2 * j - 2)) : (j + 1 < rounds ? 1 : 0);
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (ok && j < steps[t]) {
          const uint32_t v = at(sv, pv, kNarrow ? t : 0);
          const uint32_t k = at(sv, pv, kNarrow ? here + t : 1);
          const uint64_t b = desc_add(ring_v, (v & 255) * C::kStage);
          const bool next = j + 1 < steps[t];
          // the last stream to use this step's tiles lets them go
          const bool last = kNarrow || t == 1 || j >= steps[1];
          // The waits lie between the products that they hold back: the
          // tensor pipe has some four products queued meanwhile.
          if (elect_one()) {
            wait_inline(&ms->full[v & 255], v >> 8, &ms->bd);
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // P arrives in halves of 64 keys
              wait_inline(&ms->p_full[t][half], (pp >> t) & 1, &ms->bd);
              fence_after_sync();
#pragma unroll
              for (int x = 4 * half; x < 4 * half + 4; ++x)
                mma_f16_ts(tmem + C::kColO + t * D, tmem + t * 128 + x * 8, desc_add(b, x * 2048),
                           kIdO, j > 0 || x > 0);
            }
            if (next) {
              wait_inline(&ms->full[k & 255], k >> 8, &ms->bd);
              issue_s(t, k & 255);
            } else {
              mma_commit(&ms->o_full[t]);
            }
            if (last) {
              mma_commit(&ms->empty[v & 255]);
              if (kNarrow ? next : ahead > 0) mma_commit(&ms->empty[k & 255]);
              // the item's last S releases Q
              if (kNarrow ? next && 2 * (j + 1) + t == nk - 1 : j + 2 == rounds)
                mma_commit(&ms->q_empty);
            }
          }
          __syncwarp();
          pp ^= 1u << t;
        }
      }
      const uint32_t v1 = at(sv, pv, here + ahead);
      sv = v1 & 255, pv = v1 >> 8;
    }
    if (!ok) break;
    s0 = sv, p0 = pv;
  }
  if (elect_one()) mma_commit(&ms->done);          // TMEM is not freed under a running product
  __syncwarp();
  drain_bar(&ms->done, 0);
}

// Normalises and stores a warp's 32 rows of O.  Read 16 lanes x 256 bits at a
// time, a quad of threads has 8 neighbouring columns of a row; packed to 16
// bits and transposed among the quad, each thread has 16 bytes and the quad
// 64 of a row.  (Whole rows to a thread, 16 bytes a store, touched 32 lines an
// instruction: 4000 cycles of the load/store pipe to an item, during which the
// MMA warp's barrier polls waited too.)  `at`, `valid`, `seen`, w0 and w1 are
// those of the lane's own row.
template <typename T, int D>
__device__ __forceinline__ void store_rows(const AttnParams &P, uint32_t to, int64_t at,
                                           bool valid, bool seen, bool any, bool other, float w0,
                                           float w1) {
  const int lane = threadIdx.x & 31, c = lane & 3;
  const uint32_t ok = __ballot_sync(0xffffffffu, valid), has = __ballot_sync(0xffffffffu, seen);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float a[2], b[2];
    T *dst[2];
    int row[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      row[r] = 16 * half + 8 * r + (lane >> 2);
      a[r] = __shfl_sync(0xffffffffu, w0, row[r]);
      b[r] = __shfl_sync(0xffffffffu, w1, row[r]);
      dst[r] = static_cast<T *>(P.out) + __shfl_sync(0xffffffffu, at, row[r]) * D + 8 * c;
    }
    const uint32_t base = to + ((uint32_t)(16 * half) << 16);
#pragma unroll
    for (int col = 0; col < D; col += 32) {
      uint32_t o[16], o1[16];
      if (any) tmem_ld16x256b_x4(base + col, o);
      if (other) tmem_ld16x256b_x4(base + D + col, o1);
      tmem_wait_ld();
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float f[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            f[e] = (has >> row[r]) & 1 ? __uint_as_float(o[4 * k + 2 * r + e]) * a[r] : 0.f;
            if (other && ((has >> row[r]) & 1))
              f[e] = fmaf(__uint_as_float(o1[4 * k + 2 * r + e]), b[r], f[e]);
          }
          w[k] = Elem<T>::pack(f[0], f[1]);
        }
        // word k of thread c to word c of thread k
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, c & 1 ? w[k] : w[k + 1], 1);
          if (c & 1) w[k] = got; else w[k + 1] = got;
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, c & 2 ? w[k] : w[k + 2], 2);
          if (c & 2) w[k] = got; else w[k + 2] = got;
        }
        if ((ok >> row[r]) & 1)
          *reinterpret_cast<uint4 *>(dst[r] + col) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// The end of one item's stream t: row x of the tile (token i of the run, if `valid`),
// whose O is at `to` in TMEM, is normalised and stored.  kRuns: partial results are those
// of single items, number it.split (-1: none), with all rows of the item.  False if a
// wait ran out, here or before (!ok).  `any`: the stream had steps.  (Left by the caller
// where !ok, and with `any` from the item, the softmax loop in front came out slower: a
// prompt of 16384 tokens took 1409 us instead of 1381.)
template <typename T, typename C, bool kNarrow, bool kRuns = false, typename M>
__device__ __forceinline__ bool finish_item(const AttnParams &P, M *ms, const Item &it, int t,
                                            int i, bool ok, bool any, bool valid, bool rows_here,
                                            float ref, float sum, uint32_t to, uint32_t &po,
                                            uint32_t &pst) {
  constexpr int D = C::D;
  const int x = threadIdx.x & 127;
  if (ok && any) ok = wait_all(&ms->o_full[t], po, &ms->bd);
  if (!ok) return false;
  if (any) po ^= 1;
  fence_after_sync();
  // a narrow item's stream 1 hands its rows' statistics to stream 0, which
  // reads both rows of O (they are in the same lanes) and writes the output
  if (kNarrow && t == 1) {
    ms->stat[x] = make_float2(ref, sum);
    fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->stat_full);
    ok = wait_all(&ms->stat_empty, pst, &ms->bd);
    pst ^= 1;
    return ok;
  }
  float w0 = 1.f, w1 = 0.f;          // weights of the streams' rows
  bool other = false;
  if (kNarrow) {
    if (!wait_all(&ms->stat_full, pst, &ms->bd)) return false;
    pst ^= 1;
    fence_after_sync();
    other = it.steps[1] > 0;
    const float2 st = ms->stat[x];
    const float r = fmaxf(ref, st.x), base = r == -INFINITY ? 0.f : r;
    w0 = ex2(ref - base);
    w1 = ex2(st.x - base);
    sum = sum * w0 + (other ? st.y * w1 : 0.f);
    ref = r;
  }
  const bool seen = any && !(sum == 0.f);       // a NaN sum stays a NaN
  const float inv = seen ? 1.f / sum : 0.f;
  w0 *= inv, w1 *= inv;
  const float lse =
      seen ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  if (kRuns ? P.part_o && it.split >= 0 : P.splits > 0) {
    int64_t stat, elem;
    if (kRuns) {
      constexpr int kRows = kNarrow ? kTile : 2 * kTile;
      stat = (int64_t)it.split * kRows + (kNarrow ? 0 : t * kTile) + x;
      elem = (stat & ~(int64_t)31) * D + (x & 31);
    } else {
      const int64_t rows = part_rows(P.seqs.num_q, P.group);
      const int64_t at = (int64_t)(it.q0 + i) * P.group + x % P.group;
      stat = part_stat(rows, P.n_kv, it.split, it.h, at);
      elem = part_elem(rows, P.n_kv, D, it.split, it.h, at);
    }
    if (valid) {
      P.part_lse[stat] = lse;
      if (!kRuns && it.uncovered && it.split == 0) {
        const int64_t rows = part_rows(P.seqs.num_q, P.group);
        const int64_t at = (int64_t)(it.q0 + i) * P.group + x % P.group;
        for (int s = 0; s < P.cover_splits; ++s)
          P.cover_lse[part_stat(rows, P.n_kv, s, it.h, at)] = -INFINITY;
      }
    }
    if (rows_here && any) {
      float *dst = P.part_o + elem;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        float f[32];
        tmem_ld32x32b_x32(to + 32 * c, o);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) f[e] = __uint_as_float(o[e]) * w0;
        if (other) {
          tmem_ld32x32b_x32(to + D + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) f[e] = fmaf(__uint_as_float(o[e]), w1, f[e]);
        }
        if (valid && seen) {
#pragma unroll
          for (int e = 0; e < 32; ++e) dst[(32 * c + e) * 32] = f[e];
        }
      }
    }
  } else {
    const int64_t at = (int64_t)(it.q0 + i) * P.n_heads + it.h * P.group + x % P.group;
    if (valid && P.lse) P.lse[at] = lse;
    if (rows_here) store_rows<T, D>(P, to, at, valid, seen, any, other, w0, w1);
  }
  if (kNarrow) {
    fence_before_sync();
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->stat_empty);
  }
  fence_before_sync();      // O is read: the next item's first product may overwrite it
  return true;
}

// Tokens of a query tile for runs of `avg` rows on average: a tile no longer
// than they are, so that single tokens do not fetch their neighbours' queries
int tile_tokens(int64_t num_q, int64_t runs, int group) {
  const int most = kTile / group;
  int t = 1;
  while (t < most && (int64_t)t * runs < num_q) t *= 2;
  return t < most ? t : most;
}

// Single tokens of few heads go by decode_attn.cu; other runs whose rows fill no
// more than one query tile are narrow items.
enum Kind { kWideItems, kNarrowItems, kSingleTokens };

Kind kind_of(int64_t num_q, int64_t runs, int tpt, int group, bool single) {
  if (single && tpt == 1 && group <= kDecodeGroup) return kSingleTokens;
  return num_q <= runs * tpt ? kNarrowItems : kWideItems;
}

}  // namespace
}  // namespace dense
}  // namespace csa2
