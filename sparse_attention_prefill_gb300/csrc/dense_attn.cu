// Dense grouped-head attention over a K/V cache on the 5th-generation tensor
// cores: whole prompts and extends (csa2_prompt_attn), and batches that share
// prefixes (csa2_prefix_attn).
//
// Per query row x = (token, head) with keys j <= last(x):
//   l_j = c <q_x, k_j>,  out = sum_j e^{l_j} v_j / sum_j e^{l_j},
//   lse = ln sum_j e^{l_j}.
//
// An item is walked over in key tiles of 128 keys by two streams, each with a
// query tile of 128 packed rows (dense.cuh) of one key head:
//   S[t] = Q[t] K^T     (both operands in shared memory, S in TMEM)
//   O[t] += P[t] V      (P in TMEM over S's columns, V in shared memory)
// Wide items (prompts, shared prefixes) have two neighbouring query tiles that
// share the key tiles; narrow ones (decode steps, short extends: requests whose
// rows fill one tile) have one query tile, and its streams take the even and
// the odd key tiles and join their sums in the end.
//
// The softmax holds one row to a thread: it reads its row of S, keeps a
// reference maximum that moves only when a logit passes it by a margin (then
// the thread rescales its row of O; the products of that row are complete by
// then, since S of this step was issued after them), and writes P rounded to
// the inputs' type.  Row sums are taken of the unrounded P in fp32.  Warps
// without a query row leave their P as it is: rows do not mix.
//
// The MMA warp issues, step by step and stream by stream, O[t](j) and then
// S[t](j+1): while one stream's softmax runs, the other's products keep the
// tensor pipe busy.  The grid has a CTA to an item, but a CTA that runs takes
// the items of CTAs that have not started, so that an item's output overlaps
// the loads and first products of the next.
//
// A shared-prefix call runs the prefixes (wide items where a group's rows fill
// more than one query tile) and the requests' own rows (decode_attn.cu where a
// request has 16 rows at most) into partial results, which a last kernel joins.
//
// Rows of K and V outside a request's run never matter: scores past the last
// key are replaced before use, and the rows of the last V tile past the end
// are zeroed in shared memory before the product reads them (0 * NaN).
//
// Every wait is bounded; on expiry the kernel raises CSA2_DERR_TIMEOUT,
// drains its copies and products, frees TMEM and returns.
#include "dense.cuh"

namespace csa2 {
namespace dense {
namespace {

constexpr int kMaxSplits = 16;
constexpr uint32_t kMiscBytes = 1792;  // barriers and items, behind the tiles

struct AttnParams {
  Seqs seqs;
  int n_heads, n_kv, group, tpt, causal;
  int splits;        // of the key range; 0: the output itself is written
  float *part_o, *part_lse;      // partial results (dense.cuh)
  float scale_log2;
  void *out;         // [num_q, n_heads, D]
  float *lse;        // [num_q, n_heads] or null
  // shared-prefix call: rows of requests in no group get -inf in the prefix
  // part's statistics
  const int32_t *cover;
  int n_cover, cover_splits;
  float *cover_lse;
  int32_t *d_err;
  uint64_t wait_ns;
};

template <int D>
struct Cfg {
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kQTile = (D / 64) * kBlk;
  static constexpr uint32_t kStage = (D / 64) * kBlk;
  static constexpr uint32_t kOffRing = 2 * kQTile;
  static constexpr uint32_t kOffMisc = kOffRing + kStages * kStage;
  static constexpr uint32_t kSmem = kOffMisc + kMiscBytes;
  // two warpgroups of softmax; MMA, producer and item warp in a third one, which
  // gives most of its registers to them: 168 to a thread at launch, and the
  // sum stays
  static constexpr int kThreads = 3 * 128;
  static constexpr int kRegsSoftmax = 224;
  static constexpr int kRegsRest = 56;
  static_assert(2 * kRegsSoftmax + kRegsRest <= 3 * 168, "registers");
  static constexpr uint32_t kTmemCols = 512;
  // columns: S tiles (128 each; P over the first 64), then O tiles (D each)
  static constexpr uint32_t kColO = 2 * 128;
  static_assert(kSmem <= 232448, "shared memory");
};
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

template <int kStages>
struct Misc {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, q_empty, aux, s_full[2], p_full[2][2], o_full[2], done, clc;
  uint64_t item_full[kItems], item_empty[kItems];
  Bound bd;
  uint32_t tmem;
  uint64_t loaded, stat_full, stat_empty;
  alignas(16) uint64_t next[2];      // answer to the request for another CTA's work
  Item item[kItems];
  float2 stat[kTile];                // narrow items: reference and sum of stream 1's rows
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

// The item of CTA `cta` of the grid, by one warp; run = -1 if it has no work.
template <bool kNarrow>
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
      seq_keys(P.seqs, i0 + lane, start, m, err);
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
template <bool kNarrow, typename M>
__device__ void item_role(const AttnParams &P, M *ms) {
  const int lane = threadIdx.x & 31;
  uint32_t asked = 0, items = 0;
  bool ok = true, more = true, waiting = false;
  int err = 0;
  const Shares shares = count_items(P, kNarrow ? P.tpt : 2 * P.tpt, err);
  uint32_t cta = blockIdx.x;
  Item it;
  while (ok && more) {
    find_item<kNarrow>(P, cta, shares, it, err);
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

// Producer warp: an item's Q, then its K and V tiles through the ring.
template <int D, bool kNarrow, typename M>
__device__ void producer_role(const AttnParams &P, uint8_t *smem, M *ms, const CUtensorMap *mq,
                              const CUtensorMap *mk, const CUtensorMap *mv) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  uint32_t g = 0, nq = 0, naux = 0;     // uses so far
  bool ok = true, tail_open = false;
  for (uint32_t u = 0; ok; ++u) {
    if (!(ok = wait_all(&ms->item_full[u % kItems], (u / kItems) & 1, &ms->bd))) break;
    const Item cur = ms->item[u % kItems];
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms->item_empty[u % kItems]);
    if (cur.run < 0) break;
    if (cur.nk <= 0) {
      if (lane == 0) mbar_arrive(&ms->loaded);
      continue;
    }
    if (!(ok = wait_all(&ms->q_empty, (nq & 1) ^ 1, &ms->bd))) break;
    if (lane == 0) {
      const uint32_t box = (uint32_t)P.tpt * P.group * 128u;
      mbar_arrive_expect_tx(&ms->q_full, box * (D / 64) * cur.ntile);
      for (int t = 0; t < cur.ntile; ++t)
        for (int c = 0; c < D / 64; ++c)
          tma_load_3d(smem + t * C::kQTile + c * kBlk, mq, c * 64, cur.h * P.group,
                      cur.q0 + cur.tok0 + t * P.tpt, &ms->q_full);
    }
    ++nq;
    // narrow items take their key tiles in pairs: K, K, V, V
    constexpr int pair = kNarrow ? 2 : 1;
    for (int k0 = 0; k0 < cur.nk && ok; k0 += pair) {
      const int both = min(pair, cur.nk - k0);
      for (int x = 0; x < 2 * both; ++x, ++g) {
        const int kv = x >= both, kt = cur.kt0 + k0 + (kv ? x - both : x);
        const int64_t left = cur.m - (int64_t)kt * kTile;  // keys of this tile
        const uint32_t s = g % C::kStages, ph = (g / C::kStages) & 1;
        uint8_t *st = smem + C::kOffRing + s * C::kStage;
        if (!(ok = wait_all(&ms->empty[s], ph ^ 1, &ms->bd))) break;
        const bool tail = kv == 1 && left < kTile;
        if (lane == 0) {
          uint64_t *bar = tail ? &ms->aux : &ms->full[s];
          mbar_arrive_expect_tx(bar, C::kStage);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(st + c * kBlk, kv ? mv : mk, c * 64, cur.h,
                        (int)(cur.start + (int64_t)kt * kTile), bar);
        }
        if (tail) {
          // rows past the end are zeroed once the copy has landed
          __syncwarp();
          tail_open = true;
          if (!(ok = wait_all(&ms->aux, naux & 1, &ms->bd))) break;
          tail_open = false;
          ++naux;
          for (int i = (int)left * 8 + lane; i < kTile * 8; i += 32)
            for (int c = 0; c < D / 64; ++c)
              *reinterpret_cast<uint4 *>(st + c * kBlk + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->full[s]);
        }
      }
    }
    if (lane == 0) mbar_arrive(&ms->loaded);
  }
  // every copy has to land before the CTA leaves (the products wait for all
  // of them, but not once a wait has run out)
  if (lane == 0) {
    if (nq) drain_bar(&ms->q_full, (nq - 1) & 1);
    if (tail_open) drain_bar(&ms->aux, naux & 1);
    for (uint32_t i = g > (uint32_t)C::kStages ? g - C::kStages : 0; i < g; ++i)
      drain_bar(&ms->full[i % C::kStages], (i / C::kStages) & 1);
  }
  __syncwarp();
}

// One warp issues every product.
template <typename T, int D, bool kNarrow, typename M>
__device__ void mma_role(uint8_t *smem, M *ms) {
  using C = Cfg<D>;
  constexpr uint32_t kIdS = idesc_of<T>(kTile, kTile, false);
  constexpr uint32_t kIdO = idesc_of<T>(kTile, D, true);
  const uint32_t tmem = uniform(ms->tmem);
  const uint64_t ring_k = make_desc_sw128(smem_u32(smem + C::kOffRing), 16, 1024);
  const uint64_t ring_v = make_desc_sw128(smem_u32(smem + C::kOffRing), kBlk, 1024);
  const uint64_t qd = make_desc_sw128(smem_u32(smem), 16, 1024);
  uint32_t s0 = 0, p0 = 0;          // ring stage and phase of the next tile to take
  uint32_t pq = 0, pp = 0;          // phases of Q, and of P by stream (a bit each)
  // ring stage (low bits) and phase (bit 8) of the tile `n` further on
  auto at = [&](uint32_t s, uint32_t p, uint32_t n) {
    s += n;
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
      wait_inline(&ms->q_full, pq, &ms->bd);
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

// Softmax of one item's stream t and its output; one row to a thread.  False if
// a wait ran out.
template <typename T, int D, bool kNarrow, typename M>
__device__ bool softmax_item(const AttnParams &P, M *ms, const Item &it, int t, uint32_t &ps,
                             uint32_t &po, uint32_t &pst) {
  using C = Cfg<D>;
  const int x = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int tok = x / P.group;
  const int i = it.tok0 + (kNarrow ? 0 : t * P.tpt) + tok;     // token of the run
  const bool valid = tok < P.tpt && i < it.n;
  const bool rows_here = __any_sync(0xffffffffu, valid);
  const uint32_t lane_addr = (uint32_t)(32 * warp) << 16;
  const uint32_t ts = ms->tmem + t * 128 + lane_addr, to = ms->tmem + C::kColO + t * D + lane_addr;
  // keys this row sees: j <= last (rows without a token are never masked:
  // what they hold goes nowhere)
  const int last = !valid ? 0x7fffffff
                          : (int)(P.causal ? it.m - it.n + i : it.m - 1);
  const int min_last = __reduce_min_sync(0xffffffffu, last);
  // bf16 P keeps the reference at the maximum (at most 2^8 below it); f16 P
  // is scaled up by 2^8 on top of that, so that weights down to 2^-22 of the
  // largest keep full precision and the largest stays below 2^16
  constexpr float kLift = Elem<T>::kBf16 ? 0.f : 8.f;
  constexpr float kMargin = Elem<T>::kBf16 ? 8.f : 7.f;
  const uint64_t scale2 = pack2(P.scale_log2, P.scale_log2);
  float ref = -INFINITY, sum = 0.f;
  bool ok = true;
  const int steps = it.steps[t], stride = kNarrow ? 2 : 1;
  int kt = it.kt0 + (kNarrow ? t : 0);
  for (int j = 0; j < steps; ++j, kt += stride) {
    // the warp goes on or gives up as one: with a lane gone, the votes and TMEM
    // loads below would wait for it
    if (!(ok = wait_all(&ms->s_full[t], ps, &ms->bd))) break;
    ps ^= 1;
    if (!rows_here) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        mbar_arrive(&ms->p_full[t][0]);
        mbar_arrive(&ms->p_full[t][1]);
      }
      continue;
    }
    fence_after_sync();
    uint32_t s[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32x32b_x32(ts + 32 * c, s[c]);
    tmem_wait_ld();
    if (kt * kTile + kTile - 1 > min_last) {
      const int vis = last - kt * kTile;      // columns <= vis are seen
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (32 * c + e > vis) s[c][e] = 0xff800000u;
    }
    float m4[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      m4[c] = fmaxf(__uint_as_float(s[c][0]), __uint_as_float(s[c][1]));
#pragma unroll
      for (int e = 2; e < 32; e += 2)
        m4[c] = max3(m4[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
    }
    const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * P.scale_log2;
    const bool move = mx > ref + (kLift + kMargin);
    if (__any_sync(0xffffffffu, move)) {
      const float nref = move ? mx - kLift : ref;
      const float alpha = move ? ex2(ref - nref) : 1.f;     // ref = -inf: 0
      ref = nref;
      sum *= alpha;
      if (j > 0) {
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t o[32];
          tmem_ld32x32b_x16(to + 16 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32x32b_x16(to + 16 * c, o);
        }
      }
    }
    const float sub = ref == -INFINITY ? 0.f : ref;
    const uint64_t sub2 = pack2(-sub, -sub);
    uint64_t part[2] = {pack2(sum, 0.f), 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t p[32];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 x = unpack2(fma2(pack2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                      scale2, sub2));
        const float a = ex2(x.x), b = ex2(x.y);
        part[(e >> 1) & 1] = add2(part[(e >> 1) & 1], pack2(a, b));
        p[e / 2] = Elem<T>::pack(a, b);
      }
      tmem_st32x32b_x16(ts + 16 * c, p);
      if (c & 1) {                 // 64 keys written: their product may start
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->p_full[t][c >> 1]);
      }
    }
    const float2 part2 = unpack2(add2(part[0], part[1]));
    sum = part2.x + part2.y;
  }
  const bool any = steps > 0;
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
  if (P.splits > 0) {
    const int64_t rows = part_rows(P.seqs.num_q, P.group);
    const int64_t at = (int64_t)(it.q0 + i) * P.group + x % P.group;
    if (valid) {
      P.part_lse[part_stat(rows, P.n_kv, it.split, it.h, at)] = lse;
      if (it.uncovered && it.split == 0)
        for (int s = 0; s < P.cover_splits; ++s)
          P.cover_lse[part_stat(rows, P.n_kv, s, it.h, at)] = -INFINITY;
    }
    if (rows_here && any) {
      float *dst = P.part_o + part_elem(rows, P.n_kv, D, it.split, it.h, at);
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

// Items one after another, as the producer publishes them.
template <typename T, int D, bool kNarrow, typename M>
__device__ void softmax_role(const AttnParams &P, M *ms) {
  const int t = threadIdx.x >> 7;
  uint32_t ps = 0, po = 0, pst = 0;      // phases of S, O and the statistics
  for (uint32_t u = 0;; ++u) {
    const uint32_t slot = u % kItems;
    if (!wait_all(&ms->item_full[slot], (u / kItems) & 1, &ms->bd)) return;
    // the item stays in shared memory until its output is written: registers
    // are short
    const Item &it = ms->item[slot];
    if (it.run < 0) return;
    if ((kNarrow || t < it.ntile) && !softmax_item<T, D, kNarrow>(P, ms, it, t, ps, po, pst))
      return;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->item_empty[slot]);
  }
}

template <typename T, int D, bool kNarrow>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
dense_attn_kernel(const __grid_constant__ AttnParams P, const __grid_constant__ CUtensorMap mq,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<D>;
  using M = Misc<C::kStages>;
  static_assert(sizeof(M) <= kMiscBytes, "misc region");
  extern __shared__ __align__(1024) uint8_t smem[];
  M *ms = reinterpret_cast<M *>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5;
  if (warp == kMmaWarp) {
    tmem_alloc(&ms->tmem, C::kTmemCols);
    tmem_relinquish();
  } else if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&ms->full[i], 1);
      mbar_init(&ms->empty[i], 1);
    }
    mbar_init(&ms->q_full, 1);
    mbar_init(&ms->q_empty, 1);
    mbar_init(&ms->aux, 1);
    mbar_init(&ms->done, 1);
    mbar_init(&ms->clc, 1);
    mbar_init(&ms->loaded, 1);
    mbar_init(&ms->stat_full, 4);
    mbar_init(&ms->stat_empty, 4);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ms->s_full[t], 1);
      mbar_init(&ms->p_full[t][0], 4);
      mbar_init(&ms->p_full[t][1], 4);
      mbar_init(&ms->o_full[t], 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&ms->item_full[i], 1);
      mbar_init(&ms->item_empty[i], 8 + 2);          // softmax, MMA and producer warps
    }
    ms->bd.abort = 0;
    ms->bd.wait_ns = P.wait_ns;
    mbar_fence_init();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    if (warp == kProducerWarp)
      producer_role<D, kNarrow>(P, smem, ms, &mq, &mk, &mv);
    else if (warp == kMmaWarp)
      mma_role<T, D, kNarrow>(smem, ms);
    else if (warp == kItemWarp)
      item_role<kNarrow>(P, ms);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    softmax_role<T, D, kNarrow>(P, ms);
  }
  fence_before_sync();
  __syncthreads();
  // launched early, this kernel reads nothing of the one in front, but is not done
  // before it: what comes behind waits for this one only
  wait_front();
  if (threadIdx.x == 0 && ms->bd.abort) raise_err(P.d_err, CSA2_DERR_TIMEOUT);
  if (warp == kMmaWarp) {
    fence_after_sync();
    tmem_dealloc(ms->tmem, C::kTmemCols);
  }
}

// Joins the parts of a row: lse = ln sum_s e^{lse_s}, out = sum_s
// e^{lse_s - lse} out_s.  A block has 32 packed rows of a key head, a lane to a
// row, a warp to a sixteenth of the channels; parts without keys (-inf) are not
// read.  Rows that no request holds are left: nobody wrote their parts.  The
// requests' own parts, those from `own` on, say so where they ran by
// decode_attn.cu; otherwise (kLook) it takes a look at every request, since cu_q
// may be malformed.
template <typename T, int D, bool kLook>
__global__ void __launch_bounds__(512)
merge_kernel(const float *__restrict__ part_o, const float *__restrict__ part_lse, int parts,
             int own, int num_q, int n_kv, int group, const int32_t *__restrict__ cu_q, int num_req,
             T *__restrict__ out, float *__restrict__ lse) {
  constexpr int kCh = D / 16, kBatch = 4;
  __shared__ __align__(16) T tile[32][D + 8];
  __shared__ float weight[2 * kMaxSplits][32];
  __shared__ uint32_t held[16];          // by warp: bit i: row0 + i is a request's row
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const int64_t rows = part_rows(num_q, group), row0 = (int64_t)blockIdx.x * 32;
  const int64_t row = row0 + lane;
  const float *po = part_o + part_elem(rows, n_kv, D, 0, h, row) + warp * kCh * 32;
  uint32_t theirs = 0;
  for (int r = threadIdx.x; kLook && r < num_req; r += 512) {
    const int lo = cu_q[r], hi = cu_q[r + 1];
    if (lo < 0 || lo > hi || hi > num_q) continue;
    const int64_t a = max((int64_t)lo * group - row0, (int64_t)0);
    const int64_t b = min((int64_t)hi * group - row0, (int64_t)32);
    if (a < b) theirs |= (0xffffffffu >> (32 - (int)b)) & (0xffffffffu << (int)a);
  }
  wait_front();                          // the batch was there before the kernels in front
  for (int s = warp; s < parts; s += 16)
    weight[s][lane] = part_lse[part_stat(rows, n_kv, s, h, row)];
  if (kLook) {
    theirs = __reduce_or_sync(0xffffffffu, theirs);
    if (lane == 0) held[warp] = theirs;
  }
  __syncthreads();
  theirs = kLook
               ? __reduce_or_sync(0xffffffffu, held[lane & 15])
               : __ballot_sync(0xffffffffu, row < (int64_t)num_q * group &&
                                                __float_as_uint(weight[own][lane]) != kNobody);
  const bool mine = (theirs >> lane) & 1;
  if (theirs != 0xffffffffu) {           // the same in every warp
    __syncthreads();
    for (int s = warp; s < parts; s += 16)
      if (!mine) weight[s][lane] = -INFINITY;
    __syncthreads();
  }
  float top = -INFINITY, tot = 0.f;
  bool nan = false;
  for (int s = 0; s < parts; ++s) {
    const float l = weight[s][lane];
    nan |= l != l;
    top = fmaxf(top, l);
  }
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[kCh] = {};
  for (int s0 = 0; s0 < parts; s0 += kBatch) {       // the batch's loads all in flight
    float v[kBatch][kCh], w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      w[u] = s0 + u < parts ? ex2((weight[s0 + u][lane] - ref) * 1.4426950408889634f) : 0.f;
      const float *src = po + (int64_t)(s0 + u) * n_kv * rows * D;
#pragma unroll
      for (int d = 0; d < kCh; ++d) v[u][d] = w[u] != 0.f ? src[d * 32] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      tot += w[u];
#pragma unroll
      for (int d = 0; d < kCh; ++d) acc[d] = fmaf(w[u], v[u][d], acc[d]);
    }
  }
  const float inv = tot > 0.f || nan ? 1.f / tot : 0.f;
#pragma unroll
  for (int d = 0; d < kCh; d += 2)
    *reinterpret_cast<uint32_t *>(&tile[lane][warp * kCh + d]) =
        Elem<T>::pack(acc[d] * inv, acc[d + 1] * inv);
  const int64_t heads = (int64_t)n_kv * group;
  if (warp == 0 && mine && lse)
    lse[row / group * heads + (int64_t)h * group + row % group] =
        tot > 0.f || nan ? ref + log2f(tot) * 0.6931471805599453f : -INFINITY;
  __syncthreads();
  constexpr int kVec = D / 8;            // 16-byte pieces of a row
  for (int i = threadIdx.x; i < 32 * kVec; i += 512) {
    const int64_t r = row0 + i / kVec;
    if (!((theirs >> (i / kVec)) & 1)) continue;
    const int64_t at = r / group * heads + (int64_t)h * group + r % group;
    *reinterpret_cast<uint4 *>(out + at * D + (i % kVec) * 8) =
        *reinterpret_cast<const uint4 *>(&tile[i / kVec][(i % kVec) * 8]);
  }
}

template <typename T, int D, bool kNarrow>
int launch(const AttnParams &P, int items, bool early, const CUtensorMap (&m)[3],
           cudaStream_t st) {
  using C = Cfg<D>;
  allow_smem<dense_attn_kernel<T, D, kNarrow>>((int)C::kSmem);
  return launch_behind(dense_attn_kernel<T, D, kNarrow>, dim3((unsigned)items), C::kThreads,
                       (int)C::kSmem, early, st, P, m[0], m[1], m[2]);
}

template <typename T>
int launch_any(const Shape &s, const AttnParams &P, bool narrow, int items, bool early,
               const CUtensorMap (&m)[3], cudaStream_t st) {
  if (s.dim == 128)
    return narrow ? launch<T, 128, true>(P, items, early, m, st)
                  : launch<T, 128, false>(P, items, early, m, st);
  return narrow ? launch<T, 64, true>(P, items, early, m, st)
                : launch<T, 64, false>(P, items, early, m, st);
}

struct Cache {
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv, kv_rows;
};

// Tokens of a query tile for runs of `avg` rows on average: a tile no longer
// than they are, so that single tokens do not fetch their neighbours' queries
int tile_tokens(int64_t num_q, int64_t runs, int group) {
  const int most = kTile / group;
  int t = 1;
  while (t < most && (int64_t)t * runs < num_q) t *= 2;
  return t < most ? t : most;
}

int run_attn(const Shape &s, const Cache &c, const AttnParams &P, bool narrow, bool early,
             cudaStream_t st) {
  // an upper bound of the items, since the lengths are on the device
  const int64_t tok = narrow ? P.tpt : 2 * P.tpt;
  const int64_t items =
      (P.seqs.num_q / tok + P.seqs.count) * s.n_kv * (P.splits > 0 ? P.splits : 1);
  if (items > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  CUtensorMap m[3];
  const bool none = c.kv_rows == 0;   // no key row is ever fetched then
  if (!make_rows_map(&m[0], s.bf16, c.q, P.seqs.num_q, s.n_heads, s.dim, c.ldq, s.group, P.tpt) ||
      !make_rows_map(&m[1], s.bf16, none ? c.q : c.k, none ? 1 : c.kv_rows, s.n_kv, s.dim,
                     none ? c.ldq : c.ldk, 1, kTile) ||
      !make_rows_map(&m[2], s.bf16, none ? c.q : c.v, none ? 1 : c.kv_rows, s.n_kv, s.dim,
                     none ? c.ldq : c.ldv, 1, kTile))
    return CSA2_ERR_UNSUPPORTED;
  return s.bf16 ? launch_any<__nv_bfloat16>(s, P, narrow, (int)items, early, m, st)
                : launch_any<__half>(s, P, narrow, (int)items, early, m, st);
}

int check_cache(const csa2_packed *b, const Shape &s, const Cache &c) {
  int st = check_rows(c.q, c.ldq, s.n_heads, s.dim);
  if (st == CSA2_OK && c.kv_rows > 0) st = check_rows(c.k, c.ldk, s.n_kv, s.dim);
  if (st == CSA2_OK && c.kv_rows > 0) st = check_rows(c.v, c.ldv, s.n_kv, s.dim);
  return st;
}

// Whether an output or the workspace meets an input or another of them.  The
// outputs may take q's place: every item reads its own query rows before it writes
// them, and what it reads of others' goes nowhere.
bool outputs_meet(const csa2_packed *b, const csa2_prefix_groups *g, const Shape &s, const Cache &c,
                  const void *out, const void *lse, const void *ws, int64_t ws_bytes) {
  const int64_t wq = (int64_t)s.n_heads * s.dim * 2, wk = (int64_t)s.n_kv * s.dim * 2;
  const uint64_t no = (uint64_t)b->num_q * wq, nl = (uint64_t)b->num_q * s.n_heads * 4;
  const auto meets = [&](const void *p, uint64_t n, bool q_too) {
    return meets_batch(p, n, b) || meets_groups(p, n, g) ||
           meets_rows(p, n, c.k, c.kv_rows, c.ldk * 2, wk) ||
           meets_rows(p, n, c.v, c.kv_rows, c.ldv * 2, wk) ||
           (q_too && meets_rows(p, n, c.q, b->num_q, c.ldq * 2, wq));
  };
  const bool in_place = out == c.q && (c.ldq * 2 == wq || b->num_q == 1);
  return meets(out, no, !in_place) || meets(lse, nl, true) ||
         (ws && meets(ws, (uint64_t)ws_bytes, true)) || (lse && overlap(out, no, lse, nl)) ||
         (ws && (overlap(ws, (uint64_t)ws_bytes, out, no) ||
                 (lse && overlap(ws, (uint64_t)ws_bytes, lse, nl))));
}

// Single tokens of few heads go by decode_attn.cu; other runs whose rows fill no
// more than one query tile are narrow items.
enum Kind { kWideItems, kNarrowItems, kSingleTokens };

Kind kind_of(int64_t num_q, int64_t runs, int tpt, int group, bool single) {
  if (single && tpt == 1 && group <= kDecodeGroup) return kSingleTokens;
  return num_q <= runs * tpt ? kNarrowItems : kWideItems;
}

// Splits of `items` items unsplit on `places` places, of `steps` steps each: the
// waves' length in steps, `fixed` steps of fixed cost to an item, and half a
// step to a split for the join.
int plan_splits(int64_t items, int places, int64_t steps, double fixed) {
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= kMaxSplits && s <= (steps > 0 ? steps : 1); ++s) {
    const int64_t waves = (items * s + places - 1) / places;
    const double c = (double)waves * ((double)((steps + s - 1) / s) + fixed) + 0.5 * s;
    if (c < cost) cost = c, best = s;
  }
  return best;
}

struct PartPlan {
  int tpt, splits;
  Kind kind;
};

PartPlan plan_part(const Shape &s, int64_t num_q, int64_t runs, int64_t most, bool single) {
  PartPlan p;
  p.tpt = tile_tokens(num_q, runs, s.group);
  p.kind = kind_of(num_q, runs, p.tpt, s.group, single);
  const int64_t tok = p.kind == kWideItems ? 2 * p.tpt : p.tpt;
  const int64_t items = (num_q / tok > runs ? num_q / tok : runs) * s.n_kv;
  const int64_t tiles = most / kTile + (most % kTile != 0);
  if (p.kind == kSingleTokens)       // three CTAs to an SM, 64 keys a step
    p.splits = plan_splits(items, 3 * kSms, 2 * tiles, 4.0);
  else
    p.splits = plan_splits(items, kSms, p.kind == kNarrowItems ? (tiles + 1) / 2 : tiles, 3.0);
  return p;
}

struct PrefixPlan {
  PartPlan pre, own;
};

PrefixPlan plan_prefix(const Shape &s, int64_t num_q, int64_t num_req, int64_t num_groups,
                       int64_t max_prefix, int64_t max_kv) {
  PrefixPlan p{};
  p.own = plan_part(s, num_q, num_req > 0 ? num_req : 1, max_kv, true);
  if (num_groups > 0) p.pre = plan_part(s, num_q, num_groups, max_prefix, false);
  return p;
}

// One part of an attention call; early: behind single tokens' part.
int run_part(const Shape &s, const Cache &c, AttnParams &P, const PartPlan &p, bool early,
             cudaStream_t st) {
  P.tpt = p.tpt;
  if (p.kind != kSingleTokens) return run_attn(s, c, P, p.kind == kNarrowItems, early, st);
  const DecodeParams D{P.seqs,   c.q,     c.k,      c.v,        c.ldq,       c.ldk,
                       c.ldv,    P.n_heads, P.n_kv, P.group,    P.splits,    P.scale_log2,
                       P.out,    P.lse,   P.part_o, P.part_lse, P.cover,     P.n_cover,
                       P.cover_splits, P.cover_lse, P.d_err};
  return decode_attn(s, D, st);
}

int64_t part_bytes(int64_t num_q, const Shape &s) {
  return part_rows(num_q, s.group) * s.n_kv * (s.dim + 1) * 4;
}

// Cuts the splits down to `parts` parts in all, the more split side first; false
// if there is not one to each side.  (The best number of splits goes up and down
// with the batch, so that a workspace for the largest batch may be short of what
// a smaller one would like.)
bool fit_splits(PrefixPlan *p, int64_t parts) {
  int &pre = p->pre.splits, &own = p->own.splits;
  while (pre + own > parts) {
    int &most = pre > own ? pre : own;
    if (most == 1) return false;
    --most;
  }
  return true;
}

}  // namespace
}  // namespace dense
}  // namespace csa2

using namespace csa2::dense;

extern "C" CSA2_API int csa2_prompt_attn(const csa2_packed *b, int32_t n_heads,
                                         int32_t n_kv_heads, int32_t dim, int32_t dtype,
                                         const void *q, int64_t ldq, const void *k, int64_t ldk,
                                         const void *v, int64_t ldv, int64_t kv_rows,
                                         float sm_scale, void *out, float *lse, int32_t *d_err,
                                         csa2_stream_t stream) {
  Shape s;
  int st = check_packed(b, n_heads, n_kv_heads, dim, dtype, kv_rows, sm_scale, &s);
  if (st != CSA2_OK) return st;
  if (b->num_q == 0 || b->num_req == 0) return CSA2_OK;
  const Cache c{q, k, v, ldq, ldk, ldv, kv_rows};
  if (!out) return CSA2_ERR_INVALID_ARG;
  if ((st = check_cache(b, s, c)) != CSA2_OK) return st;
  if (!csa2::aligned(16, out) || !csa2::aligned(4, lse, d_err)) return CSA2_ERR_UNSUPPORTED;
  if (outputs_meet(b, nullptr, s, c, out, lse, nullptr, 0)) return CSA2_ERR_INVALID_ARG;
  AttnParams P{};
  P.seqs = Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, b->kv_start, b->kv_len,
                kv_rows};
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  P.causal = 1;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.out = out;
  P.lse = lse;
  P.d_err = d_err;
  P.wait_ns = csa2::wait_limit_ns();
  return run_part(s, c, P, plan_part(s, b->num_q, b->num_req, 0, true), false,
                  csa2::as_stream(stream));
}

extern "C" CSA2_API int csa2_prefix_attn_workspace(int32_t num_q, int32_t num_req,
                                                   int32_t num_groups, int32_t n_heads,
                                                   int32_t n_kv_heads, int32_t dim,
                                                   int64_t max_prefix, int64_t max_kv,
                                                   int64_t *bytes) {
  if (!bytes || num_q < 0 || num_req < 0 || num_groups < 0 || max_prefix < 0 || max_kv < 0)
    return CSA2_ERR_INVALID_ARG;
  Shape s;
  const csa2_packed b{};
  const int st = check_packed(&b, n_heads, n_kv_heads, dim, CSA2_DT_BF16, 0, 1.f, &s);
  if (st != CSA2_OK) return st;
  const PrefixPlan p = plan_prefix(s, num_q, num_req, num_groups, max_prefix, max_kv);
  *bytes = (p.pre.splits + p.own.splits) * part_bytes(num_q, s);
  return CSA2_OK;
}

extern "C" CSA2_API int csa2_prefix_attn(const csa2_packed *b, const csa2_prefix_groups *g,
                                         int32_t n_heads, int32_t n_kv_heads, int32_t dim,
                                         int32_t dtype, const void *q, int64_t ldq, const void *k,
                                         int64_t ldk, const void *v, int64_t ldv, int64_t kv_rows,
                                         int64_t max_kv, float sm_scale, void *out, float *lse,
                                         void *workspace, int64_t workspace_bytes, int32_t *d_err,
                                         csa2_stream_t stream) {
  Shape s;
  int st = check_packed(b, n_heads, n_kv_heads, dim, dtype, kv_rows, sm_scale, &s);
  if (st != CSA2_OK) return st;
  const int ng = g ? g->num_groups : 0;
  if (ng < 0 || max_kv < 0) return CSA2_ERR_INVALID_ARG;
  if (ng > 0 && (g->max_prefix < 0 || !g->cu_group || !g->prefix_start || !g->prefix_len))
    return CSA2_ERR_INVALID_ARG;
  if (b->num_q == 0 || b->num_req == 0) return CSA2_OK;
  const Cache c{q, k, v, ldq, ldk, ldv, kv_rows};
  if (!out) return CSA2_ERR_INVALID_ARG;
  if ((st = check_cache(b, s, c)) != CSA2_OK) return st;
  if (!csa2::aligned(16, out) || !csa2::aligned(4, lse, d_err)) return CSA2_ERR_UNSUPPORTED;
  if (ng > 0 &&
      !(csa2::aligned(4, g->cu_group) && csa2::aligned(8, g->prefix_start, g->prefix_len)))
    return CSA2_ERR_UNSUPPORTED;
  PrefixPlan p = plan_prefix(s, b->num_q, b->num_req, ng, ng ? g->max_prefix : 0, max_kv);
  if (!workspace || !fit_splits(&p, workspace_bytes / part_bytes(b->num_q, s)))
    return CSA2_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 255u) return CSA2_ERR_UNSUPPORTED;
  // (of the workspace, what the parts take)
  if (outputs_meet(b, g, s, c, out, lse, workspace,
                   (p.pre.splits + p.own.splits) * part_bytes(b->num_q, s)))
    return CSA2_ERR_INVALID_ARG;
  const cudaStream_t cs = csa2::as_stream(stream);
  const int parts = p.pre.splits + p.own.splits;
  const int64_t rows = part_rows(b->num_q, s.group) * s.n_kv;
  float *part_o = static_cast<float *>(workspace);
  float *part_lse = part_o + parts * rows * s.dim;
  AttnParams P{};
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.d_err = d_err;
  P.wait_ns = csa2::wait_limit_ns();
  // The requests' own rows, then the groups' prefixes: single tokens wait for
  // memory and run out unevenly, and the prefixes, whose time goes into products,
  // start on the SMs that they leave (48 requests in two groups 45.7 -> 35.9 us,
  // 256 requests 324 -> 318).
  P.seqs = Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, b->kv_start, b->kv_len,
                kv_rows};
  P.causal = 1;
  P.splits = p.own.splits;
  P.part_o = part_o + p.pre.splits * rows * s.dim;
  P.part_lse = part_lse + p.pre.splits * rows;
  if (ng > 0) {
    P.cover = g->cu_group;
    P.n_cover = ng;
    P.cover_splits = p.pre.splits;
    P.cover_lse = part_lse;
  }
  if ((st = run_part(s, c, P, p.own, false, cs)) != CSA2_OK) return st;
  if (ng > 0) {
    P.seqs = Seqs{ng, b->num_q, b->num_req, b->cu_q, g->cu_group, g->prefix_start, g->prefix_len,
                  kv_rows};
    P.causal = 0;
    P.splits = p.pre.splits;
    P.part_o = part_o;
    P.part_lse = part_lse;
    P.cover = nullptr;
    if ((st = run_part(s, c, P, p.pre, p.own.kind == kSingleTokens, cs)) != CSA2_OK) return st;
  }
  const int64_t blocks = part_rows(b->num_q, s.group) / 32;
  if (blocks > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  auto merge = [&](auto *o, auto dim_c) {
    using T = std::remove_pointer_t<decltype(o)>;
    constexpr int D = decltype(dim_c)::value;
    return launch_behind(
        p.own.kind == kSingleTokens ? merge_kernel<T, D, false> : merge_kernel<T, D, true>,
        dim3((unsigned)blocks, (unsigned)s.n_kv), 512, 0, true, cs, part_o, part_lse, parts,
        p.pre.splits, b->num_q, s.n_kv, s.group, b->cu_q, b->num_req, o, lse);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (s.bf16)
    return s.dim == 128 ? merge(static_cast<__nv_bfloat16 *>(out), D128{})
                        : merge(static_cast<__nv_bfloat16 *>(out), D64{});
  return s.dim == 128 ? merge(static_cast<__half *>(out), D128{})
                      : merge(static_cast<__half *>(out), D64{});
}
