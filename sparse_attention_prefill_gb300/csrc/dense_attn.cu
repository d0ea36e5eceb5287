// Dense grouped-head attention over a K/V cache on the 5th-generation tensor
// cores: whole prompts and extends (csa2_prompt_attn), and batches that share
// prefixes (csa2_prefix_attn).
//
// Per query row x = (token, head) with keys j <= last(x):
//   l_j = c <q_x, k_j>,  out = sum_j e^{l_j} v_j / sum_j e^{l_j},
//   lse = ln sum_j e^{l_j}.
//
// An item is kNT query tiles of 128 packed rows (dense.cuh) of one key head,
// walked over in key tiles of 128 keys:
//   S[t] = Q[t] K^T     (both operands in shared memory, S in TMEM)
//   O[t] += P[t] V      (P in TMEM over S's columns, V in shared memory)
// The softmax holds one row to a thread: it reads its row of S, keeps a
// reference maximum that moves only when a logit passes it by a margin (then
// the thread rescales its row of O; the products of that row are complete by
// then, since S of this step was issued after them), and writes P rounded to
// the inputs' type.  Row sums are taken of the unrounded P in fp32.
//
// The MMA warp issues, for each key tile j and query tile t, O[t](j) and
// then S[t](j+1): while one tile's softmax runs, the other tile's products
// keep the tensor pipe busy (kNT = 2), or those of the second CTA of the SM
// do (kNT = 1).  The grid has a CTA to an item, but a CTA that runs takes the
// items of CTAs that have not started, so that an item's output overlaps the
// loads and first products of the next.
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
constexpr uint32_t kMiscBytes = 640;   // barriers and items, behind the tiles

struct AttnParams {
  Seqs seqs;
  int n_heads, n_kv, group, tpt, causal, splits;
  float scale_log2;
  void *out;         // [num_q, n_heads, D]  (splits == 0)
  float *lse;        // [num_q, n_heads] or null
  float *part_o;     // [splits, num_q, n_heads, D]  (splits > 0)
  float *part_lse;   // [splits, num_q, n_heads]
  // own part of a shared-prefix call: rows of requests in no group get -inf
  // in the prefix part's statistics
  const int32_t *cover;
  int n_cover, cover_splits;
  float *cover_lse;
  int32_t *d_err;
  uint64_t wait_ns;
};

template <int D, int NT>
struct Cfg {
  static constexpr int kStages = D == 128 ? (NT == 2 ? 5 : 2) : (NT == 2 ? 8 : 5);
  static constexpr uint32_t kQTile = (D / 64) * kBlk;
  static constexpr uint32_t kStage = (D / 64) * kBlk;
  static constexpr uint32_t kOffRing = NT * kQTile;
  static constexpr uint32_t kOffMisc = kOffRing + kStages * kStage;
  static constexpr uint32_t kSmem = kOffMisc + kMiscBytes;
  // one warpgroup of softmax to a query tile; MMA and producer warp in a third
  // (second) one, which gives most of its registers to them: 168 to a thread
  // at launch (NT = 2) or 128 (NT = 1), the sum stays
  static constexpr int kThreads = (NT + 1) * 128;
  static constexpr int kRegsSoftmax = NT == 2 ? 224 : 208;
  static constexpr int kRegsRest = NT == 2 ? 56 : 48;
  static_assert(NT * kRegsSoftmax + kRegsRest <= (NT + 1) * (NT == 2 ? 168 : 128), "registers");
  static constexpr uint32_t kTmemCols = NT == 2 ? 512 : 256;
  // columns: S tiles (128 each; P over the first 64), then O tiles (D each)
  static constexpr uint32_t kColO = NT * 128;
  static_assert(kSmem <= 232448, "shared memory");
};

struct Item {
  int run, q0, n, tok0;      // run (-1: no work, -2: no more items), its first query row and
                             // rows, first token of the item
  int h, split;
  int64_t start;             // first cache row
  int64_t m;                 // cache rows
  int kt0, kt1;              // key tiles
  int nkt[2];                // key tiles that query tile t needs (end, <= kt1)
  int ntile;                 // query tiles with tokens
  int uncovered;             // a request in no group (own part of a shared-prefix call)
};

template <int kStages>
struct Misc {
  uint64_t full[kStages], empty[kStages];
  uint64_t q_full, q_empty, aux, s_full[2], p_full[2][2], o_full[2], done, clc;
  uint64_t item_full[2], item_empty[2];
  Bound bd;
  uint32_t tmem;
  alignas(16) uint64_t next[2];      // answer to the request for another CTA's work
  Item item[2];
};
// The item of CTA `cta` of the grid, by one warp; run = -1 if it has no work.
template <int NT>
__device__ void find_item(const AttnParams &P, uint32_t cta, Item &it) {
  const int ns = P.splits > 0 ? P.splits : 1, tok_cta = NT * P.tpt;
  const int split = it.split = (int)(cta % ns);
  it.h = (int)(cta / ns % P.n_kv);
  const int slot = (int)(cta / ns / P.n_kv);
  const int lane = threadIdx.x & 31;
  int base = 0, err = 0, run = -1, tile = 0, q0 = 0, n = 0;
  for (int i0 = 0; i0 < P.seqs.count; i0 += 32) {
    int a = 0, c = 0;
    if (i0 + lane < P.seqs.count) seq_rows(P.seqs, i0 + lane, a, c, err);
    const int nt_i = (c + tok_cta - 1) / tok_cta;
    int inc = nt_i;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, slot < base + inc);
    if (hit) {
      const int src = __ffs(hit) - 1;
      run = i0 + src;
      // the longest key ranges first
      tile = __shfl_sync(0xffffffffu, base + inc, src) - 1 - slot;
      q0 = __shfl_sync(0xffffffffu, a, src);
      n = __shfl_sync(0xffffffffu, c, src);
      break;
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  it.run = run;
  if (run >= 0) {
    it.q0 = q0;
    it.n = n;
    it.tok0 = tile * tok_cta;
    seq_keys(P.seqs, run, it.start, it.m, err);
    const int ntok = min(tok_cta, n - it.tok0);
    it.ntile = (ntok + P.tpt - 1) / P.tpt;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int last_tok = min(it.tok0 + (t + 1) * P.tpt, n) - 1;
      const int64_t last = P.causal ? it.m - n + last_tok : it.m - 1;
      it.nkt[t] = t < it.ntile && last >= 0 ? (int)(last / kTile) + 1 : 0;
    }
    const int total = NT == 2 ? max(it.nkt[0], it.nkt[NT - 1]) : it.nkt[0];
    if (P.splits > 0) {
      const int per = (total + P.splits - 1) / P.splits;
      it.kt0 = min(total, split * per);
      it.kt1 = min(total, it.kt0 + per);
    } else {
      it.kt0 = 0;
      it.kt1 = total;
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) it.nkt[t] = min(it.nkt[t], it.kt1);
    it.uncovered = 0;
    if (P.cover) {
      bool mine = false;
      for (int g = lane; g < P.n_cover; g += 32)
        mine |= P.cover[g] >= 0 && P.cover[g] <= run && run < P.cover[g + 1] &&
                P.cover[g + 1] <= P.seqs.num_req;
      it.uncovered = !__any_sync(0xffffffffu, mine);
    }
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane == 0) raise_err(P.d_err, err);
}

// Producer warp.  Takes this CTA's item, then those of CTAs of the grid that
// have not started (cluster launch control: the hardware hands out their
// indices), looks each up while the loads of the item in front are under way,
// and publishes it; then Q, and K and V tiles through the ring.
template <int D, int NT, typename M>
__device__ void producer_role(const AttnParams &P, uint8_t *smem, M *ms, Item cur,
                              const CUtensorMap *mq, const CUtensorMap *mk,
                              const CUtensorMap *mv) {
  using C = Cfg<D, NT>;
  const int lane = threadIdx.x & 31;
  uint32_t g = 0, nq = 0, naux = 0, nclc = 0, items = 0;     // uses so far
  bool ok = true, asked = false, tail_open = false;
  auto publish = [&](const Item &it) {
    const uint32_t s = items & 1;
    ok = wait_all(&ms->item_empty[s], ((items >> 1) & 1) ^ 1, &ms->bd);
    if (ok && lane == 0) {
      ms->item[s] = it;
      mbar_arrive(&ms->item_full[s]);
    }
    __syncwarp();
    ++items;
  };
  bool more = true;
  while (ok && more) {
    if (lane == 0) {
      mbar_arrive_expect_tx(&ms->clc, 16);
      ask_next(ms->next, &ms->clc);
    }
    asked = true;
    Item nxt;
    bool looked = false;
    auto look_ahead = [&]() {
      looked = true;
      ok = wait_all(&ms->clc, nclc & 1, &ms->bd);
      if (!ok) return;
      ++nclc;
      asked = false;
      uint32_t cta;
      more = next_cta(ms->next, cta);
      fence_proxy_async_smem();      // the next answer is written by the async proxy
      __syncwarp();
      if (more) find_item<NT>(P, cta, nxt);
    };
    if (cur.run >= 0) publish(cur);
    if (ok && cur.run >= 0 && cur.kt0 < cur.kt1) {
      ok = wait_all(&ms->q_empty, (nq & 1) ^ 1, &ms->bd);
      if (ok && lane == 0) {
        const uint32_t box = (uint32_t)P.tpt * P.group * 128u;
        mbar_arrive_expect_tx(&ms->q_full, box * (D / 64) * cur.ntile);
        for (int t = 0; t < cur.ntile; ++t)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(smem + t * C::kQTile + c * kBlk, mq, c * 64, cur.h * P.group,
                        cur.q0 + cur.tok0 + t * P.tpt, &ms->q_full);
      }
      if (ok) ++nq;
      int loads = 0;
      for (int kt = cur.kt0; kt < cur.kt1 && ok; ++kt) {
        const int row = (int)(cur.start + (int64_t)kt * kTile);
        const int64_t left = cur.m - (int64_t)kt * kTile;    // keys of this tile
        for (int kv = 0; kv < 2; ++kv, ++g) {
          if (loads++ == C::kStages) look_ahead();           // the ring is full
          if (!ok) break;
          const uint32_t s = g % C::kStages, ph = (g / C::kStages) & 1;
          uint8_t *st = smem + C::kOffRing + s * C::kStage;
          if (!(ok = wait_all(&ms->empty[s], ph ^ 1, &ms->bd))) break;
          const bool tail = kv == 1 && left < kTile;
          if (lane == 0) {
            uint64_t *bar = tail ? &ms->aux : &ms->full[s];
            mbar_arrive_expect_tx(bar, C::kStage);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(st + c * kBlk, kv ? mv : mk, c * 64, cur.h, row, bar);
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
    }
    if (ok && !looked) look_ahead();
    if (ok && more) cur = nxt;
  }
  if (ok) {
    Item end{};
    end.run = -2;
    publish(end);
  }
  // every copy has to land before the CTA leaves (the products wait for all
  // of them, but not once a wait has run out)
  if (lane == 0) {
    if (asked) drain_bar(&ms->clc, nclc & 1);
    if (nq) drain_bar(&ms->q_full, (nq - 1) & 1);
    if (tail_open) drain_bar(&ms->aux, naux & 1);
    for (uint32_t i = g > (uint32_t)C::kStages ? g - C::kStages : 0; i < g; ++i)
      drain_bar(&ms->full[i % C::kStages], (i / C::kStages) & 1);
  }
  __syncwarp();
}

// One warp issues every product.
template <typename T, int D, int NT, typename M>
__device__ void mma_role(uint8_t *smem, M *ms) {
  using C = Cfg<D, NT>;
  constexpr uint32_t kIdS = idesc_of<T>(kTile, kTile, false);
  constexpr uint32_t kIdO = idesc_of<T>(kTile, D, true);
  const uint32_t tmem = uniform(ms->tmem);
  const uint64_t ring_k = make_desc_sw128(smem_u32(smem + C::kOffRing), 16, 1024);
  const uint64_t ring_v = make_desc_sw128(smem_u32(smem + C::kOffRing), kBlk, 1024);
  const uint64_t qd = make_desc_sw128(smem_u32(smem), 16, 1024);
  // products of S[t] with the K tile of a ring stage, by the elected lane
  auto issue_s = [&](int t, uint32_t stage) {
    const uint64_t b = desc_add(ring_k, stage * C::kStage);
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k >> 2) * kBlk + (k & 3) * 32;
      mma_f16(tmem + t * 128, desc_add(qd, t * C::kQTile + off), desc_add(b, off), kIdS, k > 0);
    }
    mma_commit(&ms->s_full[t]);
  };
  uint32_t s0 = 0, p0 = 0;          // ring stage and phase of the next tile to take
  uint32_t pq = 0, pp = 0;          // phases of Q, and of P by query tile (a bit each)
  for (uint32_t u = 0;; ++u) {
    if (!wait_all(&ms->item_full[u & 1], (u >> 1) & 1, &ms->bd)) break;
    const Item &it = ms->item[u & 1];
    const int run = uniform(it.run), kt0 = uniform(it.kt0), nk = uniform(it.kt1) - kt0;
    int end[NT];                    // key tiles of query tile t, counted from kt0
#pragma unroll
    for (int t = 0; t < NT; ++t) end[t] = uniform(it.nkt[t]) - kt0;
    if (elect_one()) mbar_arrive(&ms->item_empty[u & 1]);
    __syncwarp();
    if (run < 0) break;
    if (nk <= 0) continue;
    if (elect_one()) {
      wait_inline(&ms->q_full, pq, &ms->bd);
      wait_inline(&ms->full[s0], p0, &ms->bd);
      fence_after_sync();
#pragma unroll
      for (int t = 0; t < NT; ++t)
        if (end[t] > 0) issue_s(t, s0);
      mma_commit(&ms->empty[s0]);
      if (nk == 1) mma_commit(&ms->q_empty);
    }
    __syncwarp();
    pq ^= 1;
    uint32_t sv = s0 + 1, pv = p0;  // V(j)
    if (sv == C::kStages) sv = 0, pv ^= 1;
    bool ok = true;
    for (int j = 0; j < nk && ok; ++j) {
      // once a wait has run out nothing waits any more, and the products of
      // the step at hand read whatever is there
      ok = uniform(*(volatile int *)&ms->bd.abort) == 0;
      uint32_t sk = sv + 1, pk = pv;                 // K(j + 1)
      if (sk == C::kStages) sk = 0, pk ^= 1;
      const bool more = j + 1 < nk;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if (ok && j < end[t]) {
          const uint64_t b = desc_add(ring_v, sv * C::kStage);
          // The waits lie between the products that they hold back: the
          // tensor pipe has some four products queued meanwhile.
          if (elect_one()) {
            wait_inline(&ms->full[sv], pv, &ms->bd);
#pragma unroll
            for (int half = 0; half < 2; ++half) {   // P arrives in halves of 64 keys
              wait_inline(&ms->p_full[t][half], (pp >> t) & 1, &ms->bd);
              fence_after_sync();
#pragma unroll
              for (int k = 4 * half; k < 4 * half + 4; ++k)
                mma_f16_ts(tmem + C::kColO + t * D, tmem + t * 128 + k * 8, desc_add(b, k * 2048),
                           kIdO, j > 0 || k > 0);
            }
            if (j + 1 < end[t]) {
              wait_inline(&ms->full[sk], pk, &ms->bd);
              issue_s(t, sk);
            } else {
              mma_commit(&ms->o_full[t]);
            }
            if (t == NT - 1 || j >= end[NT - 1]) {
              mma_commit(&ms->empty[sv]);
              if (more) mma_commit(&ms->empty[sk]);
              if (j + 2 == nk) mma_commit(&ms->q_empty);   // the item's last S
            }
          }
          __syncwarp();
          pp ^= 1u << t;
        }
      }
      if (more) {
        sv = sk + 1, pv = pk;
        if (sv == C::kStages) sv = 0, pv ^= 1;
      }
    }
    if (!ok) break;
    s0 = sv + 1, p0 = pv;
    if (s0 == C::kStages) s0 = 0, p0 ^= 1;
  }
  if (elect_one()) mma_commit(&ms->done);          // TMEM is not freed under a running product
  __syncwarp();
  drain_bar(&ms->done, 0);
}

// Softmax of one item's query tile t and its output; one row to a thread.
// False if a wait ran out.
template <typename T, int D, int NT, typename M>
__device__ bool softmax_item(const AttnParams &P, M *ms, const Item &it, int t, uint32_t &ps,
                             uint32_t &po) {
  using C = Cfg<D, NT>;
  const int x = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int tok = x / P.group;
  const int i = it.tok0 + t * P.tpt + tok;                 // token of the run
  const bool valid = tok < P.tpt && i < it.n;
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
  const int kt_end = it.nkt[t];
  int j = 0;
  for (int kt = it.kt0; kt < kt_end; ++kt, ++j) {
    if (!(ok = wait_bar(&ms->s_full[t], ps, &ms->bd))) break;
    ps ^= 1;
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
  const bool any = it.kt0 < kt_end;
  if (ok && any) ok = wait_bar(&ms->o_full[t], po, &ms->bd);
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) return false;
  if (any) po ^= 1;
  fence_after_sync();
  const bool seen = any && !(sum == 0.f);       // a NaN sum stays a NaN
  const float inv = seen ? 1.f / sum : 0.f;
  const float lse =
      seen ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
  const int64_t row = (int64_t)(it.q0 + i) * P.n_heads + it.h * P.group + x % P.group;
  const int64_t rows = (int64_t)P.seqs.num_q * P.n_heads;
  if (valid) {
    if (P.splits > 0) {
      P.part_lse[it.split * rows + row] = lse;
      if (it.uncovered && it.split == 0)
        for (int s = 0; s < P.cover_splits; ++s) P.cover_lse[s * rows + row] = -INFINITY;
    } else if (P.lse) {
      P.lse[row] = lse;
    }
  }
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t o[32];
    if (any) {
      tmem_ld32x32b_x32(to + 32 * c, o);
      tmem_wait_ld();
    }
    if (!seen)
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = 0;
    if (!valid) continue;
    if (P.splits > 0) {
      if (!seen) continue;
      float4 *dst = reinterpret_cast<float4 *>(P.part_o + (it.split * rows + row) * D + 32 * c);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                             __uint_as_float(o[4 * e + 2]) * inv,
                             __uint_as_float(o[4 * e + 3]) * inv);
    } else {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(P.out) + row * D + 32 * c);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          w[u] = Elem<T>::pack(__uint_as_float(o[8 * e + 2 * u]) * inv,
                               __uint_as_float(o[8 * e + 2 * u + 1]) * inv);
        dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  fence_before_sync();      // O is read: the next item's first product may overwrite it
  return true;
}

// Items one after another, as the producer publishes them.
template <typename T, int D, int NT, typename M>
__device__ void softmax_role(const AttnParams &P, M *ms) {
  const int t = threadIdx.x >> 7;
  uint32_t ps = 0, po = 0;          // phases of S and O
  for (uint32_t u = 0;; ++u) {
    if (!wait_all(&ms->item_full[u & 1], (u >> 1) & 1, &ms->bd)) return;
    // the item stays in shared memory until its output is written: registers
    // are short
    const Item &it = ms->item[u & 1];
    if (it.run < 0) return;
    if (t < it.ntile && !softmax_item<T, D, NT>(P, ms, it, t, ps, po)) return;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->item_empty[u & 1]);
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, NT == 1 ? 2 : 1)
dense_attn_kernel(AttnParams P, const __grid_constant__ CUtensorMap mq,
                  const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<D, NT>;
  using M = Misc<C::kStages>;
  static_assert(sizeof(M) <= kMiscBytes, "misc region");
  extern __shared__ __align__(1024) uint8_t smem[];
  M *ms = reinterpret_cast<M *>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5;
  Item first;
  if (warp == 4 * NT + 1) {
    find_item<NT>(P, blockIdx.x, first);
  } else if (warp == 4 * NT) {
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
    for (int t = 0; t < 2; ++t) {
      mbar_init(&ms->s_full[t], 1);
      mbar_init(&ms->p_full[t][0], 4);
      mbar_init(&ms->p_full[t][1], 4);
      mbar_init(&ms->o_full[t], 1);
      mbar_init(&ms->item_full[t], 1);
      mbar_init(&ms->item_empty[t], 4 * NT + 1);     // softmax warps, MMA warp
    }
    ms->bd.abort = 0;
    ms->bd.wait_ns = P.wait_ns;
    mbar_fence_init();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  if (warp >= 4 * NT) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    if (warp == 4 * NT + 1)
      producer_role<D, NT>(P, smem, ms, first, &mq, &mk, &mv);
    else if (warp == 4 * NT)
      mma_role<T, D, NT>(smem, ms);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    softmax_role<T, D, NT>(P, ms);
  }
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && ms->bd.abort) raise_err(P.d_err, CSA2_DERR_TIMEOUT);
  if (warp == 4 * NT) {
    fence_after_sync();
    tmem_dealloc(ms->tmem, C::kTmemCols);
  }
}

// Joins the parts of a row: lse = ln sum_s e^{lse_s}, out = sum_s
// e^{lse_s - lse} out_s.  One warp per (query row, head); parts without keys
// (-inf) are not read.  Rows in front of or behind the sequences are left.
template <typename T, int D>
__global__ void __launch_bounds__(256)
merge_kernel(const float *__restrict__ part_o, const float *__restrict__ part_lse, int parts,
             int num_q, int n_heads, const int32_t *__restrict__ cu_q, int num_req,
             T *__restrict__ out, float *__restrict__ lse) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = (int64_t)num_q * n_heads;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int q = (int)(row / n_heads);
  if (q < cu_q[0] || q >= cu_q[num_req]) return;
  float mx = -INFINITY, l = lane < parts ? part_lse[lane * rows + row] : -INFINITY;
  bool nan = l != l;
  mx = l;
#pragma unroll
  for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  nan = __any_sync(0xffffffffu, nan);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float w = ex2((l - ref) * 1.4426950408889634f);
  float tot = w;
#pragma unroll
  for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
  const float inv = tot > 0.f || nan ? 1.f / tot : 0.f;
  w *= inv;
  constexpr int V = D / 32;
  float acc[V] = {};
  for (int s = 0; s < parts; ++s) {
    const float ws = __shfl_sync(0xffffffffu, w, s);
    if (__shfl_sync(0xffffffffu, l, s) == -INFINITY) continue;
    const float *src = part_o + (s * rows + row) * D + lane * V;
    float v[V];
    if (V == 4) {
      const float4 f = *reinterpret_cast<const float4 *>(src);
      v[0] = f.x, v[1] = f.y, v[V - 2] = f.z, v[V - 1] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2 *>(src);
      v[0] = f.x, v[1] = f.y;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = fmaf(ws, v[e], acc[e]);
  }
  T *dst = out + row * D + lane * V;
#pragma unroll
  for (int e = 0; e < V; e += 2)
    *reinterpret_cast<uint32_t *>(dst + e) = Elem<T>::pack(acc[e], acc[e + 1]);
  if (lane == 0 && lse)
    lse[row] = tot > 0.f || nan ? (ref + log2f(tot) * 0.6931471805599453f) : -INFINITY;
}

template <typename T, int D, int NT>
int launch(const AttnParams &P, int slots, const CUtensorMap &mq, const CUtensorMap &mk,
           const CUtensorMap &mv, cudaStream_t st) {
  using C = Cfg<D, NT>;
  const int64_t grid = (int64_t)slots * P.n_kv * (P.splits > 0 ? P.splits : 1);
  if (grid > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  allow_smem<dense_attn_kernel<T, D, NT>>((int)C::kSmem);
  dense_attn_kernel<T, D, NT><<<(int)grid, C::kThreads, C::kSmem, st>>>(P, mq, mk, mv);
  return launch_status();
}

template <int NT>
int launch_any(const Shape &s, const AttnParams &P, int slots, const CUtensorMap &mq,
               const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st) {
  if (s.bf16)
    return s.dim == 128 ? launch<__nv_bfloat16, 128, NT>(P, slots, mq, mk, mv, st)
                        : launch<__nv_bfloat16, 64, NT>(P, slots, mq, mk, mv, st);
  return s.dim == 128 ? launch<__half, 128, NT>(P, slots, mq, mk, mv, st)
                      : launch<__half, 64, NT>(P, slots, mq, mk, mv, st);
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

int run_attn(const Shape &s, const Cache &c, AttnParams &P, bool two, cudaStream_t st) {
  const int tok = P.tpt * (two ? 2 : 1);
  const int64_t slots = P.seqs.num_q / tok + P.seqs.count;
  if (slots > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  CUtensorMap mq, mk, mv;
  const bool none = c.kv_rows == 0;   // no key row is ever fetched then
  if (!make_rows_map(&mq, s.bf16, c.q, P.seqs.num_q, s.n_heads, s.dim, c.ldq, s.group, P.tpt) ||
      !make_rows_map(&mk, s.bf16, none ? c.q : c.k, none ? 1 : c.kv_rows, s.n_kv, s.dim,
                     none ? c.ldq : c.ldk, 1, kTile) ||
      !make_rows_map(&mv, s.bf16, none ? c.q : c.v, none ? 1 : c.kv_rows, s.n_kv, s.dim,
                     none ? c.ldq : c.ldv, 1, kTile))
    return CSA2_ERR_UNSUPPORTED;
  return two ? launch_any<2>(s, P, (int)slots, mq, mk, mv, st)
             : launch_any<1>(s, P, (int)slots, mq, mk, mv, st);
}

int check_cache(const csa2_packed *b, const Shape &s, const Cache &c) {
  int st = check_rows(c.q, c.ldq, s.n_heads, s.dim);
  if (st == CSA2_OK && c.kv_rows > 0) st = check_rows(c.k, c.ldk, s.n_kv, s.dim);
  if (st == CSA2_OK && c.kv_rows > 0) st = check_rows(c.v, c.ldv, s.n_kv, s.dim);
  return st;
}

// Splits of a part with `items` CTAs unsplit on `slots` places and `tiles`
// key tiles each: the waves' length in key tiles, 3 tiles of fixed cost to a
// CTA, and half a tile to a split for the join.
int plan_splits(int64_t items, int slots, int64_t tiles) {
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= kMaxSplits && s <= (tiles > 0 ? tiles : 1); ++s) {
    const int64_t waves = (items * s + slots - 1) / slots;
    const double c = (double)waves * ((double)((tiles + s - 1) / s) + 3.0) + 0.5 * s;
    if (c < cost) cost = c, best = s;
  }
  return best;
}

struct PrefixPlan {
  int tpt_pre, tpt_own, splits_pre, splits_own;
  bool two_pre;
};

PrefixPlan plan_prefix(const Shape &s, int64_t num_q, int64_t num_req, int64_t num_groups,
                       int64_t max_prefix, int64_t max_kv) {
  PrefixPlan p{};
  p.tpt_own = tile_tokens(num_q, num_req > 0 ? num_req : 1, s.group);
  const int64_t own_items = (num_q / p.tpt_own > num_req ? num_q / p.tpt_own : num_req) * s.n_kv;
  p.splits_own = plan_splits(own_items, 2 * kSms, (max_kv + kTile - 1) / kTile);
  if (num_groups > 0) {
    p.tpt_pre = tile_tokens(num_q, num_groups, s.group);
    const int64_t tiles = num_q / p.tpt_pre > num_groups ? num_q / p.tpt_pre : num_groups;
    // two query tiles to a CTA halve the traffic of the shared keys; with a
    // single tile to a group the second would be empty
    p.two_pre = num_q > num_groups * p.tpt_pre;
    const int64_t items = (p.two_pre ? (tiles + 1) / 2 : tiles) * s.n_kv;
    p.splits_pre = plan_splits(items, p.two_pre ? kSms : 2 * kSms,
                               (max_prefix + kTile - 1) / kTile);
  }
  return p;
}

int64_t plan_bytes(const PrefixPlan &p, int64_t num_q, const Shape &s) {
  return (int64_t)(p.splits_pre + p.splits_own) * num_q * s.n_heads * (s.dim + 4) * 4 + 256;
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
  if ((uintptr_t)out & 15u) return CSA2_ERR_UNSUPPORTED;
  AttnParams P{};
  P.seqs = Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, b->kv_start, b->kv_len,
                kv_rows};
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  P.tpt = tile_tokens(b->num_q, b->num_req, s.group);
  P.causal = 1;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.out = out;
  P.lse = lse;
  P.d_err = d_err;
  P.wait_ns = csa2::wait_limit_ns();
  // one tile to a CTA where a request's rows fill no more than one
  const bool two = (int64_t)b->num_req * P.tpt < b->num_q;
  return run_attn(s, c, P, two, csa2::as_stream(stream));
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
  *bytes = plan_bytes(plan_prefix(s, num_q, num_req, num_groups, max_prefix, max_kv), num_q, s);
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
  if ((uintptr_t)out & 15u) return CSA2_ERR_UNSUPPORTED;
  const PrefixPlan p =
      plan_prefix(s, b->num_q, b->num_req, ng, ng ? g->max_prefix : 0, max_kv);
  if (!workspace || workspace_bytes < plan_bytes(p, b->num_q, s)) return CSA2_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 255u) return CSA2_ERR_UNSUPPORTED;
  const cudaStream_t cs = csa2::as_stream(stream);
  const int parts = p.splits_pre + p.splits_own;
  const int64_t rows = (int64_t)b->num_q * s.n_heads;
  float *part_o = static_cast<float *>(workspace);
  float *part_lse = part_o + parts * rows * s.dim;
  AttnParams P{};
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.d_err = d_err;
  P.wait_ns = csa2::wait_limit_ns();
  if (ng > 0) {
    P.seqs = Seqs{ng, b->num_q, b->num_req, b->cu_q, g->cu_group, g->prefix_start, g->prefix_len,
                  kv_rows};
    P.tpt = p.tpt_pre;
    P.causal = 0;
    P.splits = p.splits_pre;
    P.part_o = part_o;
    P.part_lse = part_lse;
    if ((st = run_attn(s, c, P, p.two_pre, cs)) != CSA2_OK) return st;
    P.cover = g->cu_group;
    P.n_cover = ng;
    P.cover_splits = p.splits_pre;
    P.cover_lse = part_lse;
  }
  P.seqs = Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, b->kv_start, b->kv_len,
                kv_rows};
  P.tpt = p.tpt_own;
  P.causal = 1;
  P.splits = p.splits_own;
  P.part_o = part_o + p.splits_pre * rows * s.dim;
  P.part_lse = part_lse + p.splits_pre * rows;
  if ((st = run_attn(s, c, P, false, cs)) != CSA2_OK) return st;
  const int64_t grid = (rows + 7) / 8;
  if (grid > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  auto merge = [&](auto *o, auto dim_c) {
    merge_kernel<std::remove_pointer_t<decltype(o)>, decltype(dim_c)::value>
        <<<(int)grid, 256, 0, cs>>>(part_o, part_lse, parts, b->num_q, s.n_heads, b->cu_q,
                                    b->num_req, o, lse);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  if (s.bf16)
    s.dim == 128 ? merge(static_cast<__nv_bfloat16 *>(out), D128{})
                 : merge(static_cast<__nv_bfloat16 *>(out), D64{});
  else
    s.dim == 128 ? merge(static_cast<__half *>(out), D128{})
                 : merge(static_cast<__half *>(out), D64{});
  return csa2::launch_status();
}
