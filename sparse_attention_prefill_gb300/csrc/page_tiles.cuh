// Attention over 8-bit pages on the 5th-generation tensor cores (csa2_page_attn):
// prompts, extends, and single tokens of more than 16 heads to a key head.
//
// Items, streams and products are those of dense_attn.cu, with codes for K and V and
// the scales of page_attn.cuh in the softmax.  Both products take f16 operands, in
// which codes are exact, as are bf16 queries times a power of two for each row.
// (Products of the codes themselves would need the queries and weights in 8 bits: two
// products for what two codes of a query hold, and a weight of 4 bits is too coarse.)
// So the roles are, 16 warps to a CTA:
//   0-7    softmax, a row of a query tile to a thread;
//   8      issues the products;
//   9      producer: TMA copies of Q, and of the pages' codes into a ring of raw tiles;
//          it also looks up the pages and writes the scales of each tile's 16-key groups;
//   10     hands out items;
//   12-15  converters, a key to a thread: a raw tile to an f16 tile in the products'
//          swizzle, rows behind the last and rows without a page as zeros (0 * NaN);
//          an item's bf16 queries, where they are.
// A step of 128 keys (D = 128) has 2 x 16384 codes: some 250 instructions to a
// converter thread, a tenth of what the SM can issue while the products run.
//
// Many items are handed out as in dense_attn.cu; where they are few, CTAs take equal runs of
// all their tiles (page_runs.cuh), and a second kernel joins the parts of items that were
// cut: 19 extends of 32 tokens over some ten thousand rows (152 items) take 185 us and would
// take 220 whole.  With 256 items both take the same, since parts have to be written and
// joined; beyond that items even out by themselves.
//
// Every wait is bounded; on expiry the kernel raises CSA2_DERR_TIMEOUT, drains its
// copies and products, frees TMEM and returns.
#pragma once
#include "dense_roles.cuh"
#include "page_runs.cuh"

namespace csa2 {
namespace pages {
namespace {

constexpr int kGroups = 8;           // 16-key groups of a tile, each within a page
constexpr int kSlots = 8;            // tiles whose scales are kept (see the producer)
constexpr int kConvertWarp = 12;

template <int D_>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int kStages = D == 128 ? 3 : 6;     // f16 tiles
  static constexpr int kRaw = D == 128 ? 3 : 6;        // tiles of codes
  static constexpr uint32_t kQTile = (D / 64) * kBlk;
  static constexpr uint32_t kStage = (D / 64) * kBlk;
  static constexpr uint32_t kRawStage = kTile * D;
  static constexpr uint32_t kOffRing = 2 * kQTile;
  static constexpr uint32_t kOffRaw = kOffRing + kStages * kStage;
  static constexpr uint32_t kOffMisc = kOffRaw + kRaw * kRawStage;
  static_assert(kStages + kRaw <= 12, "scales");
  static constexpr int kThreads = 4 * 128;
  // 128 registers to a thread at launch, and the sum stays
  static constexpr int kRegsSoftmax = 200;
  static constexpr int kRegsRest = 56;
  static constexpr int kRegsConvert = 56;
  static_assert(2 * kRegsSoftmax + kRegsRest + kRegsConvert <= 4 * 128, "registers");
  static constexpr uint32_t kTmemCols = 512;
  static constexpr uint32_t kColO = 2 * 128;
};

// Scales of a key tile's groups: a (times c of the softmax), log2 b and 1 / b; log2 b =
// -inf where there is no page.
struct TileScales {
  float a[kGroups], lb[kGroups], ib[kGroups];
};

template <int D>
struct Misc {
  using C = Cfg<D>;
  uint64_t full[C::kStages], empty[C::kStages];
  uint64_t raw_full[C::kRaw], raw_empty[C::kRaw], scales_full[kSlots];
  uint64_t q_full, q_ready, q_empty, s_full[2], p_full[2][2], o_full[2], done, clc;
  uint64_t item_full[kItems], item_empty[kItems];
  Bound bd;
  uint32_t tmem;
  uint64_t loaded, stat_full, stat_empty;
  alignas(16) uint64_t next[2];      // answer to the request for another CTA's work
  Item item[kItems];
  float2 stat[kTile];                // narrow items: reference and sum of stream 1's rows
  alignas(16) TileScales scales[kSlots];
  float unlift[kItems][2 * kTile];   // bf16 queries: what undoes a row's power of two
  int64_t scan[C::kThreads / 32];    // runs of tiles
  Place place;
};

// Few items: a unit is a query tile or a pair of them, a step a key tile.
struct Tiles {
  static constexpr int kFixed = 5;   // tiles' time that an item's start and end take
  static constexpr int kLeast = 4;   // cost of a share, at least
  int tok;                           // tokens of a unit
  __device__ __forceinline__ int units(const Run &u) const { return (u.n + tok - 1) / tok; }
  // key tiles that tokens up to `upto` see
  static __device__ __forceinline__ int tiles(const Run &u, int upto) {
    const int64_t last = u.m - u.n + min(upto, u.n) - 1;
    return last < 0 ? 0 : (int)(last / kTile) + 1;
  }
  // an item that sees nothing has a step, too: its output is written
  __device__ __forceinline__ int steps(const Run &u, int i) const {
    return max(1, tiles(u, (i + 1) * tok));
  }
};

// Publishes a CTA's run of items, as item_role does.
template <bool kNarrow, int D>
__device__ void run_role(const AttnParams &P, Misc<D> *ms, const Plan &plan, TileMark *marks) {
  const int lane = threadIdx.x & 31, share = (int)blockIdx.x;
  const Tiles rule{kNarrow ? P.tpt : 2 * P.tpt};
  const int64_t end = share_begin(plan, share + 1);
  Place p = ms->place;
  if (lane == 0) {
    const int parts = parts_of(rule, plan, share, p);
    TileMark mark{0, 0, 0, 0};
    if (parts)
      mark = TileMark{p.u.lo + p.i * rule.tok, min(rule.tok, p.u.n - p.i * rule.tok), p.h, parts};
    marks[share] = mark;
  }
  uint32_t items = 0;
  bool ok = true;
  for (int64_t at = share_begin(plan, share); at < end;) {
    const int all = rule.steps(p.u, p.i);
    const Steps part = steps_in<Tiles>(p, all, end - at);
    at += Tiles::kFixed + all - p.off;
    if (part.n > 0) {
      Item it{};
      it.run = p.run;
      it.q0 = p.u.lo;
      it.n = p.u.n;
      it.m = p.u.m;
      it.h = p.h;
      it.tok0 = p.i * rule.tok;
      const int t0 = Tiles::tiles(p.u, it.tok0 + P.tpt), t1 = Tiles::tiles(p.u, it.tok0 + 2 * P.tpt);
      it.ntile = min(rule.tok, it.n - it.tok0) > P.tpt ? 2 : 1;
      it.kt0 = part.from;
      it.nk = min(part.n, (kNarrow ? t0 : max(t0, t1)) - part.from);   // (0: sees nothing)
      if (kNarrow) {
        it.steps[0] = (it.nk + 1) / 2;
        it.steps[1] = it.nk / 2;
      } else {
        it.steps[0] = max(0, min(t0 - it.kt0, it.nk));
        it.steps[1] = it.ntile > 1 ? max(0, min(t1 - it.kt0, it.nk)) : 0;
      }
      it.split = part.from > 0            ? 2 * share
                 : part.from + part.n < all ? 2 * share + 1
                                            : -1;
      const uint32_t s = items % kItems;
      ok = wait_all(&ms->item_empty[s], ((items / kItems) & 1) ^ 1, &ms->bd);
      if (!ok) break;
      if (lane == 0) {
        ms->item[s] = it;
        mbar_arrive(&ms->item_full[s]);
      }
      __syncwarp();
      ++items;
    }
    if (at >= end || !next_item(rule, P.seqs, P.n_kv, p)) break;
  }
  if (ok) {
    const uint32_t s = items % kItems;
    ok = wait_all(&ms->item_empty[s], ((items / kItems) & 1) ^ 1, &ms->bd);
    if (ok && lane == 0) {
      ms->item[s].run = -2;
      mbar_arrive(&ms->item_full[s]);
    }
  }
}


template <int D>
constexpr uint32_t smem_bytes() {
  return Cfg<D>::kOffMisc + (uint32_t)sizeof(Misc<D>);
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory");

// Key tile x of an item's k-th pair (narrow) or step, as the order K, K, V, V or K, V
// of the rings goes.
struct Order {
  int both, kt;                      // tiles of this pair; tile of the item
  bool value;
};
template <bool kNarrow>
__device__ __forceinline__ Order order_of(int nk, int k0, int x) {
  const int both = min(kNarrow ? 2 : 1, nk - k0);
  return Order{both, k0 + (x >= both ? x - both : x), x >= both};
}

// Producer warp: an item's Q, then the codes of its K and V tiles, page by page.  A lane
// holds one of 32 neighbouring pages of the request and its scales.
template <int D, bool kNarrow>
__device__ void producer_role(const AttnParams &P, const Pages &C8, uint8_t *smem, Misc<D> *ms,
                              const CUtensorMap *mq, const CUtensorMap *mk,
                              const CUtensorMap *mv) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int per = kTile >> C8.shift;    // pages of a tile
  const uint32_t page_bytes = (uint32_t)C8.page * D;
  uint32_t g = 0, nq = 0, tiles = 0;    // uses so far
  int err = 0;
  bool ok = true;
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
    int id = -1;
    float a = 0.f, b = 0.f;
    const int64_t held = (cur.m + C8.page - 1) >> C8.shift;
    int64_t from = 0;                   // the first of the lanes' pages
    const auto look_up = [&](int64_t p) {
      from = p;
      const bool there = p + lane < held;
      id = there ? page_id(C8, cur.run, p + lane, err) : -1;
      a = id >= 0 ? C8.k_scale[(int64_t)id * P.n_kv + cur.h] : 0.f;
      b = id >= 0 ? C8.v_scale[(int64_t)id * P.n_kv + cur.h] : 0.f;
    };
    look_up((int64_t)cur.kt0 * per);
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
    for (int k0 = 0; k0 < cur.nk && ok; k0 += kNarrow ? 2 : 1) {
      const int both = order_of<kNarrow>(cur.nk, k0, 0).both;
      if ((int64_t)(cur.kt0 + k0 + both) * per > from + 32)
        look_up((int64_t)(cur.kt0 + k0) * per);
      for (int x = 0; x < 2 * both; ++x, ++g) {
        const Order o = order_of<kNarrow>(cur.nk, k0, x);
        const int64_t p0 = (int64_t)(cur.kt0 + o.kt) * per;
        const uint32_t s = g % C::kRaw, ph = (g / C::kRaw) & 1;
        if (!(ok = wait_all(&ms->raw_empty[s], ph ^ 1, &ms->bd))) break;
        const int off = (int)(p0 - from);
        uint8_t *to = smem + C::kOffRaw + s * C::kRawStage;
        uint64_t *bar = &ms->raw_full[s];
        const uint32_t valid =
            __ballot_sync(0xffffffffu, id >= 0 && lane >= off && lane < off + per);
        if (lane == 0) mbar_arrive_expect_tx(bar, page_bytes * __popc(valid));
        __syncwarp();
        if ((valid >> lane) & 1)         // a copy to a lane, which has the page's number
          tma_load_3d(to + (lane - off) * page_bytes, o.value ? mv : mk, 0,
                      (int)((int64_t)cur.h * C8.page * D / 128), id, bar);
        __syncwarp();
        if (!o.value) {
          // scales: the last tile that used this slot is done with.  (The rings let in
          // this tile once the product of the 12th entry before it, or an earlier one,
          // has ended, and the V tiles of eight tiles before lie further back.)
          const uint32_t tile = tiles + o.kt;
          const int src = off + ((lane % kGroups) * 16 >> C8.shift);
          const int gid = __shfl_sync(0xffffffffu, id, src);
          const float ga = __shfl_sync(0xffffffffu, a, src), gb = __shfl_sync(0xffffffffu, b, src);
          if (lane < kGroups) {
            TileScales &ts = ms->scales[tile % kSlots];
            const float sa = gid >= 0 ? scale_of(ga, err) : 0.f;
            const float sb = gid >= 0 ? scale_of(gb, err) : 0.f;
            ts.a[lane] = sa * P.scale_log2;
            ts.lb[lane] = log2f(sb);
            ts.ib[lane] = gid >= 0 ? 1.f / sb : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&ms->scales_full[tile % kSlots]);
        }
      }
    }
    tiles += cur.nk;
    if (lane == 0) mbar_arrive(&ms->loaded);
  }
  // every copy has to land before the CTA leaves
  if (lane == 0) {
    if (nq) drain_bar(&ms->q_full, (nq - 1) & 1);
    for (uint32_t i = g > (uint32_t)C::kRaw ? g - C::kRaw : 0; i < g; ++i)
      drain_bar(&ms->raw_full[i % C::kRaw], (i / C::kRaw) & 1);
  }
  __syncwarp();
  err = __reduce_or_sync(0xffffffffu, err);
  if (lane == 0) raise_err(P.d_err, err);
}

// bf16 queries of row `row` of a tile to f16, in place; what undoes their scaling.
template <int D>
__device__ __forceinline__ float convert_query(uint8_t *tile, int row) {
  uint8_t *line = tile + row * 128;
  float amax = 0.f;
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    const uint4 w = *reinterpret_cast<const uint4 *>(line + (c >> 3) * kBlk +
                                                     (((c & 7) ^ (row & 7)) << 4));
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      amax = max3(amax, fabsf(__uint_as_float(v[i] << 16)),
                  fabsf(__uint_as_float(v[i] & 0xffff0000u)));
  }
  const float lift = lift_of(amax);
#pragma unroll 4
  for (int c = 0; c < D / 8; ++c) {
    uint4 *at = reinterpret_cast<uint4 *>(line + (c >> 3) * kBlk + (((c & 7) ^ (row & 7)) << 4));
    const uint4 w = *at;
    uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = Elem<__half>::pack(__uint_as_float(v[i] << 16) * lift,
                                __uint_as_float(v[i] & 0xffff0000u) * lift);
    *at = make_uint4(v[0], v[1], v[2], v[3]);
  }
  return 1.f / lift;
}

// Converter warps, a row of a tile to a thread.  Eight neighbouring lanes have eight
// rows, whose chunks the swizzles of both tiles lay in different banks.
template <typename T, int D, bool kNarrow>
__device__ void convert_role(uint8_t *smem, Misc<D> *ms) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31, row = threadIdx.x & 127;
  uint32_t g = 0, nq = 0, tiles = 0;
  bool ok = true;
  for (uint32_t u = 0; ok; ++u) {
    const uint32_t slot = u % kItems;
    if (!wait_all(&ms->item_full[slot], (u / kItems) & 1, &ms->bd)) return;
    const Item &it = ms->item[slot];
    const int run = it.run, nk = it.nk, kt0 = it.kt0, ntile = it.ntile;
    const int64_t m = it.m;
    if (run < 0) return;
    if (nk > 0) {
      if (Elem<T>::kBf16) {
        if (!wait_all(&ms->q_full, nq & 1, &ms->bd)) return;
        for (int t = 0; t < ntile; ++t)
          ms->unlift[slot][t * kTile + row] = convert_query<D>(smem + t * C::kQTile, row);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ms->q_ready);
        ++nq;
      }
      for (int k0 = 0; k0 < nk && ok; k0 += kNarrow ? 2 : 1) {
        const int both = order_of<kNarrow>(nk, k0, 0).both;
        for (int x = 0; x < 2 * both; ++x, ++g) {
          const Order o = order_of<kNarrow>(nk, k0, x);
          const uint32_t tile = tiles + o.kt, s = g % C::kStages, r = g % C::kRaw;
          if (!(ok = wait_all(&ms->raw_full[r], (g / C::kRaw) & 1, &ms->bd))) break;
          if (!(ok = wait_all(&ms->scales_full[tile % kSlots], (tile / kSlots) & 1, &ms->bd)))
            break;
          const bool dead = (int64_t)(kt0 + o.kt) * kTile + row >= m ||
                            ms->scales[tile % kSlots].lb[row >> 4] == -INFINITY;
          const uint8_t *raw = smem + C::kOffRaw + r * C::kRawStage;
          uint8_t *to = smem + C::kOffRing + s * C::kStage + row * 128;
          uint4 w[4];
          const auto load = [&](int c0) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int line = D == 128 ? row : row >> 1;
              const int at = D == 128 ? c0 + c : (row & 1) * 4 + c;
              w[c] = *reinterpret_cast<const uint4 *>(raw + line * 128 + ((at ^ (line & 7)) << 4));
              if (dead) w[c] = make_uint4(0, 0, 0, 0);
            }
          };
          load(0);                       // while the stage may still be read
          if (!(ok = wait_all(&ms->empty[s], ((g / C::kStages) & 1) ^ 1, &ms->bd))) break;
#pragma unroll
          for (int c0 = 0; c0 < D / 16; c0 += 4) {
            if (c0) load(c0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint8_t *blk = to + ((c0 + c) >> 2) * kBlk;
              const int at = 2 * ((c0 + c) & 3);
              *reinterpret_cast<uint4 *>(blk + ((at ^ (row & 7)) << 4)) =
                  make_uint4(f16x2_of(w[c].x), f16x2_of_high(w[c].x), f16x2_of(w[c].y),
                             f16x2_of_high(w[c].y));
              *reinterpret_cast<uint4 *>(blk + (((at + 1) ^ (row & 7)) << 4)) =
                  make_uint4(f16x2_of(w[c].z), f16x2_of_high(w[c].z), f16x2_of(w[c].w),
                             f16x2_of_high(w[c].w));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&ms->full[s]);
            mbar_arrive(&ms->raw_empty[r]);
          }
        }
      }
      tiles += nk;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&ms->item_empty[slot]);
  }
}

// Softmax of one item's stream t and its output; one row to a thread.  A page has kG
// columns of a tile or a multiple.  `tiles`: key tiles of the items before.  False if a wait ran out.
template <typename T, int D, bool kNarrow, int kG>
__device__ bool softmax_item(const AttnParams &P, Misc<D> *ms, const Item &it, uint32_t slot,
                             int t, uint32_t tiles, uint32_t &ps, uint32_t &po, uint32_t &pst) {
  using C = Cfg<D>;
  const int x = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
  const int tok = x / P.group;
  const int i = it.tok0 + (kNarrow ? 0 : t * P.tpt) + tok;     // token of the run
  const bool valid = tok < P.tpt && i < it.n;
  const bool rows_here = __any_sync(0xffffffffu, valid);
  const uint32_t lane_addr = (uint32_t)(32 * warp) << 16;
  const uint32_t ts = ms->tmem + t * 128 + lane_addr, to = ms->tmem + C::kColO + t * D + lane_addr;
  // keys this row sees: j <= last (rows without a token are never masked: what they
  // hold goes nowhere)
  const int last = !valid ? 0x7fffffff : (int)(it.m - it.n + i);
  const int min_last = __reduce_min_sync(0xffffffffu, last);
  float ref = -INFINITY, sum = 0.f, unit = 1.f;
  bool ok = true;
  const int steps = it.steps[t], stride = kNarrow ? 2 : 1;
  int kt = kNarrow ? t : 0;              // tile of the item
  for (int j = 0; j < steps; ++j, kt += stride) {
    if (!(ok = wait_all(&ms->s_full[t], ps, &ms->bd))) break;
    ps ^= 1;
    const uint32_t tile = tiles + kt;
    if (!(ok = wait_all(&ms->scales_full[tile % kSlots], (tile / kSlots) & 1, &ms->bd))) break;
    if (!rows_here) {
      __syncwarp();
      if ((threadIdx.x & 31) == 0) {
        mbar_arrive(&ms->p_full[t][0]);
        mbar_arrive(&ms->p_full[t][1]);
      }
      continue;
    }
    fence_after_sync();
    // (S is there, so the queries were converted)
    if (Elem<T>::kBf16 && j == 0) unit = ms->unlift[slot][(kNarrow ? 0 : t * kTile) + x];
    const TileScales &sc = ms->scales[tile % kSlots];
    uint32_t s[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld32x32b_x32(ts + 32 * c, s[c]);
    tmem_wait_ld();
    const int key0 = (it.kt0 + kt) * kTile;
    if (key0 + kTile - 1 > min_last) {
      const int vis = last - key0;       // columns <= vis are seen
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if (32 * c + e > vis) s[c][e] = 0xff800000u;
    }
    // by blocks of kG columns: what S is multiplied by (a factor of 0 would make -inf a
    // NaN), and the largest x
    constexpr int kBlocks = kTile / kG, kEntry = kG / 16;
    float f[kBlocks], mx = -INFINITY;
#pragma unroll
    for (int k = 0; k < kBlocks; ++k) {
      f[k] = fmaxf(sc.a[k * kEntry] * unit, 1e-37f);
      float m4[kG / 16];
#pragma unroll
      for (int e = 0; e < kG; e += 2) {
        const uint32_t *y = &s[(k * kG + e) / 32][(k * kG + e) % 32];
        float &m = m4[e / 16];
        m = e % 16 ? max3(m, __uint_as_float(y[0]), __uint_as_float(y[1]))
                   : fmaxf(__uint_as_float(y[0]), __uint_as_float(y[1]));
      }
      const float mg = kG == 16 ? m4[0] : fmaxf(max3(m4[0], m4[1 % kEntry], m4[2 % kEntry]), m4[3 % kEntry]);
      mx = fmaxf(mx, fmaf(mg, f[k], sc.lb[k * kEntry]));
    }
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
    uint64_t part[2];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t p[32];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const int at = 32 * c + e, k = at / kG;
        const float l = sc.lb[k * kEntry] - sub;
        const float2 v = unpack2(fma2(pack2(__uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1])),
                                      pack2(f[k], f[k]), pack2(l, l)));
        const float a = ex2(v.x), b = ex2(v.y);
        uint64_t &sums = part[(e >> 1) & 1];
        sums = at % kG < 4 ? pack2(a, b) : add2(sums, pack2(a, b));
        p[e / 2] = Elem<__half>::pack(a, b);
        if (at % kG == kG - 2) {
          const float2 both = unpack2(add2(part[0], part[1]));
          sum = fmaf(both.x + both.y, sc.ib[k * kEntry], sum);
        }
      }
      tmem_st32x32b_x16(ts + 16 * c, p);
      if (c & 1) {                 // 64 keys written: their product may start
        tmem_wait_st();
        fence_before_sync();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->p_full[t][c >> 1]);
      }
    }
  }
  return finish_item<T, C, kNarrow, true>(P, ms, it, t, i, ok, steps > 0, valid, rows_here, ref,
                                          sum, to, po, pst);
}

template <typename T, int D, bool kNarrow, int kG>
__device__ void softmax_role(const AttnParams &P, Misc<D> *ms) {
  const int t = threadIdx.x >> 7;
  uint32_t ps = 0, po = 0, pst = 0, tiles = 0;
  for (uint32_t u = 0;; ++u) {
    const uint32_t slot = u % kItems;
    if (!wait_all(&ms->item_full[slot], (u / kItems) & 1, &ms->bd)) return;
    // the item stays in shared memory until its output is written: registers are short
    const Item &it = ms->item[slot];
    if (it.run < 0) return;
    if ((kNarrow || t < it.ntile) &&
        !softmax_item<T, D, kNarrow, kG>(P, ms, it, slot, t, tiles, ps, po, pst))
      return;
    tiles += max(it.nk, 0);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&ms->item_empty[slot]);
  }
}

template <typename T, int D, bool kNarrow, int kG>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
page_attn_kernel(const __grid_constant__ AttnParams P, const __grid_constant__ Pages C8, TileMark *marks,
                 const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<D> *ms = reinterpret_cast<Misc<D> *>(smem + C::kOffMisc);
  const int warp = threadIdx.x >> 5;
  if (warp == kMmaWarp) {
    tmem_alloc(&ms->tmem, C::kTmemCols);
    tmem_relinquish();
  } else if (threadIdx.x == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&ms->full[i], 4);                    // converter warps
      mbar_init(&ms->empty[i], 1);
    }
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&ms->raw_full[i], 1);
      mbar_init(&ms->raw_empty[i], 4);
    }
    for (int i = 0; i < kSlots; ++i) mbar_init(&ms->scales_full[i], 1);
    mbar_init(&ms->q_full, 1);
    mbar_init(&ms->q_ready, 4);
    mbar_init(&ms->q_empty, 1);
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
      mbar_init(&ms->item_empty[i], 8 + 4 + 2);      // softmax, converters, MMA, producer
    }
    ms->bd.abort = 0;
    ms->bd.wait_ns = P.wait_ns;
    mbar_fence_init();
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  Plan plan{};
  if (marks) {
    asm volatile("griddepcontrol.launch_dependents;");
    int err = 0;
    plan = find_share<C::kThreads>(Tiles{kNarrow ? P.tpt : 2 * P.tpt}, P.seqs, P.n_kv, ms->scan,
                                   ms->place, err);
    if (blockIdx.x == 0 && err) raise_err(P.d_err, err);
  }
  if (warp >= kConvertWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsConvert));
    convert_role<T, D, kNarrow>(smem, ms);
  } else if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
    if (warp == kProducerWarp)
      producer_role<D, kNarrow>(P, C8, smem, ms, &mq, &mk, &mv);
    else if (warp == kMmaWarp)
      mma_role<C, idesc_of<__half>(kTile, kTile, false), idesc_of<__half>(kTile, D, true), kNarrow>(
          smem, ms, Elem<T>::kBf16 ? &ms->q_ready : &ms->q_full);
    else if (warp == kItemWarp) {
      if (marks)
        run_role<kNarrow>(P, ms, plan, marks);
      else
        item_role<kNarrow, true>(P, ms);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsSoftmax));
    softmax_role<T, D, kNarrow, kG>(P, ms);
  }
  fence_before_sync();
  __syncthreads();
  if (threadIdx.x == 0 && ms->bd.abort) raise_err(P.d_err, CSA2_DERR_TIMEOUT);
  if (warp == kMmaWarp) {
    fence_after_sync();
    tmem_dealloc(ms->tmem, C::kTmemCols);
  }
}

// Joins the parts of items that shares cut: 32 rows of an item to a block, a lane to a
// row, a warp to a sixteenth of the channels.
template <typename T, int D>
__global__ void __launch_bounds__(512)
page_tiles_join_kernel(const __grid_constant__ AttnParams P, const TileMark *marks, int rows) {
  constexpr int kCh = D / 16, kBatch = 4;
  __shared__ __align__(16) T tile[32][D + 8];
  __shared__ float weight[kSms][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x + 1;
  wait_front();
  const TileMark mark = marks[j];
  const int row0 = (int)blockIdx.y * 32, row = row0 + lane, tok = row % kTile / P.group;
  const int token = row / kTile * P.tpt + tok;           // of the item
  const bool mine = tok < P.tpt && token < mark.tokens;
  const uint32_t theirs = __ballot_sync(0xffffffffu, mine);
  if (mark.parts == 0 || !theirs) return;
  const auto part = [&](int k) {
    return (k == 0 ? 2 * (int64_t)(j - 1) + 1 : 2 * (int64_t)(j - 1 + k)) * rows;
  };
  const float *po = P.part_o + lane + warp * kCh * 32;
  float v[kBatch][kCh];
  const auto fetch = [&](int k0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float *src = po + (part(k0 + u) + row0) * D;
#pragma unroll
      for (int d = 0; d < kCh; ++d) v[u][d] = k0 + u < mark.parts ? src[d * 32] : 0.f;
    }
  };
  fetch(0);                              // together with the statistics
  for (int k = warp; k < mark.parts; k += 16)
    weight[k][lane] = mine ? P.part_lse[part(k) + row] : -INFINITY;
  __syncthreads();
  float top = -INFINITY, tot = 0.f;
  bool nan = false;
  for (int k = 0; k < mark.parts; ++k) {
    const float l = weight[k][lane];
    nan |= l != l;
    top = fmaxf(top, l);
  }
  const float ref = top == -INFINITY ? 0.f : top;
  float acc[kCh] = {};
  for (int k0 = 0;;) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float w =
          k0 + u < mark.parts ? ex2((weight[k0 + u][lane] - ref) * 1.4426950408889634f) : 0.f;
      tot += w;
      // (what nobody saw was not written)
#pragma unroll
      for (int d = 0; d < kCh; ++d) acc[d] = w != 0.f ? fmaf(w, v[u][d], acc[d]) : acc[d];
    }
    if ((k0 += kBatch) >= mark.parts) break;
    fetch(k0);
  }
  const float inv = tot > 0.f || nan ? 1.f / tot : 0.f;
#pragma unroll
  for (int d = 0; d < kCh; d += 2)
    *reinterpret_cast<uint32_t *>(&tile[lane][warp * kCh + d]) =
        Elem<T>::pack(acc[d] * inv, acc[d + 1] * inv);
  const auto place = [&](int r) {
    const int y = (row0 + r) % kTile;
    return (int64_t)(mark.q0 + (row0 + r) / kTile * P.tpt + y / P.group) * P.n_heads +
           mark.h * P.group + y % P.group;
  };
  if (warp == 0 && mine && P.lse)
    P.lse[place(lane)] =
        tot > 0.f || nan ? ref + log2f(tot) * 0.6931471805599453f : -INFINITY;
  __syncthreads();
  constexpr int kVec = D / 8;            // 16-byte pieces of a row
  for (int i = threadIdx.x; i < 32 * kVec; i += 512) {
    if (!((theirs >> (i / kVec)) & 1)) continue;
    *reinterpret_cast<uint4 *>(static_cast<T *>(P.out) + place(i / kVec) * D + (i % kVec) * 8) =
        *reinterpret_cast<const uint4 *>(&tile[i / kVec][(i % kVec) * 8]);
  }
}

template <typename T, int D, bool kNarrow, int kG>
int launch(const AttnParams &P, const Pages &C8, const TilesWs &ws, int items, const TileMaps &m,
           cudaStream_t st) {
  allow_smem<page_attn_kernel<T, D, kNarrow, kG>>((int)smem_bytes<D>());
  page_attn_kernel<T, D, kNarrow, kG>
      <<<ws.marks ? kSms : items, Cfg<D>::kThreads, smem_bytes<D>(), st>>>(P, C8, ws.marks, m.q,
                                                                           m.k, m.v);
  const int e = launch_status();
  if (!ws.marks || e != CSA2_OK) return e;
  return launch_behind(page_tiles_join_kernel<T, D>, dim3(kSms - 1, ws.rows / 32), 512, 0, true,
                       st, P, (const TileMark *)ws.marks, ws.rows);
}

template <typename T, int D>
int launch_any(const AttnParams &P, const Pages &C8, const TilesWs &ws, bool narrow, int items,
               const TileMaps &m, cudaStream_t st) {
  if (C8.page >= 64)
    return narrow ? launch<T, D, true, 64>(P, C8, ws, items, m, st)
                  : launch<T, D, false, 64>(P, C8, ws, items, m, st);
  return narrow ? launch<T, D, true, 16>(P, C8, ws, items, m, st)
                : launch<T, D, false, 16>(P, C8, ws, items, m, st);
}

}  // namespace
}  // namespace pages
}  // namespace csa2
