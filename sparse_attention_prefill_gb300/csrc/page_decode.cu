// Attention of single tokens over 8-bit pages (csa2_page_attn), for up to 16 query
// heads to a key head.
//
// Bound by the pages' bytes, each read once: at 128 channels a key's row is 128
// bytes, and a few query rows meet it.  96 requests of 10.0 thousand rows on average
// take 295 us (6.7 TB/s, what a copy does), 61 of 2815 rows 67 us (5.3 TB/s).
//
// All (token, key head) items' blocks of 32 keys lie in one row, and each CTA (three to
// an SM) takes an equal run of them (page_runs.cuh), so that it starts once.  (A CTA to an item or an equal split of
// one: 83 and 331 us; runs equal in blocks alone: 76 and 305.)  An item that two or more
// CTAs share is left as parts, at most two to a CTA, which a second kernel joins.
//
// In a CTA one warp looks up pages and keeps a ring of blocks filled by TMA, across
// items; four warps take the blocks in turn, each with its own running maximum, sum and
// output of the item at hand, and join them at its end, while the ring holds some
// microseconds of the next.
//
// Codes become f16 in registers, exactly, on their way into m16n8k16 products whose
// wide operand the cache is:
//   S^T[key, row] = K8 Q^T: the channels' order in a dot product is free, so a
//   thread's four codes of a word are its operands of one product, and Q's fragments
//   (in shared memory, in fragment order) are laid out the same way;
//   O^T[channel, row] += V8^T P^T: V's fragments want two keys to a register: a byte
//   permutation pairs the codes of two keys, and one conversion makes a register of
//   them.  P's are S^T's accumulators, transposed 8 x 8 at a time.
// Lines of 128 bytes are swizzled by TMA (16-byte chunk i of line l lies at i ^ l %
// 8), and the keys' order within 16 is chosen so that no load of either operand meets
// a bank twice: fragment row a holds key key_of(a).
#include "page_runs.cuh"

namespace csa2 {
namespace pages {
namespace {

constexpr int kWarps = 4;                // that compute
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kKeys = 32;                // keys of a block
constexpr int kSegs = 2;                 // segments published at a time
constexpr int kBurst = 4;                // blocks asked for at a time, a lane to each

// 8 x 8 16-bit values, transposed over the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A run of blocks of one (token, key head).
struct Segment {
  int token, h;                          // token -1: no more
  int keys;                              // that the token sees
  int blk0, blocks;
  int part;                              // of the partial results; -1: the whole item
};

// Single tokens: a unit is a token, a step a block of keys.
struct Tokens {
  static constexpr int kFixed = 12;      // blocks' time that an item's start and end take
  static constexpr int kLeast = 4;       // cost of a share, at least
  static __device__ __forceinline__ int units(const Run &u) { return u.n; }
  static __device__ __forceinline__ int keys(const Run &u, int i) {
    const int64_t last = u.m - u.n + i;  // keys seen: 0 .. last
    return last < 0 ? 0 : (int)last + 1;
  }
  // a token that sees nothing has a block, too: its output is written
  static __device__ __forceinline__ int steps(const Run &u, int i) {
    return max(1, (keys(u, i) + kKeys - 1) / kKeys);
  }
};

// For the join: the item that began in the share before and goes on in this one, and its
// parts (parts_of).
struct Mark {
  int token, h, parts, pad;
};

// CTAs, by groups of 8 query rows: as many to an SM as registers allow
template <int kN>
constexpr int kToSm = kN == 1 ? 3 : 2;
template <int kN>
constexpr int kCtas = kToSm<kN> * kSms;

// kN: groups of 8 query rows
template <int D, int kN>
struct Shared {
  static constexpr int kSide = kKeys * D;            // bytes of a block's K or V
  static constexpr int kRing = D == 128 ? 8 : 16;    // blocks, 64 KB
  // A stage is one warp's for good: the warp waits for each of its phases in turn.  (A
  // wait by parity that skips a phase does not wait.)
  static_assert(kRing % kWarps == 0, "ring");
  uint8_t ring[kRing][2][kSide];
  // Q of a segment: the copy of its rows, then fragments by lane
  union {
    uint4 rows[8 * kN * D / 8];
    uint2 frag[kN][D / 16][32];
  } q[kSegs];
  float o[kWarps][8 * kN][D / 4 + 4];                // a quarter of the warps' channels
  float4 scales[kRing];                              // K's and V's of a block's halves
  float lift[8 * kN];
  float ref[kWarps][8 * kN], sum[kWarps][8 * kN];
  uint64_t full[kRing], empty[kRing], seg_full[kSegs], seg_empty[kSegs];
  Segment seg[kSegs];
  Bound bd;
  int64_t scan[kThreads / 32];
  Place place;                                       // where the CTA's share begins
};

// key of fragment row a (0..15) within 16
template <int D>
__device__ __forceinline__ int key_of(int a) {
  if (D == 128) return (a & 1) ? a ^ 4 : a;
  return 4 * ((a & 7) >> 1) + (a & 1) + ((a & 8) >> 2);
}

// byte of 16-byte chunk `chunk` of row `row` in a block's side
template <int D>
__device__ __forceinline__ int byte_of(int row, int chunk) {
  const int line = D == 128 ? row : row >> 1;
  const int at = D == 128 ? chunk : (row & 1) * 4 + chunk;
  return line * 128 + ((at ^ (line & 7)) << 4);
}

__device__ __forceinline__ void bulk_load(void *to, const void *from, uint32_t bytes,
                                          uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(to)),
      "l"(from), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The warp that fills the ring.  A lane holds one of 32 neighbouring blocks of the
// segment: the ids of its halves' pages (the same one where a page has 32 rows or more)
// and their scales.  It asks for kBurst blocks at a time: a block by itself takes some
// 1000 cycles of waits and issue, which is what a CTA has for 8 KB (one at a time, 96
// requests took 319 us instead of 306).
template <typename T, int D, int kN>
__device__ void producer_role(const PageAttnParams &P, bool whole, Shared<D, kN> &sh,
                              const CUtensorMap *mk, const CUtensorMap *mv, int64_t at, int64_t end,
                              int &err) {
  using Sh = Shared<D, kN>;
  constexpr int kSide = Sh::kSide;
  const int lane = threadIdx.x & 31;
  const Pages &C = P.cache;
  const Seqs &S = P.at.seqs;
  Place p = sh.place;
  uint32_t g = 0, segs = 0;              // blocks and segments so far
  bool ok = true;
  while (at < end) {
    const int keys = Tokens::keys(p.u, p.i), all = Tokens::steps(p.u, p.i), h = p.h;
    const int run = p.run, token = p.u.lo + p.i;
    const Steps part = steps_in<Tokens>(p, all, end - at);
    const int blk = part.from, n = whole ? (blk == 0 && part.n > 0 ? all : 0) : part.n;
    at += Tokens::kFixed + all - p.off;  // the next item
    if (n > 0) {
      const uint32_t slot = segs % kSegs;
      if (!(ok = wait_all(&sh.seg_empty[slot], ((segs / kSegs) & 1) ^ 1, &sh.bd))) break;
      if (lane == 0) {
        sh.seg[slot] = Segment{token, h, keys, blk, n,
                               blk > 0           ? 2 * (int)blockIdx.x
                               : blk + n < all ? 2 * (int)blockIdx.x + 1
                                               : -1};
        const uint32_t bytes = (uint32_t)P.at.group * D * 2;
        mbar_arrive_expect_tx(&sh.seg_full[slot], bytes);
        bulk_load(sh.q[slot].rows,
                  static_cast<const T *>(P.q) + (int64_t)token * P.ldq + (int64_t)h * P.at.group * D,
                  bytes, &sh.seg_full[slot]);
      }
      __syncwarp();
      ++segs;
    }
    int id[2] = {-1, -1};
    float a[2], b[2];
    for (int k = 0; k < n; k += kBurst) {
      if (k % 32 == 0) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int64_t key = (int64_t)(blk + k + lane) * kKeys + 16 * x;
          if (x == 1 && C.shift > 4)
            id[1] = id[0];
          else
            id[x] = k + lane < n && key < keys ? page_id(C, run, key >> C.shift, err) : -1;
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          a[x] = id[x] >= 0 ? C.k_scale[(int64_t)id[x] * P.at.n_kv + h] : 0.f;
          b[x] = id[x] >= 0 ? C.v_scale[(int64_t)id[x] * P.at.n_kv + h] : 0.f;
        }
      }
      // a block to a lane
      const int mine = lane % kBurst, some = min(kBurst, n - k);
      const bool busy = lane < some;
      const uint32_t s = (g + mine) % Sh::kRing;
      ok = !busy || wait_bar(&sh.empty[s], (((g + mine) / Sh::kRing) & 1) ^ 1, &sh.bd);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      const int p0 = __shfl_sync(0xffffffffu, id[0], (k + mine) % 32);
      const int p1 = __shfl_sync(0xffffffffu, id[1], (k + mine) % 32);
      if (busy) {
        uint8_t *to = sh.ring[s][0];
        uint64_t *bar = &sh.full[s];
        if (C.shift == 4) {
          mbar_arrive_expect_tx(bar, (uint32_t)kSide * ((p0 >= 0) + (p1 >= 0)));
          const int line = h * (16 * D / 128);
          if (p0 >= 0) tma_load_3d(to, mk, 0, line, p0, bar);
          if (p1 >= 0) tma_load_3d(to + kSide / 2, mk, 0, line, p1, bar);
          if (p0 >= 0) tma_load_3d(to + kSide, mv, 0, line, p0, bar);
          if (p1 >= 0) tma_load_3d(to + kSide + kSide / 2, mv, 0, line, p1, bar);
        } else {
          mbar_arrive_expect_tx(bar, p0 >= 0 ? 2u * kSide : 0u);
          const int line = (h * C.page + (((blk + k + mine) * kKeys) & (C.page - 1))) * D / 128;
          if (p0 >= 0) tma_load_3d(to, mk, 0, line, p0, bar);
          if (p0 >= 0) tma_load_3d(to + kSide, mv, 0, line, p0, bar);
        }
      }
      __syncwarp();
      // the scales come after the copies: they may still be on their way
      if (k % 32 == 0) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          a[x] = id[x] >= 0 ? scale_of(a[x], err) : 0.f;
          b[x] = id[x] >= 0 ? scale_of(b[x], err) : 0.f;
        }
      }
      float4 sc;
      sc.x = __shfl_sync(0xffffffffu, a[0], (k + mine) % 32);
      sc.y = __shfl_sync(0xffffffffu, a[1], (k + mine) % 32);
      sc.z = __shfl_sync(0xffffffffu, b[0], (k + mine) % 32);
      sc.w = __shfl_sync(0xffffffffu, b[1], (k + mine) % 32);
      if (busy) {
        sh.scales[s] = sc;
        mbar_arrive(&sh.full[s]);
      }
      __syncwarp();
      g += some;
    }
    if (!ok || at >= end || !next_item(Tokens{}, S, P.at.n_kv, p)) break;
  }
  if (ok) {
    const uint32_t slot = segs % kSegs;
    ok = wait_all(&sh.seg_empty[slot], ((segs / kSegs) & 1) ^ 1, &sh.bd);
    if (ok && lane == 0) {
      sh.seg[slot].token = -1;
      mbar_arrive(&sh.seg_full[slot]);
    }
  }
  // copies land before the CTA leaves: the warps that compute wait for all of them, but not
  // once a wait has run out
  if (lane == 0) {
    // (the last phase of each barrier alone can be waited for: once the end is published, it
    // is that of the slot of the segment before the last, whose copy was read by then)
    const uint32_t open = ok ? 1 : kSegs;
    for (uint32_t k = segs > open ? segs - open : 0; k < segs; ++k)
      drain_bar(&sh.seg_full[k % kSegs], (k / kSegs) & 1);
    for (uint32_t k = g > (uint32_t)Sh::kRing ? g - Sh::kRing : 0; k < g; ++k)
      drain_bar(&sh.full[k % Sh::kRing], (k / Sh::kRing) & 1);
  }
  __syncwarp();
}

// barrier of the warps that compute; whether any thread says so
__device__ __forceinline__ bool any_of_us(bool say) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)say), "n"(32 * kWarps)
      : "memory");
  return r != 0;
}

// The four warps that compute.
template <typename T, int D, int kN>
__device__ __forceinline__ void compute_role(const PageAttnParams &P, Shared<D, kN> &sh) {
  using Sh = Shared<D, kN>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  uint32_t taken = 0;                    // blocks of the segments so far
  for (uint32_t u = 0;; ++u) {
    const uint32_t slot = u % kSegs;
    bool ok = wait_all(&sh.seg_full[slot], (u / kSegs) & 1, &sh.bd);
    // (also: the last segment's sums in shared memory are read)
    if (any_of_us(!ok)) return;
    const Segment seg = sh.seg[slot];
    if (seg.token < 0) return;
    // Q's rows become fragments where they are; rows past the group's heads are zeros
    constexpr int kPieces = 8 * kN * D / 8, kEach = (kPieces + 32 * kWarps - 1) / (32 * kWarps);
    uint4 piece[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + 32 * kWarps * e, r = i / (D / 8);
      if (i >= kPieces) break;           // (whole warps)
      uint4 v = make_uint4(0, 0, 0, 0);
      if (r < P.at.group) v = sh.q[slot].rows[i];
      if (Elem<T>::kBf16) {
        uint32_t x[4] = {v.x, v.y, v.z, v.w};
        float amax = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          amax = max3(amax, fabsf(__uint_as_float(x[k] << 16)),
                      fabsf(__uint_as_float(x[k] & 0xffff0000u)));
#pragma unroll
        for (int k = 1; k < D / 8; k <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
        const float lift = lift_of(amax);
        if (i % (D / 8) == 0) sh.lift[r] = lift;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          x[k] = Elem<__half>::pack(__uint_as_float(x[k] << 16) * lift,
                                    __uint_as_float(x[k] & 0xffff0000u) * lift);
        v = make_uint4(x[0], x[1], x[2], x[3]);
      }
      piece[e] = v;
    }
    any_of_us(false);
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + 32 * kWarps * e, r = i / (D / 8), ch = i % (D / 8) * 8;
      if (i >= kPieces) break;
      const int x = 4 * (ch >> 6) + (ch >> 2 & 3), l = (r & 7) * 4 + (ch >> 4 & 3);
      sh.q[slot].frag[r >> 3][x][l] = make_uint2(piece[e].x, piece[e].y);
      sh.q[slot].frag[r >> 3][x + 1][l] = make_uint2(piece[e].z, piece[e].w);
    }
    any_of_us(false);

    // this thread's rows: 8 y + 2 c + r
    float o[kN][D / 16][4] = {}, ref[kN][2], sum[kN][2], unit[kN][2];
#pragma unroll
    for (int y = 0; y < kN; ++y)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ref[y][r] = -INFINITY, sum[y][r] = 0.f;
        unit[y][r] = P.at.scale_log2 / (Elem<T>::kBf16 ? sh.lift[8 * y + 2 * c + r] : 1.f);
      }
    for (int k = (int)((warp - taken) & (kWarps - 1)); k < seg.blocks; k += kWarps) {
      const uint32_t s = (taken + k) % Sh::kRing;
      if (!(ok = wait_all(&sh.full[s], ((taken + k) / Sh::kRing) & 1, &sh.bd))) break;
      uint8_t *kt = sh.ring[s][0], *vt = sh.ring[s][1];
      const int key0 = (seg.blk0 + k) * kKeys;
      const float4 sc = sh.scales[s];
      const float ka[2] = {sc.x, sc.y}, vb[2] = {sc.z, sc.w};
      const bool all = key0 + kKeys <= seg.keys && vb[0] != 0.f && vb[1] != 0.f;
      if (!all) {
        // rows behind the last and rows without a page may hold NaN: 0 * NaN
        for (int r = 0; r < kKeys; ++r)
          if (key0 + r >= seg.keys || vb[r >> 4] == 0.f)
            for (int d = lane; d < D / 16; d += 32)
              *reinterpret_cast<uint4 *>(vt + byte_of<D>(r, d)) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();          // the next copy into them comes later
        __syncwarp();
      }
      // S^T: accumulator e: fragment row g + 8 (e / 2), query row 2 c + e % 2
      float st[2][kN][4] = {};
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int ch = 0; ch < D / 64; ++ch) {
          uint4 w[2];
#pragma unroll
          for (int t = 0; t < 2; ++t)
            w[t] = *reinterpret_cast<const uint4 *>(
                kt + byte_of<D>(16 * x + key_of<D>(g + 8 * t), c + 4 * ch));
          const uint32_t *w0 = &w[0].x, *w1 = &w[1].x;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = f16x2_of(w0[j]), a1 = f16x2_of(w1[j]);
            const uint32_t a2 = f16x2_of_high(w0[j]), a3 = f16x2_of_high(w1[j]);
#pragma unroll
            for (int y = 0; y < kN; ++y) {
              const uint2 qv = sh.q[slot].frag[y][4 * ch + j][lane];
              mma16816(st[x][y], a0, a1, a2, a3, qv.x, qv.y);
            }
          }
        }
      }
      float lb[2], ib[2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        lb[x] = log2f(vb[x]);              // -inf without a page: masked below
        ib[x] = vb[x] != 0.f ? 1.f / vb[x] : 0.f;
#pragma unroll
        for (int y = 0; y < kN; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            st[x][y][e] = fmaf(st[x][y][e], unit[y][e & 1] * ka[x], lb[x]);
      }
      if (!all) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 16 * x + key_of<D>(g + 8 * (e >> 1)) >= seg.keys || vb[x] == 0.f)
#pragma unroll
              for (int y = 0; y < kN; ++y) st[x][y][e] = -INFINITY;
      }
      uint32_t pt[2][kN][2];
#pragma unroll
      for (int y = 0; y < kN; ++y) {
        float alpha[2];
        bool moved = false;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float mx = -INFINITY;
#pragma unroll
          for (int x = 0; x < 2; ++x) mx = max3(mx, st[x][y][r], st[x][y][2 + r]);
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
          alpha[r] = 1.f;
          if (mx > ref[y][r] + (kLift + kMargin)) {
            alpha[r] = ex2(ref[y][r] - (mx - kLift));
            ref[y][r] = mx - kLift;
            moved = true;
          }
        }
        if (__any_sync(0xffffffffu, moved)) {
          sum[y][0] *= alpha[0], sum[y][1] *= alpha[1];
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            o[y][d][0] *= alpha[0], o[y][d][1] *= alpha[1];
            o[y][d][2] *= alpha[0], o[y][d][3] *= alpha[1];
          }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float base = ref[y][e & 1] == -INFINITY ? 0.f : ref[y][e & 1];
            w[e] = ex2(st[x][y][e] - base);
          }
          sum[y][0] = fmaf(w[0] + w[2], ib[x], sum[y][0]);
          sum[y][1] = fmaf(w[1] + w[3], ib[x], sum[y][1]);
          pt[x][y][0] = transpose8(Elem<__half>::pack(w[0], w[1]));
          pt[x][y][1] = transpose8(Elem<__half>::pack(w[2], w[3]));
        }
      }
      // O^T: product d has channels (D / 8) g + 2 d (rows g) and + 1 (rows g + 8)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int row = 16 * x + key_of<D>(2 * c + (u & 1) + 8 * (u >> 1));
          if (D == 128) {
            *reinterpret_cast<uint4 *>(v[u]) =
                *reinterpret_cast<const uint4 *>(vt + byte_of<D>(row, g));
          } else {
            *reinterpret_cast<uint2 *>(v[u]) =
                *reinterpret_cast<const uint2 *>(vt + byte_of<D>(row, g >> 1) + 8 * (g & 1));
          }
        }
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t p = __byte_perm(v[0][j], v[1][j], e ? 0x7362 : 0x5140);
            const uint32_t r = __byte_perm(v[2][j], v[3][j], e ? 0x7362 : 0x5140);
            const uint32_t a0 = f16x2_of(p), a1 = f16x2_of_high(p);
            const uint32_t a2 = f16x2_of(r), a3 = f16x2_of_high(r);
#pragma unroll
            for (int y = 0; y < kN; ++y)
              mma16816(o[y][2 * j + e], a0, a1, a2, a3, pt[x][y][0], pt[x][y][1]);
          }
        }
      }
      __syncwarp();                        // every lane has read the stage
      if (lane == 0) mbar_arrive(&sh.empty[s]);
    }
    taken += seg.blocks;

    // join the warps: each row's statistics and sums, weighted, by quarters of the products
    // (the channels (D / 8) g + 2 d and + 1 of products d)
    fence_proxy_async_smem();            // the next copy of Q into the slot comes later
    if (any_of_us(!ok)) return;          // (and Q is done with)
    if (threadIdx.x == 0) mbar_arrive(&sh.seg_empty[slot]);
#pragma unroll
    for (int y = 0; y < kN; ++y)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) sum[y][r] += __shfl_xor_sync(0xffffffffu, sum[y][r], k);
        const int row = 8 * y + 2 * c + r;
        if (g == 0) sh.ref[warp][row] = ref[y][r], sh.sum[warp][row] = sum[y][r];
      }
    constexpr int kRows = 8 * kN, kTeam = kWarps * 32 / kRows;       // threads of a row
    constexpr int kPart = D / 32;        // channels of a lane group in a quarter
    const int row = threadIdx.x / kTeam, col = threadIdx.x % kTeam;
    const bool mine = row < P.at.group;
    const int64_t part = (int64_t)seg.part * kRows + row;
    const int64_t at = (int64_t)seg.token * P.at.n_heads + seg.h * P.at.group + row;
    float w[kWarps];
#pragma unroll
    for (int z = 0; z < 4; ++z) {
      if (z) any_of_us(false);           // the quarter before is read
#pragma unroll
      for (int y = 0; y < kN; ++y)
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int d = 0; d < D / 64; ++d)
            *reinterpret_cast<float2 *>(&sh.o[warp][8 * y + 2 * c + r][kPart * g + 2 * d]) =
                make_float2(o[y][z * (D / 64) + d][r], o[y][z * (D / 64) + d][2 + r]);
      any_of_us(false);
      if (z == 0) {
        float top = -INFINITY, tot = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, sh.ref[k][row]);
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          w[k] = ex2(sh.ref[k][row] - base);
          tot += sh.sum[k][row] * w[k];
        }
        const bool seen = !(tot == 0.f);   // a NaN stays a NaN
        const float inv = seen ? 1.f / tot : 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) w[k] = seen ? w[k] * inv : 0.f;
        const float lse = seen ? (base + log2f(tot)) * 0.6931471805599453f : -INFINITY;
        if (col == 0 && mine) {
          if (seg.part >= 0)
            P.at.part_lse[part] = lse;
          else if (P.at.lse)
            P.at.lse[at] = lse;
        }
      }
      if (mine) {
#pragma unroll
        for (int x = 2 * col; x < D / 4; x += 2 * kTeam) {
          const int d = x / kPart * (D / 8) + z * kPart + x % kPart;
          float f[2] = {0.f, 0.f};
#pragma unroll
          for (int k = 0; k < kWarps; ++k) {
            const float2 v = *reinterpret_cast<const float2 *>(&sh.o[k][row][x]);
            f[0] = fmaf(w[k], v.x, f[0]), f[1] = fmaf(w[k], v.y, f[1]);
          }
          if (seg.part >= 0)
            *reinterpret_cast<float2 *>(P.at.part_o + part * D + d) = make_float2(f[0], f[1]);
          else
            *reinterpret_cast<uint32_t *>(static_cast<T *>(P.at.out) + at * D + d) =
                Elem<T>::pack(f[0], f[1]);
        }
      }
      __syncwarp();
    }
  }
}

template <typename T, int D, int kN>
__global__ void __launch_bounds__(kThreads, kToSm<kN>)
page_decode_kernel(const __grid_constant__ PageAttnParams P, Mark *marks,
                   const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  // the join may start on the SMs that the last CTAs leave
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<D, kN> &sh = *reinterpret_cast<Shared<D, kN> *>(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < Shared<D, kN>::kRing; ++s) {
      mbar_init(&sh.full[s], 2);         // copies asked for, scales written
      mbar_init(&sh.empty[s], 1);
    }
    for (int s = 0; s < kSegs; ++s) {
      mbar_init(&sh.seg_full[s], 1);
      mbar_init(&sh.seg_empty[s], 1);
    }
    sh.bd.abort = 0;
    sh.bd.wait_ns = P.at.wait_ns;
    mbar_fence_init();
  }
  int err = 0;
  const Plan plan =
      find_share<kThreads>(Tokens{}, P.at.seqs, P.at.n_kv, sh.scan, sh.place, err);
  const int share = (int)blockIdx.x;
  const int64_t begin = share_begin(plan, share), end = share_begin(plan, share + 1);
  if (share > 0) err = 0;                // one CTA speaks of the requests
  if (marks && threadIdx.x == 32 * kWarps - 1) {
    Mark mark{-1, 0, 0, 0};
    const Place &p = sh.place;
    if (const int parts = parts_of(Tokens{}, plan, share, p))
      mark = Mark{p.u.lo + p.i, p.h, parts, 0};
    marks[share] = mark;
  }
  if (begin < end) {
    if (threadIdx.x >= 32 * kWarps)
      producer_role<T>(P, !marks, sh, &mk, &mv, begin, end, err);
    else
      compute_role<T>(P, sh);
    __syncthreads();
    if (threadIdx.x == 0 && sh.bd.abort) err |= CSA2_DERR_TIMEOUT;
  }
  if (err) raise_err(P.at.d_err, err);
}

// Joins the parts of items that shares cut, an item to a block.  A chain of loads in the
// main: the first parts are asked for together with all statistics.
constexpr int kJoin = 256, kBatch = 8;

template <typename T, int D, int kN>
__global__ void __launch_bounds__(kJoin)
page_join_kernel(const __grid_constant__ PageAttnParams P, const Mark *marks) {
  constexpr int kRows = 8 * kN;
  __shared__ float weight[kCtas<kN>][kRows];         // by part
  __shared__ float total[kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = blockIdx.x + 1;
  wait_front();
  const Mark mark = marks[j];
  if (mark.token < 0) return;
  const int parts = mark.parts;
  const auto part = [&](int k) {
    return (k == 0 ? 2 * (int64_t)(j - 1) + 1 : 2 * (int64_t)(j - 1 + k)) * kRows;
  };
  constexpr int kQuads = kRows * D / 4, kEach = (kQuads + kJoin - 1) / kJoin;
  float4 v[kEach][kBatch];
  const auto fetch = [&](int k0) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int i = threadIdx.x + e * kJoin, r = i / (D / 4), d = i % (D / 4) * 4;
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        v[e][k] = r < P.at.group && k0 + k < parts
                      ? *reinterpret_cast<const float4 *>(P.at.part_o + (part(k0 + k) + r) * D + d)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  fetch(0);
  for (int r = warp; r < P.at.group; r += kJoin / 32) {
    float most = -INFINITY, tot = 0.f;
    bool nan = false;
    for (int k = lane; k < parts; k += 32) {
      const float l = P.at.part_lse[part(k) + r];
      weight[k][r] = l;
      nan |= l != l;
      most = fmaxf(most, l);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float ref = most == -INFINITY ? 0.f : most;
    for (int k = lane; k < parts; k += 32) {
      const float w = ex2((weight[k][r] - ref) * 1.4426950408889634f);
      weight[k][r] = w;
      tot += w;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
    nan = __any_sync(0xffffffffu, nan);
    if (lane == 0) {
      total[r] = tot;
      if (P.at.lse)
        P.at.lse[(int64_t)mark.token * P.at.n_heads + mark.h * P.at.group + r] =
            tot > 0.f || nan ? ref + log2f(tot) * 0.6931471805599453f : -INFINITY;
    }
  }
  __syncthreads();
  float f[kEach][4] = {};
  for (int k0 = 0;;) {
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int r = min((int)(threadIdx.x + e * kJoin) / (D / 4), P.at.group - 1);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float w = k0 + k < parts ? weight[k0 + k][r] : 0.f;
        f[e][0] = fmaf(w, v[e][k].x, f[e][0]), f[e][1] = fmaf(w, v[e][k].y, f[e][1]);
        f[e][2] = fmaf(w, v[e][k].z, f[e][2]), f[e][3] = fmaf(w, v[e][k].w, f[e][3]);
      }
    }
    if ((k0 += kBatch) >= parts) break;
    fetch(k0);
  }
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = threadIdx.x + e * kJoin, r = i / (D / 4), d = i % (D / 4) * 4;
    if (r >= P.at.group) break;
    const float inv = total[r] == 0.f ? 0.f : 1.f / total[r];
    const int64_t at = (int64_t)mark.token * P.at.n_heads + mark.h * P.at.group + r;
    *reinterpret_cast<uint2 *>(static_cast<T *>(P.at.out) + at * D + d) =
        make_uint2(Elem<T>::pack(f[e][0] * inv, f[e][1] * inv),
                   Elem<T>::pack(f[e][2] * inv, f[e][3] * inv));
  }
}

template <typename T, int D, int kN>
int launch(PageAttnParams P, int64_t max_kv, const CUtensorMap &mk, const CUtensorMap &mv,
           void *ws, cudaStream_t st) {
  constexpr int kSmem = (int)sizeof(Shared<D, kN>);
  static_assert(kSmem <= 232448 / kToSm<kN> - 1024, "CTAs to an SM");
  allow_smem<page_decode_kernel<T, D, kN>>(kSmem);
  // no more CTAs than the blocks may need
  const double most =
      (double)P.at.seqs.num_q * P.at.n_kv * (double)(max_kv / kKeys + 1 + Tokens::kFixed);
  const int grid = most >= (double)Tokens::kLeast * kCtas<kN> ? kCtas<kN>
                                                                : (int)(most / Tokens::kLeast) + 1;
  Mark *marks = static_cast<Mark *>(ws);
  if (ws) {
    P.at.part_lse = reinterpret_cast<float *>(marks + kCtas<kN>);
    P.at.part_o = P.at.part_lse + 2 * kCtas<kN> * 8 * kN;
  }
  page_decode_kernel<T, D, kN><<<grid, kThreads, kSmem, st>>>(P, marks, mk, mv);
  const int e = launch_status();
  if (e != CSA2_OK || !ws || grid == 1) return e;
  return launch_behind(page_join_kernel<T, D, kN>, dim3(grid - 1), kJoin, 0, true, st, P,
                       (const Mark *)marks);
}

template <typename T>
int launch_any(const Shape &s, const PageAttnParams &P, int64_t max_kv, const CUtensorMap &mk,
               const CUtensorMap &mv, void *ws, cudaStream_t st) {
  if (s.dim == 128)
    return s.group <= 8 ? launch<T, 128, 1>(P, max_kv, mk, mv, ws, st)
                        : launch<T, 128, 2>(P, max_kv, mk, mv, ws, st);
  return s.group <= 8 ? launch<T, 64, 1>(P, max_kv, mk, mv, ws, st)
                      : launch<T, 64, 2>(P, max_kv, mk, mv, ws, st);
}

}  // namespace

int64_t page_decode_bytes(const Shape &s) {
  const int rows = s.group <= 8 ? 8 : 16;
  const int64_t ctas = s.group <= 8 ? kCtas<1> : kCtas<2>;
  return ctas * (int64_t)sizeof(Mark) + 2 * ctas * rows * (s.dim + 1) * 4;
}

int page_decode(const Shape &s, const PageAttnParams &P, int64_t max_kv, const csa2_pages *c,
                void *ws, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!make_cache_maps(&mk, &mv, c, P.q, s, kKeys)) return CSA2_ERR_UNSUPPORTED;
  return s.bf16 ? launch_any<__nv_bfloat16>(s, P, max_kv, mk, mv, ws, st)
                : launch_any<__half>(s, P, max_kv, mk, mv, ws, st);
}

}  // namespace pages
}  // namespace csa2
