// Attention of single tokens over 8-bit pages (csa2_page_attn), for up to 16 query
// heads to a key head.
//
// Bound by the pages' bytes, each read once: at 128 channels a key's row is 128
// bytes, and a few query rows meet it.  A CTA has one (token, key head, split); its
// four warps take blocks of 32 keys in turn, each with its own running maximum, sum
// and output, which are joined once at the end.  Each warp has a ring of kStages
// blocks of its own in shared memory, filled by TMA: 24 copies of 8 KB in flight to
// an SM, with no registers under them.
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
#include "decode_rows.cuh"
#include "page_attn.cuh"

namespace csa2 {
namespace pages {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 32;                // keys of a block
constexpr int kStages = 2;

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

// kN: groups of 8 query rows
template <int D, int kN>
struct Shared {
  static constexpr int kSide = kKeys * D;            // bytes of a block's K or V
  union {
    uint8_t ring[kWarps][kStages][2][kSide];
    float o[kWarps][8 * kN][D + 4];                  // once the ring is done with
  };
  uint2 q[kN][D / 16][32];                           // Q in fragment order, by lane
  float lift[8 * kN], unlift[8 * kN];
  float ref[kWarps][8 * kN], sum[kWarps][8 * kN];
  uint64_t full[kWarps][kStages];
  Bound bd;
  uint32_t runs[kWarps];
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

// One item: the token's rows of key head h over a split of its request's m rows,
// whose n query rows begin at q0.  `used`: blocks that this warp's ring has had.
template <typename T, int D, int kN>
__device__ __forceinline__ void decode_item(const PageAttnParams &P, const CUtensorMap *mk,
                                            const CUtensorMap *mv, Shared<D, kN> &sh, int token,
                                            int run, int q0, int n, int64_t m, int h, int split,
                                            uint32_t &used, int &err) {
  constexpr int kSide = Shared<D, kN>::kSide;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int ns = P.at.splits > 0 ? P.at.splits : 1;
  const Pages &C = P.cache;
  const int64_t last = m - n + (token - q0);           // keys seen: 0 .. last
  const int keys = last < 0 ? 0 : (int)last + 1;
  const int blocks = (keys + kKeys - 1) / kKeys, each = (blocks + ns - 1) / ns;
  const int b0 = min(blocks, split * each), b1 = min(blocks, b0 + each);
  const int mine = b1 - b0 > warp ? (b1 - b0 - warp + kWarps - 1) / kWarps : 0;

  // Pages of this warp's next 32 blocks, a block to a lane: ids of the pages of its
  // halves (the same one where a page has 32 rows or more), and their scales, which
  // are asked for with the copies and used two blocks later.
  int id[2] = {-1, -1};
  float na[2], nb[2], a[2], b[2];
  bool checked[2];
  const auto look_up = [&](int i0) {
    const int64_t blk = b0 + warp + (int64_t)kWarps * (i0 + lane);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int64_t key = blk * kKeys + 16 * x;
      if (x == 1 && C.shift > 4) {
        id[1] = id[0];
        continue;
      }
      id[x] = i0 + lane < mine && key < keys ? page_id(C, run, key >> C.shift, err) : -1;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      checked[x] = id[x] >= 0;
      na[x] = checked[x] ? C.k_scale[(int64_t)id[x] * P.at.n_kv + h] : 0.f;
      nb[x] = checked[x] ? C.v_scale[(int64_t)id[x] * P.at.n_kv + h] : 0.f;
    }
  };
  const auto fetch = [&](int i) {
    if (i % 32 == 0) look_up(i);
    const int p0 = __shfl_sync(0xffffffffu, id[0], i % 32);
    const int p1 = __shfl_sync(0xffffffffu, id[1], i % 32);
    if (lane == 0) {
      const uint32_t s = used % kStages;
      uint8_t *to = &sh.ring[warp][s][0][0];
      uint64_t *bar = &sh.full[warp][s];
      const int blk = b0 + warp + kWarps * i;
      if (C.shift == 4) {
        mbar_arrive_expect_tx(bar, (uint32_t)kSide * ((p0 >= 0) + (p1 >= 0)));
        const int line = h * (16 * D / 128);
        if (p0 >= 0) tma_load_3d(to, mk, 0, line, p0, bar);
        if (p1 >= 0) tma_load_3d(to + kSide / 2, mk, 0, line, p1, bar);
        if (p0 >= 0) tma_load_3d(to + kSide, mv, 0, line, p0, bar);
        if (p1 >= 0) tma_load_3d(to + kSide + kSide / 2, mv, 0, line, p1, bar);
      } else {
        mbar_arrive_expect_tx(bar, p0 >= 0 ? 2u * kSide : 0u);
        const int line = (h * C.page + ((blk * kKeys) & (C.page - 1))) * D / 128;
        if (p0 >= 0) tma_load_3d(to, mk, 0, line, p0, bar);
        if (p0 >= 0) tma_load_3d(to + kSide, mv, 0, line, p0, bar);
      }
    }
    ++used;
  };
  const uint32_t used0 = used;
  for (int i = 0; i < kStages && i < mine; ++i) fetch(i);

  // Q's fragments; rows past the group's heads are zeros
  const T *q = static_cast<const T *>(P.q) + (int64_t)token * P.ldq + (int64_t)h * P.at.group * D;
  if (Elem<T>::kBf16) {
    for (int r = warp; r < 8 * kN; r += kWarps) {
      float amax = 0.f;
      if (r < P.at.group)
        for (int d = lane; d < D; d += 32) amax = fmaxf(amax, fabsf((float)q[r * D + d]));
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
      if (lane == 0) {
        const float lift = lift_of(amax);
        sh.lift[r] = lift;
        sh.unlift[r] = 1.f / lift;
      }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < kN * D / 16 * 32; i += kWarps * 32) {
    const int l = i & 31, x = (i >> 5) % (D / 16), r = (i >> 5) / (D / 16) * 8 + (l >> 2);
    const int ch = 16 * ((l & 3) + 4 * (x >> 2)) + 4 * (x & 3);
    uint2 w = make_uint2(0, 0);
    if (r < P.at.group) {
      w = *reinterpret_cast<const uint2 *>(q + r * D + ch);
      if (Elem<T>::kBf16) {
        const float f = sh.lift[r];
        w = make_uint2(Elem<__half>::pack(__uint_as_float(w.x << 16) * f,
                                          __uint_as_float(w.x & 0xffff0000u) * f),
                       Elem<__half>::pack(__uint_as_float(w.y << 16) * f,
                                          __uint_as_float(w.y & 0xffff0000u) * f));
      }
    }
    (&sh.q[0][0][0])[i] = w;
  }
  __syncthreads();

  // this thread's rows: 8 y + 2 c + r
  float o[kN][D / 16][4] = {}, ref[kN][2], sum[kN][2], unit[kN][2];
#pragma unroll
  for (int y = 0; y < kN; ++y)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      ref[y][r] = -INFINITY, sum[y][r] = 0.f;
      unit[y][r] = P.at.scale_log2 * (Elem<T>::kBf16 ? sh.unlift[8 * y + 2 * c + r] : 1.f);
    }
  bool ok = true;
  int i = 0;
  for (; i < mine; ++i) {
    if (i % 32 == 0) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        a[x] = checked[x] ? scale_of(na[x], err) : 0.f;
        b[x] = checked[x] ? scale_of(nb[x], err) : 0.f;
      }
    }
    const uint32_t s = (used0 + i) % kStages;
    if (!(ok = wait_all(&sh.full[warp][s], ((used0 + i) / kStages) & 1, &sh.bd))) break;
    uint8_t *kt = &sh.ring[warp][s][0][0], *vt = kt + kSide;
    const int key0 = (b0 + warp + kWarps * i) * kKeys;
    float ka[2], vb[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      ka[x] = __shfl_sync(0xffffffffu, a[x], i % 32);
      vb[x] = __shfl_sync(0xffffffffu, b[x], i % 32);
    }
    const bool whole = key0 + kKeys <= keys && vb[0] != 0.f && vb[1] != 0.f;
    if (!whole) {
      // rows behind the last and rows without a page may hold NaN: 0 * NaN
      for (int r = 0; r < kKeys; ++r)
        if (key0 + r >= keys || vb[r >> 4] == 0.f)
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
            const uint2 qv = sh.q[y][4 * ch + j][lane];
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
    if (!whole) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 16 * x + key_of<D>(g + 8 * (e >> 1)) >= keys || vb[x] == 0.f)
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
    if (i + kStages < mine) fetch(i + kStages);
  }
  if (!ok && lane == 0)                  // copies land before the CTA leaves
    for (uint32_t u = used0 + i; u != used; ++u)
      drain_bar(&sh.full[warp][u % kStages], (u / kStages) & 1);
  __syncthreads();                       // the ring is done with

  // join the warps: each row's statistics and sums, weighted
#pragma unroll
  for (int y = 0; y < kN; ++y) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) sum[y][r] += __shfl_xor_sync(0xffffffffu, sum[y][r], k);
      const int row = 8 * y + 2 * c + r;
      if (g == 0) sh.ref[warp][row] = ref[y][r], sh.sum[warp][row] = sum[y][r];
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
        *reinterpret_cast<float2 *>(&sh.o[warp][row][D / 8 * g + 2 * d]) =
            make_float2(o[y][d][r], o[y][d][2 + r]);
    }
  }
  __syncthreads();
  // a result's rows are channel-innermost, a partial result's blocks row-innermost
  const bool part = P.at.splits > 0;
  constexpr int kRows = 8 * kN, kTeam = kWarps * 32 / kRows;       // threads of a row
  const int row = part ? threadIdx.x % kRows : threadIdx.x / kTeam;
  const int col = part ? threadIdx.x / kRows : threadIdx.x % kTeam;
  if (row >= P.at.group) return;
  float top = -INFINITY, tot = 0.f, w[kWarps];
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
  const float lse = seen ? (base + log2f(tot)) * 0.6931471805599453f : -INFINITY;
  if (part) {
    const int64_t rows = part_rows(P.at.seqs.num_q, P.at.group), at = (int64_t)token * P.at.group + row;
    if (col == 0) P.at.part_lse[part_stat(rows, P.at.n_kv, split, h, at)] = lse;
    if (!seen) return;
    float *dst = P.at.part_o + part_elem(rows, P.at.n_kv, D, split, h, at);
#pragma unroll 4
    for (int d = col; d < D; d += kTeam) {
      float f = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) f = fmaf(w[k], sh.o[k][row][d], f);
      dst[d * 32] = f * inv;
    }
  } else {
    const int64_t at = (int64_t)token * P.at.n_heads + h * P.at.group + row;
    if (col == 0 && P.at.lse) P.at.lse[at] = lse;
#pragma unroll
    for (int d = 4 * col; d < D; d += 4 * kTeam) {
      float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        const float4 v = *reinterpret_cast<const float4 *>(&sh.o[k][row][d]);
        f[0] = fmaf(w[k], v.x, f[0]), f[1] = fmaf(w[k], v.y, f[1]);
        f[2] = fmaf(w[k], v.z, f[2]), f[3] = fmaf(w[k], v.w, f[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = seen ? f[e] * inv : 0.f;
      *reinterpret_cast<uint2 *>(static_cast<T *>(P.at.out) + at * D + d) =
          make_uint2(Elem<T>::pack(f[0], f[1]), Elem<T>::pack(f[2], f[3]));
    }
  }
}

template <typename T, int D, int kN>
__global__ void __launch_bounds__(kWarps * 32, kN == 2 ? 2 : 3)
page_decode_kernel(const __grid_constant__ PageAttnParams P, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv) {
  // the join may start on the SMs that the last items leave
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(1024) uint8_t smem[];
  Shared<D, kN> &sh = *reinterpret_cast<Shared<D, kN> *>(smem);
  if (threadIdx.x == 0) {
    for (int w = 0; w < kWarps; ++w)
      for (int s = 0; s < kStages; ++s) mbar_init(&sh.full[w][s], 1);
    sh.bd.abort = 0;
    sh.bd.wait_ns = P.at.wait_ns;
    mbar_fence_init();
  }
  __syncthreads();
  uint32_t used = 0;
  int err = 0;
  bool again = false;
  each_item<kWarps, true>(P.at.seqs, P.at.n_kv, P.at.group, P.at.splits, P.at.part_lse, P.at.d_err, sh.runs,
                          [&](int token, int run, int q0, int n, int64_t, int64_t m, int h,
                              int split) {
                            if (again) {  // the ring held a join's sums
                              fence_proxy_async_smem();
                              __syncthreads();
                            }
                            again = true;
                            decode_item<T, D, kN>(P, &mk, &mv, sh, token, run, q0, n, m, h,
                                                  split, used, err);
                          });
  if (*(volatile int *)&sh.bd.abort) err |= CSA2_DERR_TIMEOUT;
  if (err) raise_err(P.at.d_err, err);
}

template <typename T, int D, int kN>
int launch(const PageAttnParams &P, int grid, const CUtensorMap &mk, const CUtensorMap &mv,
           cudaStream_t st) {
  constexpr int kSmem = (int)sizeof(Shared<D, kN>);
  allow_smem<page_decode_kernel<T, D, kN>>(kSmem);
  page_decode_kernel<T, D, kN><<<grid, kWarps * 32, kSmem, st>>>(P, mk, mv);
  return launch_status();
}

template <typename T>
int launch_any(const Shape &s, const PageAttnParams &P, int grid, const CUtensorMap &mk,
               const CUtensorMap &mv, cudaStream_t st) {
  if (s.dim == 128)
    return s.group <= 8 ? launch<T, 128, 1>(P, grid, mk, mv, st)
                        : launch<T, 128, 2>(P, grid, mk, mv, st);
  return s.group <= 8 ? launch<T, 64, 1>(P, grid, mk, mv, st)
                      : launch<T, 64, 2>(P, grid, mk, mv, st);
}

}  // namespace

int page_decode(const Shape &s, const PageAttnParams &P, const csa2_pages *c, cudaStream_t st) {
  // an item to a block, and one that looks the batch over
  const int64_t grid = (int64_t)P.at.seqs.num_q * P.at.n_kv * (P.at.splits > 0 ? P.at.splits : 1) + 1;
  if (grid > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  CUtensorMap mk, mv;
  if (!make_cache_maps(&mk, &mv, c, P.q, s, kKeys)) return CSA2_ERR_UNSUPPORTED;
  return s.bf16 ? launch_any<__nv_bfloat16>(s, P, (int)grid, mk, mv, st)
                : launch_any<__half>(s, P, (int)grid, mk, mv, st);
}

}  // namespace pages
}  // namespace csa2
