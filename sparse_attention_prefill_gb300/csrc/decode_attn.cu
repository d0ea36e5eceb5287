// Attention of single tokens over their own cache rows (the own part of
// csa2_prefix_attn, and csa2_prompt_attn on decode batches), for up to 16 query
// heads to a key head.
//
// Bound by the cache rows, each read once: a few query rows meet every 256-byte
// row, so the kernel is built to keep loads in flight, not around the tensor
// pipe.  A CTA has one (token, key head, split); its four warps take blocks of
// 16 keys in turn, each with its own running maximum, sum and output, which
// are joined once at the end.  K and V go from memory straight into the
// registers that m16n8k16 products want as their wide operand, 16 bytes a
// load, without shared memory or any exchange between warps:
//   S^T[key, row] = K Q^T: the order of the channels in a dot product is free,
//   so thread c of a quad takes channels 32 x + 8 c .. + 7 of its keys, and Q's
//   fragments (in shared memory, in fragment order) are laid out the same way;
//   O^T[channel, row] += V^T P^T: V's fragments want two keys to a register,
//   which a byte permutation makes of the rows of two keys; P's are S^T's
//   accumulators, transposed 8 x 8 at a time.  Row r of product (j, e) is
//   channel 64 j + 8 (r % 8) + 2 e + r / 8, so that a thread's channels of a
//   key are 16 bytes of it.
// With the rows as the wide operand (16 of them, half unused by groups of 8)
// the output took 64 registers a thread instead of 32, and what that spilled
// were the loads: 143 us for 256 requests x 8 key heads x 512 rows (537 MB).
// Those take 92 us now, the join included; 256 requests of 693 rows on average
// (731 MB) 131 us without it, 5.6 TB/s, and 125 us where nothing is split.  The
// next block's K is asked for as soon as S is done, its V once O is.
//
// (On the tcgen05 path of dense_attn.cu a decode item is a chain of copies,
// products of 128 rows with G of them in use, barriers and a TMEM epilogue: 108
// us for the 537 MB with the join, 171 for the 731 MB where nothing is split.)
#include "dense.cuh"

namespace csa2 {
namespace dense {
namespace {

constexpr int kWarps = 4;
constexpr int kKeys = 16;            // keys of a block

__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// 8 x 8 16-bit values, transposed over the warp
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint4 &a, uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint4 &a, uint32_t b0,
                                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint4 &a, uint32_t b0,
                                                 uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b0), "r"(b1));
}

// kN: groups of 8 query rows
template <int D, int kN>
struct Shared {
  uint2 q[kN][D / 16][32];           // Q in fragment order, by lane
  float o[kWarps][8 * kN][D + 4];
  float ref[kWarps][8 * kN], sum[kWarps][8 * kN];
  bool uncovered;                    // the request is in no group (split 0)
  uint32_t runs[kWarps];
};

// The run that holds query row `token`, by the block; -1: none.
__device__ int run_of(const Seqs &S, int token, uint32_t (&tmp)[kWarps]) {
  uint32_t run = 0xffffffffu;
#pragma unroll 4
  for (int r = threadIdx.x; r < S.count; r += kWarps * 32) {
    const int lo = S.cu_q[r], hi = S.cu_q[r + 1];
    if (lo >= 0 && lo <= token && token < hi && hi <= S.num_q) run = min(run, (uint32_t)r);
  }
  run = __reduce_min_sync(0xffffffffu, run);
  if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = run;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i) run = min(run, tmp[i]);
  return (int)run;
}

// One item: the token's rows of key head h over a split of the cached rows
// [start, start + m) of its run, whose n query rows begin at q0.
template <typename T, int D, int kN>
__device__ __forceinline__ void decode_item(const DecodeParams &P, Shared<D, kN> &sh, int token,
                                            int run, int q0, int n, int64_t start, int64_t m,
                                            int h, int split) {
  constexpr int kQ = D / 32, kJ = D / 64;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int ns = P.splits > 0 ? P.splits : 1;
  const Seqs &S = P.seqs;
  const int64_t last = m - n + (token - q0);           // keys seen: 0 .. last
  const int keys = last < 0 ? 0 : (int)last + 1;
  // Q's fragments; rows past the group's heads are zeros
  const T *q = static_cast<const T *>(P.q) + (int64_t)token * P.ldq + (int64_t)h * P.group * D;
  for (int i = threadIdx.x; i < kN * D / 16 * 32; i += kWarps * 32) {
    const int l = i & 31, s = (i >> 5) % (D / 16), r = (i >> 5) / (D / 16) * 8 + (l >> 2);
    const int ch = (s >> 1) * 32 + (l & 3) * 8 + (s & 1) * 4;
    (&sh.q[0][0][0])[i] = r < P.group ? *reinterpret_cast<const uint2 *>(q + r * D + ch)
                                      : make_uint2(0, 0);
  }
  __syncthreads();

  const int blocks = (keys + kKeys - 1) / kKeys, each = (blocks + ns - 1) / ns;
  const int b1 = min(blocks, split * each + each);
  const T *kb = static_cast<const T *>(P.k) + start * P.ldk + (int64_t)h * D + c * 8;
  const T *vb = static_cast<const T *>(P.v) + start * P.ldv + (int64_t)h * D + g * 8;
  uint4 kr[2][kQ], vr[4][kJ];
  // keys past the request's last row are read as that row: their weights are 0
  const int top_row = (int)m - 1;
  auto load_k = [&](int b) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const T *p = kb + (int64_t)min(b * kKeys + t * 8 + g, top_row) * P.ldk;
#pragma unroll
      for (int x = 0; x < kQ; ++x) kr[t][x] = ld_stream(p + x * 32);
    }
  };
  auto load_v = [&](int b) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int key = b * kKeys + 2 * c + (u & 1) + (u >> 1) * 8;
      const T *p = vb + (int64_t)min(key, top_row) * P.ldv;
#pragma unroll
      for (int j = 0; j < kJ; ++j) vr[u][j] = ld_stream(p + j * 64);
    }
  };
  // The block after the next, for which there are no registers yet: into L2, a
  // 128-byte line to a lane (731 MB of rows 135 -> 131 us; two blocks ahead: 133).
  auto prefetch = [&](int b) {
    constexpr int kLines = D / 64;
    if (lane < kKeys * kLines) {
      const int64_t row = start + min(b * kKeys + lane / kLines, top_row);
      const int64_t at = (int64_t)h * D + lane % kLines * 64;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T *>(P.k) + row * P.ldk + at));
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const T *>(P.v) + row * P.ldv + at));
    }
  };
  constexpr float kLift = Elem<T>::kBf16 ? 0.f : 8.f;    // as in dense_attn.cu
  constexpr float kMargin = Elem<T>::kBf16 ? 8.f : 7.f;
  // this thread's rows: 8 y + 2 c + r
  float o[kN][D / 16][4] = {}, ref[kN][2], sum[kN][2];
#pragma unroll
  for (int y = 0; y < kN; ++y)
#pragma unroll
    for (int r = 0; r < 2; ++r) ref[y][r] = -INFINITY, sum[y][r] = 0.f;
  int b = split * each + warp;
  if (b < b1) {
    load_k(b);
    load_v(b);
    if (b + kWarps < b1) prefetch(b + kWarps);
  }
  // while the first rows are on their way, by the warp that has the fewest blocks
  if (P.cover && split == 0 && warp == kWarps - 1) {
    const bool in = in_groups(P.cover, P.n_cover, run, S);
    if (lane == 0) sh.uncovered = !in;
  }
  for (; b < b1; b += kWarps) {
    // accumulator e: key g + 8 (e / 2), row 2 c + e % 2; even and odd channel
    // steps apart, for shorter chains of products
    float s[kN][4];
#pragma unroll
    for (int y = 0; y < kN; ++y) {
      float s0[4] = {}, s1[4] = {};
#pragma unroll
      for (int x = 0; x < kQ; ++x) {
        const uint2 q0v = sh.q[y][2 * x][lane], q1v = sh.q[y][2 * x + 1][lane];
        mma16816<T>(s0, make_uint4(kr[0][x].x, kr[1][x].x, kr[0][x].y, kr[1][x].y), q0v.x, q0v.y);
        mma16816<T>(s1, make_uint4(kr[0][x].z, kr[1][x].z, kr[0][x].w, kr[1][x].w), q1v.x, q1v.y);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) s[y][e] = s0[e] + s1[e];
    }
    const int nb = b + kWarps;
    if (nb < b1) load_k(nb);
    if (nb + kWarps < b1) prefetch(nb + kWarps);
    if (b * kKeys + kKeys > keys) {
#pragma unroll
      for (int y = 0; y < kN; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (b * kKeys + g + 8 * (e >> 1) >= keys) s[y][e] = -INFINITY;
    }
    uint32_t pt[kN][2];
#pragma unroll
    for (int y = 0; y < kN; ++y) {
      float alpha[2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float mx = fmaxf(s[y][r], s[y][2 + r]);
#pragma unroll
        for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
        mx *= P.scale_log2;
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
        for (int i = 0; i < D / 16; ++i) {
          o[y][i][0] *= alpha[0], o[y][i][1] *= alpha[1];
          o[y][i][2] *= alpha[0], o[y][i][3] *= alpha[1];
        }
      }
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float base = ref[y][e & 1] == -INFINITY ? 0.f : ref[y][e & 1];
        w[e] = ex2(fmaf(s[y][e], P.scale_log2, -base));
        sum[y][e & 1] += w[e];
      }
      pt[y][0] = transpose8(Elem<T>::pack(w[0], w[1]));
      pt[y][1] = transpose8(Elem<T>::pack(w[2], w[3]));
    }
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const uint32_t *v0 = &vr[0][j].x, *v1 = &vr[1][j].x, *v2 = &vr[2][j].x, *v3 = &vr[3][j].x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint4 a =
            make_uint4(__byte_perm(v0[e], v1[e], 0x5410), __byte_perm(v0[e], v1[e], 0x7632),
                       __byte_perm(v2[e], v3[e], 0x5410), __byte_perm(v2[e], v3[e], 0x7632));
#pragma unroll
        for (int y = 0; y < kN; ++y) mma16816<T>(o[y][4 * j + e], a, pt[y][0], pt[y][1]);
      }
    }
    if (nb < b1) load_v(nb);
  }

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
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<float2 *>(&sh.o[warp][row][64 * j + 8 * g + 2 * e]) =
              make_float2(o[y][4 * j + e][r], o[y][4 * j + e][2 + r]);
    }
  }
  __syncthreads();
  // a result's rows are channel-innermost, a partial result's blocks row-innermost
  const bool part = P.splits > 0;
  constexpr int kRows = 8 * kN, kTeam = kWarps * 32 / kRows;       // threads of a row
  const int row = part ? threadIdx.x % kRows : threadIdx.x / kTeam;
  const int col = part ? threadIdx.x / kRows : threadIdx.x % kTeam;
  if (row >= P.group) return;
  float top = -INFINITY, tot = 0.f, w[kWarps];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sh.ref[i][row]);
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    w[i] = ex2(sh.ref[i][row] - base);
    tot += sh.sum[i][row] * w[i];
  }
  const bool seen = !(tot == 0.f);   // a NaN stays a NaN
  const float inv = seen ? 1.f / tot : 0.f;
  const float lse = seen ? (base + log2f(tot)) * 0.6931471805599453f : -INFINITY;
  if (part) {
    const int64_t rows = part_rows(S.num_q, P.group), at = (int64_t)token * P.group + row;
    if (col == 0) {
      P.part_lse[part_stat(rows, P.n_kv, split, h, at)] = lse;
      if (P.cover && split == 0 && sh.uncovered)
        for (int i = 0; i < P.cover_splits; ++i)
          P.cover_lse[part_stat(rows, P.n_kv, i, h, at)] = -INFINITY;
    }
    if (!seen) return;
    float *dst = P.part_o + part_elem(rows, P.n_kv, D, split, h, at);
#pragma unroll 4
    for (int d = col; d < D; d += kTeam) {
      float f = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) f = fmaf(w[i], sh.o[i][row][d], f);
      dst[d * 32] = f * inv;
    }
  } else {
    const int64_t at = (int64_t)token * P.n_heads + h * P.group + row;
    if (col == 0 && P.lse) P.lse[at] = lse;
#pragma unroll
    for (int d = 4 * col; d < D; d += 4 * kTeam) {
      float f[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(&sh.o[i][row][d]);
        f[0] = fmaf(w[i], v.x, f[0]), f[1] = fmaf(w[i], v.y, f[1]);
        f[2] = fmaf(w[i], v.z, f[2]), f[3] = fmaf(w[i], v.w, f[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = seen ? f[e] * inv : 0.f;
      *reinterpret_cast<uint2 *>(static_cast<T *>(P.out) + at * D + d) =
          make_uint2(Elem<T>::pack(f[0], f[1]), Elem<T>::pack(f[2], f[3]));
    }
  }
}

template <typename T, int D, int kN>
__global__ void __launch_bounds__(kWarps * 32, kN == 2 ? 2 : D == 128 ? 3 : 4)
decode_attn_kernel(const __grid_constant__ DecodeParams P) {
  // a kernel launched with launch_behind may start on the SMs that the last items
  // leave (every item has started by then)
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(16) uint8_t smem[];
  Shared<D, kN> &sh = *reinterpret_cast<Shared<D, kN> *>(smem);
  const int ns = P.splits > 0 ? P.splits : 1;
  int split = blockIdx.x % ns, h = blockIdx.x / ns % P.n_kv;
  const Seqs &S = P.seqs;
  int err = 0;
  if (blockIdx.x == gridDim.x - 1) {         // no item: looks at every request's rows
    for (int r = threadIdx.x, a, b; r < S.count; r += kWarps * 32) seq_rows(S, r, a, b, err);
    err = __reduce_or_sync(0xffffffffu, err);
    if ((threadIdx.x & 31) == 0) raise_err(P.d_err, err);
    return;
  }
  // Query row `token`: the rows from the first request's on, then those in front
  // of it.  In a batch of single tokens row number i of these is run i's, and
  // everything of it is asked for at once; otherwise its run is looked for.
  const int slot = blockIdx.x / ns / P.n_kv, first = S.cu_q[0], end = S.cu_q[S.count];
  int run = min(slot, S.count - 1);
  int q0 = S.cu_q[run], behind = S.cu_q[run + 1];
  int64_t start = S.kv_start[run], m = S.kv_len[run];
  const uint32_t at = (uint32_t)slot + (first > 0 && first < S.num_q ? (uint32_t)first : 0u);
  const int token = (int)(at < (uint32_t)S.num_q ? at : at - S.num_q);
  const auto holds = [&]() {
    return q0 >= 0 && q0 <= token && token < behind && behind <= S.num_q;
  };
  bool sweep = false;
  if (!holds()) {
    // Rows in front of the first request and behind the last are nobody's, unless
    // the batch is malformed: one block to a row makes sure, and has all items
    // of the row if it is somebody's after all.  (With a look by every block,
    // 256 tokens in a batch of 4096 rows took 236 us instead of 188.)
    sweep = token < first || token >= end;
    if (sweep && (h > 0 || split > 0)) return;
    run = run_of(S, token, sh.runs);
    if (run < 0) {
      // the join leaves the row
      if (P.splits > 0 && split == 0) {
        const int64_t rows = part_rows(S.num_q, P.group), row = (int64_t)token * P.group;
        for (int i = threadIdx.x; i < (sweep ? P.n_kv : 1) * P.group; i += kWarps * 32)
          P.part_lse[part_stat(rows, P.n_kv, 0, h + i / P.group, row + i % P.group)] =
              __uint_as_float(kNobody);
      }
      return;
    }
    q0 = S.cu_q[run], behind = S.cu_q[run + 1];
  }
  seq_keys(S, run, start, m, err);
  if (err && threadIdx.x == 0) raise_err(P.d_err, err);
  for (;;) {
    decode_item<T, D, kN>(P, sh, token, run, q0, behind - q0, start, m, h, split);
    if (!sweep) return;
    __syncthreads();
    if (++split == ns) {
      split = 0;
      if (++h == P.n_kv) return;
    }
  }
}

}  // namespace

template <typename T, int D, int kN>
int decode_launch(const DecodeParams &P, int grid, cudaStream_t st) {
  constexpr int kSmem = (int)sizeof(Shared<D, kN>);
  allow_smem<decode_attn_kernel<T, D, kN>>(kSmem);
  decode_attn_kernel<T, D, kN><<<grid, kWarps * 32, kSmem, st>>>(P);
  return launch_status();
}

template <typename T>
int decode_any(const Shape &s, const DecodeParams &P, int grid, cudaStream_t st) {
  if (s.dim == 128)
    return s.group <= 8 ? decode_launch<T, 128, 1>(P, grid, st)
                        : decode_launch<T, 128, 2>(P, grid, st);
  return s.group <= 8 ? decode_launch<T, 64, 1>(P, grid, st) : decode_launch<T, 64, 2>(P, grid, st);
}

int decode_attn(const Shape &s, const DecodeParams &P, cudaStream_t st) {
  // an item to a block, and one that looks the batch over
  const int64_t grid = (int64_t)P.seqs.num_q * P.n_kv * (P.splits > 0 ? P.splits : 1) + 1;
  if (grid > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  return s.bf16 ? decode_any<__nv_bfloat16>(s, P, (int)grid, st)
                : decode_any<__half>(s, P, (int)grid, st);
}

}  // namespace dense
}  // namespace csa2
