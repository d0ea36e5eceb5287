// Partial results of attention calls that split the cache: how many, how large,
// and the kernel that joins them.
#pragma once
#include "dense.cuh"

namespace csa2 {
namespace dense {

constexpr int kMaxSplits = 16;

// Splits of `items` items unsplit on `places` places, of `steps` steps each: the
// waves' length in steps, `fixed` steps of fixed cost to an item, and half a
// step to a split for the join.
inline int plan_splits(int64_t items, int places, int64_t steps, double fixed) {
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= kMaxSplits && s <= (steps > 0 ? steps : 1); ++s) {
    const int64_t waves = (items * s + places - 1) / places;
    const double c = (double)waves * ((double)((steps + s - 1) / s) + fixed) + 0.5 * s;
    if (c < cost) cost = c, best = s;
  }
  return best;
}

inline int64_t part_bytes(int64_t num_q, const Shape &s) {
  return part_rows(num_q, s.group) * s.n_kv * (s.dim + 1) * 4;
}

namespace {

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

struct Join {
  const float *part_o, *part_lse;
  int parts, own;                // parts in all; the first of the requests' own
  int num_q, num_req;
  const int32_t *cu_q;
  void *out;
  float *lse;
};

template <typename T, int D>
int launch_join(const Shape &s, const Join &j, bool look, unsigned blocks, cudaStream_t st) {
  return launch_behind(look ? merge_kernel<T, D, true> : merge_kernel<T, D, false>,
                       dim3(blocks, (unsigned)s.n_kv), 512, 0, true, st, j.part_o, j.part_lse,
                       j.parts, j.own, j.num_q, s.n_kv, s.group, j.cu_q, j.num_req,
                       static_cast<T *>(j.out), j.lse);
}

int join_parts(const Shape &s, const Join &j, bool look, cudaStream_t st) {
  const int64_t blocks = part_rows(j.num_q, s.group) / 32;
  if (blocks > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  const unsigned n = (unsigned)blocks;
  if (s.bf16)
    return s.dim == 128 ? launch_join<__nv_bfloat16, 128>(s, j, look, n, st)
                        : launch_join<__nv_bfloat16, 64>(s, j, look, n, st);
  return s.dim == 128 ? launch_join<__half, 128>(s, j, look, n, st)
                      : launch_join<__half, 64>(s, j, look, n, st);
}

}  // namespace
}  // namespace dense
}  // namespace csa2
