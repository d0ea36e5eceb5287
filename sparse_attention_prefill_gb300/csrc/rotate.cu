// Rotary positions of rows [num_q, n_heads, dim] (csa2_rotate), and with the sign
// turned round the gradient.
//
// Bound by memory: two bytes read and written for each channel; 16001 rows of 64 heads x
// 128 channels take 82 us (6.4 TB/s).  A thread has eight
// pairs of one row's channels (rope.cuh) and goes over the row's heads with them, so
// that an angle's reduction, sine and cosine are spent once for all of the heads that
// it does.
#include "rope.cuh"

namespace csa2 {
namespace rope {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 4;                // heads of a row that a block does at a time
constexpr int kAhead = 4;                // heads that a thread has in flight
// rows of a block (with 8 heads at a time and half the rows, 12345 rows of 24 heads x 64
// took 17.7 us instead of 15.8; with 2 and twice the rows, 16001 of 64 x 128 85 instead of
// 82)
template <int D>
constexpr int kRows = kThreads / (D / 16) / kSlots;

struct RotateParams {
  int num_q, num_req, n_heads;
  const int32_t *cu_q;
  const int64_t *kv_len;
  const void *x;
  void *out;
  int64_t ldx, ldo;
  Rope rope;
  float sign;
  int each;                              // heads of a block
  int32_t *d_err;
};

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const __grid_constant__ RotateParams P) {
  constexpr int kTeam = D / 16;                          // threads of a row and head
  __shared__ uint64_t turn[D / 2];
  __shared__ int64_t pos[kRows<D>];
  __shared__ int held[kRows<D>];
  const int64_t row0 = (int64_t)blockIdx.x * kRows<D>;
  if (threadIdx.x < kRows<D>) {
    const int64_t row = row0 + threadIdx.x;
    held[threadIdx.x] = P.rope.pos && row < P.num_q;
    if (P.rope.pos && row < P.num_q) pos[threadIdx.x] = P.rope.pos[row];
  }
  load_turns(P.rope, turn);
  __syncthreads();
  if (!P.rope.pos) {
    int err = 0;
#pragma unroll 4
    for (int r = threadIdx.x; r < P.num_req; r += kThreads) {
      const int lo = P.cu_q[r], hi = P.cu_q[r + 1];
      if (lo < 0 || hi < lo || hi > P.num_q) {
        err |= CSA2_DERR_BAD_EXTEND;
        continue;
      }
      const int64_t a = max((int64_t)lo, row0), b = min((int64_t)hi, row0 + kRows<D>);
      if (a >= b) continue;
      const int64_t first = P.kv_len[r] - (hi - lo) - lo;
      for (int64_t i = a; i < b; ++i) {
        pos[i - row0] = first + i;
        held[i - row0] = 1;
      }
    }
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      err = __reduce_or_sync(0xffffffffu, err);
      if ((threadIdx.x & 31) == 0) raise_err(P.d_err, err);
    }
    __syncthreads();
  }
  const int t = threadIdx.x % kTeam, row = threadIdx.x / kTeam % kRows<D>;
  if (!held[row]) return;
  const Place at = place_of<D, kInterleaved>(t, P.rope.rot);
  float c[kUnit], s[kUnit];
  angles<D, kInterleaved>(turn, t, at, pos[row], P.rope.amplitude, P.sign, c, s);
  const T *x = static_cast<const T *>(P.x) + (row0 + row) * P.ldx;
  T *out = static_cast<T *>(P.out) + (row0 + row) * P.ldo;
  const int h1 = min(P.n_heads, ((int)blockIdx.y + 1) * P.each);
  for (int h0 = (int)blockIdx.y * P.each + threadIdx.x / kTeam / kRows<D>; h0 < h1;
       h0 += kAhead * kSlots) {
    uint4 a[kAhead], b[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * kSlots;
      if (h < h1) {
        a[i] = *reinterpret_cast<const uint4 *>(x + (int64_t)h * D + at.a);
        b[i] = *reinterpret_cast<const uint4 *>(x + (int64_t)h * D + at.b);
      }
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = h0 + i * kSlots;
      if (h >= h1) break;
      if (at.ta || at.tb) {
        float v[2 * kUnit];
        unpack8<T>(a[i], v);
        unpack8<T>(b[i], v + kUnit);
        turn16<kInterleaved>(v, at, c, s);
        a[i] = make_uint4(Elem<T>::pack(v[0], v[1]), Elem<T>::pack(v[2], v[3]),
                          Elem<T>::pack(v[4], v[5]), Elem<T>::pack(v[6], v[7]));
        b[i] = make_uint4(Elem<T>::pack(v[8], v[9]), Elem<T>::pack(v[10], v[11]),
                          Elem<T>::pack(v[12], v[13]), Elem<T>::pack(v[14], v[15]));
      }
      *reinterpret_cast<uint4 *>(out + (int64_t)h * D + at.a) = a[i];
      *reinterpret_cast<uint4 *>(out + (int64_t)h * D + at.b) = b[i];
    }
  }
}

template <typename T, int D>
int launch(const RotateParams &P, dim3 grid, cudaStream_t st) {
  if (P.rope.interleaved)
    rotate_kernel<T, D, true><<<grid, kThreads, 0, st>>>(P);
  else
    rotate_kernel<T, D, false><<<grid, kThreads, 0, st>>>(P);
  return launch_status();
}

}  // namespace
}  // namespace rope
}  // namespace csa2

using namespace csa2;

extern "C" CSA2_API int csa2_rotate(const csa2_packed *b, int32_t n_heads, int32_t dim,
                                    int32_t dtype, const void *x, int64_t ldx,
                                    const csa2_rope *r, int32_t inverse, void *out, int64_t ldo,
                                    int32_t *d_err, csa2_stream_t stream) {
  if (!b || !r || b->num_q < 0 || b->num_req < 0 || n_heads < 1) return CSA2_ERR_INVALID_ARG;
  if (dtype != CSA2_DT_BF16 && dtype != CSA2_DT_F16) return CSA2_ERR_UNSUPPORTED;
  if ((dim != 64 && dim != 128) || n_heads > 65535) return CSA2_ERR_UNSUPPORTED;
  int st = rope::check_rope(r, dim);
  if (st != CSA2_OK) return st;
  if (b->num_q == 0 || (!r->pos && b->num_req == 0)) return CSA2_OK;
  if (!r->pos && (!b->cu_q || !b->kv_len)) return CSA2_ERR_INVALID_ARG;
  if (!r->pos && !(aligned(4, b->cu_q) && aligned(8, b->kv_len))) return CSA2_ERR_UNSUPPORTED;
  if ((st = dense::check_rows(x, ldx, n_heads, dim)) != CSA2_OK) return st;
  if ((st = dense::check_rows(out, ldo, n_heads, dim)) != CSA2_OK) return st;
  if (!aligned(4, d_err)) return CSA2_ERR_UNSUPPORTED;
  const uint64_t wide = (uint64_t)n_heads * dim * 2, nq = (uint64_t)b->num_q;
  const uint64_t nx = (nq - 1) * ldx * 2 + wide, no = (nq - 1) * ldo * 2 + wide;
  const bool in_place = x == out && (ldx == ldo || nq == 1);
  if (!in_place && overlap(out, no, x, nx) &&
      (ldx != ldo || dense::meets_rows(out, wide, x, b->num_q, ldx * 2, (int64_t)wide) ||
       dense::meets_rows(x, wide, out, b->num_q, ldo * 2, (int64_t)wide)))
    return CSA2_ERR_INVALID_ARG;
  if (dense::meets_rows(r->freq, (uint64_t)r->rot * 4, out, b->num_q, ldo * 2, (int64_t)wide) ||
      dense::meets_rows(r->pos, nq * 8, out, b->num_q, ldo * 2, (int64_t)wide))
    return CSA2_ERR_INVALID_ARG;
  if (!r->pos) {
    const uint64_t nr = (uint64_t)b->num_req;
    if (dense::meets_rows(b->cu_q, 4 * (nr + 1), out, b->num_q, ldo * 2, (int64_t)wide) ||
        dense::meets_rows(b->kv_len, 8 * nr, out, b->num_q, ldo * 2, (int64_t)wide))
      return CSA2_ERR_INVALID_ARG;
  }
  rope::RotateParams P{};
  P.num_q = b->num_q;
  P.num_req = b->num_req;
  P.n_heads = n_heads;
  P.cu_q = b->cu_q;
  P.kv_len = b->kv_len;
  P.x = x;
  P.out = out;
  P.ldx = ldx;
  P.ldo = ldo;
  P.rope = rope::Rope{r->freq, r->pos, r->rot, r->interleaved, r->amplitude};
  P.sign = inverse ? -1.f : 1.f;
  P.d_err = d_err;
  // all heads of a row in one block, unless there are too few rows to fill the GPU
  const int rows = dim == 128 ? rope::kRows<128> : rope::kRows<64>;
  const int64_t blocks = ((int64_t)b->num_q + rows - 1) / rows;
  int chunks = 1;
  while (chunks * rope::kSlots < n_heads && blocks * chunks < 4 * dense::kSms) chunks *= 2;
  P.each = (n_heads + chunks - 1) / chunks;
  const dim3 grid((unsigned)blocks, (unsigned)((n_heads + P.each - 1) / P.each));
  const cudaStream_t cs = as_stream(stream);
  if (dtype == CSA2_DT_BF16)
    return dim == 128 ? rope::launch<__nv_bfloat16, 128>(P, grid, cs)
                      : rope::launch<__nv_bfloat16, 64>(P, grid, cs);
  return dim == 128 ? rope::launch<__half, 128>(P, grid, cs)
                    : rope::launch<__half, 64>(P, grid, cs);
}
