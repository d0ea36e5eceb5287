// New keys and values into 8-bit pages (csa2_page_append).
//
// A block (page, head, side) has one scale s, the smallest power of two with |x| <=
// 448 s, so that rescaling older rows by old / new is exact but below 2^-6.
//
// Bound by memory: two bytes read and one written for each channel.
//
// Which page a block of the grid has: the pages that request r's new rows touch
// take the places from floor(cu_q[r] / page) + 2 r on.  (n rows touch at most
// floor((n - 1) / page) + 2 pages, which is what lies between there and the next
// request's first place, so no prefix sum is needed.)
//
// A page to a CTA; its blocks are shared out among the CTA's warps.
#include "pages.cuh"
#include "rope.cuh"

namespace csa2 {
namespace pages {
namespace {

using rope::kUnit;

struct AppendParams {
  int num_q, num_req, n_kv;
  const int32_t *cu_q;
  const int64_t *kv_len;
  const void *k, *v;
  int64_t ldk, ldv;
  Pages cache;
  rope::Rope rope;                       // freq null: keys are not rotated
  int32_t *d_err;
};

// Rows of a request and what they touch.
struct Touched {
  int q0;                                // first query row
  int64_t row0, m;                       // first new row (0 and up), rows
  int64_t place;                         // of its first page
  int pages;                             // 0: nothing to do
};

__device__ __forceinline__ Touched touched_by(const AppendParams &P, int r, int lo, int hi,
                                              int &err) {
  Touched t{lo, 0, 0, (int64_t)(lo >> P.cache.shift) + 2ll * r, 0};
  if (lo < 0 || hi < lo || hi > P.num_q) {
    err |= CSA2_DERR_BAD_EXTEND;
    return t;
  }
  if (hi == lo) return t;
  const int64_t m = P.kv_len[r], n = hi - lo;
  if (m < 0 || m > P.cache.most) {
    err |= CSA2_DERR_RANGE_ROW;
    return t;
  }
  t.m = m;
  t.row0 = m - n;
  if (m < n) {
    err |= CSA2_DERR_BAD_EXTEND;
    t.q0 = (int)(lo + (n - m));
    t.row0 = 0;
  }
  if (m > 0) t.pages = (int)(((m - 1) >> P.cache.shift) - (t.row0 >> P.cache.shift)) + 1;
  return t;
}

// smallest power of two s with amax <= 448 s, within the scales' range
__device__ __forceinline__ float need_of(float amax, int &err) {
  if (!(amax > kTop * kLowScale)) return kLowScale;
  if (amax > kTop * kHighScale) {
    err |= CSA2_DERR_SCALE;
    return kHighScale;
  }
  const uint32_t u = __float_as_uint(amax);              // 448 = 1.75 * 2^8
  const uint32_t e = (u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u);
  return __uint_as_float(e << 23);
}

// x / scale: by the reciprocal where that is exact
struct Divider {
  float scale, inv;
  bool exact;
  __device__ __forceinline__ float operator()(float x) const {
    return exact ? x * inv : __fdiv_rn(x, scale);
  }
};

__device__ __forceinline__ Divider by_scale(float s) {
  return Divider{s, 1.f / s, (__float_as_uint(s) & 0x7fffffu) == 0};
}

__device__ __forceinline__ uint2 codes8(const float *x, const Divider &by) {
  return make_uint2(e4m3x2_of(by(x[0]), by(x[1])) | (e4m3x2_of(by(x[2]), by(x[3])) << 16),
                    e4m3x2_of(by(x[4]), by(x[5])) | (e4m3x2_of(by(x[6]), by(x[7])) << 16));
}

// 16 codes times `ratio`, rounded again
__device__ __forceinline__ uint4 rescaled(uint4 w, float ratio) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = f16x2_of(v[i]), b = f16x2_of_high(v[i]);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    v[i] = e4m3x2_of(x.x * ratio, x.y * ratio) | (e4m3x2_of(y.x * ratio, y.y * ratio) << 16);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// 16 channels of a row: loaded, rotated, and zeros where the row's head (the lanes
// of a team) has anything that is not finite; its largest magnitude.
template <typename T, int D>
__device__ __forceinline__ float load_row(const T *src, const rope::Place &at, bool turns,
                                          bool interleaved, const float (&c)[kUnit],
                                          const float (&s)[kUnit], float (&x)[2 * kUnit],
                                          bool there, int &err) {
  constexpr int kTeam = D / 16;
  if (there) {
    rope::unpack8<T>(*reinterpret_cast<const uint4 *>(src + at.a), x);
    rope::unpack8<T>(*reinterpret_cast<const uint4 *>(src + at.b), x + kUnit);
    if (turns) rope::turn16(x, interleaved, c, s);
  } else {
#pragma unroll
    for (int i = 0; i < 2 * kUnit; ++i) x[i] = 0.f;
  }
  bool fine = true;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * kUnit; ++i) {
    fine &= fabsf(x[i]) <= 3.402823466e38f;
    amax = fmaxf(amax, fabsf(x[i]));
  }
  const uint32_t bad = __ballot_sync(0xffffffffu, !fine);
  const int lane = threadIdx.x & 31, team = lane / kTeam * kTeam;
  if ((bad >> team) & ((1u << kTeam) - 1)) {
    err |= CSA2_DERR_NONFINITE;
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * kUnit; ++i) x[i] = 0.f;
  }
  return amax;
}

constexpr int kWarps = 16;

// One block by a warp: its rows are gone over twice, for the scale and for the
// codes (the last of them stay in registers).
template <typename T, int D>
__device__ void append_block(const AppendParams &P, const uint64_t *turn, const Touched &t,
                             int64_t p, int id, int h, int side, int &err) {
  constexpr int kTeam = D / 16, kStep = 32 / kTeam;      // lanes of a row, rows at a time
  const Pages &C = P.cache;
  const int lane = threadIdx.x & 31, i = lane % kTeam;
  const int64_t base = p << C.shift;
  const int first = (int)max(t.row0 - base, (int64_t)0), end = (int)min(t.m - base, (int64_t)C.page);
  const bool rot = side == 0 && P.rope.freq;
  const rope::Place at =
      rot ? rope::place_of(i, P.rope.rot, P.rope.interleaved) : rope::place_of(i, 0, true);
  const int64_t ld = side ? P.ldv : P.ldk;
  const T *src = static_cast<const T *>(side ? P.v : P.k) + (int64_t)h * D;
  uint8_t *codes = (side ? C.v + id * C.v_stride : C.k + id * C.k_stride) +
                   (int64_t)h * C.page * D;
  float x[2 * kUnit];
  const auto load = [&](int row) {
    const bool there = row < end;
    const int64_t q = t.q0 + (base + row - t.row0);
    float c[kUnit], s[kUnit];
    const bool turns = rot && at.turns && there;
    if (turns)
      rope::angles(turn, i, P.rope.pos ? P.rope.pos[q] : base + row, P.rope.amplitude, 1.f, c, s);
    return load_row<T, D>(src + (there ? q * ld : 0), at, turns, P.rope.interleaved, c, s, x,
                          there, err);
  };
  float amax = 0.f;
  int row0 = first;
  for (int r = first; r < end; r += kStep) {
    row0 = r;
    amax = fmaxf(amax, load(r + lane / kTeam));
  }
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, k));
  float *scale = (side ? C.v_scale : C.k_scale) + (int64_t)id * P.n_kv + h;
  float now = need_of(amax, err);
  if (first > 0) {
    const float old = scale_of(*scale, err);
    if (now > old) {
      uint4 *w = reinterpret_cast<uint4 *>(codes);
      for (int j = lane; j < first * (D / 16); j += 32) w[j] = rescaled(w[j], old / now);
    } else {
      now = old;
    }
    __syncwarp();                        // every lane has read the scale
  }
  if (lane == 0) *scale = now;
  const Divider by = by_scale(now);
  for (int r = row0;; r -= kStep) {
    const int row = r + lane / kTeam;
    if (row < end) {
      *reinterpret_cast<uint2 *>(codes + row * D + at.a) = codes8(x, by);
      *reinterpret_cast<uint2 *>(codes + row * D + at.b) = codes8(x + kUnit, by);
    }
    if (r == first) break;
    load(r - kStep + lane / kTeam);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32)
append_kernel(const __grid_constant__ AppendParams P) {
  __shared__ uint64_t turn[D / 2];
  __shared__ int found, matches;
  const int64_t place = blockIdx.x;
  int err = 0;
  if (blockIdx.x == gridDim.x - 1) {         // no page: looks at every request
    for (int r = threadIdx.x; r < P.num_req; r += kWarps * 32)
      touched_by(P, r, P.cu_q[r], P.cu_q[r + 1], err);
    err = __reduce_or_sync(0xffffffffu, err);
    if ((threadIdx.x & 31) == 0) raise_err(P.d_err, err);
    return;
  }
  if (P.rope.freq) rope::load_turns(P.rope, turn);
  // The request that has this place; in a malformed batch more than one may.
  for (int from = 0;;) {
    if (threadIdx.x == 0) found = 0x7fffffff, matches = 0;
    __syncthreads();
#pragma unroll 4
    for (int r = from + threadIdx.x; r < P.num_req; r += kWarps * 32) {
      const int lo = P.cu_q[r], hi = P.cu_q[r + 1];
      const int64_t off = place - ((lo >> P.cache.shift) + 2ll * r);
      if (off < 0 || lo < 0 || hi < lo || off > ((int64_t)hi - lo) / P.cache.page + 1) continue;
      int ignored = 0;
      if (off < touched_by(P, r, lo, hi, ignored).pages) {
        atomicMin(&found, r);
        atomicAdd(&matches, 1);
      }
    }
    __syncthreads();
    const int r = found, n = matches;
    if (n == 0) break;
    int ignored = 0;
    const Touched t = touched_by(P, r, P.cu_q[r], P.cu_q[r + 1], ignored);
    const int64_t p = (t.row0 >> P.cache.shift) + (place - t.place);
    const int id = page_id(P.cache, r, p, err);
    if (id >= 0)
      for (int i = threadIdx.x >> 5; i < 2 * P.n_kv; i += kWarps)
        append_block<T, D>(P, turn, t, p, id, i >> 1, i & 1, err);
    if (n == 1) break;
    from = r + 1;
    __syncthreads();
  }
  err = __reduce_or_sync(0xffffffffu, err);
  if ((threadIdx.x & 31) == 0) raise_err(P.d_err, err);
}

template <typename T, int D>
int launch(const AppendParams &P, int places, cudaStream_t st) {
  append_kernel<T, D><<<places + 1, kWarps * 32, 0, st>>>(P);
  return launch_status();
}

// n bytes from p on against rows of one side's codes, page by page
bool meets_side(const void *p, uint64_t n, const csa2_pages *c, int n_kv, int dim, bool v) {
  return meets_rows(p, n, v ? c->v : c->k, c->num_pages,
                    side_stride(c, n_kv, dim, v ? c->v_stride : c->k_stride),
                    (int64_t)n_kv * c->page * dim);
}

// Whether what the call writes meets what it reads, or itself.
bool cache_meets(const csa2_packed *b, const csa2_pages *c, int n_kv, int dim, const void *k,
                 int64_t ldk, const void *v, int64_t ldv, const csa2_rope *r) {
  const int64_t wide = (int64_t)n_kv * dim * 2;
  const uint64_t nq = (uint64_t)b->num_q, nr = (uint64_t)b->num_req;
  const uint64_t ns = (uint64_t)c->num_pages * n_kv * 4;
  const auto written = [&](const void *p, uint64_t n) {
    return p && (meets_side(p, n, c, n_kv, dim, false) || meets_side(p, n, c, n_kv, dim, true) ||
                 overlap(p, n, c->k_scale, ns) || overlap(p, n, c->v_scale, ns));
  };
  if (written(k, (nq - 1) * ldk * 2 + wide) || written(v, (nq - 1) * ldv * 2 + wide)) return true;
  if (written(b->cu_q, 4 * (nr + 1)) || written(b->kv_len, 8 * nr) ||
      written(c->table, nr * c->table_ld * 4))
    return true;
  if (r && (written(r->freq, (uint64_t)r->rot * 4) || written(r->pos, nq * 8))) return true;
  // the four arrays
  if (overlap(c->k_scale, ns, c->v_scale, ns)) return true;
  for (int i = 0; i < 2; ++i) {
    const float *s = i ? c->v_scale : c->k_scale;
    if (meets_side(s, ns, c, n_kv, dim, false) || meets_side(s, ns, c, n_kv, dim, true))
      return true;
  }
  const int64_t side = (int64_t)n_kv * c->page * dim;
  const int64_t sk = side_stride(c, n_kv, dim, c->k_stride),
                sv = side_stride(c, n_kv, dim, c->v_stride);
  if (!overlap(c->k, (uint64_t)(c->num_pages - 1) * sk + side, c->v,
               (uint64_t)(c->num_pages - 1) * sv + side))
    return false;
  return sk != sv || meets_side(c->k, side, c, n_kv, dim, true) ||
         meets_side(c->v, side, c, n_kv, dim, false);
}

}  // namespace
}  // namespace pages
}  // namespace csa2

using namespace csa2;

extern "C" CSA2_API int csa2_page_append(const csa2_packed *b, int32_t n_kv_heads, int32_t dim,
                                         int32_t dtype, const void *k, int64_t ldk,
                                         const void *v, int64_t ldv, const csa2_rope *r,
                                         const csa2_pages *c, int32_t *d_err,
                                         csa2_stream_t stream) {
  if (n_kv_heads < 1) return CSA2_ERR_INVALID_ARG;
  if (dtype != CSA2_DT_BF16 && dtype != CSA2_DT_F16) return CSA2_ERR_UNSUPPORTED;
  if ((dim != 64 && dim != 128) || n_kv_heads > 1024) return CSA2_ERR_UNSUPPORTED;
  int st = pages::check_paged(b, c, n_kv_heads, dim);
  if (st == CSA2_OK && r) st = rope::check_rope(r, dim);
  if (st != CSA2_OK) return st;
  if (b->num_q == 0 || b->num_req == 0) return CSA2_OK;
  if ((st = dense::check_rows(k, ldk, n_kv_heads, dim)) != CSA2_OK) return st;
  if ((st = dense::check_rows(v, ldv, n_kv_heads, dim)) != CSA2_OK) return st;
  if (!aligned(4, d_err)) return CSA2_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && pages::cache_meets(b, c, n_kv_heads, dim, k, ldk, v, ldv, r))
    return CSA2_ERR_INVALID_ARG;
  pages::AppendParams P{};
  P.num_q = b->num_q;
  P.num_req = b->num_req;
  P.n_kv = n_kv_heads;
  P.cu_q = b->cu_q;
  P.kv_len = b->kv_len;
  P.k = k;
  P.v = v;
  P.ldk = ldk;
  P.ldv = ldv;
  P.cache = pages::to_device_view(c);
  if (r) P.rope = rope::Rope{r->freq, r->pos, r->rot, r->interleaved, r->amplitude};
  P.d_err = d_err;
  const int64_t places = (b->num_q >> P.cache.shift) + 2ll * b->num_req;
  if (places >= 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  const cudaStream_t cs = as_stream(stream);
  if (dtype == CSA2_DT_BF16)
    return dim == 128 ? pages::launch<__nv_bfloat16, 128>(P, (int)places, cs)
                      : pages::launch<__nv_bfloat16, 64>(P, (int)places, cs);
  return dim == 128 ? pages::launch<__half, 128>(P, (int)places, cs)
                    : pages::launch<__half, 64>(P, (int)places, cs);
}
