// New keys and values into 8-bit pages (csa2_page_append).
//
// A block (page, head, side) has one scale s, the smallest power of two with |x| <=
// 448 s, so that rescaling older rows by old / new is exact but below 2^-6.
//
// Bound by memory in the end, two bytes read and one written for each channel, but short of
// it by what 16 warps to an SM cover (126 registers): eight prompts of 8192 rows, 8 heads x
// 128, take 82 us (4.9 TB/s; one row to a thread 87.6, of which the rotation was 15) with
// issue slots 58 % busy; 256 single rows 8.0, in two waves of CTAs of 512 threads.
//
// Which page a block of the grid has: the pages that request r's new rows touch
// take the places from floor(cu_q[r] / page) + 2 r on.  (n rows touch at most
// floor((n - 1) / page) + 2 pages, which is what lies between there and the next
// request's first place, so no prefix sum is needed.)
//
// Two kernels do the pages.  No more rows than requests (decode steps): a block to a warp,
// and a CTA to two places (one request's, most of the time); four rows at a time, gone over
// twice where there are more.  Otherwise a CTA has one side of a page and some of its heads,
// and a thread 16 channels of two rows (of one in the smallest pages), so that an angle's
// sine and cosine are spent once for all of the heads; a head's rows stay in registers
// between the maximum, which the CTA finds together, and the codes, while the next heads'
// are on their way.
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
  int each;                              // heads of a CTA (many rows)
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
                                              int64_t m, int &err) {
  Touched t{lo, 0, 0, (int64_t)(lo >> P.cache.shift) + 2ll * r, 0};
  if (lo < 0 || hi < lo || hi > P.num_q) {
    err |= CSA2_DERR_BAD_EXTEND;
    return t;
  }
  if (hi == lo) return t;
  const int64_t n = hi - lo;
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

// x / scale, by the reciprocal where that is exact.  (Divisions take a path of their
// own: chosen for each value, they cost 14 of 20 instructions a value.)
struct Divider {
  float scale, inv;
  bool exact;
};
__device__ __forceinline__ Divider by_scale(float s) {
  const uint32_t u = __float_as_uint(s);                 // 2^e: 2^-e has 254 - its exponent
  return Divider{s, __uint_as_float((254u << 23) - u), (u & 0x7fffffu) == 0};
}

// codes of four values
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3) {
  uint32_t r;
  asm("{ .reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h}; }"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

// a thread's 16 channels, divided
__device__ __forceinline__ void divide16(float (&x)[2 * kUnit], const Divider &by) {
  if (by.exact) {
    const uint64_t inv = pack2(by.inv, by.inv);
#pragma unroll
    for (int i = 0; i < 2 * kUnit; i += 2) {
      const float2 y = unpack2(rope::mul2(pack2(x[i], x[i + 1]), inv));
      x[i] = y.x, x[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * kUnit; ++i) x[i] = __fdiv_rn(x[i], by.scale);
  }
}
__device__ __forceinline__ void store16(uint8_t *row, const rope::Place &at,
                                        const float (&x)[2 * kUnit]) {
  *reinterpret_cast<uint2 *>(row + at.a) =
      make_uint2(codes4(x[0], x[1], x[2], x[3]), codes4(x[4], x[5], x[6], x[7]));
  *reinterpret_cast<uint2 *>(row + at.b) =
      make_uint2(codes4(x[8], x[9], x[10], x[11]), codes4(x[12], x[13], x[14], x[15]));
}

// 16 codes times `ratio`, rounded again
__device__ __forceinline__ uint4 rescaled(uint4 w, float ratio) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = f16x2_of(v[i]), b = f16x2_of_high(v[i]);
    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    v[i] = codes4(x.x * ratio, x.y * ratio, y.x * ratio, y.y * ratio);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// 16 channels as they lie in memory
struct Raw {
  uint4 a, b;
};
template <typename T>
__device__ __forceinline__ Raw load_raw(const T *src, const rope::Place &at) {
  return Raw{*reinterpret_cast<const uint4 *>(src + at.a), *reinterpret_cast<const uint4 *>(src + at.b)};
}

// The channels, rotated, and as zeros where the row's head (the lanes of a team) has
// anything that is not finite; their largest magnitude.
template <typename T, int D, bool kInterleaved>
__device__ __forceinline__ float open_row(const Raw &raw, const rope::Place &at,
                                          const float (&c)[kUnit], const float (&s)[kUnit],
                                          float (&x)[2 * kUnit], int &err) {
  constexpr int kTeam = D / 16;
  rope::unpack8<T>(raw.a, x);
  rope::unpack8<T>(raw.b, x + kUnit);
  rope::turn16<kInterleaved>(x, at, c, s);
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 2 * kUnit; i += 2)                 // (a NaN stays)
    asm("max.NaN.f32 %0, %1, %2, %3;"
        : "=f"(amax)
        : "f"(amax), "f"(fabsf(x[i])), "f"(fabsf(x[i + 1])));
  const uint32_t bad = __ballot_sync(0xffffffffu, !(amax <= 3.402823466e38f));
  if (bad) {
    const int lane = threadIdx.x & 31, team = lane / kTeam * kTeam;
    if ((bad >> team) & ((1u << kTeam) - 1)) {
      err |= CSA2_DERR_NONFINITE;
      amax = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * kUnit; ++i) x[i] = 0.f;
    }
  }
  return amax;
}

// The page that a CTA has: request, its rows, page number in the request, id (-1: none).
struct Found {
  Touched t;
  int run, id;
  int64_t p;
};

// Calls f(found) for each page of a request that has one of `places` places from `place`
// on.  In a malformed batch places may be several requests'; of more than kMost the first
// are served, or a batch whose requests all lie over one another would take requests times
// pages of time.
constexpr int kMost = 32;

template <typename F>
__device__ __forceinline__ void each_page(const AppendParams &P, int64_t place, int places,
                                          const F &f) {
  __shared__ Touched held;
  __shared__ int found, matches;
  for (int from = 0, served = 0; served < kMost; ++served) {
    if (threadIdx.x == 0) found = 0x7fffffff, matches = 0;
    __syncthreads();
    int mine = 0x7fffffff;
    Touched t;
#pragma unroll 2
    for (int r = from + threadIdx.x; r < P.num_req; r += blockDim.x) {
      int ignored = 0;
      const Touched u = touched_by(P, r, P.cu_q[r], P.cu_q[r + 1], P.kv_len[r], ignored);
      if (place + places > u.place && place - u.place < u.pages) {
        if (mine == 0x7fffffff) mine = r, t = u;
        atomicMin(&found, r);
        atomicAdd(&matches, 1);
      }
    }
    __syncthreads();
    const int r = found, n = matches;
    if (n == 0) return;
    if (r == mine) held = t;
    __syncthreads();
    const Touched u = held;
    const int i1 = (int)min((int64_t)u.pages, place + places - u.place);
    for (int i = (int)max(place - u.place, (int64_t)0); i < i1; ++i) {
      const int64_t p = (u.row0 >> P.cache.shift) + i;
      f(Found{u, r, P.cache.table[r * P.cache.table_ld + p], p});
    }
    if (n == 1) return;
    from = r + 1;
    __syncthreads();
  }
}

__device__ __forceinline__ bool is_page(const AppendParams &P, int id, int &err) {
  if (id >= 0 && id < P.cache.num_pages) return true;
  err |= CSA2_DERR_RANGE_ROW;
  return false;
}

// the last block of a grid has no page: it looks at every request
__device__ __forceinline__ void check_batch(const AppendParams &P) {
  int err = 0;
  for (int r = threadIdx.x; r < P.num_req; r += blockDim.x)
    touched_by(P, r, P.cu_q[r], P.cu_q[r + 1], P.kv_len[r], err);
  if (err) raise_err(P.d_err, err);
}

// ---------------------------------------------------------------------------
// no more rows than requests: a block to a warp
// ---------------------------------------------------------------------------
constexpr int kWarps = 16;

template <typename T, int D, bool kInterleaved>
__device__ __forceinline__ void append_block(const AppendParams &P, const uint64_t *turn,
                                             const Found &F, int h, int side, int &err) {
  constexpr int kTeam = D / 16, kStep = 32 / kTeam;      // lanes of a row, rows at a time
  const Pages &C = P.cache;
  const Touched &t = F.t;
  const int lane = threadIdx.x & 31, i = lane % kTeam;
  const int64_t base = F.p << C.shift;
  const int first = (int)max(t.row0 - base, (int64_t)0), end = (int)min(t.m - base, (int64_t)C.page);
  const rope::Place at = rope::place_of<D, kInterleaved>(i, side == 0 && P.rope.freq ? P.rope.rot : 0);
  const int64_t ld = side ? P.ldv : P.ldk;
  const T *src = static_cast<const T *>(side ? P.v : P.k) + (int64_t)h * D;
  const auto query = [&](int row) { return t.q0 + (base + row - t.row0); };
  const auto raw_of = [&](int row) {
    return row < end ? load_raw(src + query(row) * ld, at) : Raw{};
  };
  float x[2 * kUnit];
  const auto open = [&](const Raw &raw, int row) {
    float c[kUnit], s[kUnit];
    if ((at.ta || at.tb) && row < end)
      rope::angles<D, kInterleaved>(turn, i, at, P.rope.pos ? P.rope.pos[query(row)] : base + row,
                                    P.rope.amplitude, 1.f, c, s);
    else
      for (int k = 0; k < kUnit; ++k) c[k] = s[k] = 0.f;       // of zeros
    return open_row<T, D, kInterleaved>(raw, at, c, s, x, err);
  };
  // the first rows are asked for before the page is known to be one
  const Raw first_rows = raw_of(first + lane / kTeam);
  if (!is_page(P, F.id, err)) return;
  float *scale = (side ? C.v_scale : C.k_scale) + (int64_t)F.id * P.n_kv + h;
  const float stored = first > 0 ? *scale : 0.f;
  uint8_t *codes = (side ? C.v + F.id * C.v_stride : C.k + F.id * C.k_stride) +
                   (int64_t)h * C.page * D;
  float amax = open(first_rows, first + lane / kTeam);
  int row0 = first;
  for (int r = first + kStep; r < end; r += kStep) {
    row0 = r;
    amax = fmaxf(amax, open(raw_of(r + lane / kTeam), r + lane / kTeam));
  }
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  float now = need_of(amax, err);
  if (first > 0) {
    const float old = scale_of(stored, err);
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
    divide16(x, by);
    if (row < end) store16(codes + row * D, at, x);
    if (r == first) break;
    open(raw_of(row - kStep), row - kStep);
  }
}

template <typename T, int D, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32)
append_few_kernel(const __grid_constant__ AppendParams P) {
  __shared__ uint64_t turn[D / 2];
  if (blockIdx.x == gridDim.x - 1) return check_batch(P);
  int err = 0;
  if (P.rope.freq) rope::load_turns(P.rope, turn);       // (a barrier follows)
  each_page(P, 2 * (int64_t)blockIdx.x, 2, [&](const Found &F) {
    for (int i = threadIdx.x >> 5; i < 2 * P.n_kv; i += kWarps)
      append_block<T, D, kInterleaved>(P, turn, F, i >> 1, i & 1, err);
  });
  if (err) raise_err(P.d_err, err);
}

// ---------------------------------------------------------------------------
// many rows: a side of a page to a CTA, kRows rows of 16 channels to a thread
// ---------------------------------------------------------------------------
constexpr int kAhead = 4;                // heads whose rows are on their way or there

// 16 bytes into shared memory, or zeros
__device__ __forceinline__ void copy16(void *to, const void *from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from),
               "r"(there ? 16 : 0)
               : "memory");
}

template <typename T, int D, bool kInterleaved, int kRows>
__global__ void __launch_bounds__(kRows == 1 ? 128 : 512, kRows == 1 ? 8 : 1)
append_many_kernel(const __grid_constant__ AppendParams P) {
  constexpr int kTeam = D / 16;
  __shared__ uint64_t turn[D / 2];
  __shared__ uint32_t top[3];                            // a head's maximum, by head modulo 3
  extern __shared__ __align__(16) uint4 staged[];        // [kAhead][kRows][2][threads]
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0) check_batch(P);
    return;
  }
  const Pages &C = P.cache;
  const int side = blockIdx.y & 1;
  const int h0 = (int)(blockIdx.y >> 1) * P.each, h1 = min(P.n_kv, h0 + P.each);
  int err = 0;
  const bool rot = side == 0 && P.rope.freq;
  if (rot) rope::load_turns(P.rope, turn);               // (a barrier follows)
  if (threadIdx.x < 3) top[threadIdx.x] = 0;
  each_page(P, blockIdx.x, 1, [&](const Found &F) {
    if (!is_page(P, F.id, err)) return;
    const Touched &t = F.t;
    const int64_t base = F.p << C.shift;
    const int first = (int)max(t.row0 - base, (int64_t)0);
    const int end = (int)min(t.m - base, (int64_t)C.page);
    const int i = threadIdx.x % kTeam, mine = threadIdx.x / kTeam, step = blockDim.x / kTeam;
    const rope::Place at = rope::place_of<D, kInterleaved>(i, rot ? P.rope.rot : 0);
    const int64_t ld = side ? P.ldv : P.ldk;
    const T *src[kRows];
    bool there[kRows];
    float c[kRows][kUnit], s[kRows][kUnit];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const int row = mine + k * step;
      const int64_t q = t.q0 + (base + row - t.row0);
      there[k] = row >= first && row < end;
      src[k] = static_cast<const T *>(side ? P.v : P.k) + (there[k] ? q * ld : 0) +
               (int64_t)h0 * D;
#pragma unroll
      for (int e = 0; e < kUnit; ++e) c[k][e] = s[k][e] = 0.f;
      if ((at.ta || at.tb) && there[k])
        rope::angles<D, kInterleaved>(turn, i, at, P.rope.pos ? P.rope.pos[q] : base + row,
                                      P.rope.amplitude, 1.f, c[k], s[k]);
    }
    float *scale = (side ? C.v_scale : C.k_scale) + (int64_t)F.id * P.n_kv;
    uint8_t *page = side ? C.v + F.id * C.v_stride : C.k + F.id * C.k_stride;
    // a thread copies what it reads itself, so that no barrier is needed for it
    uint4 *const own = staged + threadIdx.x;
    const int unit = blockDim.x, stage = 2 * kRows * unit;
    int to = 0, from = 0, next = h0;                     // stages, and the next head to copy
    const auto fetch = [&]() {
      if (next < h1) {
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
          copy16(own + to + 2 * k * unit, src[k] + at.a, there[k]);
          copy16(own + to + (2 * k + 1) * unit, src[k] + at.b, there[k]);
          src[k] += D;
        }
        to = to == (kAhead - 1) * stage ? 0 : to + stage;
        ++next;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int h = 0; h < kAhead - 1; ++h) fetch();
    for (int h = h0, slot = 0; h < h1; ++h, slot = slot == 2 ? 0 : slot + 1) {
      const float kept = first > 0 ? scale[h] : 0.f;
      fetch();
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      float x[kRows][2 * kUnit], amax = 0.f;
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        amax = fmaxf(amax, open_row<T, D, kInterleaved>(Raw{own[from + 2 * k * unit], own[from + (2 * k + 1) * unit]}, at, c[k], s[k], x[k], err));
      from = from == (kAhead - 1) * stage ? 0 : from + stage;
      const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
      if ((threadIdx.x & 31) == 0) atomicMax(&top[slot], most);
      __syncthreads();
      float now = need_of(__uint_as_float(top[slot]), err);
      // the slot before this was read before the barrier, and is next used after another
      if (threadIdx.x == 0) top[slot == 0 ? 2 : slot - 1] = 0;
      uint8_t *codes = page + (int64_t)h * C.page * D;
      if (first > 0) {
        const float old = scale_of(kept, err);
        if (now > old) {
          uint4 *w = reinterpret_cast<uint4 *>(codes);
          for (int j = threadIdx.x; j < first * (D / 16); j += blockDim.x)
            w[j] = rescaled(w[j], old / now);
        } else {
          now = old;
        }
      }
      if (threadIdx.x == 0) scale[h] = now;
      const Divider by = by_scale(now);
#pragma unroll
      for (int k = 0; k < kRows; ++k)
        if (there[k]) {
          divide16(x[k], by);
          store16(codes + (mine + k * step) * D, at, x[k]);
        }
    }
    __syncthreads();
    if (threadIdx.x < 3) top[threadIdx.x] = 0;           // for another page
    __syncthreads();
  });
  if (err) raise_err(P.d_err, err);
}

template <typename T, int D, bool kInterleaved>
int launch_many(const AppendParams &P, dim3 grid, cudaStream_t st) {
  const int threads = P.cache.page * (D / 16);
  const int smem = kAhead * 2 * 16 * threads;
  if (threads < 256) {
    allow_smem<append_many_kernel<T, D, kInterleaved, 1>>(kAhead * 2 * 16 * 128);
    append_many_kernel<T, D, kInterleaved, 1><<<grid, threads, smem, st>>>(P);
  } else {
    allow_smem<append_many_kernel<T, D, kInterleaved, 2>>(kAhead * 2 * 16 * 1024);
    append_many_kernel<T, D, kInterleaved, 2><<<grid, threads / 2, smem, st>>>(P);
  }
  return launch_status();
}

template <typename T, int D>
int launch(AppendParams &P, int places, cudaStream_t st) {
  // (128 requests of two rows each on average, some of them with more, take 12 us by the
  // one kernel and 8 to 14 by the other, 128 single rows 5 and 8 to 14)
  if (P.num_q <= P.num_req) {
    const int grid = (places + 1) / 2 + 1;
    if (P.rope.freq && P.rope.interleaved)
      append_few_kernel<T, D, true><<<grid, kWarps * 32, 0, st>>>(P);
    else
      append_few_kernel<T, D, false><<<grid, kWarps * 32, 0, st>>>(P);
    return launch_status();
  }
  // all heads of a side in one CTA, unless the pages are too few to fill the GPU with
  // 1024 threads to an SM
  int chunks = 1;
  const int64_t pages = (P.num_q >> P.cache.shift) + P.num_req;
  while (chunks < P.n_kv && pages * 4 * chunks * P.cache.page * (D / 16) <= 1024ll * kSms)
    chunks *= 2;
  P.each = (P.n_kv + chunks - 1) / chunks;
  const dim3 grid((unsigned)places + 1, 2u * (unsigned)((P.n_kv + P.each - 1) / P.each));
  return P.rope.freq && P.rope.interleaved ? launch_many<T, D, true>(P, grid, st)
                                           : launch_many<T, D, false>(P, grid, st);
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
