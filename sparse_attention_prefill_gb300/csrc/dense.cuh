// What the dense-cache kernels share (prompt and shared-prefix attention,
// accumulated attention weight): the packed batch on the device, the tensor
// maps of Q, K and V, and bounded waits.
//
// Packed rows.  n_heads query heads share n_kv_heads key heads, G = n_heads /
// n_kv_heads to each.  A query tile holds the rows (token, head of the group)
// of one key head, token-major: row x is token x / G, head h * G + x % G, so
// that short extends and decode steps fill a tile with heads, and the causal
// edge crosses few tiles.  A tile has tpt tokens (tpt * G <= 128 rows); TMA
// fetches it as one box (64 channels, G heads, tpt tokens) per 64 channels,
// which lands as consecutive 128-byte rows.
#pragma once
#include "common.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace csa2 {
namespace dense {

using namespace tc;

constexpr int kTile = 128;            // rows of a query tile, keys of a key tile
constexpr uint32_t kBlk = 128 * 128;  // bytes of a 128-row, 64-channel operand block
constexpr int kSms = 152;             // GB300: split plans are made for this count
constexpr uint64_t kDrainNs = 2000000000ull;

// ---------------------------------------------------------------------------
// waits: bounded, and left early once another role has given up
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t gtimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
  return t;
}

struct Bound {
  uint64_t wait_ns;
  int abort;
};

// poll without suspending
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_slow(uint64_t *bar, uint32_t parity, Bound *bd) {
  // the hardware suspends a try_wait for some microseconds: a bound shorter
  // than that is polled for
  const uint64_t t0 = gtimer(), limit = bd->wait_ns;
  while (limit < 100000 ? !mbar_test(bar, parity) : !mbar_try_wait(bar, parity)) {
    if (*(volatile int *)&bd->abort) return false;
    if (gtimer() - t0 > limit) {
      atomicExch(&bd->abort, 1);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, Bound *bd) {
  if (mbar_test(bar, parity)) return true;
  return wait_slow(bar, parity, bd);
}

// the same without a call, for the elected lane between its products
__device__ __forceinline__ void wait_inline(uint64_t *bar, uint32_t parity, Bound *bd) {
  if (mbar_test(bar, parity)) return;
  const uint64_t t0 = gtimer(), limit = bd->wait_ns;
  while (!mbar_test(bar, parity)) {
    if (*(volatile int *)&bd->abort) return;
    if (gtimer() - t0 > limit) {
      atomicExch(&bd->abort, 1);
      return;
    }
  }
}

// the same by a whole warp, which goes on or gives up together
__device__ __forceinline__ bool wait_all(uint64_t *bar, uint32_t parity, Bound *bd) {
  return __all_sync(0xffffffffu, wait_bar(bar, parity, bd));
}

// One lane of a converged warp (the same one every time).  Products are issued
// by the elected lane of a warp that runs its whole loop together: operands of
// an MMA live in uniform registers, which only warp-uniform code computes in
// place.  From a lane-0 branch each is moved over first, which holds the
// tensor pipe at 70 cycles for an M = N = 128, K = 16 product with both
// operands in shared memory and 107 with A in TMEM; issued this way it runs
// at its own 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Cluster launch control: asks for the index of a CTA of this grid that has not
// started, which then does not start; the answer (16 bytes) completes on `bar`.
__device__ __forceinline__ void ask_next(uint64_t *answer, uint64_t *bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], "
      "[%1];" ::"r"(smem_u32(answer)),
      "r"(smem_u32(bar))
      : "memory");
}
// The answer: false if no CTA is left (no further request may be made then).
__device__ __forceinline__ bool next_cta(const uint64_t *answer, uint32_t &cta) {
  uint32_t got;
  asm volatile(
      "{\n\t.reg .b128 a;\n\t.reg .pred p;\n\t"
      "mov.b128 a, {%2, %3};\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, a;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, a;\n\t}"
      : "=r"(got), "=r"(cta)
      : "l"(((const volatile uint64_t *)answer)[0]), "l"(((const volatile uint64_t *)answer)[1]));
  return got != 0;
}

// the value of lane 0, known to be the same in every lane
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// wait that ignores the abort flag, for work that has to land before the CTA
// leaves
__device__ __forceinline__ void drain_bar(uint64_t *bar, uint32_t parity) {
  const uint64_t t0 = gtimer();
  while (!mbar_try_wait(bar, parity) && gtimer() - t0 < kDrainNs) {
  }
}

// 2^x on the special-function unit (ex2.approx: relative error ~2^-22)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// two fp32 operations in one instruction, on register pairs
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// A operand in TMEM (16-bit elements, two per 32-bit column), B in shared memory
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

template <typename T> struct Elem;
template <> struct Elem<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
};
template <> struct Elem<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float lo, float hi) {
    __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
  }
};

template <typename T>
__host__ __device__ constexpr uint32_t idesc_of(uint32_t m, uint32_t n, bool b_mn) {
  return make_idesc_f16(m, n, false, b_mn) | (Elem<T>::kBf16 ? (1u << 7) | (1u << 10) : 0u);
}

// ---------------------------------------------------------------------------
// sequences on the device: `count` runs of query rows, each with its run of
// cache rows.  With cu_group set, run i is a group of requests: its query
// rows are those of the requests cu_group[i] .. cu_group[i+1] - 1.
// ---------------------------------------------------------------------------
struct Seqs {
  int count, num_q, num_req;
  const int32_t *cu_q;
  const int32_t *cu_group;
  const int64_t *kv_start, *kv_len;
  int64_t kv_rows;
};

__device__ __forceinline__ void seq_rows(const Seqs &S, int i, int &q0, int &n, int &err) {
  int a = i, b = i + 1;
  if (S.cu_group) {
    a = S.cu_group[i];
    b = S.cu_group[i + 1];
    if (a < 0 || b < a || b > S.num_req) {
      q0 = n = 0;
      err |= CSA2_DERR_BAD_EXTEND;
      return;
    }
  }
  const int lo = S.cu_q[a], hi = S.cu_q[b];
  if (lo < 0 || hi < lo || hi > S.num_q) {
    q0 = n = 0;
    err |= CSA2_DERR_BAD_EXTEND;
    return;
  }
  q0 = lo;
  n = hi - lo;
}

__device__ __forceinline__ void seq_keys(const Seqs &S, int i, int64_t &start, int64_t &m,
                                         int &err) {
  start = S.kv_start[i];
  m = S.kv_len[i];
  if (m < 0 || start < 0 || start > S.kv_rows || m > S.kv_rows - start) {
    start = m = 0;
    err |= CSA2_DERR_RANGE_ROW;
  }
}

// Partial results: by split and key head, blocks of 32 packed rows (query row *
// group + head of the group), each [D, 32]: lanes with neighbouring rows store
// neighbours, and whoever joins the parts reads a block front to back.  (With
// all rows of a head innermost the channels lay a power of two apart, and the
// join took 20 us instead of 13.4 for 2048 rows x 8 heads x 8 parts.)
__host__ __device__ __forceinline__ int64_t part_rows(int64_t num_q, int group) {
  return (num_q * group + 31) / 32 * 32;
}
// Statistic of a row that no request holds: a NaN that no computation gives.
// decode_attn.cu looks at every query row and writes it for the first split; where
// the own part runs by dense_attn.cu the join looks for the rows' requests.
constexpr uint32_t kNobody = 0x7fffdeadu;
// statistics of packed row `at`; and the element of its channel 0 (channel d: 32 d on)
__device__ __forceinline__ int64_t part_stat(int64_t rows, int n_kv, int split, int h,
                                             int64_t at) {
  return ((int64_t)split * n_kv + h) * rows + at;
}
__device__ __forceinline__ int64_t part_elem(int64_t rows, int n_kv, int dim, int split, int h,
                                             int64_t at) {
  return (((int64_t)split * n_kv + h) * rows + (at & ~(int64_t)31)) * dim + (at & 31);
}

// Whether request r lies in one of the groups that are not skipped, by one warp:
// seq_rows' conditions, or a request of a skipped group would wait in the join for
// a prefix part that nobody wrote.
__device__ __forceinline__ bool in_groups(const int32_t *cu_group, int groups, int r,
                                          const Seqs &S) {
  bool mine = false;
  for (int g = threadIdx.x & 31; g < groups; g += 32) {
    const int a = cu_group[g], b = cu_group[g + 1];
    if (a < 0 || a > r || r >= b || b > S.num_req) continue;
    const int lo = S.cu_q[a], hi = S.cu_q[b];
    mine |= lo >= 0 && lo <= hi && hi <= S.num_q;
  }
  return __any_sync(0xffffffffu, mine);
}

// ---------------------------------------------------------------------------
// tensor maps (host)
// ---------------------------------------------------------------------------
// [rows, heads, dim] with `ld` elements between rows, as boxes of 64 channels
// x box_heads heads x box_rows rows in the 128-byte swizzle
inline bool make_rows_map(CUtensorMap *map, bool bf16, const void *base, int64_t rows, int heads,
                          int dim, int64_t ld, int box_heads, int box_rows) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)ld * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
            const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---------------------------------------------------------------------------
// host checks shared by the entry points
// ---------------------------------------------------------------------------
struct Shape {
  int n_heads, n_kv, dim, group;
  bool bf16;
};

inline int check_packed(const csa2_packed *b, int32_t n_heads, int32_t n_kv_heads, int32_t dim,
                        int32_t dtype, int64_t kv_rows, float sm_scale, Shape *s) {
  if (!b || b->num_q < 0 || b->num_req < 0 || kv_rows < 0) return CSA2_ERR_INVALID_ARG;
  if (n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads) return CSA2_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || !(sm_scale <= 3.402823466e38f)) return CSA2_ERR_INVALID_ARG;
  if (dtype != CSA2_DT_BF16 && dtype != CSA2_DT_F16) return CSA2_ERR_UNSUPPORTED;
  if (dim != 64 && dim != 128) return CSA2_ERR_UNSUPPORTED;
  if (n_heads / n_kv_heads > kTile || n_kv_heads > 1024) return CSA2_ERR_UNSUPPORTED;
  if (kv_rows > 0x7fffffffll - 2 * kTile) return CSA2_ERR_UNSUPPORTED;
  if (b->num_q > 0 && b->num_req > 0 && (!b->cu_q || !b->kv_start || !b->kv_len))
    return CSA2_ERR_INVALID_ARG;
  if (!aligned(4, b->cu_q) || !aligned(8, b->kv_start, b->kv_len)) return CSA2_ERR_UNSUPPORTED;
  *s = Shape{n_heads, n_kv_heads, dim, n_heads / n_kv_heads, dtype == CSA2_DT_BF16};
  return CSA2_OK;
}

// Launches a kernel; with `early` it may start before the kernel in front of it
// in the stream has ended, and must wait for that itself (wait_front).
template <typename... A, typename... B>
int launch_behind(void (*f)(A...), dim3 grid, int threads, int smem, bool early, cudaStream_t st,
                  const B &...args) {
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = &at;
  cfg.numAttrs = early ? 1 : 0;
  cudaLaunchKernelEx(&cfg, f, A(args)...);
  return launch_status();
}

// Waits for the kernel in front and all that it wrote; returns at once in a
// kernel that was not launched early.
__device__ __forceinline__ void wait_front() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Single tokens over their own rows (decode_attn.cu): groups of at most
// kDecodeGroup heads; results or partial results as in dense_attn.cu.
constexpr int kDecodeGroup = 16;
struct DecodeParams {
  Seqs seqs;
  const void *q, *k, *v;
  int64_t ldq, ldk, ldv;
  int n_heads, n_kv, group;
  int splits;
  float scale_log2;
  void *out;
  float *lse, *part_o, *part_lse;
  const int32_t *cover;
  int n_cover, cover_splits;
  float *cover_lse;
  int32_t *d_err;
};
int decode_attn(const Shape &s, const DecodeParams &P, cudaStream_t st);

// rows with `ld` elements between them: TMA wants 16-byte rows and bases
inline int check_rows(const void *p, int64_t ld, int heads, int dim) {
  if (!p || ld < (int64_t)heads * dim) return CSA2_ERR_INVALID_ARG;
  if (((uintptr_t)p & 15u) || (ld & 7) || ld > (1ll << 31)) return CSA2_ERR_UNSUPPORTED;
  return CSA2_OK;
}

// Whether n bytes from p on meet rows of `width` bytes, `step` bytes apart (they
// may lie between two of them).
inline bool meets_rows(const void *p, uint64_t n, const void *rows, int64_t count, int64_t step,
                       int64_t width) {
  if (!p || !rows || count == 0) return false;
  if (!overlap(p, n, rows, (uint64_t)(count - 1) * step + width)) return false;
  const uint64_t x = (uint64_t)(uintptr_t)p, y = (uint64_t)(uintptr_t)rows;
  if (x < y) return true;
  const uint64_t off = (x - y) % (uint64_t)step;
  return off < (uint64_t)width || off + n > (uint64_t)step;
}

// An output (or workspace) of n bytes against what a call reads of a batch.
inline bool meets_batch(const void *p, uint64_t n, const csa2_packed *b) {
  const uint64_t r = (uint64_t)b->num_req;
  return p && (overlap(p, n, b->cu_q, 4 * (r + 1)) || overlap(p, n, b->kv_start, 8 * r) ||
               overlap(p, n, b->kv_len, 8 * r));
}
inline bool meets_groups(const void *p, uint64_t n, const csa2_prefix_groups *g) {
  if (!p || !g || g->num_groups < 1) return false;
  const uint64_t c = (uint64_t)g->num_groups;
  return overlap(p, n, g->cu_group, 4 * (c + 1)) || overlap(p, n, g->prefix_start, 8 * c) ||
         overlap(p, n, g->prefix_len, 8 * c);
}

}  // namespace dense
}  // namespace csa2
