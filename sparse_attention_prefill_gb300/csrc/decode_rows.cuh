// Which query row, key head and split a block of the single-token kernels has.
#pragma once
#include "dense.cuh"

namespace csa2 {
namespace dense {
namespace {

// The run that holds query row `token`, by the block; -1: none.
template <int kWarps>
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

// Calls item(token, run, first query row and rows of the run, its first cache row
// and cache rows, key head, split) for what block blockIdx.x of a grid of num_q *
// n_kv * splits + 1 has to do.  kPaged: runs have no first row, and at most
// S.kv_rows rows.
template <int kWarps, bool kPaged, typename F>
__device__ __forceinline__ void each_item(const Seqs &S, int n_kv, int group, int splits,
                                          float *part_lse, int32_t *d_err,
                                          uint32_t (&tmp)[kWarps], const F &item) {
  const int ns = splits > 0 ? splits : 1;
  int split = blockIdx.x % ns, h = blockIdx.x / ns % n_kv;
  int err = 0;
  if (blockIdx.x == gridDim.x - 1) {         // no item: looks at every request's rows
    for (int r = threadIdx.x, a, b; r < S.count; r += kWarps * 32) seq_rows(S, r, a, b, err);
    err = __reduce_or_sync(0xffffffffu, err);
    if ((threadIdx.x & 31) == 0) raise_err(d_err, err);
    return;
  }
  // Query row `token`: the rows from the first request's on, then those in front
  // of it.  In a batch of single tokens row number i of these is run i's, and
  // everything of it is asked for at once; otherwise its run is looked for.
  const int slot = blockIdx.x / ns / n_kv, first = S.cu_q[0], end = S.cu_q[S.count];
  int run = min(slot, S.count - 1);
  int q0 = S.cu_q[run], behind = S.cu_q[run + 1];
  int64_t start = kPaged ? 0 : S.kv_start[run], m = S.kv_len[run];
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
    run = run_of<kWarps>(S, token, tmp);
    if (run < 0) {
      // the join leaves the row
      if (splits > 0 && split == 0) {
        const int64_t rows = part_rows(S.num_q, group), row = (int64_t)token * group;
        for (int i = threadIdx.x; i < (sweep ? n_kv : 1) * group; i += kWarps * 32)
          part_lse[part_stat(rows, n_kv, 0, h + i / group, row + i % group)] =
              __uint_as_float(kNobody);
      }
      return;
    }
    q0 = S.cu_q[run], behind = S.cu_q[run + 1];
  }
  if (kPaged) {
    start = 0;
    m = S.kv_len[run];
    if (m < 0 || m > S.kv_rows) m = 0, err |= CSA2_DERR_RANGE_ROW;
  } else {
    seq_keys(S, run, start, m, err);
  }
  if (err && threadIdx.x == 0) raise_err(d_err, err);
  for (;;) {
    item(token, run, q0, behind - q0, start, m, h, split);
    if (!sweep) return;
    __syncthreads();
    if (++split == ns) {
      split = 0;
      if (++h == n_kv) return;
    }
  }
}

}  // namespace
}  // namespace dense
}  // namespace csa2
