// Equal runs of all items' work, one to a CTA, for the attention kernels on pages.
//
// A request's items (by a rule U: units of it, each with n_kv heads) lie in one row of
// costs, and a CTA's share is an equal run of that row, whatever items it crosses: lengths
// of any mixture fill the GPU evenly.  An item's cost is a fixed one, what its start and end
// take, and one for each step; the steps lie behind the fixed cost, so that every step is in
// one share, and a share that ends within an item's fixed cost has none of its steps.
#pragma once
#include "page_attn.cuh"

namespace csa2 {
namespace pages {
namespace {

// Query rows of a request, and its cache rows.
struct Run {
  int lo, n;                             // (n = 0: none, or skipped)
  int64_t m;
};
// A point of the row: unit i of run `run`, its head, and how far into the item; the query
// rows of the runs in front.
struct Place {
  int run, i, h, off;
  Run u;
  int64_t rows;
};

__device__ __forceinline__ Run run_at(const Seqs &S, int r, int &err) {
  Run u;
  const int64_t m = S.kv_len[r];
  seq_rows(S, r, u.lo, u.n, err);
  u.m = m;
  if (m < 0 || m > S.kv_rows) {
    if (u.n) err |= CSA2_DERR_RANGE_ROW;
    u.m = 0;
  }
  return u;
}

// Equal shares of the cost: `more` of them have one more.
struct Plan {
  int64_t share;
  int shares, more;
};
__device__ __forceinline__ Plan plan_of(int64_t total, int least) {
  Plan p;
  p.shares = max(1, (int)min((int64_t)gridDim.x, total / least));
  // (32 bits divide in a fifth of the time)
  p.share = total >> 32 ? total / p.shares : (int64_t)((uint32_t)total / (uint32_t)p.shares);
  p.more = (int)(total - p.share * p.shares);
  return p;
}
__device__ __forceinline__ int64_t share_begin(const Plan &p, int s) {
  return s < p.shares ? s * p.share + min(s, p.more) : p.shares * p.share + p.more;
}
__device__ __forceinline__ int share_of(const Plan &p, int64_t at) {
  const int64_t big = p.more * (p.share + 1);
  const int64_t off = at < big ? at : at - big, by = at < big ? p.share + 1 : p.share;
  return (at < big ? 0 : p.more) +
         (int)(off >> 32 || by >> 32 ? off / by : (int64_t)((uint32_t)off / (uint32_t)by));
}

// of one head of a run
template <typename U>
__device__ __forceinline__ int64_t cost_of(const U &rule, const Run &u) {
  int64_t c = 0;
  for (int i = 0; i < rule.units(u); ++i) c += U::kFixed + rule.steps(u, i);
  return c;
}

// The place of a run's point `at`.
template <typename U>
__device__ __forceinline__ Place place_in(const U &rule, const Run &u, int run, int n_kv,
                                          int64_t at) {
  Place p{run, 0, 0, 0, u, 0};
  for (int64_t c; at >= (c = U::kFixed + rule.steps(u, p.i)) * n_kv; ++p.i) at -= c * n_kv;
  const int c = U::kFixed + rule.steps(u, p.i);
  for (; at >= c; ++p.h) at -= c;
  p.off = (int)at;
  return p;
}

// Sum of the threads' values in front of this one's, and of all, by the whole CTA.
template <int kThreads>
__device__ __forceinline__ int64_t sum_before(int64_t own, int64_t (&scan)[kThreads / 32],
                                              int64_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t upto = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  __syncthreads();
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) upto += scan[w];
    total += scan[w];
  }
  return upto - own;
}

// The shares, and the place of the CTA's own, by the whole CTA of kThreads threads.
//
// In a malformed batch requests may lie over one another and have any number of rows
// together; they are served in order as long as that is num_q at most.
template <int kThreads, typename U>
__device__ Plan find_share(const U &rule, const Seqs &S, int n_kv,
                           int64_t (&scan)[kThreads / 32], Place &place, int &err) {
  const int per = (S.count + kThreads - 1) / kThreads;
  const int r0 = min(S.count, (int)threadIdx.x * per), r1 = min(S.count, r0 + per);
  int64_t own = 0, rows = 0;
  Run u{0, 0, 0};
#pragma unroll 4
  for (int r = r0; r < r1; ++r) {
    u = run_at(S, r, err);
    rows += u.n;
    if (rows <= S.num_q) own += cost_of(rule, u) * n_kv;
  }
  int64_t total, all;
  int64_t before = sum_before<kThreads>(rows, scan, all);      // query rows in front
  if (all > S.num_q) {                   // (the same in every thread)
    own = 0;
    int64_t upto = before;
    int ignored = 0;
    for (int r = r0; r < r1; ++r) {
      u = run_at(S, r, ignored);
      upto += u.n;
      if (upto <= S.num_q) own += cost_of(rule, u) * n_kv;
    }
  }
  int64_t base = sum_before<kThreads>(own, scan, total);       // of this thread's first run
  const Plan plan = plan_of(total, U::kLeast);
  const int64_t begin = share_begin(plan, (int)blockIdx.x);
  if (base <= begin && begin < base + own) {
    int ignored = 0;
    for (int r = r0; r < r1; ++r) {
      if (per > 1) u = run_at(S, r, ignored);
      const int64_t c = cost_of(rule, u) * n_kv;
      if (begin < base + c) {
        place = place_in(rule, u, r, n_kv, begin - base);
        place.rows = before;
        break;
      }
      base += c;
      before += u.n;
    }
  }
  __syncthreads();
  return plan;
}

// Behind the item at `p`, by a warp; false if there is none.
template <typename U>
__device__ __forceinline__ bool next_item(const U &rule, const Seqs &S, int n_kv, Place &p) {
  const int lane = threadIdx.x & 31;
  p.off = 0;
  if (++p.h < n_kv) return true;
  p.h = 0;
  if (++p.i < rule.units(p.u)) return true;
  p.i = 0;
  int ignored = 0;
  p.rows += p.u.n;
  for (++p.run; p.run < S.count; p.run += 32) {
    int lo = 0, c = 0;
    if (p.run + lane < S.count) seq_rows(S, p.run + lane, lo, c, ignored);
    const uint32_t some = __ballot_sync(0xffffffffu, c > 0);
    if (some) {
      const int src = __ffs(some) - 1;
      if (p.rows + __shfl_sync(0xffffffffu, c, src) > S.num_q) return false;
      p.run += src;
      p.u = run_at(S, p.run, ignored);
      return true;
    }
  }
  return false;
}

// Steps [from, from + n) of the item at `p` in a share that ends `left` behind p.
struct Steps {
  int from, n;
};
template <typename U>
__device__ __forceinline__ Steps steps_in(const Place &p, int all, int64_t left) {
  const int from = max(0, p.off - U::kFixed);
  const int upto = (int)min((int64_t)(U::kFixed + all), p.off + left);
  return Steps{from, max(0, upto - U::kFixed) - from};
}

// How many parts an item has whose steps share `share` cuts at its beginning, if it began
// in the share before; else 0.  The first is the share before's second part, the others are
// first parts.
template <typename U>
__device__ __forceinline__ int parts_of(const U &rule, const Plan &plan, int share,
                                        const Place &p) {
  const int64_t begin = share_begin(plan, share);
  if (begin >= share_begin(plan, share + 1) || p.off <= U::kFixed) return 0;
  const int64_t first = begin - p.off + U::kFixed;   // of the item's steps
  const int64_t last = first + rule.steps(p.u, p.i) - 1;
  return first >= share_begin(plan, share - 1) ? share_of(plan, last) - share + 2 : 0;
}

}  // namespace
}  // namespace pages
}  // namespace csa2
