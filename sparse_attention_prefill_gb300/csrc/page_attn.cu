// Entry points of the attention over 8-bit pages (csa2_page_attn).
#include "dense_join.cuh"
#include "page_attn.cuh"

namespace csa2 {
namespace pages {
namespace {

// Splits of single tokens: three CTAs to an SM, 128 keys a step.
int plan(const Shape &s, int64_t num_q, int64_t num_req, int64_t max_kv) {
  return plan_splits(num_q * s.n_kv, 3 * kSms, (max_kv + kTile - 1) / kTile, 4.0);
}

int check_call(const csa2_packed *b, int32_t n_heads, int32_t n_kv_heads, int32_t dim,
               int32_t dtype, float sm_scale, Shape *s) {
  csa2_packed none{};
  if (!b || b->num_q < 0 || b->num_req < 0) return CSA2_ERR_INVALID_ARG;
  return check_packed(&none, n_heads, n_kv_heads, dim, dtype, 0, sm_scale, s);
}

}  // namespace
}  // namespace pages
}  // namespace csa2

using namespace csa2;

extern "C" CSA2_API int csa2_page_attn_workspace(int32_t num_q, int32_t num_req, int32_t n_heads,
                                                 int32_t n_kv_heads, int32_t dim, int64_t max_kv,
                                                 int64_t *bytes) {
  if (!bytes || max_kv < 0) return CSA2_ERR_INVALID_ARG;
  csa2_packed b{};
  b.num_q = num_q;
  b.num_req = num_req;
  dense::Shape s;
  const int st = pages::check_call(&b, n_heads, n_kv_heads, dim, CSA2_DT_BF16, 1.f, &s);
  if (st != CSA2_OK) return st;
  const int splits = pages::plan(s, num_q, num_req, max_kv);
  *bytes = splits > 1 ? splits * dense::part_bytes(num_q, s) : 0;
  return CSA2_OK;
}

extern "C" CSA2_API int csa2_page_attn(const csa2_packed *b, int32_t n_heads, int32_t n_kv_heads,
                                       int32_t dim, int32_t dtype, const void *q, int64_t ldq,
                                       const csa2_pages *c, int64_t max_kv, float sm_scale,
                                       void *out, float *lse, void *workspace,
                                       int64_t workspace_bytes, int32_t *d_err,
                                       csa2_stream_t stream) {
  dense::Shape s;
  int st = pages::check_call(b, n_heads, n_kv_heads, dim, dtype, sm_scale, &s);
  if (st == CSA2_OK) st = pages::check_paged(b, c, n_kv_heads, dim);
  if (st != CSA2_OK) return st;
  if (max_kv < 0 || workspace_bytes < 0 || (workspace_bytes > 0 && !workspace))
    return CSA2_ERR_INVALID_ARG;
  if (b->num_q == 0 || b->num_req == 0) return CSA2_OK;
  if ((st = dense::check_rows(q, ldq, n_heads, dim)) != CSA2_OK) return st;
  if (!out) return CSA2_ERR_INVALID_ARG;
  if (!aligned(16, out) || !aligned(4, lse, d_err) || ((uintptr_t)workspace & 255u))
    return CSA2_ERR_UNSUPPORTED;
  const int64_t part = dense::part_bytes(b->num_q, s);
  int splits = pages::plan(s, b->num_q, b->num_req, max_kv);
  if (splits > workspace_bytes / part) splits = (int)(workspace_bytes / part);
  const uint64_t ws = splits > 1 ? (uint64_t)(splits * part) : 0;
  // outputs and workspace against the inputs and each other; out may be q
  const int64_t wide = (int64_t)n_heads * dim * 2;
  const uint64_t no = (uint64_t)b->num_q * wide, nl = (uint64_t)b->num_q * n_heads * 4;
  const bool in_place = out == q && (ldq * 2 == wide || b->num_q == 1);
  const auto meets = [&](const void *p, uint64_t n, bool q_too) {
    return p && n &&
           (overlap(p, n, b->cu_q, 4 * ((uint64_t)b->num_req + 1)) ||
            overlap(p, n, b->kv_len, 8 * (uint64_t)b->num_req) ||
            pages::meets_pages(p, n, c, n_kv_heads, dim, b->num_req) ||
            (q_too && dense::meets_rows(p, n, q, b->num_q, ldq * 2, wide)));
  };
  if (meets(out, no, !in_place) || meets(lse, nl, true) || meets(workspace, ws, true) ||
      (lse && overlap(out, no, lse, nl)) || overlap(workspace, ws, out, no) ||
      (lse && overlap(workspace, ws, lse, nl)))
    return CSA2_ERR_INVALID_ARG;
  pages::PageAttnParams P{};
  P.cache = pages::to_device_view(c);
  P.seqs = dense::Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, nullptr, b->kv_len,
                       P.cache.most};
  P.q = q;
  P.ldq = ldq;
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.out = out;
  P.lse = lse;
  P.d_err = d_err;
  P.wait_ns = wait_limit_ns();
  if (splits > 1) {
    const int64_t rows = dense::part_rows(b->num_q, s.group) * s.n_kv;
    P.splits = splits;
    P.part_o = static_cast<float *>(workspace);
    P.part_lse = P.part_o + splits * rows * s.dim;
  }
  const cudaStream_t cs = as_stream(stream);
  if (s.group > dense::kDecodeGroup) return CSA2_ERR_UNSUPPORTED;
  if ((st = pages::page_decode(s, P, c, cs)) != CSA2_OK || splits <= 1) return st;
  const dense::Join j{P.part_o, P.part_lse, splits, 0, b->num_q, b->num_req, b->cu_q, out, lse};
  return dense::join_parts(s, j, false, cs);
}
