// Entry points of the attention over 8-bit pages (csa2_page_attn), and the choice among its
// kernels: page_decode.cu for single tokens, page_tiles.cuh for the rest.
#include "dense_roles.cuh"
#include "page_attn.cuh"

namespace csa2 {
namespace pages {
namespace {

constexpr int kMostRuns = 2;         // items to an SM, up to which they are cut

int run_tiles(const Shape &s, const csa2_pages *c, const Pages &C8, const void *q, int64_t ldq,
              const AttnParams &P, const TilesWs &ws, bool narrow, cudaStream_t st) {
  // an upper bound of the items, since the lengths are on the device
  const int64_t tok = narrow ? P.tpt : 2 * P.tpt;
  const int64_t items = (P.seqs.num_q / tok + P.seqs.count) * s.n_kv;
  if (items > 0x7fffffffll) return CSA2_ERR_UNSUPPORTED;
  TileMaps m;
  if (!make_rows_map(&m.q, s.bf16, q, P.seqs.num_q, s.n_heads, s.dim, ldq, s.group, P.tpt) ||
      !make_cache_maps(&m.k, &m.v, c, q, s, kTile))
    return CSA2_ERR_UNSUPPORTED;
  return s.dim == 128 ? page_tiles_128(s.bf16, P, C8, ws, narrow, (int)items, m, st)
                      : page_tiles_64(s.bf16, P, C8, ws, narrow, (int)items, m, st);
}

// How a call runs, and the workspace that it would like.
struct CallPlan {
  int tpt;
  Kind kind;
  int64_t bytes;                         // 0: items whole
};

CallPlan plan(const Shape &s, int64_t num_q, int64_t num_req, int64_t max_kv) {
  CallPlan p{};
  const int64_t runs = num_req > 0 ? num_req : 1;
  p.tpt = tile_tokens(num_q, runs, s.group);
  p.kind = kind_of(num_q, runs, p.tpt, s.group, true);
  if (num_q == 0 || num_req == 0) return p;
  if (p.kind == kSingleTokens) {
    p.bytes = page_decode_bytes(s);
    return p;
  }
  // Runs of tiles where the items are few and there is something to cut; handed out whole,
  // more items even out by themselves, and none is joined.
  const int64_t tok = p.kind == kWideItems ? 2 * p.tpt : p.tpt;
  const int64_t items = (num_q / tok > runs ? num_q / tok : runs) * s.n_kv;
  const int64_t rows = p.kind == kWideItems ? 2 * kTile : kTile;
  if (items <= kMostRuns * kSms && max_kv > 2 * kTile)
    p.bytes = kSms * ((int64_t)sizeof(TileMark) + 2 * rows * (s.dim + 1) * 4);
  return p;
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
  *bytes = pages::plan(s, num_q, num_req, max_kv).bytes;
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
  const pages::CallPlan plan = pages::plan(s, b->num_q, b->num_req, max_kv);
  const uint64_t ws = workspace_bytes >= plan.bytes ? (uint64_t)plan.bytes : 0;
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
  dense::AttnParams P{};
  const pages::Pages C8 = pages::to_device_view(c);
  P.seqs = dense::Seqs{b->num_req, b->num_q, b->num_req, b->cu_q, nullptr, nullptr, b->kv_len,
                       C8.most};
  P.n_heads = s.n_heads;
  P.n_kv = s.n_kv;
  P.group = s.group;
  P.tpt = plan.tpt;
  P.causal = 1;
  P.scale_log2 = sm_scale * 1.4426950408889634f;
  P.out = out;
  P.lse = lse;
  P.d_err = d_err;
  P.wait_ns = wait_limit_ns();
  const cudaStream_t cs = as_stream(stream);
  if (plan.kind == dense::kSingleTokens)
    return pages::page_decode(s, pages::PageAttnParams{P, C8, q, ldq}, max_kv, c,
                              ws ? workspace : nullptr, cs);
  const bool narrow = plan.kind == dense::kNarrowItems;
  pages::TilesWs parts{nullptr, narrow ? dense::kTile : 2 * dense::kTile};
  if (ws) {
    parts.marks = static_cast<pages::TileMark *>(workspace);
    P.part_lse = reinterpret_cast<float *>(parts.marks + dense::kSms);
    P.part_o = P.part_lse + 2 * dense::kSms * parts.rows;
  }
  return pages::run_tiles(s, c, C8, q, ldq, P, parts, narrow, cs);
}
