// What the calls on 8-bit pages share: the cache on the device, its tensor maps,
// E4M3 conversions and host checks.
#pragma once
#include "dense.cuh"

namespace csa2 {
namespace pages {

using namespace dense;

constexpr float kLowScale = 0x1p-32f, kHighScale = 0x1p32f;
constexpr float kTop = 448.f;            // the largest E4M3 value

struct Pages {
  int num_pages, page, shift;            // shift: log2 of page
  uint8_t *k, *v;
  int64_t k_stride, v_stride;
  float *k_scale, *v_scale;
  const int32_t *table;
  int64_t table_ld, most;                // rows that a request may have
};

inline Pages to_device_view(const csa2_pages *c) {
  Pages p;
  p.num_pages = c->num_pages;
  p.page = c->page;
  p.shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  p.k = static_cast<uint8_t *>(c->k);
  p.v = static_cast<uint8_t *>(c->v);
  p.k_stride = c->k_stride;
  p.v_stride = c->v_stride;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.table = c->table;
  p.table_ld = c->table_ld;
  p.most = c->table_ld * c->page;
  return p;
}

// a stored scale, brought into its range
__device__ __forceinline__ float scale_of(float s, int &err) {
  if (s >= kLowScale && s <= kHighScale) return s;
  err |= CSA2_DERR_SCALE;
  return s > kHighScale ? kHighScale : kLowScale;
}

// page `p` of request r; -1 where the table names none
__device__ __forceinline__ int page_id(const Pages &C, int r, int64_t p, int &err) {
  const int id = C.table[r * C.table_ld + p];
  if (id >= 0 && id < C.num_pages) return id;
  err |= CSA2_DERR_RANGE_ROW;
  return -1;
}

// two E4M3 codes (low byte first) to f16, exact
__device__ __forceinline__ uint32_t f16x2_of(uint32_t two) {
  uint32_t h;
  asm("{ .reg .b16 c; cvt.u16.u32 c, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(h) : "r"(two));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_of_high(uint32_t four) {
  uint32_t h;
  asm("{ .reg .b16 l, c; mov.b32 {l, c}, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(h) : "r"(four));
  return h;
}

// [pages, lines of 128 bytes] of one side, as boxes of `rows` rows of a page (a row
// of 64 channels is half a line) in the 128-byte swizzle
inline bool make_pages_map(CUtensorMap *map, const void *base, int64_t num_pages, int n_kv,
                           int page, int dim, int64_t stride, int rows) {
  EncodeTiled fn = encode_tiled();
  if (!fn) return false;
  const cuuint64_t dims[3] = {128, (cuuint64_t)n_kv * page * dim / 128, (cuuint64_t)num_pages};
  const cuuint64_t strides[2] = {128, (cuuint64_t)stride};
  const cuuint32_t box[3] = {128, (cuuint32_t)(rows * dim / 128), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The maps of both sides, with boxes of `rows` rows or a page, whichever is fewer.
// Without pages nothing is ever fetched, and the maps are of `any`.
inline bool make_cache_maps(CUtensorMap *mk, CUtensorMap *mv, const csa2_pages *c,
                            const void *any, const Shape &s, int rows) {
  const bool none = c->num_pages == 0;
  const int64_t wide = (int64_t)s.n_kv * c->page * s.dim;
  const auto make = [&](CUtensorMap *m, const void *p, int64_t stride) {
    return make_pages_map(m, none ? any : p, none ? 1 : c->num_pages, s.n_kv, c->page, s.dim,
                          stride < wide ? wide : stride, rows < c->page ? rows : c->page);
  };
  return make(mk, c->k, c->k_stride) && make(mv, c->v, c->v_stride);
}

// ---------------------------------------------------------------------------
// host checks
// ---------------------------------------------------------------------------
inline int check_pages(const csa2_pages *c, int n_kv, int dim) {
  if (!c || c->num_pages < 0 || c->table_ld < 0) return CSA2_ERR_INVALID_ARG;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128)
    return CSA2_ERR_UNSUPPORTED;
  if (c->table_ld > (0x7fffffffll - 2 * kTile) / c->page) return CSA2_ERR_UNSUPPORTED;
  if (c->table_ld > 0 && !c->table) return CSA2_ERR_INVALID_ARG;
  if (c->num_pages > 0) {
    const int64_t wide = (int64_t)n_kv * c->page * dim;
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return CSA2_ERR_INVALID_ARG;
    if (c->num_pages > 1 && (c->k_stride < wide || c->v_stride < wide))
      return CSA2_ERR_INVALID_ARG;
    if (!aligned(16, c->k, c->v) || (c->k_stride & 15) || (c->v_stride & 15) ||
        c->k_stride > (1ll << 39) || c->v_stride > (1ll << 39))
      return CSA2_ERR_UNSUPPORTED;
  }
  return aligned(4, c->k_scale, c->v_scale, c->table) ? CSA2_OK : CSA2_ERR_UNSUPPORTED;
}

// the bytes between one side's pages (with one page they do not matter)
inline int64_t side_stride(const csa2_pages *c, int n_kv, int dim, int64_t stride) {
  const int64_t wide = (int64_t)n_kv * c->page * dim;
  return stride < wide ? wide : stride;
}

// n bytes from p on against the codes, scales and table of a cache
inline bool meets_pages(const void *p, uint64_t n, const csa2_pages *c, int n_kv, int dim,
                        int num_req) {
  if (!p) return false;
  const int64_t wide = (int64_t)n_kv * c->page * dim;
  const uint64_t ns = (uint64_t)c->num_pages * n_kv * 4;
  return meets_rows(p, n, c->k, c->num_pages, side_stride(c, n_kv, dim, c->k_stride), wide) ||
         meets_rows(p, n, c->v, c->num_pages, side_stride(c, n_kv, dim, c->v_stride), wide) ||
         overlap(p, n, c->k_scale, ns) || overlap(p, n, c->v_scale, ns) ||
         overlap(p, n, c->table, (uint64_t)num_req * c->table_ld * 4);
}

// a packed batch whose requests lie in pages
inline int check_paged(const csa2_packed *b, const csa2_pages *c, int n_kv, int dim) {
  if (!b || b->num_q < 0 || b->num_req < 0) return CSA2_ERR_INVALID_ARG;
  if (b->num_q > 0 && b->num_req > 0 && (!b->cu_q || !b->kv_len)) return CSA2_ERR_INVALID_ARG;
  if (!aligned(4, b->cu_q) || !aligned(8, b->kv_len)) return CSA2_ERR_UNSUPPORTED;
  return check_pages(c, n_kv, dim);
}

}  // namespace pages
}  // namespace csa2
