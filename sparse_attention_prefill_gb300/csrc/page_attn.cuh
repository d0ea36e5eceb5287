// Attention over 8-bit pages: what its kernels and its entry point share.
//
// A block's codes K8, V8 have the scales a and b (rows are a K8 and b V8).  With
//   x_j = c a_j <q, K8_j> + log2 b_j        (c: sm_scale log2 e)
// the weight of V8_j is 2^x_j, and that of the softmax's sum 2^x_j / b_j: the scales
// of V ride in the exponent, and the running maximum is that of x, so that weights fit
// f16 whatever the scales are.
#pragma once
#include "pages.cuh"

namespace csa2 {
namespace pages {

struct PageAttnParams {
  dense::AttnParams at;          // seqs.kv_start is null, kv_rows what the table has room for
  Pages cache;
  const void *q;
  int64_t ldq;
};

// f16 weights: scaled up by 2^kLift, so that those down to 2^-22 of the largest keep
// full precision; the reference moves when a logit passes it by kMargin, and the
// largest weight stays below 2^16.
constexpr float kLift = 8.f, kMargin = 7.f;

// Single tokens (page_decode.cu); ws: page_decode_bytes, or null: items are not shared
// among CTAs.
int64_t page_decode_bytes(const Shape &s);
int page_decode(const Shape &s, const PageAttnParams &P, int64_t max_kv, const csa2_pages *c,
                void *ws, cudaStream_t st);

// Tiles (page_tiles.cuh).  For the join: the item that began in the share before and goes on
// in this one: its first query row, tokens, key head and parts.
struct TileMark {
  int q0, tokens, h, parts;
};
struct TilesWs {
  TileMark *marks;                       // null: items are handed out whole
  int rows;                              // of a part
};
struct TileMaps {
  CUtensorMap q, k, v;
};
int page_tiles_64(bool bf16, const AttnParams &P, const Pages &C8, const TilesWs &ws, bool narrow,
                  int items, const TileMaps &m, cudaStream_t st);
int page_tiles_128(bool bf16, const AttnParams &P, const Pages &C8, const TilesWs &ws, bool narrow,
                   int items, const TileMaps &m, cudaStream_t st);

// Power of two that takes a query row's largest magnitude to [2^14, 2^15), so that
// its bf16 channels are f16 ones.
__device__ __forceinline__ float lift_of(float amax) {
  const int e = (int)(__float_as_uint(amax) >> 23) - 127;
  return __uint_as_float((uint32_t)(min(14 - e, 100) + 127) << 23);
}

}  // namespace pages
}  // namespace csa2
