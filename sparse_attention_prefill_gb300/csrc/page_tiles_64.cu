// The tensor-core attention over 8-bit pages for head size 64 (page_tiles.cuh); a file to a
// size, for the build's time.
#include "page_tiles.cuh"

namespace csa2 {
namespace pages {

int page_tiles_64(bool bf16, const AttnParams &P, const Pages &C8, const TilesWs &ws, bool narrow,
                 int items, const TileMaps &m, cudaStream_t st) {
  return bf16 ? launch_any<__nv_bfloat16, 64>(P, C8, ws, narrow, items, m, st)
              : launch_any<__half, 64>(P, C8, ws, narrow, items, m, st);
}

}  // namespace pages
}  // namespace csa2
