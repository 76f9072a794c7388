// paged_tiles_window.cu -- the launches of the tile kernel (paged_tiles.cuh) over a window.

#include "paged_tiles.cuh"

namespace q8a {

cudaError_t launch_paged_tiles_window(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                      cudaStream_t stream) {
  return plan.pair ? launch_tiles_mode<true, kWindow>(a, dtype, head_dim, plan, stream)
                   : launch_tiles_mode<false, kWindow>(a, dtype, head_dim, plan, stream);
}

}  // namespace q8a
