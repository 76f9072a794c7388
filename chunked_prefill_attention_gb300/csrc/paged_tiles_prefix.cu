// paged_tiles_prefix.cu -- the launches of the tile kernel (paged_tiles.cuh) over a shared prefix and over the keys
// behind it.

#include "paged_tiles.cuh"

namespace q8a {

cudaError_t launch_paged_tiles_prefix(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                      cudaStream_t stream) {
  return plan.pair ? launch_tiles_mode<true, kPrefix>(a, dtype, head_dim, plan, stream)
                   : launch_tiles_mode<false, kPrefix>(a, dtype, head_dim, plan, stream);
}
cudaError_t launch_paged_tiles_own(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                   cudaStream_t stream) {
  return plan.pair ? launch_tiles_mode<true, kOwn>(a, dtype, head_dim, plan, stream) : cudaErrorInvalidValue;
}

}  // namespace q8a
