// paged_tiles_prefix.cu -- the launches of the tile kernel (paged_tiles.cuh) over a shared prefix and over the keys
// behind it.  The rows of the whole batch (tokens x heads of a group) fill its tiles, so a key of the prefix is
// dequantised once for every 256 rows instead of once a sequence.  64 single tokens, 8 x 128 bf16, 32,768 keys: 47 us
// (1.3 us a tile of 64 keys, 14 us to start and end), and 5 us for the join; 16 bursts of 2 to 8 tokens, 8 x 64 fp16,
// 100,001 keys (320 rows, two units): 136 us, 1.1 us a tile of 96.

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
