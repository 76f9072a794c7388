// paged_few_range.cu -- the launches of the few-row kernel (paged_few.cuh) over a window, and over the keys behind a
// shared prefix.  What bounds them is what bounds the kernel over whole sequences: HBM and, close behind, the issue slots.
// 64 single tokens in windows of 4,096 keys, 8 x 128 bf16: 118 us, 4.7 TB/s (512 units on 304 places, 84 % of two waves);
// 38 of them (304 units) 61 us, 5.55 TB/s; a test of every copied piece and positions by two
// products had cost 3 us each.

#include "paged_few.cuh"

namespace q8a {

cudaError_t launch_paged_few_range(const PagedArgs& a, int mode, int32_t dtype, int32_t head_dim, int64_t rows,
                                   bool direct, cudaStream_t stream) {
  return mode == kWindow ? launch_few_mode<kWindow>(a, dtype, head_dim, rows, direct, stream)
                         : launch_few_mode<kOwn>(a, dtype, head_dim, rows, direct, stream);
}

}  // namespace q8a
