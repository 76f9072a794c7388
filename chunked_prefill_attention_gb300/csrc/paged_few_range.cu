// paged_few_range.cu -- the launches of the few-row kernel (paged_few.cuh) over a window, and over the keys behind a
// shared prefix.

#include "paged_few.cuh"

namespace q8a {

cudaError_t launch_paged_few_range(const PagedArgs& a, int mode, int32_t dtype, int32_t head_dim, int64_t rows,
                                   bool direct, cudaStream_t stream) {
  return mode == kWindow ? launch_few_mode<kWindow>(a, dtype, head_dim, rows, direct, stream)
                         : launch_few_mode<kOwn>(a, dtype, head_dim, rows, direct, stream);
}

}  // namespace q8a
