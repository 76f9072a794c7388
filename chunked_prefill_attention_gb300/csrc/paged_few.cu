// paged_few.cu -- the launches of the few-row kernel (paged_few.cuh) where rows see all keys up to their own.

#include "paged_few.cuh"

namespace q8a {

// Whether every unit is one CTA's: no unit has more than four tiles a warp.  The shares
// and their join would spread so few tiles further, but cost a second launch.
bool paged_few_direct(int64_t batch, int32_t kv_heads, int64_t max_kv, int32_t head_dim) {
  const int64_t tile = head_dim == 64 ? Shape<64, 1>::KT : Shape<128, 1>::KT;
  return max_kv <= 4 * kWarps * tile && batch * kv_heads <= 0x7FFFFFFF;
}

int64_t paged_few_floats(int32_t head_dim, int64_t rows) {
  const int64_t r = rows <= 8 ? 8 : 16;
  return kMaxWarps * (kDescInts + 2 * (r * head_dim + 2 * r));
}

cudaError_t launch_paged_few(const PagedArgs& a, int32_t dtype, int32_t head_dim, int64_t rows, bool direct,
                             cudaStream_t stream) {
  return launch_few_mode<kPlain>(a, dtype, head_dim, rows, direct, stream);
}

}  // namespace q8a
