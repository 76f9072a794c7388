// Stands in for the attention launches of attn_paged_prefix when it is preloaded before the library, and writes down
// how the launch over the sequences' own keys is cut.  No CUDA call is made.
#include <cstdint>

#include "../chunked_prefill_attention_gb300/csrc/internal.h"
#include "../chunked_prefill_attention_gb300/csrc/paged.h"

namespace {
int64_t g_own[9];   // kind (0 few rows, 1 tiles, -1 none), direct, cluster, row tiles, rows, shares, CTAs, shared, only
uint32_t g_words[64];
}  // namespace

namespace q8a {
uint32_t* host_status_words() { return g_words; }
cudaError_t launch_paged_few(const PagedArgs&, int32_t, int32_t, int64_t, bool, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_paged_few_range(const PagedArgs& a, int mode, int32_t, int32_t, int64_t rows, bool direct, cudaStream_t) {
  if (mode == kOwn) g_own[0] = 0, g_own[1] = direct, g_own[2] = a.cluster, g_own[3] = a.row_tiles, g_own[4] = rows, g_own[8] = a.only;
  return cudaSuccess;
}
cudaError_t launch_paged_tiles(const PagedArgs&, int32_t, int32_t, const TilesPlan&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_paged_tiles_window(const PagedArgs&, int32_t, int32_t, const TilesPlan&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_paged_tiles_own(const PagedArgs&, int32_t, int32_t, const TilesPlan& p, cudaStream_t) {
  g_own[0] = 1, g_own[5] = p.shares, g_own[6] = p.ctas;
  return cudaSuccess;
}
cudaError_t launch_paged_tiles_prefix(const PagedArgs&, int32_t, int32_t, const TilesPlan&, cudaStream_t) {
  g_own[7] = 1;
  return cudaSuccess;
}
}  // namespace q8a

extern "C" void record_own(int64_t* out) {
  for (int i = 0; i < 9; ++i) {
    out[i] = g_own[i];
    g_own[i] = i == 0 ? -1 : 0;
  }
}
