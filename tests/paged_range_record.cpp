// Stands in for the launches of attn_paged_window, attn_paged_prefix, q8kv_extend_paged and attn_norm_rope when it is
// preloaded before the library: it writes down what the C-ABI layer asks of the attention kernels.  No CUDA call is made.
#include <cstdint>

#include "../chunked_prefill_attention_gb300/csrc/internal.h"
#include "../chunked_prefill_attention_gb300/csrc/paged.h"

namespace {
// kind: 0 few rows, 1 tiles; mode as in paged.h; part: floats before the kernel's workspace
struct Launch {
  int64_t kind, mode, part, rows, direct, pair, shares, share_tiles, ctas, floats, batch, seqs, window, sinks, state, most, join;
};
Launch g_log[8];
int g_n;
const float* g_base;
uint32_t g_words[64];

cudaError_t log(int64_t kind, int64_t mode, const q8a::PagedArgs& a, int64_t rows, bool direct, const q8a::TilesPlan* p) {
  if (g_n < 8)
    g_log[g_n++] = Launch{kind, mode, a.part - g_base, rows, direct, p ? p->pair : 0, p ? p->shares : 0, p ? p->share_tiles : 0,
                          p ? p->ctas : 0, p ? p->floats : 0, a.batch, a.seqs, a.window, a.sinks,
                          a.state ? a.state - g_base : -1, a.prefix_most, a.join_rows};
  return cudaSuccess;
}
}  // namespace

namespace q8a {
uint32_t* host_status_words() { return g_words; }
cudaError_t launch_norm_rope(const NormRopeArgs&, int32_t, int32_t, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_extend(const ExtendArgs&, cudaStream_t) { return cudaSuccess; }
cudaError_t launch_paged_few(const PagedArgs& a, int32_t, int32_t, int64_t rows, bool direct, cudaStream_t) {
  return log(0, kPlain, a, rows, direct, nullptr);
}
cudaError_t launch_paged_few_range(const PagedArgs& a, int mode, int32_t, int32_t, int64_t rows, bool direct, cudaStream_t) {
  return log(0, mode, a, rows, direct, nullptr);
}
cudaError_t launch_paged_tiles(const PagedArgs& a, int32_t, int32_t, const TilesPlan& p, cudaStream_t) {
  return log(1, kPlain, a, 0, false, &p);
}
cudaError_t launch_paged_tiles_window(const PagedArgs& a, int32_t, int32_t, const TilesPlan& p, cudaStream_t) {
  return log(1, kWindow, a, 0, false, &p);
}
cudaError_t launch_paged_tiles_own(const PagedArgs& a, int32_t, int32_t, const TilesPlan& p, cudaStream_t) {
  return log(1, kOwn, a, 0, false, &p);
}
cudaError_t launch_paged_tiles_prefix(const PagedArgs& a, int32_t, int32_t, const TilesPlan& p, cudaStream_t) {
  return log(1, kPrefix, a, 0, false, &p);
}
}  // namespace q8a

extern "C" {
void record_start(const void* workspace) {
  g_n = 0;
  g_base = static_cast<const float*>(workspace);
}
int record_take(int64_t* out) {
  for (int i = 0; i < g_n; ++i) {
    const int64_t* from = reinterpret_cast<const int64_t*>(&g_log[i]);
    for (int k = 0; k < 17; ++k) out[17 * i + k] = from[k];
  }
  return g_n;
}
}
