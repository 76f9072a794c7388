// Stands in for the launches of the paged calls when it is preloaded before the library: it
// writes down what the C-ABI layer asks of attn_paged's.  No CUDA call is made.
#include <cstdint>

#include "../chunked_prefill_attention_gb300/csrc/internal.h"
#include "../chunked_prefill_attention_gb300/csrc/paged.h"

namespace {
struct Record {
  int64_t few_calls, few_rows, few_direct, few_limit;
  int64_t tiles_calls, tiles_floats, tiles_part;   // part: floats before the tile kernel's workspace
  int64_t shares, share_tiles;
};
Record g_rec;
const float* g_part;
uint32_t g_words[64];
}  // namespace

namespace q8a {
uint32_t* host_status_words() { return g_words; }
cudaError_t launch_rope(const void*, void*, int32_t, int64_t, int32_t, int32_t, int64_t, int64_t, const RopeArgs&,
                        cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_append(const void*, const void*, int32_t, int64_t, int32_t, int64_t, int64_t, const int64_t*,
                          const RopeArgs&, const PagePool&, uint32_t*, cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_read(void*, void*, int32_t, int64_t, int32_t, const int64_t*, const PagePool&, uint32_t*,
                        cudaStream_t) {
  return cudaSuccess;
}
cudaError_t launch_paged_few(const PagedArgs& a, int32_t, int32_t, int64_t rows, bool direct, cudaStream_t) {
  g_rec.few_calls++;
  g_rec.few_rows = rows;
  g_rec.few_direct = direct;
  g_rec.few_limit = a.row_limit;
  return cudaSuccess;
}
cudaError_t launch_paged_tiles(const PagedArgs& a, int32_t, int32_t, const TilesPlan& plan, cudaStream_t) {
  g_rec.tiles_calls++;
  g_rec.tiles_floats = plan.floats;
  g_rec.tiles_part = a.part - g_part;
  g_rec.shares = plan.shares;
  g_rec.share_tiles = plan.share_tiles;
  return cudaSuccess;
}
}  // namespace q8a

extern "C" {
void record_start(const void* workspace) {
  g_rec = Record{};
  g_part = static_cast<const float*>(workspace);
}
void record_take(int64_t* out) {
  const int64_t v[9] = {g_rec.few_calls, g_rec.few_rows, g_rec.few_direct, g_rec.few_limit,
                        g_rec.tiles_calls, g_rec.tiles_floats, g_rec.tiles_part, g_rec.shares, g_rec.share_tiles};
  for (int i = 0; i < 9; ++i) out[i] = v[i];
}
}
