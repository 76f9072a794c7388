// paged_tiles.cu -- the plans of the tile kernel (paged_tiles.cuh), and its launches where rows see all keys up to
// their own.

#include "paged_tiles.cuh"

namespace q8a {

TilesPlan plan_paged_tiles(int64_t batch, int64_t total_rows, int64_t max_rows, int32_t kv_heads, int64_t max_kv,
                           int32_t head_dim) {
  TilesPlan p;
  p.pair = max_rows <= BM;
  const int64_t per = p.pair ? BM : 2 * BM;
  int64_t units = batch * ((max_rows + per - 1) / per);
  if (units > total_rows / per + batch) units = total_rows / per + batch;
  p.slots = units * kv_heads;
  // Few pairs of row unit and K/V head are cut into shares of their key tiles: by the lengths
  // themselves, on the device, or for many sequences by the bounds.  Up to 76 pairs fill
  // one wave of SMs with at least two shares each; 77 to 101 two waves with three; from there
  // on only lengths that differ give anything to share.  4 sequences of 8,192 to 32,768
  // keys, 64 rows, 8 K/V heads: 75 us by the bounds, 54 by the lengths (64 channels), 117
  // and 78 (128 channels).
  const int64_t bn = head_dim == 64 ? Geo<64, false>::BN : Geo<128, false>::BN;
  const int64_t tiles = (max_kv + bn - 1) / bn;
  p.shares = tiles >= 8 && (p.slots <= kSms * 2 / 3 || (batch > 1 && p.slots <= kSms));
  p.share_tiles = p.pair ? 0x3FFFFFFF : 0;
  p.ctas = p.slots;
  if (p.shares) {
    p.ctas = p.slots > kSms / 2 && p.slots <= kSms * 2 / 3 ? 2 * kSms : kSms;
    const int64_t n = p.ctas / p.slots;
    p.share_tiles = batch <= kPlanned ? 0 : static_cast<int32_t>((tiles + n - 1) / n);
  }
  const int64_t states = p.shares || p.pair ? p.ctas * 2 * BM : 0;
  p.part_ml = states * head_dim;
  p.floats = states * (head_dim + 2);
  return p;
}

int64_t window_tiles(int64_t kv, int64_t window, int64_t sinks, int32_t group, bool pair, int32_t head_dim) {
  const int rows = pair ? BM : 2 * BM;
  return head_dim == 64 ? window_bound<Geo<64, false>::BN>(kv, window, sinks, group, rows)
                        : window_bound<Geo<128, false>::BN>(kv, window, sinks, group, rows);
}

cudaError_t launch_paged_tiles(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                               cudaStream_t stream) {
  return plan.pair ? launch_tiles_mode<true, kPlain>(a, dtype, head_dim, plan, stream)
                   : launch_tiles_mode<false, kPlain>(a, dtype, head_dim, plan, stream);
}

}  // namespace q8a
