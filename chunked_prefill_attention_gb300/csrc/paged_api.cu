// paged_api.cu -- the extern "C" entry points of the paged Q8_0 cache and of the
// rotary positions (declared in include/q8attn.h): host-side argument validation
// and the launches.  Every argument is checked before the first CUDA call.
//
// All kernels of these calls are launched with programmatic stream serialization: a
// step of a server is a chain of short kernels, and each may be scheduled while its
// predecessor's last CTAs run.  Each waits for the predecessor's completion before it
// touches memory (pdl_wait), so nothing else changes.  What a predecessor may have written
// (queries, pages, slots, lengths) is never read through the non-coherent path, whose data
// must not change while the kernel is resident, the wait included.

#include <cmath>

#include "../../include/q8attn.h"
#include "internal.h"
#include "paged.h"
#include "paged_check.h"

extern "C" {

int attn_rope(const void* x, void* out, int32_t dtype, int64_t n_tokens, int32_t heads, int32_t head_dim,
              int64_t x_token_stride, int64_t out_token_stride, const int64_t* positions, const double* inv_freq,
              int32_t rot_dim, int32_t layout, float mscale, int32_t inverse, void* stream) {
  q8a::NvtxRange nvtx_range("attn_rope");
  q8a::PdlScope early;   // see the top of this file
  const char* fn = "attn_rope";
  if (int rc = check_heads(fn, heads, head_dim, dtype, true)) return rc;
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "n_tokens must be 0..2^31 (got %lld)", (long long)n_tokens);
  if (int rc = check_stride(fn, "x", x_token_stride, heads, head_dim)) return rc;
  if (int rc = check_stride(fn, "out", out_token_stride, heads, head_dim)) return rc;
  if (n_tokens == 0) return q8a::clear_error();
  if (!x || !out) return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  if (x == out && x_token_stride != out_token_stride)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "in place, x and out must have the same token stride");
  if (!aligned(x, elem_bytes(dtype)) || !aligned(out, elem_bytes(dtype)))
    return refuse(Q8A_ERR_MISALIGNED, fn, "x and out need their element's alignment");
  if (int rc = check_rope(fn, positions, inv_freq, rot_dim, head_dim, layout, mscale)) return rc;
  const int64_t width = heads * static_cast<int64_t>(head_dim) * elem_bytes(dtype);
  if (x != out && meet(rows_at(x, n_tokens, width, x_token_stride * elem_bytes(dtype)),
                       rows_at(out, n_tokens, width, out_token_stride * elem_bytes(dtype))))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "x and out overlap");
  const q8a::RopeArgs r{positions, inv_freq, rot_dim, layout == Q8A_ROPE_INTERLEAVED, mscale,
                        inverse ? -1.0f : 1.0f};
  const cudaError_t e = q8a::launch_rope(x, out, dtype, n_tokens, heads, head_dim, x_token_stride, out_token_stride,
                                         r, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

int q8kv_append_paged(const void* k, const void* v, int32_t dtype, int64_t n_tokens, int32_t kv_heads,
                      int32_t head_dim, int64_t k_token_stride, int64_t v_token_stride, const int64_t* slots,
                      void* k_pages, void* v_pages, int64_t n_pages, int32_t page_tokens, int64_t page_stride_bytes,
                      const int64_t* positions, const double* inv_freq, int32_t rot_dim, int32_t layout, float mscale,
                      void* stream) {
  q8a::NvtxRange nvtx_range("q8kv_append_paged");
  q8a::PdlScope early;   // see the top of this file
  const char* fn = "q8kv_append_paged";
  if (int rc = check_heads(fn, kv_heads, head_dim, dtype, true)) return rc;
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "n_tokens must be 0..2^31 (got %lld)", (long long)n_tokens);
  if (int rc = check_stride(fn, "k", k_token_stride, kv_heads, head_dim)) return rc;
  if (int rc = check_stride(fn, "v", v_token_stride, kv_heads, head_dim)) return rc;
  if (n_tokens == 0) return q8a::clear_error();
  q8a::PagePool pool;
  if (int rc = check_pool(fn, k_pages, v_pages, n_pages, page_tokens, page_stride_bytes, kv_heads, head_dim, &pool))
    return rc;
  if (!k || !v || !slots) return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  const int64_t per16 = 16 / elem_bytes(dtype);
  if (!aligned(k, 16) || !aligned(v, 16) || k_token_stride % per16 || v_token_stride % per16 || !aligned(slots, 8))
    return refuse(Q8A_ERR_MISALIGNED, fn, "k, v and their token strides need 16-byte, slots 8-byte alignment");
  {
    const int64_t page = static_cast<int64_t>(kv_heads) * page_tokens * row_bytes(head_dim);
    if (meet(rows_at(k_pages, n_pages, page, page_stride_bytes), rows_at(v_pages, n_pages, page, page_stride_bytes)))
      return refuse(Q8A_ERR_INVALID_ARG, fn, "k_pages and v_pages overlap");
  }
  q8a::RopeArgs r{};
  if (positions || inv_freq) {
    if (int rc = check_rope(fn, positions, inv_freq, rot_dim, head_dim, layout, mscale)) return rc;
    r = q8a::RopeArgs{positions, inv_freq, rot_dim, layout == Q8A_ROPE_INTERLEAVED, mscale, 1.0f};
  }
  uint32_t* status = nullptr;
  if (int rc = status_words(fn, &status)) return rc;
  const cudaError_t e = q8a::launch_append(k, v, dtype, n_tokens, head_dim, k_token_stride, v_token_stride, slots, r,
                                           pool, status, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

int q8kv_read_paged(const void* k_pages, const void* v_pages, int64_t n_pages, int32_t page_tokens,
                    int64_t page_stride_bytes, const int64_t* slots, int64_t n_tokens, int32_t kv_heads,
                    int32_t head_dim, void* k_out, void* v_out, int32_t dtype, void* stream) {
  q8a::NvtxRange nvtx_range("q8kv_read_paged");
  q8a::PdlScope early;   // see the top of this file
  const char* fn = "q8kv_read_paged";
  if (int rc = check_heads(fn, kv_heads, head_dim, dtype, true)) return rc;
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "n_tokens must be 0..2^31 (got %lld)", (long long)n_tokens);
  if (n_tokens == 0) return q8a::clear_error();
  q8a::PagePool pool;
  if (int rc = check_pool(fn, k_pages, v_pages, n_pages, page_tokens, page_stride_bytes, kv_heads, head_dim, &pool))
    return rc;
  if (!k_out || !v_out || !slots) return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(slots, 8))
    return refuse(Q8A_ERR_MISALIGNED, fn, "k_out and v_out need 16-byte, slots 8-byte alignment");
  const int64_t bytes = n_tokens * kv_heads * head_dim * elem_bytes(dtype);
  if (meet(rows_at(k_out, 1, bytes, bytes), rows_at(v_out, 1, bytes, bytes)))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "k_out and v_out overlap");
  uint32_t* status = nullptr;
  if (int rc = status_words(fn, &status)) return rc;
  const cudaError_t e = q8a::launch_read(k_out, v_out, dtype, n_tokens, head_dim, slots, pool, status,
                                         static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

}  // extern "C"

namespace {

// Sequences of at most so many rows (tokens * group) go to the few-row kernel.  Both
// kernels at 16 rows, 16 sequences of 8 K/V heads: 142 us against 257 for 32,768 keys of 64
// channels, 277 against 419 of 128; for 2,048 keys 28 against 30 and 51 against 42.  At 32 rows
// a few-row kernel made for them took 310 and 430 (50 and 61 for 2,048 keys), the tile
// kernel 257 and 421 (30 and 42), so from 17 rows on the tile kernel takes them.
constexpr int64_t kFewRows = 16;

// A number of keys, cut to the most that a sequence can have.
int64_t keys_at_most(int64_t n) { return n < q8a::kMaxKeys ? n : q8a::kMaxKeys; }

// Where the keys of a sequence are bounded, by a window or behind a prefix, the few-row kernel can take a cluster of
// CTAs per (sequence, K/V head): no second launch then, but the longest unit sets the time.  The CTAs of a cluster, or 0:
// shares of all tiles and a join.  As many as fit one wave of two CTAs an SM (the CTAs beyond cost a wave, and a
// cluster's start) and have two tiles a warp.  Us of shares, 1, 2, 4, 8 CTAs, single tokens, 8 K/V heads:
//   one sequence, windows of 1,024, 4,096, 16,384 keys of 64 channels   15  9  8  8  8 | 16 22 15 11 11 | 18 73 40 24 19
//   4 sequences, 4,096 keys of 64, of 128 channels                      17 22 17 14 13 | 23 40 27 22 18
//   16 sequences, 4,096                                                 26 31 21 28 46 | 46 60 38 47 69
//   38 sequences (304 units)                                            51 35 43 64 104 | 86 64 73 100 150
//   64 sequences (512 units, 84 % of two waves)                         69 65 72 99 170 | 125 121 124 155 244
// Of more than 8 rows at most four CTAs, whose states are twice as large (one sequence of 16 rows, 4,096 keys of 64 channels,
// 1, 2, 4, 8 CTAs 31 21 18 19; 4 sequences 34 27 23 26; 2,048 keys of 128 channels 36 27 25 29, 36 30 28 34).
// 16 rows of 128 channels in one CTA an SM, shares, 1, 2, 4 CTAs: one sequence, 1,024 and 4,096 keys 31 19 16 16 | 30 47 30 23;
// 4: 32 19 16 16 | 39 48 31 24; 8, with at most 2: 34 20 17 26 | 50 48 31 39; 16, with 1: 45 20 26 | 80 51 56.
// Longer units than 8 tiles a warp only where they fill their waves, and up to 40: a batch with one long sequence
// waits 50 us for it (38 sequences of 512 to 4,096 keys of 128 channels: 60 in shares, 61 so).  Both bounds are for such batches;
// of sequences of one length a CTA a unit still gains beyond them.  Us of shares and of one CTA, 128 channels, windows of 4,096:
// 64 sequences (84 % of two waves) 124 116, 70 133 117, 76 (100 %) 143 118, 80 (70 % of three) 148 146, but 60 (79 %) 116 116, 56 (74 %)
// 111 95, 30 (79 % of one) 71 61; 76 sequences in windows of 5,000 (40 tiles a warp) 168 140, of 5,200 (41) 173 144, of 8,000 249 211.
// Around 8 tiles, 2 sequences in clusters of eight: windows of 14,400 23 23, of 16,384 24 25, of 20,800 26 28.
// `most` (behind a prefix): keys that a sequence can have beyond `keys`, which are those that it has where the prefix is as
// long as its bound.  The clusters are made for them as far as they fit one wave, since the CTAs that a sequence has no tiles
// for leave at once (ranks_of): single tokens, 8 x 128 bf16, max_kv 32,768, max_prefix 32,000, us for prefixes of 0, 64, 2,048, 16,384
// and 32,000 keys, in clusters made for `keys` and for `most` (attn_paged whatever the prefix):
//   4 sequences   170 202 187 119 45 |  66  74  73  60 45 (61)      16 sequences, 2 heads  168 200 194 118 35 |  68  73  74  57 34 (61)
//   8 sequences   198 203 195 123 46 | 112 118 115  83 46 (106)     32 sequences, 1 head   136 145 142 120 36 |  65  74  75  57 36 (61)
// and 4 bursts of 4 tokens (16 rows) 169 178 171 115 55 | 97 108 105 81 55 (88).
// Sequences that differ are not evened out: 63 of 500 to 934 keys and one of 32,768, nothing shared, 265, but 57 in the shares
// that max_prefix = max_kv plans (attn_paged 48).
struct Cluster {
  int32_t ctas;
  bool only;   // each has an SM for itself: the instance of the few-row kernel for that
};
Cluster few_cluster(int64_t batch, int32_t kv_heads, int64_t rows, int64_t keys, int32_t head_dim, int64_t most) {
  const int64_t units = batch * kv_heads, keys_of_warps = 8 * (2048 / head_dim);   // a tile each
  const bool only = rows > 8 && head_dim == 128 && units <= q8a::kSms;   // see kOnly there
  const int64_t slots = only ? q8a::kSms : 2 * q8a::kSms;
  const int64_t tiles = (keys + keys_of_warps - 1) / keys_of_warps;   // of a warp of one CTA
  int32_t ctas = 1;
  const int64_t at_most = (most + keys_of_warps - 1) / keys_of_warps;
  while (ctas < (rows <= 8 ? 8 : 4) && units * 2 * ctas <= slots && at_most >= 4 * ctas) ctas *= 2;
  const int64_t waves = (units * ctas + slots - 1) / slots, each = (tiles + ctas - 1) / ctas;
  if (units * ctas > 0x7FFFFFFF) return Cluster{0, false};
  const bool takes = each <= (only ? 12 : 8) || (each <= 40 && units * ctas * 100 >= waves * slots * 84);
  return takes ? Cluster{ctas, only} : Cluster{0, false};
}

// Whether sequences of more than 16 rows per K/V head, with bounded keys, go to the few-row kernel as well, a cluster for
// every 16 rows: it reads the keys again for each, but needs neither the tile kernel's start nor its join.  Tile kernel and
// few-row kernel, us, 8 K/V heads; windows of 512, 1,024, 4,096 keys:
//   32 rows, 64 channels: one sequence 21 14 | 19 16 | 23 20; 4: 23 14 | 21 18 | 28 24; 16: 28 16 | 36 21 | 62 45;
//     64: 104 52 | 123 64 | 225 150.  128 channels: 20 13 | 21 17 | 27 24; 21 15 | 23 17 | 33 31; 37 25 | 43 33 | 87 88;
//     123 80 | 150 114 | 307 294
//   64 rows, 64 channels: 22 15 | 20 17 | 23 27; 24 16 | 21 20 | 28 30; 30 29 | 38 40 | 64 87; 112 98 | 132 123 | 235 291.
//     128 channels: 21 13 | 22 17 | 28 24; 22 15 | 23 20 | 33 48; 40 44 | 46 62 | 90 168; 64 of 128 keys 115 100
// On both sides of the edges, 64 rows.  64 channels, windows of 500, 640, 800, 1,100 keys: 4 sequences 24 16 | 22 17 | 22 19 | 22 20;
//   16: 30 34 | 36 33 | 36 34 | 39 41; 64: 112 104 | 119 105 | 122 113 | 132 133.  128 channels, of 120, 200, 300 keys: 8 sequences
//   26 17 | 26 19 | 28 21; 16: 32 31 | 31 34 | 34 39; 64: 120 101 | 120 109 | 130 123; of 1,100, 1,400 keys: 4 (128 clusters) 24 20 | 25 24,
//   8 (256) 31 35 | 33 41; of 2,200, 3,000: 2 (64) 25 22 | 27 25, 4 28 31 | 30 38.  32 rows of 128 channels have no edge of their own: windows
//   of 8,192, 4 sequences, 47 51, is the most that they lose.
// `units`: pairs of sequence and K/V head.
bool few_takes(int64_t rows, int64_t units, int64_t keys, int32_t head_dim) {
  if (rows <= 32) return true;
  if (rows > 64) return false;
  if (head_dim == 64) return keys <= 640;
  const int64_t clusters = units * ((rows + 15) / 16);
  return keys <= 200 || (clusters <= q8a::kSms && keys <= 1100) || (clusters <= q8a::kSms / 2 && keys <= 2200);
}

// The launches of a call, from its bounds alone.
struct Plan {
  bool few, direct, tiles;
  Cluster cluster;
  int32_t row_tiles;
  q8a::TilesPlan t;
  int64_t few_rows;   // rows a K/V head of the few-row kernel's sequences, at most: it sizes its tiles
                      // and their partial states, so workspace and launch both take it from here
  int64_t few_floats, floats;
};
// `window`, `sinks`: of attn_paged_window, else 0.
Plan plan_paged(int64_t batch, int64_t total_q, int64_t max_q, int64_t group, int32_t kv_heads, int64_t max_kv,
                int32_t head_dim, int64_t window = 0, int64_t sinks = 0) {
  Plan p{};
  if (max_q > total_q) max_q = total_q;
  if (max_kv > q8a::kMaxKeys) max_kv = q8a::kMaxKeys;
  int64_t few_kv = max_kv;
  if (window) {   // the keys that a unit takes, at most
    const int64_t bn = head_dim == 64 ? 96 : 64;
    const int64_t most = window + sinks + max_q;
    if (few_kv > most) few_kv = most;
    max_kv = q8a::window_tiles(max_kv, window, sinks, static_cast<int32_t>(group), max_q * group <= 128, head_dim) * bn;
  }
  p.tiles = max_q * group > kFewRows;
  p.row_tiles = 1;
  if (window && p.tiles && few_takes(max_q * group, batch * kv_heads, few_kv, head_dim)) {
    const int32_t row_tiles = static_cast<int32_t>((max_q * group + kFewRows - 1) / kFewRows);
    p.cluster = few_cluster(batch, kv_heads * row_tiles, max_q * group, few_kv, head_dim, few_kv);
    if (p.cluster.ctas > 0) {
      p.tiles = false;
      p.few = p.direct = true;
      p.row_tiles = row_tiles;
      p.few_rows = max_q * group;
      return p;
    }
  }
  if (p.tiles) p.t = q8a::plan_paged_tiles(batch, total_q * group, max_q * group, kv_heads, max_kv, head_dim);
  // The tile kernel takes every sequence of a call of at most 128 rows each (one of few
  // rows costs it no more than one of many, the other kernel's launches 8 us), and of a
  // call whose bounds leave no room for a short one.  Single tokens beside prompts keep their
  // own kernel: there a long cache would be one CTA's.  So it is in pairs too where there are
  // too many for shares, and the lengths, which would tell, are the device's: 20 sequences on 8
  // K/V heads, one with a burst of 5 tokens, one with 262,144 keys take 2,112 us so and 128 with
  // the short ones in the few-row kernel; but without the long one (2,000 keys) 50 and 60, and
  // 63 single tokens and a burst of 16 (300 to 16,384 keys, 128 channels) 395 and 452.
  p.few = !p.tiles || (!p.t.pair && (total_q - (batch - 1) * max_q) * group <= kFewRows);
  p.few_rows = p.tiles ? kFewRows : max_q * group;
  p.cluster = window ? few_cluster(batch, kv_heads, max_q * group, few_kv, head_dim, few_kv) : Cluster{};
  p.direct = window ? p.cluster.ctas > 0 : q8a::paged_few_direct(batch, kv_heads, few_kv, head_dim);
  p.few_floats = p.few && !p.direct ? q8a::paged_few_floats(head_dim, p.few_rows) : 0;
  p.floats = p.few_floats + p.t.floats;
  return p;
}

}  // namespace

extern "C" {

int64_t q8a_paged_workspace_floats(int64_t batch, int64_t total_q, int32_t heads, int32_t kv_heads, int64_t max_q,
                                   int64_t max_kv, int32_t head_dim) {
  if (batch < 0 || batch > (1 << 20) || total_q < 0 || total_q >= kMaxTokens || heads <= 0 || kv_heads <= 0 ||
      heads % kv_heads || max_q < 0 || max_kv < 0 || (head_dim != 64 && head_dim != 128))
    return -1;
  if (batch == 0 || max_q == 0 || total_q == 0) return 0;
  return plan_paged(batch, total_q, max_q, heads / kv_heads, kv_heads, max_kv, head_dim).floats;
}

}  // extern "C"

namespace {

// The arguments that the attention calls share.
struct Call {
  const void* q;
  int32_t dtype;
  int64_t q_token_stride, total_q;
  int32_t heads, kv_heads, head_dim;
  const void *k_pages, *v_pages;
  int64_t n_pages;
  int32_t page_tokens;
  int64_t page_stride_bytes;
  const int32_t* block_table;
  int64_t table_stride;
  const int32_t *kv_lens, *cu_q;
  int64_t batch, max_q, max_kv;
  float scale;
  int32_t causal;
  void* out;
  float* workspace;
  int64_t workspace_floats;
  bool empty() const { return batch == 0 || total_q == 0 || max_q == 0; }
};

// Checks what does not depend on the plan; fills in the kernels' arguments.  An empty call (Call::empty) is accepted
// before its pointers are looked at.
int check_call(const char* fn, const Call& c, q8a::PagedArgs* a) {
  if (int rc = check_heads(fn, c.heads, c.head_dim, c.dtype, false)) return rc;
  if (c.kv_heads <= 0 || c.heads % c.kv_heads)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "heads (%d) must be a positive multiple of kv_heads (%d)", c.heads, c.kv_heads);
  if (c.batch < 0 || c.batch > (1 << 20) || c.total_q < 0 || c.total_q >= kMaxTokens || c.max_q < 0 || c.max_kv < 0)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "batch must be 0..2^20, total_q 0..2^31-1, max_q and max_kv not negative");
  const float scale_log2 = c.scale * 1.4426950408889634f;   // log2(e)
  if (!(c.scale > 0.0f) || !std::isfinite(scale_log2))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "scale must be > 0 and finite, also times log2(e)");
  if (int rc = check_stride(fn, "q", c.q_token_stride, c.heads, c.head_dim)) return rc;
  if (c.empty()) return Q8A_OK;
  q8a::PagePool pool;
  if (int rc = check_pool(fn, c.k_pages, c.v_pages, c.n_pages, c.page_tokens, c.page_stride_bytes, c.kv_heads, c.head_dim, &pool))
    return rc;
  if (!c.q || !c.out || !c.kv_lens || !c.cu_q || (c.table_stride > 0 && !c.block_table))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  if (c.out == c.q) return refuse(Q8A_ERR_INVALID_ARG, fn, "out must not be q");
  if (c.table_stride < 0 || c.table_stride > 0x7FFFFFFFll)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "table stride must be 0..2^31-1 (got %lld)", (long long)c.table_stride);
  if (c.max_kv > c.table_stride * c.page_tokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "max_kv %lld: the table's rows hold %lld keys", (long long)c.max_kv,
                  (long long)(c.table_stride * c.page_tokens));
  if (!aligned(c.q, 16) || !aligned(c.out, 16) || !aligned(c.workspace, 16) || c.q_token_stride % 8 ||
      !aligned(c.kv_lens, 4) || !aligned(c.cu_q, 4) || !aligned(c.block_table, 4))
    return refuse(Q8A_ERR_MISALIGNED, fn,
                  "q, its token stride, out and workspace need 16-byte, the index arrays 4-byte alignment");
  if (c.total_q * (c.heads / c.kv_heads) >= kMaxTokens)
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "total_q * heads / kv_heads must be below 2^31");
  *a = q8a::PagedArgs{};
  a->q = c.q;
  a->out = c.out;
  a->k = pool.k;
  a->v = pool.v;
  a->table = c.block_table;
  a->kv_lens = c.kv_lens;
  a->cu_q = c.cu_q;
  a->part = c.workspace;
  a->n_pages = c.n_pages;
  a->page_stride = c.page_stride_bytes;
  a->q_stride = c.q_token_stride;
  a->table_stride = c.table_stride;
  a->total_q = c.total_q;
  a->batch = static_cast<int32_t>(c.batch);
  a->heads = c.heads;
  a->kv_heads = c.kv_heads;
  a->group = c.heads / c.kv_heads;
  a->page_shift = pool.page_shift;
  a->causal = c.causal ? 1 : 0;
  a->scale_log2 = scale_log2;
  a->timeout_ns = q8a::wait_timeout_ns();
  return Q8A_OK;
}

// Checks the workspace against what the plan needs of it, and that no buffers overlap; takes the status words.
int check_workspace(const char* fn, const Call& c, int64_t need, q8a::PagedArgs* a) {
  if (need > 0 && !c.workspace) return refuse(Q8A_ERR_INVALID_ARG, fn, "null workspace");
  if (c.workspace_floats < need)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "workspace of %lld floats < %lld needed", (long long)c.workspace_floats,
                  (long long)need);
  const int64_t row = static_cast<int64_t>(c.heads) * c.head_dim * 2;
  const Rows q_rows = rows_at(c.q, c.total_q, row, c.q_token_stride * 2), o_rows = rows_at(c.out, c.total_q, row, row);
  if (meet(q_rows, o_rows)) return refuse(Q8A_ERR_INVALID_ARG, fn, "q and out overlap");
  const Rows ws = rows_at(c.workspace, 1, need * 4, need * 4);
  if (need > 0 && (meet(q_rows, ws) || meet(o_rows, ws)))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "the workspace overlaps q or out");
  return status_words(fn, &a->status);
}

// The tile kernel's share of a call, with its states at `part`.
q8a::PagedArgs tiles_args(const q8a::PagedArgs& a, const q8a::TilesPlan& t, int32_t row_limit, float* part) {
  q8a::PagedArgs b = a;
  b.row_limit = row_limit;
  b.shares = t.shares;
  b.share_tiles = t.share_tiles;
  b.ctas = t.ctas;
  b.part = part;
  b.part_ml = t.part_ml;
  auto even = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 32 == 0; };
  b.wide = (even(a.q) && a.q_stride % 16 == 0 ? q8a::kWideQ : 0) | (even(a.out) ? q8a::kWideOut : 0) |
           (even(part) ? q8a::kWidePart : 0);
  return b;
}

// attn_paged, or where `window` is not 0 attn_paged_window (not causal: of a window beyond every length).
int run_paged(const char* fn, const Call& c, int64_t window, int64_t sinks, cudaStream_t st) {
  q8a::PagedArgs a{};
  if (int rc = check_call(fn, c, &a)) return rc;
  if (c.empty()) return q8a::clear_error();
  const Plan plan = plan_paged(c.batch, c.total_q, c.max_q, a.group, c.kv_heads, c.max_kv, c.head_dim, window, sinks);
  if (int rc = check_workspace(fn, c, plan.floats, &a)) return rc;
  a.window = static_cast<int32_t>(window);
  a.sinks = static_cast<int32_t>(sinks);
  a.cluster = plan.cluster.ctas;
  a.only = plan.cluster.only;
  a.row_tiles = plan.row_tiles;
  cudaError_t e = cudaSuccess;
  if (plan.tiles) {
    const q8a::PagedArgs b =
        tiles_args(a, plan.t, plan.few ? static_cast<int32_t>(kFewRows) : 0, c.workspace + plan.few_floats);
    e = window ? q8a::launch_paged_tiles_window(b, c.dtype, c.head_dim, plan.t, st)
               : q8a::launch_paged_tiles(b, c.dtype, c.head_dim, plan.t, st);
  }
  if (plan.few && e == cudaSuccess) {
    a.row_limit = plan.tiles ? static_cast<int32_t>(kFewRows) : 0x7FFFFFFF;
    e = window ? q8a::launch_paged_few_range(a, q8a::kWindow, c.dtype, c.head_dim, plan.few_rows, plan.direct, st)
               : q8a::launch_paged_few(a, c.dtype, c.head_dim, plan.few_rows, plan.direct, st);
  }
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

// A call behind a shared prefix: first the rows' states over their own keys (own_few or own), then all rows together
// over the prefix, whose join takes those states in.  Not `share`: attn_paged, or where clusters of the few-row
// kernel take the call (4 sequences of 2,250 keys, 8 x 64: 16 us, 11 so) a window that hides nothing.
struct PrefixPlan {
  int64_t window;   // not `share`: run_paged's
  bool share, own_few, own_direct;
  int32_t join_rows, row_tiles;
  Cluster cluster;
  int64_t own_rows;
  q8a::TilesPlan own, prefix;
  int64_t state_floats, floats;
};
// Sequences of more rows per K/V head than this fill the tiles of the tensor cores by themselves.
constexpr int64_t kShareRows = 128;
// Whether sharing pays.  Read for each sequence, a key of the prefix costs (relative to one of the few-row kernel for up
// to 8 rows) 1, 1.35 for up to 16 rows, 2.4 in the tile kernel; read once, 2.4 for every 256 rows of the batch (what bounds the
// tile kernel there is dequantisation, whose cost a byte is that much above the few-row kernel's).  The gain has to
// outweigh the launches that sharing adds, 12 us, which is 3e7 channels, and twice that where the own keys are the tile
// kernel's (32 rows a sequence, one K/V head, 128 channels, 64 sequences of 2,048 keys 40 and 32, of 8,192 44 and 70).  Shared and not, us: 8 K/V
// heads, group 4, 64 channels, single tokens, 4 sequences of 32,768 keys 38 and 35; 16 of 2,048 24 and 20, of 8,192 23 and
// 36, of 32,768 33 and 101; 64 of 512 30 and 17, of 2,048 29 and 39, of 32,768 47 and 361; 128 channels, 64 of
// 32,768 72 and 724, 4 of 32,768 43 and 62.
bool share_pays(int64_t batch, int64_t total_rows, int64_t max_rows, int32_t kv_heads, int64_t max_prefix, int32_t head_dim) {
  const double each = max_rows <= 8 ? 1.0 : max_rows <= kFewRows ? 1.35 : 2.4;
  const double units = static_cast<double>((total_rows + 255) / 256);
  return static_cast<double>(max_prefix) * kv_heads * head_dim * (each * batch - 2.4 * units) > (max_rows <= kFewRows ? 3e7 : 6e7);
}
PrefixPlan plan_prefix(int64_t batch, int64_t total_q, int64_t max_q, int64_t group, int32_t kv_heads, int64_t max_kv,
                       int64_t max_prefix, int32_t head_dim) {
  PrefixPlan p{};
  if (max_q > total_q) max_q = total_q;
  if (max_kv > q8a::kMaxKeys) max_kv = q8a::kMaxKeys;
  if (max_prefix > max_kv) max_prefix = max_kv;
  p.share = max_q * group <= kShareRows && share_pays(batch, total_q * group, max_q * group, kv_heads, max_prefix, head_dim);
  if (!p.share) {
    const Plan w = plan_paged(batch, total_q, max_q, group, kv_heads, max_kv, head_dim, q8a::kMaxKeys, 0);
    const Plan plain = plan_paged(batch, total_q, max_q, group, kv_heads, max_kv, head_dim);
    p.window = !w.tiles && w.direct && !plain.direct ? q8a::kMaxKeys : 0;
    p.floats = p.window ? w.floats : plain.floats;
    return p;
  }
  // the own keys are those behind the prefix if it is as long as its bound; the launches have to do with any from there to
  // max_kv, where a bound serves shorter prefixes too
  const int64_t own_kv = max_kv > max_prefix ? max_kv - max_prefix : max_kv;
  int64_t own_floats = 0;
  p.own_rows = max_q * group;
  p.row_tiles = 1;
  // 32 rows a K/V head of few keys too, where that is one launch less (16 bursts of up to 8 tokens: 166 us, 159 so).  The whole
  // call behind 65,536 keys, 8 x 64, 32 rows, the tile kernel and so, us, 200, 900, 1,100, 1,400, 2,000 own keys: 4 sequences 58 55 | 59 61 |
  // 60 60 | 59 60 | 61 62; 16: 110 109 | 118 114 | 120 116 | 122 119 | 126 123; 32: 222 217 | 231 225 | 234 231 | 238 234 | 246 242.  With 128
  // channels 82 82 | 83 88 | 84 88; 182 187 | 196 196 | 198 198; 378 377 | 394 402 | 400 406: no gain.
  if (p.own_rows > kFewRows && p.own_rows <= 32 && head_dim == 64 && own_kv <= 1100) p.row_tiles = 2;
  p.cluster = few_cluster(batch, kv_heads * p.row_tiles, p.own_rows, own_kv, head_dim, max_kv);
  p.own_few = p.own_rows <= kFewRows || (p.row_tiles > 1 && p.cluster.ctas > 0);
  if (p.own_few) {
    p.own_direct = p.cluster.ctas > 0;
    own_floats = p.own_direct ? 0 : q8a::paged_few_floats(head_dim, p.own_rows);
  } else {
    // Shares for the keys that a sequence can have: up to 64 sequences cut them on the device, by what they have, and of more
    // the shares are planned here.  But of more than two thirds of a wave of units, shares for few keys are not worth their
    // grid.  By own_kv and by max_kv, bounds and prefixes as at few_cluster, 200 own keys, us:
    //   4 sequences of 64 rows, 8 x 128 (32 units)   419 430 413 248  71 | 124 135 135 102  71 (attn_paged 118)
    //   8 sequences of 64 rows, 8 x 64 (64 units)    255 264 251 161  67 | 138 148 142 106  69 (131)
    //   16 sequences of 32 rows, 8 x 128 (128 units) 427 439 418 269 109 | 431 444 422 274 113 (413)
    p.own = q8a::plan_paged_tiles(batch, total_q * group, p.own_rows, kv_heads, max_kv, head_dim);
    if (batch <= 64 && p.own.slots > q8a::kSms * 2 / 3)
      p.own = q8a::plan_paged_tiles(batch, total_q * group, p.own_rows, kv_heads, own_kv, head_dim);
    own_floats = p.own.floats;
  }
  p.prefix = q8a::plan_paged_tiles(1, total_q * group, total_q * group, kv_heads, max_prefix, head_dim);
  if (!p.prefix.shares) {   // whole units leave their states too, for the join
    p.prefix.share_tiles = 0x3FFFFFFF;
    p.prefix.part_ml = p.prefix.ctas * 256 * head_dim;
    p.prefix.floats = p.prefix.ctas * 256 * (head_dim + 2);
  }
  // a warp a row where they are enough for the machine, else a block a row
  p.join_rows = total_q * group * kv_heads >= q8a::kSms * 8 ? 8 : 1;
  p.state_floats = (total_q * group * kv_heads * (head_dim + 1) + 7) / 8 * 8;
  p.floats = p.state_floats + (own_floats > p.prefix.floats ? own_floats : p.prefix.floats);
  return p;
}

}  // namespace

extern "C" {

int attn_paged(const void* q, int32_t dtype, int64_t q_token_stride, int64_t total_q, int32_t heads, int32_t kv_heads,
               int32_t head_dim, const void* k_pages, const void* v_pages, int64_t n_pages, int32_t page_tokens,
               int64_t page_stride_bytes, const int32_t* block_table, int64_t table_stride, const int32_t* kv_lens,
               const int32_t* cu_q, int64_t batch, int64_t max_q, int64_t max_kv, float scale, int32_t causal,
               void* out, float* workspace, int64_t workspace_floats, void* stream) {
  q8a::NvtxRange nvtx_range("attn_paged");
  q8a::PdlScope early;   // see the top of this file
  const Call c{q, dtype, q_token_stride, total_q, heads, kv_heads, head_dim, k_pages, v_pages, n_pages, page_tokens,
               page_stride_bytes, block_table, table_stride, kv_lens, cu_q, batch, max_q, max_kv, scale, causal, out,
               workspace, workspace_floats};
  return run_paged("attn_paged", c, 0, 0, static_cast<cudaStream_t>(stream));
}

int64_t q8a_paged_window_workspace_floats(int64_t batch, int64_t total_q, int32_t heads, int32_t kv_heads, int64_t max_q,
                                          int64_t max_kv, int64_t window, int64_t sinks, int32_t head_dim) {
  if (q8a_paged_workspace_floats(batch, total_q, heads, kv_heads, max_q, max_kv, head_dim) < 0 || window < 1 || sinks < 0)
    return -1;
  if (batch == 0 || max_q == 0 || total_q == 0) return 0;
  return plan_paged(batch, total_q, max_q, heads / kv_heads, kv_heads, max_kv, head_dim, keys_at_most(window),
                    keys_at_most(sinks)).floats;
}

int attn_paged_window(const void* q, int32_t dtype, int64_t q_token_stride, int64_t total_q, int32_t heads,
                      int32_t kv_heads, int32_t head_dim, const void* k_pages, const void* v_pages, int64_t n_pages,
                      int32_t page_tokens, int64_t page_stride_bytes, const int32_t* block_table, int64_t table_stride,
                      const int32_t* kv_lens, const int32_t* cu_q, int64_t batch, int64_t max_q, int64_t max_kv,
                      int64_t window, int64_t sinks, float scale, void* out, float* workspace, int64_t workspace_floats,
                      void* stream) {
  q8a::NvtxRange nvtx_range("attn_paged_window");
  q8a::PdlScope early;   // see the top of this file
  const char* fn = "attn_paged_window";
  if (window < 1 || sinks < 0)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "window must be at least 1, sinks not negative (got %lld, %lld)",
                  (long long)window, (long long)sinks);
  const Call c{q, dtype, q_token_stride, total_q, heads, kv_heads, head_dim, k_pages, v_pages, n_pages, page_tokens,
               page_stride_bytes, block_table, table_stride, kv_lens, cu_q, batch, max_q, max_kv, scale, 1, out,
               workspace, workspace_floats};
  return run_paged(fn, c, keys_at_most(window), keys_at_most(sinks), static_cast<cudaStream_t>(stream));
}

int64_t q8a_paged_prefix_workspace_floats(int64_t batch, int64_t total_q, int32_t heads, int32_t kv_heads, int64_t max_q,
                                          int64_t max_kv, int64_t max_prefix, int32_t head_dim) {
  if (q8a_paged_workspace_floats(batch, total_q, heads, kv_heads, max_q, max_kv, head_dim) < 0 || max_prefix < 0) return -1;
  if (batch == 0 || max_q == 0 || total_q == 0) return 0;
  return plan_prefix(batch, total_q, max_q, heads / kv_heads, kv_heads, max_kv, max_prefix, head_dim).floats;
}

int attn_paged_prefix(const void* q, int32_t dtype, int64_t q_token_stride, int64_t total_q, int32_t heads,
                      int32_t kv_heads, int32_t head_dim, const void* k_pages, const void* v_pages, int64_t n_pages,
                      int32_t page_tokens, int64_t page_stride_bytes, const int32_t* block_table, int64_t table_stride,
                      const int32_t* kv_lens, const int32_t* cu_q, int64_t batch, int64_t max_q, int64_t max_kv,
                      const int32_t* prefix_table, int64_t prefix_pages, const int32_t* prefix_len, int64_t max_prefix,
                      float scale, int32_t causal, void* out, float* workspace, int64_t workspace_floats, void* stream) {
  q8a::NvtxRange nvtx_range("attn_paged_prefix");
  q8a::PdlScope early;   // see the top of this file
  const char* fn = "attn_paged_prefix";
  const Call c{q, dtype, q_token_stride, total_q, heads, kv_heads, head_dim, k_pages, v_pages, n_pages, page_tokens,
               page_stride_bytes, block_table, table_stride, kv_lens, cu_q, batch, max_q, max_kv, scale, causal, out,
               workspace, workspace_floats};
  if (prefix_pages < 0 || prefix_pages > 0x7FFFFFFFll || max_prefix < 0)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "prefix_pages must be 0..2^31-1, max_prefix not negative (got %lld, %lld)",
                  (long long)prefix_pages, (long long)max_prefix);
  q8a::PagedArgs a{};
  if (int rc = check_call(fn, c, &a)) return rc;
  if (c.empty()) return q8a::clear_error();
  if (max_prefix > 0 && (!prefix_table || !prefix_len)) return refuse(Q8A_ERR_INVALID_ARG, fn, "null prefix");
  if (max_prefix > prefix_pages * page_tokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "max_prefix %lld: the prefix's pages hold %lld keys", (long long)max_prefix,
                  (long long)(prefix_pages * page_tokens));
  if (!aligned(prefix_table, 4) || !aligned(prefix_len, 4))
    return refuse(Q8A_ERR_MISALIGNED, fn, "prefix_table and prefix_len need 4-byte alignment");
  const PrefixPlan plan = plan_prefix(batch, total_q, max_q, a.group, kv_heads, max_kv, max_prefix, head_dim);
  if (!plan.share) return run_paged(fn, c, plan.window, 0, static_cast<cudaStream_t>(stream));
  if (int rc = check_workspace(fn, c, plan.floats, &a)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  a.prefix_len = prefix_len;
  a.prefix_most = keys_at_most(max_prefix);
  a.state = workspace;
  a.cluster = plan.cluster.ctas;
  a.only = plan.cluster.only;
  a.row_tiles = plan.row_tiles;
  a.part = workspace + plan.state_floats;
  cudaError_t e;
  if (plan.own_few) {
    a.row_limit = 0x7FFFFFFF;
    e = q8a::launch_paged_few_range(a, q8a::kOwn, dtype, head_dim, plan.own_rows, plan.own_direct, st);
  } else {
    e = q8a::launch_paged_tiles_own(tiles_args(a, plan.own, 0, a.part), dtype, head_dim, plan.own, st);
  }
  if (e == cudaSuccess) {
    q8a::PagedArgs b = tiles_args(a, plan.prefix, 0, a.part);
    b.seqs = b.batch;
    b.batch = 1;
    b.table = prefix_table;
    b.table_stride = prefix_pages;
    b.join_rows = plan.join_rows;
    e = q8a::launch_paged_tiles_prefix(b, dtype, head_dim, plan.prefix, st);
  }
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

}  // extern "C"
