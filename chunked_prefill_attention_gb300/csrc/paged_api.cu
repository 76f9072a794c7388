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
#include <cstdarg>
#include <cstdio>

#include "../../include/q8attn.h"
#include "internal.h"
#include "paged.h"

namespace {

int refuse(int code, const char* fn, const char* fmt, ...) {
  char msg[384];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return q8a::set_error(code, fn, msg);
}
int cuda_refuse(cudaError_t e, const char* fn) {
  cudaGetLastError();   // a refused launch leaves no error behind for the caller's next check
  return refuse(Q8A_ERR_CUDA, fn, "%s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
}
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
int64_t row_bytes(int32_t head_dim) { return static_cast<int64_t>(head_dim / 32) * 34; }
int64_t elem_bytes(int32_t dtype) { return dtype == Q8A_F32 ? 4 : 2; }

constexpr int64_t kMaxTokens = int64_t{1} << 31;
constexpr int64_t kMaxStride = int64_t{1} << 32;   // elements between tokens

// n rows of `width` bytes, `stride` apart.
struct Rows {
  uintptr_t at;
  int64_t stride, width, n;
  uintptr_t end() const {   // cut to the last address: the sizes that are accepted can pass it
    const unsigned __int128 e = static_cast<unsigned __int128>(n - 1) * static_cast<uint64_t>(stride) + at +
                                static_cast<uint64_t>(width);
    return e > UINTPTR_MAX ? UINTPTR_MAX : static_cast<uintptr_t>(e);
  }
};
// Whether a row of r has a byte of [lo, hi).
bool meets(const Rows& r, uintptr_t lo, uintptr_t hi) {
  if (hi <= r.at || lo >= r.end()) return false;
  const int64_t gap = static_cast<int64_t>(lo - r.at) - r.width;   // the first row that ends behind lo
  const int64_t first = lo <= r.at || gap < 0 ? 0 : gap / r.stride + 1;
  return r.at + static_cast<uintptr_t>(first * r.stride) < hi;     // the last row ends at r.end() > lo
}
// Whether two sets of rows (both not empty) share a byte.  Slices of one buffer lie between each other
// without; those have one stride, so that two rows of b stand for all.
bool meet(const Rows& a, const Rows& b) {
  if (a.end() <= b.at || b.end() <= a.at) return false;
  if (a.n > 1 && b.n > 1 && a.stride == b.stride) {
    if (b.at < a.at) return meet(b, a);
    return meets(a, b.at, b.at + b.width);   // a's rows from here on and b's go on in step
  }
  const Rows &few = a.n < b.n ? a : b, &many = a.n < b.n ? b : a;
  for (int64_t i = 0; i < few.n; ++i) {
    const uintptr_t lo = few.at + static_cast<uintptr_t>(i) * static_cast<uintptr_t>(few.stride);
    if (lo >= many.end()) return false;
    if (meets(many, lo, lo + few.width)) return true;
  }
  return false;
}
Rows rows_at(const void* p, int64_t n, int64_t width, int64_t stride) {
  return Rows{reinterpret_cast<uintptr_t>(p), stride, width, n};
}

int check_heads(const char* fn, int32_t heads, int32_t head_dim, int32_t dtype, bool f32) {
  if (heads <= 0 || heads > 65535) return refuse(Q8A_ERR_INVALID_ARG, fn, "heads must be 1..65535 (got %d)", heads);
  if (head_dim != 64 && head_dim != 128)
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "head_dim must be 64 or 128 (got %d)", head_dim);
  if (dtype != Q8A_F16 && dtype != Q8A_BF16 && !(f32 && dtype == Q8A_F32))
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "dtype must be Q8A_F16%s Q8A_BF16%s (got %d)", f32 ? "," : " or",
                  f32 ? " or Q8A_F32" : "", dtype);
  return Q8A_OK;
}

int check_stride(const char* fn, const char* name, int64_t stride, int32_t heads, int32_t head_dim) {
  if (stride < static_cast<int64_t>(heads) * head_dim || stride > kMaxStride)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "%s token stride %lld: at least heads*head_dim = %lld elements, at most 2^32",
                  name, (long long)stride, (long long)heads * head_dim);
  return Q8A_OK;
}

int check_rope(const char* fn, const int64_t* positions, const double* inv_freq, int32_t rot_dim, int32_t head_dim,
               int32_t layout, float mscale) {
  if (!positions || !inv_freq) return refuse(Q8A_ERR_INVALID_ARG, fn, "null positions or inv_freq");
  if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 2)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "rot_dim must be even, 2..head_dim (got %d)", rot_dim);
  if (layout != Q8A_ROPE_HALF && layout != Q8A_ROPE_INTERLEAVED)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "layout must be Q8A_ROPE_HALF or Q8A_ROPE_INTERLEAVED (got %d)", layout);
  if (!std::isfinite(mscale) || mscale == 0.0f)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "mscale must be finite and not 0");
  if (!aligned(positions, 8) || !aligned(inv_freq, 8))
    return refuse(Q8A_ERR_MISALIGNED, fn, "positions and inv_freq need 8-byte alignment");
  return Q8A_OK;
}

int check_pool(const char* fn, const void* k_pages, const void* v_pages, int64_t n_pages, int32_t page_tokens,
               int64_t page_stride_bytes, int32_t kv_heads, int32_t head_dim, q8a::PagePool* pool) {
  if (page_tokens < 16 || page_tokens > 4096 || (page_tokens & (page_tokens - 1)))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "page_tokens must be a power of two, 16..4096 (got %d)", page_tokens);
  if (n_pages <= 0 || n_pages > 0x7FFFFFFFll)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "n_pages must be 1..2^31-1 (got %lld)", (long long)n_pages);
  const int64_t need = static_cast<int64_t>(kv_heads) * page_tokens * row_bytes(head_dim);
  if (page_stride_bytes < need || page_stride_bytes > (int64_t{1} << 40))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "page stride %lld < kv_heads*page_tokens*%lld = %lld, or beyond 2^40",
                  (long long)page_stride_bytes, (long long)row_bytes(head_dim), (long long)need);
  if (!k_pages || !v_pages) return refuse(Q8A_ERR_INVALID_ARG, fn, "null pages");
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || page_stride_bytes % 16)
    return refuse(Q8A_ERR_MISALIGNED, fn, "pages and the page stride must be 16-byte aligned");
  pool->k = static_cast<uint8_t*>(const_cast<void*>(k_pages));
  pool->v = static_cast<uint8_t*>(const_cast<void*>(v_pages));
  pool->n_pages = n_pages;
  pool->page_stride = page_stride_bytes;
  pool->kv_heads = kv_heads;
  pool->page_shift = 0;
  while ((1 << pool->page_shift) < page_tokens) ++pool->page_shift;
  return Q8A_OK;
}

int status_words(const char* fn, uint32_t** out) {
  *out = q8a::host_status_words();
  if (!*out) return refuse(Q8A_ERR_CUDA, fn, "the host-mapped status words could not be registered");
  return Q8A_OK;
}

}  // namespace

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

// The launches of a call, from its bounds alone.
struct Plan {
  bool few, direct, tiles;
  q8a::TilesPlan t;
  int64_t few_rows;   // rows a K/V head of the few-row kernel's sequences, at most: it sizes its tiles
                      // and their partial states, so workspace and launch both take it from here
  int64_t few_floats, floats;
};
Plan plan_paged(int64_t batch, int64_t total_q, int64_t max_q, int64_t group, int32_t kv_heads, int64_t max_kv,
                int32_t head_dim) {
  Plan p{};
  if (max_q > total_q) max_q = total_q;
  if (max_kv > q8a::kMaxKeys) max_kv = q8a::kMaxKeys;
  p.tiles = max_q * group > kFewRows;
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
  p.direct = q8a::paged_few_direct(batch, kv_heads, max_kv, head_dim);
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

int attn_paged(const void* q, int32_t dtype, int64_t q_token_stride, int64_t total_q, int32_t heads, int32_t kv_heads,
               int32_t head_dim, const void* k_pages, const void* v_pages, int64_t n_pages, int32_t page_tokens,
               int64_t page_stride_bytes, const int32_t* block_table, int64_t table_stride, const int32_t* kv_lens,
               const int32_t* cu_q, int64_t batch, int64_t max_q, int64_t max_kv, float scale, int32_t causal,
               void* out, float* workspace, int64_t workspace_floats, void* stream) {
  q8a::NvtxRange nvtx_range("attn_paged");
  q8a::PdlScope early;   // see the top of this file
  const char* fn = "attn_paged";
  if (int rc = check_heads(fn, heads, head_dim, dtype, false)) return rc;
  if (kv_heads <= 0 || heads % kv_heads)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "heads (%d) must be a positive multiple of kv_heads (%d)", heads, kv_heads);
  if (batch < 0 || batch > (1 << 20) || total_q < 0 || total_q >= kMaxTokens || max_q < 0 || max_kv < 0)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "batch must be 0..2^20, total_q 0..2^31-1, max_q and max_kv not negative");
  const float scale_log2 = scale * 1.4426950408889634f;   // log2(e)
  if (!(scale > 0.0f) || !std::isfinite(scale_log2))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "scale must be > 0 and finite, also times log2(e)");
  if (int rc = check_stride(fn, "q", q_token_stride, heads, head_dim)) return rc;
  if (batch == 0 || total_q == 0 || max_q == 0) return q8a::clear_error();
  q8a::PagePool pool;
  if (int rc = check_pool(fn, k_pages, v_pages, n_pages, page_tokens, page_stride_bytes, kv_heads, head_dim, &pool))
    return rc;
  if (!q || !out || !kv_lens || !cu_q || (table_stride > 0 && !block_table))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  if (out == q) return refuse(Q8A_ERR_INVALID_ARG, fn, "out must not be q");
  if (table_stride < 0 || table_stride > 0x7FFFFFFFll)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "table stride must be 0..2^31-1 (got %lld)", (long long)table_stride);
  if (max_kv > table_stride * page_tokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "max_kv %lld: the table's rows hold %lld keys", (long long)max_kv,
                  (long long)(table_stride * page_tokens));
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) || q_token_stride % 8 ||
      !aligned(kv_lens, 4) || !aligned(cu_q, 4) || !aligned(block_table, 4))
    return refuse(Q8A_ERR_MISALIGNED, fn,
                  "q, its token stride, out and workspace need 16-byte, the index arrays 4-byte alignment");
  if (total_q * (heads / kv_heads) >= kMaxTokens)
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "total_q * heads / kv_heads must be below 2^31");
  const Plan plan = plan_paged(batch, total_q, max_q, heads / kv_heads, kv_heads, max_kv, head_dim);
  const int64_t need = plan.floats;
  if (need > 0 && !workspace) return refuse(Q8A_ERR_INVALID_ARG, fn, "null workspace");
  if (workspace_floats < need)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "workspace of %lld floats < %lld needed", (long long)workspace_floats,
                  (long long)need);
  {
    const int64_t row = static_cast<int64_t>(heads) * head_dim * 2;
    const Rows q_rows = rows_at(q, total_q, row, q_token_stride * 2), o_rows = rows_at(out, total_q, row, row);
    if (meet(q_rows, o_rows)) return refuse(Q8A_ERR_INVALID_ARG, fn, "q and out overlap");
    const Rows ws = rows_at(workspace, 1, need * 4, need * 4);
    if (need > 0 && (meet(q_rows, ws) || meet(o_rows, ws)))
      return refuse(Q8A_ERR_INVALID_ARG, fn, "the workspace overlaps q or out");
  }
  q8a::PagedArgs a{};
  a.q = q;
  a.out = out;
  a.k = pool.k;
  a.v = pool.v;
  a.table = block_table;
  a.kv_lens = kv_lens;
  a.cu_q = cu_q;
  a.part = workspace;
  a.n_pages = n_pages;
  a.page_stride = page_stride_bytes;
  a.q_stride = q_token_stride;
  a.table_stride = table_stride;
  a.total_q = total_q;
  a.batch = static_cast<int32_t>(batch);
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.page_shift = pool.page_shift;
  a.causal = causal ? 1 : 0;
  a.scale_log2 = scale_log2;
  a.timeout_ns = q8a::wait_timeout_ns();
  if (int rc = status_words(fn, &a.status)) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (plan.tiles) {
    q8a::PagedArgs b = a;
    b.row_limit = plan.few ? static_cast<int32_t>(kFewRows) : 0;
    b.shares = plan.t.shares;
    b.share_tiles = plan.t.share_tiles;
    b.ctas = plan.t.ctas;
    b.part = workspace + plan.few_floats;
    b.part_ml = plan.t.part_ml;
    auto even = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 32 == 0; };
    b.wide = (even(q) && q_token_stride % 16 == 0 ? q8a::kWideQ : 0) | (even(out) ? q8a::kWideOut : 0) |
             (even(b.part) ? q8a::kWidePart : 0);
    e = q8a::launch_paged_tiles(b, dtype, head_dim, plan.t, st);
  }
  if (plan.few && e == cudaSuccess) {
    a.row_limit = plan.tiles ? static_cast<int32_t>(kFewRows) : 0x7FFFFFFF;
    e = q8a::launch_paged_few(a, dtype, head_dim, plan.few_rows, plan.direct, st);
  }
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

}  // extern "C"
