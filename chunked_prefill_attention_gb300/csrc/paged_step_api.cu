// paged_step_api.cu -- the extern "C" entry points of a step's tables and of the norms with rotary positions
// (declared in include/q8attn.h): host-side argument validation and the launches, as in paged_api.cu.

#include "paged_check.h"

namespace {

// Whether two runs of bytes share one.
bool share(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  if (a_bytes <= 0 || b_bytes <= 0 || !a || !b) return false;
  return meet(rows_at(a, 1, a_bytes, a_bytes), rows_at(b, 1, b_bytes, b_bytes));
}

}  // namespace

extern "C" {

int q8kv_extend_paged(const int32_t* new_lens, const int32_t* kv_lens, int64_t batch, int32_t* block_table,
                      int64_t table_stride, const int32_t* free_pages, int64_t free_capacity, const int32_t* n_free,
                      int32_t page_tokens, int64_t total_q, int32_t* kv_lens_out, int32_t* cu_q, int64_t* slots,
                      int64_t* positions, int32_t* n_free_out, void* stream) {
  q8a::NvtxRange nvtx_range("q8kv_extend_paged");
  q8a::PdlScope early;
  const char* fn = "q8kv_extend_paged";
  if (batch < 0 || batch > (1 << 20) || total_q < 0 || total_q >= kMaxTokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "batch must be 0..2^20, total_q 0..2^31-1 (got %lld, %lld)", (long long)batch,
                  (long long)total_q);
  if (page_tokens < 16 || page_tokens > 4096 || (page_tokens & (page_tokens - 1)))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "page_tokens must be a power of two, 16..4096 (got %d)", page_tokens);
  if (table_stride < 0 || table_stride > 0x7FFFFFFFll)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "table stride must be 0..2^31-1 (got %lld)", (long long)table_stride);
  if (free_capacity < 0 || free_capacity > 0x7FFFFFFFll)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "free_capacity must be 0..2^31-1 (got %lld)", (long long)free_capacity);
  if (!n_free || !n_free_out || !cu_q || (batch > 0 && (!new_lens || !kv_lens || !kv_lens_out)) ||
      (total_q > 0 && (!slots || !positions)) || (batch > 0 && table_stride > 0 && !block_table) ||
      (free_capacity > 0 && !free_pages))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  if (!aligned(new_lens, 4) || !aligned(kv_lens, 4) || !aligned(block_table, 4) || !aligned(free_pages, 4) ||
      !aligned(n_free, 4) || !aligned(kv_lens_out, 4) || !aligned(cu_q, 4) || !aligned(n_free_out, 4) ||
      !aligned(slots, 8) || !aligned(positions, 8))
    return refuse(Q8A_ERR_MISALIGNED, fn, "slots and positions need 8-byte, the other arrays 4-byte alignment");
  // what is written shares no byte with anything else, but the lengths and the number of free pages with themselves
  struct Run {
    const void* at;
    int64_t bytes;
  };
  const Run out[6] = {{kv_lens_out, 4 * batch},   {cu_q, 4 * (batch + 1)},
                      {slots, 8 * total_q},       {positions, 8 * total_q},
                      {n_free_out, 4},            {block_table, 4 * batch * table_stride}};
  const Run in[4] = {{kv_lens, 4 * batch}, {n_free, 4}, {new_lens, 4 * batch}, {free_pages, 4 * free_capacity}};
  for (int i = 0; i < 6; ++i) {
    for (int j = i + 1; j < 6; ++j)
      if (share(out[i].at, out[i].bytes, out[j].at, out[j].bytes))
        return refuse(Q8A_ERR_INVALID_ARG, fn, "two of the outputs and the table overlap");
    for (int j = 0; j < 4; ++j) {
      const bool same = out[i].at == in[j].at && ((i == 0 && j == 0) || (i == 4 && j == 1));
      if (!same && share(out[i].at, out[i].bytes, in[j].at, in[j].bytes))
        return refuse(Q8A_ERR_INVALID_ARG, fn, "an output or the table overlaps an input");
    }
  }
  q8a::ExtendArgs a{};
  a.new_lens = new_lens;
  a.kv_lens = kv_lens;
  a.table = block_table;
  a.free_pages = free_pages;
  a.n_free = n_free;
  a.kv_out = kv_lens_out;
  a.cu_q = cu_q;
  a.slots = slots;
  a.positions = positions;
  a.n_free_out = n_free_out;
  a.batch = batch;
  a.table_stride = table_stride;
  a.free_capacity = free_capacity;
  a.total_q = total_q;
  while ((1 << a.page_shift) < page_tokens) ++a.page_shift;
  if (int rc = status_words(fn, &a.status)) return rc;
  const cudaError_t e = q8a::launch_extend(a, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

int attn_norm_rope(const void* q, void* q_out, int32_t heads, int64_t q_token_stride, int64_t q_out_token_stride,
                   const void* k, void* k_out, int32_t kv_heads, int64_t k_token_stride, int64_t k_out_token_stride,
                   int32_t dtype, int64_t n_tokens, int32_t head_dim, const void* q_weight, const void* k_weight,
                   int32_t weight_dtype, float eps, const int64_t* positions, int32_t n_axes, const int32_t* axes,
                   const double* inv_freq, int32_t rot_dim, int32_t layout, float mscale, void* stream) {
  q8a::NvtxRange nvtx_range("attn_norm_rope");
  q8a::PdlScope early;
  const char* fn = "attn_norm_rope";
  if (int rc = check_heads(fn, heads, head_dim, dtype, true)) return rc;
  if (kv_heads < 0 || kv_heads > 65535)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "kv_heads must be 0..65535 (got %d)", kv_heads);
  if (n_tokens < 0 || n_tokens > kMaxTokens)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "n_tokens must be 0..2^31 (got %lld)", (long long)n_tokens);
  if (weight_dtype != Q8A_F16 && weight_dtype != Q8A_BF16 && weight_dtype != Q8A_F32)
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "weight_dtype must be Q8A_F16, Q8A_BF16 or Q8A_F32 (got %d)", weight_dtype);
  if (!(eps >= 0.0f) || !std::isfinite(eps))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "eps must be finite and not negative");
  if (int rc = check_stride(fn, "q", q_token_stride, heads, head_dim)) return rc;
  if (int rc = check_stride(fn, "q_out", q_out_token_stride, heads, head_dim)) return rc;
  if (kv_heads > 0) {
    if (int rc = check_stride(fn, "k", k_token_stride, kv_heads, head_dim)) return rc;
    if (int rc = check_stride(fn, "k_out", k_out_token_stride, kv_heads, head_dim)) return rc;
  }
  if (n_axes < 0 || n_axes > 65535 || (n_axes > 1 && !axes))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "n_axes must be 0..65535, with axes where it is above 1 (got %d)", n_axes);
  const bool turns = positions || inv_freq;
  if (!turns && !q_weight && !(k_weight && kv_heads > 0))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "neither a weight nor positions: nothing to do");
  if (n_tokens == 0) return q8a::clear_error();
  if (!q || !q_out || (kv_heads > 0 && (!k || !k_out))) return refuse(Q8A_ERR_INVALID_ARG, fn, "null pointer");
  const int64_t size = elem_bytes(dtype);
  if (!aligned(q, size) || !aligned(q_out, size) || (kv_heads > 0 && (!aligned(k, size) || !aligned(k_out, size))) ||
      !aligned(q_weight, elem_bytes(weight_dtype)) || !aligned(k_weight, elem_bytes(weight_dtype)) || !aligned(axes, 4))
    return refuse(Q8A_ERR_MISALIGNED, fn, "q, k, the outputs, the weights and axes need their element's alignment");
  if (turns) {
    if (int rc = check_rope(fn, positions, inv_freq, rot_dim, head_dim, layout, mscale)) return rc;
    if (n_axes < 1) return refuse(Q8A_ERR_INVALID_ARG, fn, "positions of at least one axis are needed");
  }
  if ((q == q_out && q_token_stride != q_out_token_stride) ||
      (kv_heads > 0 && k == k_out && k_token_stride != k_out_token_stride))
    return refuse(Q8A_ERR_INVALID_ARG, fn, "in place, input and output must have the same token stride");
  {
    const int64_t wq = static_cast<int64_t>(heads) * head_dim * size, wk = static_cast<int64_t>(kv_heads) * head_dim * size;
    const Rows rq = rows_at(q, n_tokens, wq, q_token_stride * size), oq = rows_at(q_out, n_tokens, wq, q_out_token_stride * size);
    if (q != q_out && meet(rq, oq)) return refuse(Q8A_ERR_INVALID_ARG, fn, "q and q_out overlap");
    if (kv_heads > 0) {
      const Rows rk = rows_at(k, n_tokens, wk, k_token_stride * size), ok = rows_at(k_out, n_tokens, wk, k_out_token_stride * size);
      if (k != k_out && meet(rk, ok)) return refuse(Q8A_ERR_INVALID_ARG, fn, "k and k_out overlap");
      if (meet(oq, ok) || meet(oq, rk) || meet(ok, rq))
        return refuse(Q8A_ERR_INVALID_ARG, fn, "an output overlaps the other output or input");
    }
  }
  q8a::NormRopeArgs a{};
  a.x[0] = q;
  a.x[1] = k;
  a.out[0] = q_out;
  a.out[1] = k_out;
  a.x_stride[0] = q_token_stride;
  a.x_stride[1] = k_token_stride;
  a.out_stride[0] = q_out_token_stride;
  a.out_stride[1] = k_out_token_stride;
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.n_tokens = n_tokens;
  a.heads[0] = heads;
  a.heads[1] = kv_heads;
  a.weight_dtype = weight_dtype;
  a.eps = eps;
  a.positions = positions;
  a.axes = axes;
  a.inv_freq = inv_freq;
  a.n_axes = n_axes;
  a.rot = turns ? rot_dim : 0;
  a.interleaved = layout == Q8A_ROPE_INTERLEAVED;
  a.mscale = mscale;
  if (int rc = status_words(fn, &a.status)) return rc;
  const cudaError_t e = q8a::launch_norm_rope(a, dtype, head_dim, static_cast<cudaStream_t>(stream));
  return e != cudaSuccess ? cuda_refuse(e, fn) : q8a::clear_error();
}

}  // extern "C"
