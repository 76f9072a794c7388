// paged_check.h -- the argument checks that the C-ABI layers of the paged calls share: refusals with a message,
// the sizes and alignments of packed tensors, tables of angles and pools, and whether buffers share memory.
#pragma once

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "../../include/q8attn.h"
#include "internal.h"
#include "paged.h"

namespace {

inline int refuse(int code, const char* fn, const char* fmt, ...) {
  char msg[384];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return q8a::set_error(code, fn, msg);
}
inline int cuda_refuse(cudaError_t e, const char* fn) {
  cudaGetLastError();   // a refused launch leaves no error behind for the caller's next check
  return refuse(Q8A_ERR_CUDA, fn, "%s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
}
inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int64_t row_bytes(int32_t head_dim) { return static_cast<int64_t>(head_dim / 32) * 34; }
inline int64_t elem_bytes(int32_t dtype) { return dtype == Q8A_F32 ? 4 : 2; }

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
inline bool meets(const Rows& r, uintptr_t lo, uintptr_t hi) {
  if (hi <= r.at || lo >= r.end()) return false;
  const int64_t gap = static_cast<int64_t>(lo - r.at) - r.width;   // the first row that ends behind lo
  const int64_t first = lo <= r.at || gap < 0 ? 0 : gap / r.stride + 1;
  return r.at + static_cast<uintptr_t>(first * r.stride) < hi;     // the last row ends at r.end() > lo
}
// Whether two sets of rows (both not empty) share a byte.  Slices of one buffer lie between each other
// without; those have one stride, so that two rows of b stand for all.
inline bool meet(const Rows& a, const Rows& b) {
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
inline Rows rows_at(const void* p, int64_t n, int64_t width, int64_t stride) {
  return Rows{reinterpret_cast<uintptr_t>(p), stride, width, n};
}

inline int check_heads(const char* fn, int32_t heads, int32_t head_dim, int32_t dtype, bool f32) {
  if (heads <= 0 || heads > 65535) return refuse(Q8A_ERR_INVALID_ARG, fn, "heads must be 1..65535 (got %d)", heads);
  if (head_dim != 64 && head_dim != 128)
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "head_dim must be 64 or 128 (got %d)", head_dim);
  if (dtype != Q8A_F16 && dtype != Q8A_BF16 && !(f32 && dtype == Q8A_F32))
    return refuse(Q8A_ERR_UNSUPPORTED, fn, "dtype must be Q8A_F16%s Q8A_BF16%s (got %d)", f32 ? "," : " or",
                  f32 ? " or Q8A_F32" : "", dtype);
  return Q8A_OK;
}

inline int check_stride(const char* fn, const char* name, int64_t stride, int32_t heads, int32_t head_dim) {
  if (stride < static_cast<int64_t>(heads) * head_dim || stride > kMaxStride)
    return refuse(Q8A_ERR_INVALID_ARG, fn, "%s token stride %lld: at least heads*head_dim = %lld elements, at most 2^32",
                  name, (long long)stride, (long long)heads * head_dim);
  return Q8A_OK;
}

inline int check_rope(const char* fn, const int64_t* positions, const double* inv_freq, int32_t rot_dim, int32_t head_dim,
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

inline int check_pool(const char* fn, const void* k_pages, const void* v_pages, int64_t n_pages, int32_t page_tokens,
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

inline int status_words(const char* fn, uint32_t** out) {
  *out = q8a::host_status_words();
  if (!*out) return refuse(Q8A_ERR_CUDA, fn, "the host-mapped status words could not be registered");
  return Q8A_OK;
}

}  // namespace
