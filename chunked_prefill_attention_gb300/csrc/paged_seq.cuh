// paged_seq.cuh -- what the paged kernels share on the device: the record of a failure
// and the reading of a batch's lengths.
#pragma once

#include "internal.h"
#include "paged.h"
#include "ptx.cuh"

namespace q8a {

// Plain stores: each word has one code, so it does not matter who stores it, or how often.
__device__ __forceinline__ void record_timeout(uint32_t* status) {
  *reinterpret_cast<volatile uint32_t*>(status + kHostPagedTimeout) = kStatusTimeout;
}
__device__ __forceinline__ void record_index(uint32_t* status) {
  *reinterpret_cast<volatile uint32_t*>(status + kHostPagedIndex) = kStatusIndex;
}

// A sequence as the device arrays give it, with every bound checked: rows that
// do not exist and keys beyond the table are left out and recorded.
struct Seq {
  int64_t q0;      // first query row
  int32_t n_q, kv;
};
__device__ __forceinline__ Seq read_seq(const PagedArgs& a, int b) {
  Seq s;
  int64_t q0 = a.cu_q[b], q1 = a.cu_q[b + 1];
  const int64_t kv = a.kv_lens[b], most = i64min(a.table_stride << a.page_shift, kMaxKeys);
  const bool wrong = q0 < 0 || q1 < q0 || q1 > a.total_q || kv < 0 || kv > most;
  if (wrong) record_index(a.status);
  q0 = i64max(0, i64min(q0, a.total_q));
  q1 = i64max(q0, i64min(q1, a.total_q));
  s.q0 = q0;
  s.n_q = static_cast<int32_t>(q1 - q0);
  s.kv = static_cast<int32_t>(i64max(0, i64min(kv, most)));
  return s;
}

// Keys of the shared prefix: whole pages of it, so that what is left of it is every sequence's own.
__device__ __forceinline__ int prefix_keys(const PagedArgs& a) {
  const int64_t n = a.prefix_len[0];
  if (n < 0 || n > a.prefix_most) record_index(a.status);
  return static_cast<int>(i64max(0, i64min(n, a.prefix_most)) >> a.page_shift << a.page_shift);
}

// The key tiles of a run of rows: `sink` tiles from key 0 on, the others `skip` keys further on than they would be;
// the first of these starts a piece of a page (kPlain: all from key 0 on).
struct Span {
  int32_t sink, skip;
  int32_t low;   // kWindow: where the pieces of the first row's window start
};
template <int kMode, int KT>
__device__ __forceinline__ int key_of(const Span& s, int tile) {
  if (kMode == kPlain || kMode == kPrefix) return tile * KT;
  return tile * KT + (kMode == kWindow && tile < s.sink ? 0 : s.skip);
}
// Whether any row needs the piece that starts at `key`.  Those between the sinks and the window are not copied (their
// pages may have been given away), so a tile has there whatever its buffer held.
template <int kMode>
__device__ __forceinline__ bool piece_needed(const PagedArgs& a, const Span& s, int key) {
  return kMode != kWindow || key >= s.low || key < a.sinks;
}
// Of rows whose first token is at position p0 and whose last sees the keys before `end`; start: the first own key.
template <int kMode, int KT>
__device__ __forceinline__ Span span_of(const PagedArgs& a, int64_t p0, int end, int start, int piece_shift) {
  if (kMode == kOwn) return Span{0, start, 0};
  if (kMode != kWindow) return Span{0, 0, 0};
  Span s;
  s.low = static_cast<int32_t>(i64max(0, p0 - a.window + 1) >> piece_shift << piece_shift);
  s.sink = (max(0, min(a.sinks, end)) + KT - 1) / KT;
  const int64_t skip = s.low - static_cast<int64_t>(s.sink) * KT;
  s.skip = static_cast<int32_t>(i64max(0, skip));
  if (skip <= 0) s.sink = 0;   // one run
  return s;
}
// Tiles that reach the keys before `end`.
template <int kMode, int KT>
__device__ __forceinline__ int span_tiles(const Span& s, int end) {
  return (max(end - (kMode == kPlain || kMode == kPrefix ? 0 : s.skip), kMode == kWindow ? s.sink * KT : 0) + KT - 1) / KT;
}

// Weight of a partial state (reference m, sum l) under the joint reference top.  A row whose scores
// are all NaN has no reference, and keeps its NaN.
__device__ __forceinline__ float state_weight(float m, float l, float top) {
  return m == -INFINITY ? (l != l ? l : 0.0f) : (m == top ? 1.0f : ex2_approx(m - top));
}
// The logarithm of a row's sum of weights; -infinity of a row that sees nothing.
__device__ __forceinline__ float state_log(float m, float l) {
  return l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) + log2f(l);
}

}  // namespace q8a
