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

}  // namespace q8a
