// paged.h -- launchers of the paged Q8_0 cache and of the rotary positions,
// shared by the C-ABI layer (paged_api.cu) and the kernel translation units.
// Not part of the public ABI.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace q8a {

// Element types of the paged calls (Q8A_F16, Q8A_BF16, Q8A_F32 of the ABI).
enum : int32_t { kF16 = 0, kBF16 = 1, kF32 = 2 };

// Codes that the paged kernels store into the device's host-mapped status words, each
// into its own (kHostPagedTimeout, kHostPagedIndex): bit 0 a wait that ran out, bit 1 an
// index or length out of range; bits 8..15 the role.
enum : uint32_t { kRolePaged = 6, kRoleIndex = 7 };
constexpr uint32_t kStatusTimeout = 1u | (kRolePaged << 8);
constexpr uint32_t kStatusIndex = 2u | (kRoleIndex << 8);

// Rotary positions of packed tokens: channel pairs of the first `rot` channels
// turned by position * inv_freq.  inv_freq null (append only): no rotation.
struct RopeArgs {
  const int64_t* positions;   // [n_tokens]
  const double* inv_freq;     // [rot / 2], radians per position
  int32_t rot;
  int32_t interleaved;
  float mscale;
  float sign;                 // +1, or -1 for the inverse rotation
};

cudaError_t launch_rope(const void* x, void* out, int32_t dtype, int64_t n_tokens, int32_t heads,
                        int32_t head_dim, int64_t x_stride, int64_t out_stride, const RopeArgs& r,
                        cudaStream_t stream);

// A pool of pages: page p holds, for each K/V head, page_tokens rows.
struct PagePool {
  uint8_t* k;
  uint8_t* v;
  int64_t n_pages;
  int64_t page_stride;   // bytes between pages
  int32_t page_shift;    // log2(page_tokens)
  int32_t kv_heads;
};

cudaError_t launch_append(const void* k, const void* v, int32_t dtype, int64_t n_tokens, int32_t head_dim,
                          int64_t k_stride, int64_t v_stride, const int64_t* slots, const RopeArgs& r,
                          const PagePool& pool, uint32_t* status, cudaStream_t stream);

cudaError_t launch_read(void* k, void* v, int32_t dtype, int64_t n_tokens, int32_t head_dim,
                        const int64_t* slots, const PagePool& pool, uint32_t* status, cudaStream_t stream);

// Queries and keys of packed tokens, each head row divided by its root mean square and rotated.
struct NormRopeArgs {
  const void* x[2];           // q, k: [n_tokens][heads][D], token strides x_stride
  void* out[2];
  int64_t x_stride[2];
  int64_t out_stride[2];
  const void* weight[2];      // [D] of weight_dtype; null: that tensor is not normalised
  int64_t n_tokens;
  int32_t heads[2];           // heads[1] may be 0
  int32_t weight_dtype;
  float eps;
  const int64_t* positions;   // [n_axes][n_tokens]
  const int32_t* axes;        // [rot / 2] axis of each pair, or null: axis 0
  const double* inv_freq;     // [rot / 2], radians per position
  int32_t n_axes;
  int32_t rot;                // 0: no rotation
  int32_t interleaved;
  float mscale;
  uint32_t* status;
};
cudaError_t launch_norm_rope(const NormRopeArgs& a, int32_t dtype, int32_t head_dim, cudaStream_t stream);

// Lengths, tables and slots of a step.
struct ExtendArgs {
  const int32_t* new_lens;    // [batch]
  const int32_t* kv_lens;     // [batch] keys before the step
  int32_t* table;             // [batch][table_stride]
  const int32_t* free_pages;  // [free_capacity], the next page last
  const int32_t* n_free;      // [1]
  int32_t* kv_out;            // [batch], may be kv_lens
  int32_t* cu_q;              // [batch + 1]
  int64_t* slots;             // [total_q]
  int64_t* positions;         // [total_q]
  int32_t* n_free_out;        // [1], may be n_free
  int64_t batch;
  int64_t table_stride;
  int64_t free_capacity;
  int64_t total_q;
  int32_t page_shift;
  uint32_t* status;
};
cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream);

constexpr int kSms = 152;   // of a GB300: what the rules fill waves of

// Most keys of a sequence: lengths are int32, and a tile's end must not pass 2^31.
constexpr int64_t kMaxKeys = 0x7FFF0000;

// Arguments of the attention over pages.
struct PagedArgs {
  const void* q;              // [total_q][heads][D], token stride q_stride elements
  void* out;                  // [total_q][heads][D], contiguous
  const uint8_t* k;
  const uint8_t* v;
  const int32_t* table;       // [batch][table_stride] page numbers
  const int32_t* kv_lens;     // [batch], the new tokens included
  const int32_t* cu_q;        // [batch + 1], first query row of each sequence
  float* part;                // partial states of the split units
  uint32_t* status;           // device address of the device's host-mapped status words
  int64_t n_pages;
  int64_t page_stride;
  int64_t q_stride;
  int64_t table_stride;
  int64_t total_q;
  int32_t batch;
  int32_t heads;
  int32_t kv_heads;
  int32_t group;              // heads / kv_heads
  int32_t page_shift;
  int32_t causal;
  float scale_log2;           // scale * log2(e)
  int32_t row_limit;          // sequences of at most so many rows (tokens * group) are the few-row
                              // kernel's, the others the tile kernel's
  int32_t shares;             // tile kernel: units are cut into shares of their key tiles
  int32_t share_tiles;        // key tiles of a share; 0: from the lengths, on the device
  int64_t part_ml;            // tile kernel: floats of `part` before the shares' (m, l)
  int64_t ctas;               // tile kernel: its grid
  int32_t wide;               // tile kernel: whose rows start 32-byte aligned (kWide...)
  uint64_t timeout_ns;
  // kWindow: a row sees the keys of the last `window` positions up to its own, and the first `sinks`
  int32_t window, sinks;
  // kOwn, kPrefix: the keys before prefix_len (down to a whole page) are every sequence's
  const int32_t* prefix_len;  // [1] on the device
  int64_t prefix_most;        // what it may be at most
  int32_t seqs;               // kPrefix: sequences of kv_lens and cu_q (batch is 1)
  int32_t row_tiles;          // few-row kernel, direct, kWindow and kOwn: tiles of 16 rows (8 where one is enough) of a unit
  int32_t cluster;            // few-row kernel, direct, kWindow and kOwn: CTAs of a unit (1, 2, 4 or 8)
  int32_t only;               // and whether each has an SM for itself, by the plan
  int32_t join_rows;          // kPrefix: rows of a block of the join, 8 (a warp each) or 1
  float* state;               // [total_q][heads][D] and then [total_q][heads]: outputs over the own keys,
                              // and the logarithms (base 2) of their sums of weights
};

// Which keys the rows of a launch see.
enum : int {
  kPlain = 0,
  kWindow = 1,   // window and sinks
  kOwn = 2,      // those behind the shared prefix; the rows' states go to PagedArgs::state
  kPrefix = 3    // the shared prefix: all rows of all sequences are one sequence's, whose join takes the
                 // rows' states over their own keys in and writes `out`
};

constexpr int32_t kWideQ = 1, kWideOut = 2, kWidePart = 4;

// Few query rows per K/V head: one launch over key tiles plus the merge.
// `rows`: the largest tokens * group of the sequences it takes (a bound).
// `direct`: a CTA per (sequence, K/V head), no workspace.
cudaError_t launch_paged_few(const PagedArgs& a, int32_t dtype, int32_t head_dim, int64_t rows, bool direct,
                             cudaStream_t stream);
bool paged_few_direct(int64_t batch, int32_t kv_heads, int64_t max_kv, int32_t head_dim);
// Floats of PagedArgs::part that launch_paged_few needs when not direct.
int64_t paged_few_floats(int32_t head_dim, int64_t rows);

// Many query rows per K/V head.  The plan of a call from its bounds.
struct TilesPlan {
  bool pair;        // no sequence of more than 128 rows
  bool shares;
  int32_t share_tiles;
  int64_t slots;    // (row unit, K/V head) pairs, at most
  int64_t ctas;
  int64_t part_ml;
  int64_t floats;
};
TilesPlan plan_paged_tiles(int64_t batch, int64_t total_rows, int64_t max_rows, int32_t kv_heads, int64_t max_kv,
                           int32_t head_dim);
cudaError_t launch_paged_tiles(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                               cudaStream_t stream);
// Key tiles that a row unit of a sequence of kv keys can take in a window, at most (`group` query heads a K/V head).
int64_t window_tiles(int64_t kv, int64_t window, int64_t sinks, int32_t group, bool pair, int32_t head_dim);

// The same launches where rows see other keys than all before them (the tile kernel's kOwn in pairs only).
cudaError_t launch_paged_few_range(const PagedArgs& a, int mode, int32_t dtype, int32_t head_dim, int64_t rows,
                                   bool direct, cudaStream_t stream);   // kWindow or kOwn
cudaError_t launch_paged_tiles_window(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                      cudaStream_t stream);
cudaError_t launch_paged_tiles_own(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                   cudaStream_t stream);
cudaError_t launch_paged_tiles_prefix(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                                      cudaStream_t stream);

}  // namespace q8a
