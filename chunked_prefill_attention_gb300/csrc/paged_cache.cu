// paged_cache.cu -- rotary positions, and the Q8_0 cache in pages: rows appended
// (rotated, quantised, scattered by slot) and read back (gathered, dequantised).
//
// All three kernels read and write each value once, and every thread has 32 to 128
// bytes in flight before the first use.  HBM bounds the rotation (81 % of the copy rate) and the
// read (85 %); the append waits for its loads and barriers (43 %, see there).
// This unit must not be built with fast-math (IEEE divides in the quantiser).

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.h"
#include "paged_seq.cuh"
#include "ptx.cuh"
#include "q8_codes.cuh"
#include "rotary.cuh"

namespace q8a {
namespace {

// One item of a head row: a pair of vectors, one vector of whole pairs
// (interleaved), or one vector that passes through.
constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 64;

// N: elements of one access.  kInter: pairs (2i, 2i + 1), else (i, i + rot / 2).
// A thread has one item (threadIdx.x) of one token and turns it in heads_per_thread
// heads, so its angles are formed once, in registers; the fp64 part of them, which does
// not depend on the token, once per block.
// Four resident blocks and up to 16 heads a thread: 16,384 tokens, 32 x 128 bf16, half of the
// channels turned in interleaved pairs, 49 us (three blocks and 8 heads 53, five blocks 54, eight
// heads in flight 67), 65,536 tokens 176 us, 6.1 TB/s (203); all channels in halves 63 us
// (three blocks 66, five 87), where two vectors and eight pairs of angles a thread leave bf16 with
// spills of 60 bytes of stores and 80 of loads (fp16 and fp32 none).
template <typename T, int N, bool kInter>
__global__ void __launch_bounds__(kRopeThreads, 4)
rope_kernel(const T* x, T* out, int64_t n_tokens, int32_t heads, int32_t head_dim, int64_t x_stride,
            int64_t out_stride, const RopeArgs r, int32_t heads_per_thread) {
  constexpr bool kTwo = !(kInter && N > 1);         // a rotating item is two vectors
  constexpr int kAngles = kTwo ? N : N / 2;
  constexpr int kU = kTwo && N > 1 ? 2 : 4;         // heads in flight
  __shared__ uint64_t steps[kMaxPairs];
  pdl_launch_dependents();
  pdl_wait();
  using V = Vec<T, N>;
  const int pairs = r.rot / 2;
  const int turning = kTwo ? pairs / N : r.rot / N;   // items that rotate
  const int item = threadIdx.x;
  const bool turns = item < turning;
  int c0, c1 = 0, pair0 = 0;
  if (turns) {
    c0 = kTwo ? (kInter ? 2 * item : item * N) : item * N;
    c1 = kInter ? c0 + 1 : c0 + pairs;
    pair0 = kTwo ? item * N : c0 / 2;
  } else {
    c0 = r.rot + (item - turning) * N;
  }
  const int64_t t = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  const int h0 = blockIdx.y * heads_per_thread;
  const int h1 = min(heads, h0 + heads_per_thread);
  const bool live = t < n_tokens && (turns || x != out);   // in place, the rest stays
  const T* px = x + t * x_stride + static_cast<int64_t>(h0) * head_dim;
  T* po = out + t * out_stride + static_cast<int64_t>(h0) * head_dim;
  V a[kU], b[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u)
    if (live && h0 + u < h1) {
      a[u] = *reinterpret_cast<const V*>(px + u * head_dim + c0);
      if (kTwo && turns) b[u] = *reinterpret_cast<const V*>(px + u * head_dim + c1);
    }
  const int64_t position = live ? r.positions[t] : 0;
  for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < pairs; i += blockDim.x * blockDim.y)
    steps[i] = turn_step(r.inv_freq[i]);
  __syncthreads();
  if (!live) return;
  float2 cs[kAngles];
  if (turns) {
#pragma unroll
    for (int e = 0; e < kAngles; ++e) cs[e] = rotation(position, steps[pair0 + e], r.mscale, r.sign);
  }
  for (int h = h0;;) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (h + u >= h1) break;
      if (turns) {
        if (kTwo) {
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float va = Elem<T>::get(a[u].e[e]), vb = Elem<T>::get(b[u].e[e]);
            const float2 y = turn_pair(va, vb, cs[e]);
            a[u].e[e] = Elem<T>::put(y.x);
            b[u].e[e] = Elem<T>::put(y.y);
          }
          *reinterpret_cast<V*>(po + u * head_dim + c1) = b[u];
        } else {
#pragma unroll
          for (int e = 0; e < N / 2; ++e) {
            const float va = Elem<T>::get(a[u].e[2 * e]), vb = Elem<T>::get(a[u].e[2 * e + 1]);
            const float2 y = turn_pair(va, vb, cs[e]);
            a[u].e[2 * e] = Elem<T>::put(y.x);
            a[u].e[2 * e + 1] = Elem<T>::put(y.y);
          }
        }
      }
      *reinterpret_cast<V*>(po + u * head_dim + c0) = a[u];
    }
    h += kU;
    if (h >= h1) break;
    px += kU * head_dim;
    po += kU * head_dim;
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (h + u < h1) {
        a[u] = *reinterpret_cast<const V*>(px + u * head_dim + c0);
        if (kTwo && turns) b[u] = *reinterpret_cast<const V*>(px + u * head_dim + c1);
      }
  }
}

template <typename T, int N>
cudaError_t launch_rope_n(const T* x, T* out, int64_t n_tokens, int32_t heads, int32_t head_dim,
                          int64_t x_stride, int64_t out_stride, const RopeArgs& r, cudaStream_t stream) {
  const bool two = !(r.interleaved && N > 1);
  const int items = (two ? r.rot / 2 / N : r.rot / N) + (head_dim - r.rot) / N;
  const int tokens = kRopeThreads / items;
  // as many heads a thread as leave every SM its threads
  constexpr int64_t kFill = kSms * 2048;
  int hpt = 16;
  while (hpt > 1 && n_tokens * items * ((heads + hpt - 1) / hpt) < kFill) hpt /= 2;
  const int64_t blocks = (n_tokens + tokens - 1) / tokens;
  const int64_t groups = (heads + hpt - 1) / hpt;
  if (blocks > 0x7FFFFFFF || groups > 65535) return cudaErrorInvalidValue;
  auto kernel = r.interleaved ? rope_kernel<T, N, true> : rope_kernel<T, N, false>;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(groups)), dim3(items, tokens), 0,
                       stream, x, out, n_tokens, heads, head_dim, x_stride, out_stride, r, hpt);
}

template <typename T>
cudaError_t launch_rope_t(const void* x, void* out, int64_t n_tokens, int32_t heads, int32_t head_dim,
                          int64_t x_stride, int64_t out_stride, const RopeArgs& r, cudaStream_t stream) {
  constexpr int kN = 16 / sizeof(T);
  const T* xt = static_cast<const T*>(x);
  T* ot = static_cast<T*>(out);
  // 16-byte accesses where a vector lies in one half of the rotated channels
  // and every row starts 16-byte aligned; single elements otherwise
  const bool wide = r.rot % (2 * kN) == 0 && x_stride % kN == 0 && out_stride % kN == 0 &&
                    (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(out)) % 16 == 0;
  return wide ? launch_rope_n<T, kN>(xt, ot, n_tokens, heads, head_dim, x_stride, out_stride, r, stream)
              : launch_rope_n<T, 1>(xt, ot, n_tokens, heads, head_dim, x_stride, out_stride, r, stream);
}

// ---------------------------------------------------------------- append --

constexpr int kAppThreads = 256;
constexpr int kAppHeads = kAppThreads / 32;   // (tensor, head) rows of a block, one warp each
constexpr int kStageBytes = 1088;             // one warp's rows: 16 x 68 or 8 x 136 bytes

// Eight consecutive elements, 16-byte aligned, as floats.
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  constexpr int kN = 16 / sizeof(T);
#pragma unroll
  for (int h = 0; h < 8 / kN; ++h) {
    const Vec<T, kN> v = *reinterpret_cast<const Vec<T, kN>*>(p + h * kN);
#pragma unroll
    for (int e = 0; e < kN; ++e) f[h * kN + e] = Elem<T>::get(v.e[e]);
  }
}

// A warp takes 32 / (D / 32) tokens of one head of K or V, a lane one block of
// 32 channels (lane = blocks * token + block).  The lane loads its block, and
// the block's partners of the half layout (another part of the same row, in L1
// or L2 by then), rotates in registers, quantises, and the warp's rows go
// through shared memory so that each row leaves as consecutive words.
// It waits most of the time (16,384 tokens, 32 x 64 fp16, interleaved, 61 us: issue slots 67 %
// busy, 43 % of the copy rate, long scoreboard the largest stall): every block forms the angles
// of its tokens anew for eight rows, behind two barriers.  The half layout in whole runs of eight took 36 us,
// with a test per channel 40 (16,384 tokens, 8 x 128 bf16, all channels turned).  Resident
// blocks an SM: five without rotation (65,536 tokens, 8 x 128 bf16: 79 us; with four 88), four
// with it.
// kRope: 0 none, 1 half, 2 interleaved.
template <typename T, int kD, int kRope>
__global__ void __launch_bounds__(kAppThreads, kRope ? 4 : 5)
append_kernel(const T* k, const T* v, int64_t n_tokens, int64_t k_stride,
              int64_t v_stride, const int64_t* slots, const RopeArgs r, const PagePool pool, uint32_t* status,
              int32_t row_tiles) {
  constexpr int kBlk = kD / 32;
  constexpr int kRow = kBlk * 34;
  constexpr int kTok = 32 / kBlk;
  static_assert(kTok * kRow == kStageBytes, "one warp's rows");
  __shared__ __align__(16) uint8_t stage[kAppHeads][kStageBytes];
  // (cos, sin) of (token, pair); a row of pairs + 1, so that the lanes of different tokens
  // read different banks
  __shared__ float2 cs[kRope ? kTok * (kD / 2 + 1) : 1];
  __shared__ uint64_t steps[kRope ? kD / 2 : 1];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) / row_tiles * kTok;
  const int first = static_cast<int>(blockIdx.x % row_tiles) * kAppHeads;   // of the block's 2 * kv_heads rows
  const int n_tok = static_cast<int>(i64min(kTok, n_tokens - t0));
  const int pairs = r.rot / 2;
  const int row = first + warp;
  const bool have = row < 2 * pool.kv_heads;
  const bool is_v = row >= pool.kv_heads;
  const int head = is_v ? row - pool.kv_heads : row;
  const int tok = lane / kBlk, bb = lane % kBlk;
  const bool valid = have && tok < n_tok;
  // the block's values are on their way while the angles are formed
  const T* src = nullptr;
  float x[32];
  if (valid) {
    src = (is_v ? v + (t0 + tok) * v_stride : k + (t0 + tok) * k_stride) + static_cast<int64_t>(head) * kD;
#pragma unroll
    for (int i = 0; i < 4; ++i) load8(src + 32 * bb + 8 * i, x + 8 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = 0.0f;
  }
  int64_t slot = -1;   // lane t < n_tok: token t's
  if (have && lane < n_tok) slot = slots[t0 + lane];
  if (kRope && first < pool.kv_heads) {   // uniform: the block has key heads
    for (int i = threadIdx.x; i < pairs; i += kAppThreads) steps[i] = turn_step(r.inv_freq[i]);
    __syncthreads();
    for (int i = threadIdx.x; i < n_tok * pairs; i += kAppThreads) {
      const int t = i / pairs;
      cs[i + t] = rotation(r.positions[t0 + t], steps[i - t * pairs], r.mscale, r.sign);
    }
    __syncthreads();
  }
  if (!have) return;
  if (valid) {
    if (kRope && !is_v) {
      const float2* turn = cs + tok * (pairs + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = 32 * bb + 8 * i;   // first of eight channels
        if (kRope == 2) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            if (c + e < r.rot) {
              const float2 q = turn[(c + e) / 2];
              const float2 y = turn_pair(x[8 * i + e], x[8 * i + e + 1], q);
              x[8 * i + e] = y.x;
              x[8 * i + e + 1] = y.y;
            }
          }
        } else if (c < r.rot && pairs % 8 == 0) {
          // the eight channels lie on one side and their partners are one 16-byte aligned run
          const bool low = c < pairs;
          float y[8];
          load8(src + (low ? c + pairs : c - pairs), y);
          const float2* q = turn + (low ? c : c - pairs);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            // low: a cos - b sin; high: b cos + a sin, the same rounding as attn_rope's
            x[8 * i + e] = low ? fmaf(x[8 * i + e], q[e].x, -y[e] * q[e].y) : fmaf(y[e], q[e].y, x[8 * i + e] * q[e].x);
          }
        } else if (c < r.rot) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (c + e < r.rot) {
              const bool low = c + e < pairs;
              const float2 q = turn[low ? c + e : c + e - pairs];
              const float y = Elem<T>::get(src[low ? c + e + pairs : c + e - pairs]);
              x[8 * i + e] = low ? fmaf(x[8 * i + e], q.x, -y * q.y) : fmaf(y, q.y, x[8 * i + e] * q.x);
            }
          }
        }
      }
    }
  }
  uint32_t w[8];
  const uint32_t d = q8_block(x, w);
  if (valid) q8_put_block(&stage[warp][tok * kRow], bb, d, w);
  // lane t < kTok knows where token t's row goes (-1: nowhere)
  int64_t at = -1;
  if (slot >= 0) {
    const int64_t page = slot >> pool.page_shift;
    if (page < pool.n_pages) {
      const int64_t off = slot & ((1ll << pool.page_shift) - 1);
      at = page * pool.page_stride + ((static_cast<int64_t>(head) << pool.page_shift) + off) * kRow;
    } else {
      record_index(status);
    }
  }
  __syncwarp();
  uint8_t* base = is_v ? pool.v : pool.k;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(stage[warp]);
  constexpr int kWords = kRow / 4;
  // A prompt's tokens mostly fill consecutive rows of a page: then the warp's rows are
  // one run of bytes (they end 16-byte aligned where they start so).
  const int64_t at0 = __shfl_sync(0xFFFFFFFFu, at, 0);
  if (__all_sync(0xFFFFFFFFu, lane >= n_tok || at == at0 + lane * kRow) && at0 >= 0) {
    uint8_t* dst = base + at0;
    const int n_words = n_tok * kWords;
    if ((at0 & 15) == 0 && n_tok == kTok) {
      for (int i = lane; i < kStageBytes / 16; i += 32)
        reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(words)[i];
    } else {
      for (int i = lane; i < n_words; i += 32) reinterpret_cast<uint32_t*>(dst)[i] = words[i];
    }
    return;
  }
#pragma unroll
  for (int i0 = 0; i0 < kTok * kWords; i0 += 32) {
    const int i = i0 + lane;
    const int t = i / kWords;   // warp-wide shuffle: every lane takes part
    const int64_t dst = __shfl_sync(0xFFFFFFFFu, at, t < kTok ? t : 0);
    if (i < kTok * kWords && dst >= 0) *reinterpret_cast<uint32_t*>(base + dst + 4 * (i - t * kWords)) = words[i];
  }
}

template <typename T, int kD>
cudaError_t launch_append_d(const void* k, const void* v, int64_t n_tokens, int64_t k_stride, int64_t v_stride,
                            const int64_t* slots, const RopeArgs& r, const PagePool& pool, uint32_t* status,
                            cudaStream_t stream) {
  constexpr int kTok = 32 / (kD / 32);
  const int64_t row_tiles = (2 * static_cast<int64_t>(pool.kv_heads) + kAppHeads - 1) / kAppHeads;
  const int64_t blocks = (n_tokens + kTok - 1) / kTok * row_tiles;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kernel = !r.inv_freq ? append_kernel<T, kD, 0>
                : r.interleaved ? append_kernel<T, kD, 2> : append_kernel<T, kD, 1>;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kAppThreads), 0, stream,
                       static_cast<const T*>(k), static_cast<const T*>(v), n_tokens, k_stride, v_stride, slots, r,
                       pool, status, static_cast<int32_t>(row_tiles));
}

template <typename T>
cudaError_t launch_append_t(const void* k, const void* v, int64_t n_tokens, int32_t head_dim, int64_t k_stride,
                            int64_t v_stride, const int64_t* slots, const RopeArgs& r, const PagePool& pool,
                            uint32_t* status, cudaStream_t stream) {
  return head_dim == 64
             ? launch_append_d<T, 64>(k, v, n_tokens, k_stride, v_stride, slots, r, pool, status, stream)
             : launch_append_d<T, 128>(k, v, n_tokens, k_stride, v_stride, slots, r, pool, status, stream);
}

// ------------------------------------------------------------------ read --

constexpr int kReadThreads = 256;
constexpr int kReadRows = 4;   // rows of a thread, in flight together

// A thread takes eight channels of a head row: eight codes (two words, or
// three where an even block's codes straddle words) and the block's scale, all
// from one or two 32-byte sectors that its neighbours read as well.
template <typename T, int kD>
__global__ void __launch_bounds__(kReadThreads)
read_kernel(T* k, T* v, int64_t n_rows, const int64_t* slots, const PagePool pool, uint32_t* status) {
  constexpr int kRow = kD / 32 * 34;
  constexpr int kPer = kD / 8;                     // threads of a row
  constexpr int kPass = kReadThreads / kPer;       // rows of a block and pass
  constexpr int kU = kReadRows;
  pdl_launch_dependents();
  pdl_wait();
  const int j = threadIdx.x % kPer;
  const int bb = j / 4;                            // block of 32 channels
  const int code0 = 34 * bb + 2 + 8 * (j % 4);     // first code's byte of the row
  const uint8_t* base = blockIdx.y ? pool.v : pool.k;
  T* out = blockIdx.y ? v : k;
  // row = token * kv_heads + head: one division for the thread's first row, the others
  // kPass further each
  const int64_t block0 = static_cast<int64_t>(blockIdx.x) * (kPass * kU);
  const int64_t row0 = block0 + threadIdx.x / kPer;
  const uint32_t heads = static_cast<uint32_t>(pool.kv_heads);
  int64_t t = block0 / pool.kv_heads;   // uniform
  uint32_t h = static_cast<uint32_t>(block0 - t * pool.kv_heads) + threadIdx.x / kPer;
  t += h / heads;
  h %= heads;
  const uint32_t dt = kPass / heads, dh = kPass % heads;
  int64_t slot[kU];
  uint32_t head[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    slot[u] = row0 + u * kPass < n_rows ? slots[t] : -1;
    head[u] = h;
    t += dt;
    h += dh;
    if (h >= heads) {
      h -= heads;
      ++t;
    }
  }
  const uint8_t* at[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    at[u] = nullptr;
    const int64_t page = slot[u] >> pool.page_shift;
    if (slot[u] >= 0 && page < pool.n_pages) {
      const uint32_t off = static_cast<uint32_t>(slot[u]) & ((1u << pool.page_shift) - 1);
      at[u] = base + page * pool.page_stride + ((static_cast<int64_t>(head[u]) << pool.page_shift) + off) * kRow;
    } else if (slot[u] >= 0) {
      record_index(status);
    }
  }
  uint32_t w[kU][3], d[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (at[u]) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(at[u] + (code0 & ~3));
      w[u][0] = p[0];
      w[u][1] = p[1];
      w[u][2] = (bb & 1) ? 0u : p[2];
      d[u] = *reinterpret_cast<const unsigned short*>(at[u] + 34 * bb);
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    if (!at[u]) continue;
    const uint32_t c0 = (bb & 1) ? w[u][0] : __funnelshift_r(w[u][0], w[u][1], 16);
    const uint32_t c1 = (bb & 1) ? w[u][1] : __funnelshift_r(w[u][1], w[u][2], 16);
    const float scale = __half2float(__ushort_as_half(static_cast<unsigned short>(d[u])));
    constexpr int kN = 16 / sizeof(T);
    T* dst = out + (row0 + u * kPass) * kD + 8 * j;
    T y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t word = e < 4 ? c0 : c1;
      y[e] = Elem<T>::put(static_cast<float>(static_cast<int8_t>(word >> (8 * (e & 3)))) * scale);
    }
#pragma unroll
    for (int h = 0; h < 8 / kN; ++h) {
      Vec<T, kN> o;
#pragma unroll
      for (int e = 0; e < kN; ++e) o.e[e] = y[h * kN + e];
      *reinterpret_cast<Vec<T, kN>*>(dst + h * kN) = o;
    }
  }
}

template <typename T>
cudaError_t launch_read_t(void* k, void* v, int64_t n_tokens, int32_t head_dim, const int64_t* slots,
                          const PagePool& pool, uint32_t* status, cudaStream_t stream) {
  const int64_t rows = n_tokens * pool.kv_heads;
  const int64_t per = kReadRows * (kReadThreads / (head_dim / 8));
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  auto kernel = head_dim == 64 ? read_kernel<T, 64> : read_kernel<T, 128>;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(blocks), 2), dim3(kReadThreads), 0, stream,
                       static_cast<T*>(k), static_cast<T*>(v), rows, slots, pool, status);
}

}  // namespace

cudaError_t launch_rope(const void* x, void* out, int32_t dtype, int64_t n_tokens, int32_t heads,
                        int32_t head_dim, int64_t x_stride, int64_t out_stride, const RopeArgs& r,
                        cudaStream_t stream) {
  if (dtype == kF16) return launch_rope_t<__half>(x, out, n_tokens, heads, head_dim, x_stride, out_stride, r, stream);
  if (dtype == kBF16)
    return launch_rope_t<__nv_bfloat16>(x, out, n_tokens, heads, head_dim, x_stride, out_stride, r, stream);
  return launch_rope_t<float>(x, out, n_tokens, heads, head_dim, x_stride, out_stride, r, stream);
}

cudaError_t launch_append(const void* k, const void* v, int32_t dtype, int64_t n_tokens, int32_t head_dim,
                          int64_t k_stride, int64_t v_stride, const int64_t* slots, const RopeArgs& r,
                          const PagePool& pool, uint32_t* status, cudaStream_t stream) {
  if (dtype == kF16)
    return launch_append_t<__half>(k, v, n_tokens, head_dim, k_stride, v_stride, slots, r, pool, status, stream);
  if (dtype == kBF16)
    return launch_append_t<__nv_bfloat16>(k, v, n_tokens, head_dim, k_stride, v_stride, slots, r, pool, status, stream);
  return launch_append_t<float>(k, v, n_tokens, head_dim, k_stride, v_stride, slots, r, pool, status, stream);
}

cudaError_t launch_read(void* k, void* v, int32_t dtype, int64_t n_tokens, int32_t head_dim,
                        const int64_t* slots, const PagePool& pool, uint32_t* status, cudaStream_t stream) {
  if (dtype == kF16) return launch_read_t<__half>(k, v, n_tokens, head_dim, slots, pool, status, stream);
  if (dtype == kBF16) return launch_read_t<__nv_bfloat16>(k, v, n_tokens, head_dim, slots, pool, status, stream);
  return launch_read_t<float>(k, v, n_tokens, head_dim, slots, pool, status, stream);
}

}  // namespace q8a
