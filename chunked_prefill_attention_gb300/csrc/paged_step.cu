// paged_step.cu -- what a step of a server does around its attention: lengths, block tables and slots of its new
// tokens, and the norms of its queries and keys with their rotary positions.

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.h"
#include "paged_seq.cuh"
#include "ptx.cuh"
#include "rotary.cuh"

namespace q8a {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// ---------------------------------------------------------------- extend --
//
// Sequence b gets new_lens[b] tokens behind its kv_lens[b] keys.  With P tokens a page it needs
//   ceil((kv + n) / P) - ceil(kv / P)
// more pages; the sums of the rows and of the pages before b (two exclusive scans) say where its rows start
// and which of the free pages are its own, so nothing depends on the order in which blocks run.  The pages' scan counts what
// refused sequences lack too, so that a sequence's pages suffice if all before it had theirs as well: pages go to the first ones, and
// nobody overtakes a sequence that waits for more than are left.  A new page's first row is a new token's, and that token's
// thread writes the page's number into the table.
//
// A step's work is a few kilobytes: latency bounds it.  Every block scans the lengths itself, so no block waits
// for another's results.  Many tokens are dealt to blocks, the first of which writes the lengths and the number of free
// pages too (kWhole); but where these lie in the place of those that the other blocks read, a second
// launch does that (kTokens, then kLens).  On the device: 64 sequences, a token each, 2.4 us (with 1,024 threads instead of
// 256 5.7); 1,000 sequences, 8,500 rows, 6.8; 48 prompts, 197,000 tokens, 6.8 (in place 10.9; one cluster of
// eight blocks 36).

constexpr int kExtThreads = 1024;
enum : int { kWhole, kTokens, kLens };

template <int kPart>
__global__ void __launch_bounds__(kExtThreads, 1) extend_kernel(const ExtendArgs a) {
  __shared__ int64_t sums[2][32];
  __shared__ int32_t row0[kExtThreads], kv0[kExtThreads], page0[kExtThreads];
  __shared__ int32_t taken;
  pdl_launch_dependents();
  pdl_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
  const bool lead = blockIdx.x == 0;
  const int64_t page = int64_t{1} << a.page_shift;
  const int64_t most = i64min(a.table_stride << a.page_shift, kMaxKeys);
  const int64_t n_raw = a.n_free[0];
  const int64_t n_free = i64max(0, i64min(n_raw, a.free_capacity));
  bool wrong = n_raw != n_free;
  int64_t rows = 0, pages = 0;   // of the sequences before this round's
  const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + tid, stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  if (tid == 0) taken = 0;
  if (kPart != kLens && lead && tid == 0) a.cu_q[0] = 0;
  for (int64_t b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int64_t b = b0 + tid;
    const bool have = b < a.batch;
    const int64_t n_in = have ? a.new_lens[b] : 0, kv = have ? a.kv_lens[b] : 0;
    const int64_t n = i64max(n_in, 0);
    const bool valid = n_in >= 0 && kv >= 0 && kv + n <= most;
    const int64_t had = (kv + page - 1) >> a.page_shift;
    const int64_t need = valid ? ((kv + n + page - 1) >> a.page_shift) - had : 0;
    int64_t r = n, p = need;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(kFull, r, o), w = __shfl_up_sync(kFull, p, o);
      if (lane >= o) {
        r += v;
        p += w;
      }
    }
    if (lane == 31) {
      sums[0][warp] = r;
      sums[1][warp] = p;
    }
    __syncthreads();
    int64_t all_r = rows, all_p = pages;
    r += rows;
    p += pages;
    for (int w = 0; w < warps; ++w) {
      const int64_t x = sums[0][w], y = sums[1][w];
      if (w < warp) {
        r += x;
        p += y;
      }
      all_r += x;
      all_p += y;
    }
    const bool granted = valid && (need == 0 || p <= n_free) && (n == 0 || r <= a.total_q);
    if (have && !granted) wrong = true;
    if (have && granted && need > 0) atomicMax(&taken, static_cast<int32_t>(p));   // the granted ones come first
    const int64_t start = i64min(r - n, a.total_q);
    row0[tid] = static_cast<int32_t>(have ? start : a.total_q);
    kv0[tid] = granted ? static_cast<int32_t>(kv) : -1;
    page0[tid] = static_cast<int32_t>(p - need - had);   // page i of the sequence is the free one page0 + i
    if (kPart != kLens && lead && have) a.cu_q[b + 1] = static_cast<int32_t>(i64min(r, a.total_q));
    __syncthreads();
    if (kPart != kTokens && lead && have) a.kv_out[b] = static_cast<int32_t>(granted ? kv + n : kv);
    const int64_t end = i64min(all_r, a.total_q);
    int half = 1;   // of the search: the sequences of this round are at most 2 * half
    while (2 * half < i64min(a.batch - b0, blockDim.x)) half *= 2;
    for (int64_t t = i64min(rows, a.total_q) + first; kPart != kLens && t < end; t += stride) {
      int lo = 0;   // the last sequence that starts at or before t: of those that start there, the one with rows
      for (int step = half; step > 0; step /= 2)
        if (row0[lo + step] <= t) lo += step;
      int64_t slot = -1, pos = 0;
      if (kv0[lo] >= 0) {
        pos = kv0[lo] + (t - row0[lo]);
        const int64_t i = pos >> a.page_shift, off = pos & (page - 1);
        int32_t* entry = a.table + (b0 + lo) * a.table_stride + i;
        int32_t at;
        if (i >= (kv0[lo] + page - 1) >> a.page_shift) {
          at = a.free_pages[n_free - 1 - (page0[lo] + i)];
          if (off == 0) *entry = at;
        } else {
          at = *entry;
        }
        if (at >= 0)
          slot = (static_cast<int64_t>(at) << a.page_shift) + off;
        else
          wrong = true;
      }
      a.slots[t] = slot;
      a.positions[t] = pos;
    }
    rows = all_r;
    pages = all_p;
    __syncthreads();   // the tables of this round are used no more
  }
  for (int64_t t = i64min(rows, a.total_q) + first; kPart != kLens && t < a.total_q; t += stride) {
    a.slots[t] = -1;
    a.positions[t] = 0;
  }
  if (a.batch == 0) __syncthreads();
  if (kPart != kTokens && lead && tid == 0) a.n_free_out[0] = static_cast<int32_t>(n_free - taken);
  if (wrong) record_index(a.status);
}

// ------------------------------------------------------------- norm, rope --
//
// A head row x of D channels becomes
//   y = x / sqrt(mean(x^2) + eps) * w,   then its channel pairs (a, b) -> (a cos t - b sin t, a sin t + b cos t),
// t = position * f, the position that of the pair's axis; everything in fp32, rounded once.

// A warp per token and run of heads, pairs (lane, lane + 32) of each row: any rotated width, any alignment.
template <typename T, int kD>
__global__ void __launch_bounds__(256) norm_rope_any_kernel(const NormRopeArgs a, int32_t heads_per_warp) {
  constexpr int kP = kD / 64;   // pairs of a lane
  __shared__ float weight[2][kD];
  __shared__ uint64_t steps[kD / 2];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int pairs = a.rot / 2;
  for (int i = threadIdx.x; i < 2 * kD; i += blockDim.x) {
    const void* w = a.weight[i / kD];
    const int c = i % kD;
    weight[i / kD][c] = !w ? 1.0f
                        : a.weight_dtype == kF16  ? __half2float(static_cast<const __half*>(w)[c])
                        : a.weight_dtype == kBF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[c])
                                                  : static_cast<const float*>(w)[c];
  }
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) steps[i] = turn_step(a.inv_freq[i]);
  __syncthreads();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + warp;
  if (t >= a.n_tokens) return;
  float2 cs[kP];
  int c0[kP], c1[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) {
    const int p = lane + 32 * i;
    cs[i] = make_float2(1.0f, 0.0f);
    c0[i] = 2 * p;
    c1[i] = 2 * p + 1;
    if (p < pairs) {
      int axis = a.axes ? a.axes[p] : 0;
      if (axis < 0 || axis >= a.n_axes) {
        record_index(a.status);
        axis = 0;
      }
      cs[i] = rotation(a.positions[axis * a.n_tokens + t], steps[p], a.mscale, 1.0f);
      if (!a.interleaved) {
        c0[i] = p;
        c1[i] = p + pairs;
      }
    }
  }
  const int h0 = blockIdx.y * heads_per_warp, h1 = min(a.heads[0] + a.heads[1], h0 + heads_per_warp);
  for (int h = h0; h < h1; ++h) {
    const int which = h >= a.heads[0];
    const int head = which ? h - a.heads[0] : h;
    const T* x = static_cast<const T*>(a.x[which]) + t * a.x_stride[which] + static_cast<int64_t>(head) * kD;
    T* y = static_cast<T*>(a.out[which]) + t * a.out_stride[which] + static_cast<int64_t>(head) * kD;
    float u[kP], v[kP], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      u[i] = Elem<T>::get(x[c0[i]]);
      v[i] = Elem<T>::get(x[c1[i]]);
      ss = fmaf(u[i], u[i], fmaf(v[i], v[i], ss));
    }
#pragma unroll
    for (int o = 1; o < 32; o *= 2) ss += __shfl_xor_sync(kFull, ss, o);
    const float r = a.weight[which] ? rsqrtf(fmaf(ss, 1.0f / kD, a.eps)) : 1.0f;
#pragma unroll
    for (int i = 0; i < kP; ++i) {
      const float p = u[i] * r * weight[which][c0[i]], q = v[i] * r * weight[which][c1[i]];
      const float2 z = turn_pair(p, q, cs[i]);
      const bool turns = lane + 32 * i < pairs;   // the other channels keep their value, whatever it is
      y[c0[i]] = Elem<T>::put(turns ? z.x : p);
      y[c1[i]] = Elem<T>::put(turns ? z.y : q);
    }
  }
}

// Eight halves or four floats of one 16-byte access as floats, and back (one rounding).
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float* f);
template <>
__device__ __forceinline__ void unpack<float>(const uint4& v, float* f) {
  f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
}
template <>
__device__ __forceinline__ void unpack<__half>(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    f[2 * i] = x.x, f[2 * i + 1] = x.y;
  }
}
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(w[i] << 16), f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float* f);
template <>
__device__ __forceinline__ uint4 pack<float>(const float* f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack<__half>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack<__nv_bfloat16>(const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The same with 16-byte accesses: a head row is 2 L vectors of N elements, L lanes each take two.  Of the turned
// channels in halves a lane's vectors are each other's partners; in interleaved pairs every vector holds whole ones.
// A thread keeps to one token, its two vectors and the heads of one tensor (a block's), so its angles are formed
// once, and with them the weights: a pair becomes r (a A - b B), r (a C + b E), r the row's factor, with
//   A = w_a cos t, B = w_b sin t, C = w_a sin t, E = w_b cos t
// in registers.  HBM bounds it: 16,384 tokens, 32 + 8 heads x 128 bf16, all channels turned in halves, 54 us, 91 % of the
// copy rate; three axes, interleaved, 9,001 tokens, 24 + 24 x 64 fp16, 17 us, 95 %.  Folding the weights into the angles and
// keeping to one tensor a block took the first from 113 to 57 us (the issue slots were 57 % busy), four heads in
// flight instead of two to 54 (with three blocks an SM and two heads 57, one 65).
template <typename T, int kD, bool kInter>
__global__ void __launch_bounds__(256, 2)
norm_rope_kernel(const NormRopeArgs a, int32_t heads_per_thread, int32_t q_groups) {
  constexpr int N = 16 / sizeof(T), L = kD / (2 * N);
  constexpr int kU = 4;   // heads in flight
  __shared__ uint64_t steps[kD / 2];
  __shared__ int32_t axis_of[kD / 2];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x % L;
  const int pairs = a.rot / 2;
  const int which = static_cast<int>(blockIdx.y) >= q_groups;
  const int h0 = (blockIdx.y - (which ? q_groups : 0)) * heads_per_thread;
  const int n = min(a.heads[which] - h0, heads_per_thread);
  const int64_t t_own = static_cast<int64_t>(blockIdx.x) * (blockDim.x / L) + threadIdx.x / L;
  const bool live = t_own < a.n_tokens;
  const int64_t t = live ? t_own : a.n_tokens - 1;   // the lanes behind the last token read it too, and write nothing
  int c0, c1;
  bool turn0, turn1;
  if (kInter) {
    c0 = N * lane;
    c1 = kD / 2 + N * lane;
    turn0 = c0 < a.rot;
    turn1 = c1 < a.rot;
  } else {
    const int turning = pairs / N;
    turn0 = turn1 = lane < turning;
    c0 = turn0 ? N * lane : a.rot + N * (lane - turning);
    c1 = c0 + (turn0 ? pairs : (kD - a.rot) / 2);
  }
  const T* x = static_cast<const T*>(a.x[which]) + t * a.x_stride[which] + static_cast<int64_t>(h0) * kD;
  T* y = static_cast<T*>(a.out[which]) + t * a.out_stride[which] + static_cast<int64_t>(h0) * kD;
  uint4 x0[kU], x1[kU];
  auto load = [&](int h) {
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (h + u < n) {
        x0[u] = *reinterpret_cast<const uint4*>(x + u * kD + c0);
        x1[u] = *reinterpret_cast<const uint4*>(x + u * kD + c1);
      }
    x += kU * kD;
  };
  load(0);
  for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
    steps[i] = turn_step(a.inv_freq[i]);
    int axis = a.axes ? a.axes[i] : 0;
    if (axis < 0 || axis >= a.n_axes) {
      record_index(a.status);
      axis = 0;
    }
    axis_of[i] = axis;
  }
  __syncthreads();
  const void* weight = a.weight[which];
  float wa[N], wb[N];   // of the two vectors; A and E of the pairs in their place later
  float B[N], C[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    auto get = [&](int c) {
      return !weight                     ? 1.0f
             : a.weight_dtype == kF16    ? __half2float(static_cast<const __half*>(weight)[c])
             : a.weight_dtype == kBF16   ? __bfloat162float(static_cast<const __nv_bfloat16*>(weight)[c])
                                         : static_cast<const float*>(weight)[c];
    };
    wa[e] = get(c0 + e);
    wb[e] = get(c1 + e);
    B[e] = C[e] = 0.0f;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    // pair e: (first vector, second vector) at e; interleaved: 2 e and 2 e + 1 of the first vector, then of the second
    const bool turns = kInter && e >= N / 2 ? turn1 : turn0;
    const int p = kInter ? (e < N / 2 ? c0 / 2 + e : c1 / 2 + e - N / 2) : c0 + e;
    if (turns) {
      const float2 cs = rotation(a.positions[axis_of[p] * a.n_tokens + t], steps[p], a.mscale, 1.0f);
      float& fa = kInter ? (e < N / 2 ? wa[2 * e] : wb[2 * e - N]) : wa[e];
      float& fb = kInter ? (e < N / 2 ? wa[2 * e + 1] : wb[2 * e + 1 - N]) : wb[e];
      B[e] = fb * cs.y;
      C[e] = fa * cs.y;
      fa *= cs.x;
      fb *= cs.x;
    }
  }
  for (int h = 0; h < n; h += kU) {
    uint4 y0[kU], y1[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      y0[u] = x0[u];
      y1[u] = x1[u];
    }
    load(h + kU);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (h + u >= n) break;   // uniform
      float p[N], q[N];
      unpack<T>(y0[u], p);
      unpack<T>(y1[u], q);
      if (weight) {   // uniform
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          s0 = fmaf(p[e], p[e], s0);
          s1 = fmaf(q[e], q[e], s1);
        }
        s0 += s1;
#pragma unroll
        for (int o = 1; o < L; o *= 2) s0 += __shfl_xor_sync(kFull, s0, o);
        const float r = rsqrtf(fmaf(s0, 1.0f / kD, a.eps));
#pragma unroll
        for (int e = 0; e < N; ++e) {
          p[e] *= r;
          q[e] *= r;
        }
      }
      if (kInter) {
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
          const float a0 = p[2 * e], b0 = p[2 * e + 1], a1 = q[2 * e], b1 = q[2 * e + 1];
          p[2 * e] = a0 * wa[2 * e];
          p[2 * e + 1] = b0 * wa[2 * e + 1];
          q[2 * e] = a1 * wb[2 * e];
          q[2 * e + 1] = b1 * wb[2 * e + 1];
          if (turn0) {   // a channel that is not turned takes nothing from its neighbour, not even 0 times infinity
            p[2 * e] = fmaf(a0, wa[2 * e], -b0 * B[e]);
            p[2 * e + 1] = fmaf(a0, C[e], p[2 * e + 1]);
          }
          if (turn1) {
            q[2 * e] = fmaf(a1, wb[2 * e], -b1 * B[N / 2 + e]);
            q[2 * e + 1] = fmaf(a1, C[N / 2 + e], q[2 * e + 1]);
          }
        }
      } else if (turn0) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float a0 = p[e], b0 = q[e];
          p[e] = fmaf(a0, wa[e], -b0 * B[e]);
          q[e] = fmaf(a0, C[e], b0 * wb[e]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          p[e] *= wa[e];
          q[e] *= wb[e];
        }
      }
      if (live) {
        *reinterpret_cast<uint4*>(y + u * kD + c0) = pack<T>(p);
        *reinterpret_cast<uint4*>(y + u * kD + c1) = pack<T>(q);
      }
    }
    y += kU * kD;
  }
}

template <typename T, int kD>
cudaError_t launch_norm_rope_d(const NormRopeArgs& a, cudaStream_t stream) {
  const int heads = a.heads[0] + a.heads[1];
  // 16-byte accesses where a vector lies in one half of the turned channels and every row starts 16-byte aligned
  constexpr int N = 16 / sizeof(T), L = kD / (2 * N);
  bool wide = a.rot % (2 * N) == 0;
  for (int i = 0; i < (a.heads[1] ? 2 : 1); ++i)
    wide = wide && (a.x_stride[i] | a.out_stride[i]) % N == 0 &&
           (reinterpret_cast<uintptr_t>(a.x[i]) | reinterpret_cast<uintptr_t>(a.out[i])) % 16 == 0;
  if (wide) {
    // The fewest heads a thread with which the blocks are one wave, two an SM: every block starts with its
    // angles, and a few blocks beyond a wave cost another.  32 + 8 heads x 128 bf16, us with 1, 2, 3, 5, 8, 12, 16, 24, 32:
    //   256 tokens 6.3 4.8 4.8 4.4 5.1 6.1 7.1 9.2 11; 512: 9.1 6.9 5.3 5.6 5.8 6.2 7.2 9.1 11; 1,024: 14 9.8 7.7 6.1 6.9 7.9 8.7 11 11;
    //   2,048: 26 16 12 10 10 8.5 9.8 12 15; 4,096: 48 29 22 18 15 14 14 13 16; 16,384: 181 106 82 67 56 55 55 55 55
    // More than 16 only where the wave is full of rows, too (9,001 tokens, 24 + 24 x 64: 19 with 16, 17 with 24); else
    // 16, or 32 for many waves.
    constexpr int64_t kWave = 2 * kSms;
    auto groups_of = [&](int hpt) { return (a.heads[0] + hpt - 1) / hpt + (a.heads[1] + hpt - 1) / hpt; };
    const int64_t blocks = (a.n_tokens + 256 / L - 1) / (256 / L);
    int hpt = 1;
    while (hpt < 32 && blocks * groups_of(hpt) > kWave) ++hpt;
    if (blocks * groups_of(hpt) > kWave || (hpt > 16 && blocks * heads * 10 < kWave * hpt * 7))
      hpt = blocks * groups_of(32) > 2 * kWave ? 32 : 16;
    const int64_t groups = groups_of(hpt);
    if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
    return launch_kernel(a.interleaved ? norm_rope_kernel<T, kD, true> : norm_rope_kernel<T, kD, false>,
                         dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(groups)), dim3(256), 0, stream, a,
                         static_cast<int32_t>(hpt), static_cast<int32_t>((a.heads[0] + hpt - 1) / hpt));
  }
  constexpr int64_t kFill = kSms * 64;   // warps
  int hpw = 16;
  while (hpw > 2 && a.n_tokens * ((heads + hpw - 1) / hpw) < kFill) hpw /= 2;   // 2: at most 65,535 groups
  const int64_t blocks = (a.n_tokens + 7) / 8, groups = (heads + hpw - 1) / hpw;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  return launch_kernel(norm_rope_any_kernel<T, kD>, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(groups)),
                       dim3(256), 0, stream, a, static_cast<int32_t>(hpw));
}
template <typename T>
cudaError_t launch_norm_rope_t(const NormRopeArgs& a, int32_t head_dim, cudaStream_t stream) {
  return head_dim == 64 ? launch_norm_rope_d<T, 64>(a, stream) : launch_norm_rope_d<T, 128>(a, stream);
}

}  // namespace

cudaError_t launch_extend(const ExtendArgs& a, cudaStream_t stream) {
  if (a.total_q <= 4096)
    return launch_kernel(extend_kernel<kWhole>, dim3(1), dim3(a.batch <= 256 && a.total_q <= 1024 ? 256 : kExtThreads), 0, stream, a);
  const int64_t most = (a.total_q + kExtThreads - 1) / kExtThreads, blocks = most < kSms ? most : kSms;
  if (a.kv_out != a.kv_lens && a.n_free_out != a.n_free)
    return launch_kernel(extend_kernel<kWhole>, dim3(static_cast<unsigned>(blocks)), dim3(kExtThreads), 0, stream, a);
  const cudaError_t e = launch_kernel(extend_kernel<kTokens>, dim3(static_cast<unsigned>(blocks)), dim3(kExtThreads), 0, stream, a);
  return e != cudaSuccess ? e : launch_kernel(extend_kernel<kLens>, dim3(1), dim3(kExtThreads), 0, stream, a);
}

cudaError_t launch_norm_rope(const NormRopeArgs& a, int32_t dtype, int32_t head_dim, cudaStream_t stream) {
  if (dtype == kF16) return launch_norm_rope_t<__half>(a, head_dim, stream);
  if (dtype == kBF16) return launch_norm_rope_t<__nv_bfloat16>(a, head_dim, stream);
  return launch_norm_rope_t<float>(a, head_dim, stream);
}

}  // namespace q8a
