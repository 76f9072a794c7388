// paged_few.cu -- attention of few query rows per K/V head over a paged Q8_0
// cache: single tokens, bursts, short tails of prompts.
//
//   out_i = sum_j e^(S_ij - m_i) V_j / sum_j e^(S_ij - m_i),  S_ij = scale Q_i.K_j
// with K_j = d c and V_j = d c per block of 32 channels (Q8_0) and the key j
// visible when j < kv_len and, causal, j <= kv_len - n_q + token(i).
//
// What bounds it: HBM.  Each key and head is 2 * 34 * D / 32 bytes for at most
// 16 rows (token, query head of the group), so the arithmetic has to stay under
// one SM's share of the memory rate (about 23 bytes a cycle): 5.8 cycles per key
// and head at D = 64.
//
// Products.  mma.sync m16n8k16 with the keys (or channels) on the side of 16
// and the query rows on the side of 8, so that one row wastes the least:
//   S^T = K Q^T  (A = codes of 16 keys x 16 channels, B = Q^T),
//   O^T = V^T P^T  (A = codes of 16 channels x 16 keys, B = P^T).
// The codes enter as fp16, exactly; the block scales d are applied in fp32 to
// the block's partial scores, and for V they are folded into the weights before
// those are rounded to fp16 (one rounding a weight, 2^-11 relative): the codes
// of both tensors are never scaled in memory or rounded.  bf16 queries enter as
// fp16 after scaling a row by a power of two (its largest value to [2^14,
// 2^15)), which keeps their 8 bits down to 2^-31 of that value (fp16's smallest
// step is 2^-24).
// (tcgen05 wants 64 or 128 rows and fp16 operands in shared memory: the codes
// would have to be converted and stored at more than twice their bytes, for
// at most 16 useful rows.)
//
// Layout.  The order of keys inside a tile and of channels inside a block is
// free as long as both operands agree, and is chosen so that every shared
// memory load is one aligned word of four codes of one row and the 32 lanes of
// a load touch 32 banks, although rows are 68 or 136 bytes: lane (g, t) = (lane
// / 4, lane % 4) takes key S g + j for the scores and keys 2 S t + j for the
// values, S = 4 (D = 64) or 2 (D = 128) keys of a group.  An even block's codes
// straddle words by two bytes: the word left over is made of the row's first
// and ninth words.  The weights come from the score fragments by one 8 x 8
// transposition in registers (movmatrix).
//
// Work.  All key tiles of all (sequence, K/V head, row tile) units are laid end
// to end and cut into equal shares, one per warp (16 warps per SM), so ragged
// batches and single long sequences both fill the machine.  A warp works alone:
// its own ring of asynchronous copies (page rows are contiguous: one copy per page
// and tensor), its own running softmax, no barrier with other warps, so the start
// and end of a unit in one warp hide behind the others' tiles (64 sequences of 256
// to 16,384 keys, 8 heads x 64: 157 us with shares and barriers of whole CTAs, 127 us
// so).  A unit cut between warps leaves partial states, which a second kernel joins
// in order: no atomics, the same result every time.  Where a CTA's eight shares all
// lie in one unit, the CTA joins them first, which leaves an eighth of the parts.

#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged.h"
#include "paged_seq.cuh"
#include "ptx.cuh"
#include "q8_codes.cuh"

namespace q8a {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 320;      // two per SM of 160 SMs
constexpr int kMaxWarps = kMaxCtas * kWarps;
constexpr int kMinShare = 2;       // tiles of a warp's share
constexpr int kDescInts = 8;       // join record of a share boundary
constexpr float kLazy = 8.0f;      // the reference moves when exceeded by more than 2^8
// Powers of two of V's scales: of subnormal ones (below 2^-14), and of 65504 and beyond.
constexpr float kMostUp = 2097152.0f, kLeastUp = 1.0f / 1024.0f;
constexpr uint32_t kFull = 0xFFFFFFFFu;

template <int D, int NT>
struct Shape {
  static constexpr int S = 256 / D;              // keys of a lane group and tile
  static constexpr int KT = 8 * S;               // keys of a tile: 32 or 16
  static constexpr int P = D / 64;               // pairs of Q8_0 blocks
  static constexpr int RW = 17 * P;              // words of a row
  static constexpr int TILE = KT * RW * 4;       // bytes of a tensor's tile: 2176
  static constexpr int STAGE = 2 * TILE;
  // 16 rows of 128 channels: Q^T's fragments stay in shared memory and take a stage of the ring
  // (16 sequences of 32,768 keys: 334 us with them in registers, 275 so).  O's registers and the
  // weights still spill: 180 bytes of stores and 392 of loads a thread (16 rows of 64 channels:
  // 72 and 192; 8 rows of 128: 24 and 56).
  static constexpr bool QS = NT * D >= 256;
  static constexpr int STAGES = QS ? 2 : 3;
  static constexpr int RING = kWarps * STAGES * STAGE;
  static constexpr int QBYTES = QS ? P * 4 * NT * 32 * 8 : 0;   // of a warp
  static constexpr int SMEM = RING + kWarps * QBYTES;
};

template <int D, int NT>
struct Part {
  static constexpr int R = 8 * NT;               // rows of a tile
  static constexpr int NREG = D / 16 * NT * 4;   // O registers of a lane
  static constexpr int FLOATS = NREG * 32 + 2 * R;
};

// Bounded waits of a warp on its own copies.  A wait that runs out is recorded;
// the warp then starts no further copy and waits (again bounded) only for those
// it has started, so that it never leaves one in flight.
struct Waiter {
  uint64_t budget;   // cycles
  uint32_t* status;
  bool bad;
  __device__ __forceinline__ void wait(uint32_t bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return;
    const long long t0 = clock64();
    while (!__all_sync(kFull, mbar_try_wait_sleep(bar, parity, 100000u))) {
      const int out = static_cast<uint64_t>(clock64() - t0) > budget;
      if (__any_sync(kFull, out)) {
        bad = true;
        if ((threadIdx.x & 31) == 0) record_timeout(status);
        return;
      }
    }
  }
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 x 8 transposition of 16-bit values held two to a lane (lane 4 r + c: row r,
// columns 2 c and 2 c + 1).
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  __half2 l, h;
  q8a::codes_to_half2(w, l, h);
  lo = h2u(l);
  hi = h2u(h);
}

__device__ __forceinline__ float half_bits(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
}
// Weight of a partial state with reference m under the joint reference top.
__device__ __forceinline__ float join_weight(float m, float top) {
  return m == -INFINITY ? 0.0f : (m == top ? 1.0f : ex2_approx(m - top));
}

template <int D, int NT>
struct Units {
  int32_t tiles;   // key tiles of one unit (at least 1, so that a row without keys is written)
  int32_t row_tiles;
  int64_t all;     // tiles of the sequence's units
};
template <int D, int NT>
__device__ __forceinline__ Units<D, NT> units_of(const PagedArgs& a, const Seq& s) {
  Units<D, NT> u;
  const int64_t rows = static_cast<int64_t>(s.n_q) * a.group;
  u.tiles = max(1, (s.kv + Shape<D, NT>::KT - 1) / Shape<D, NT>::KT);
  u.row_tiles = rows > a.row_limit ? 0 : static_cast<int32_t>((rows + 8 * NT - 1) / (8 * NT));
  u.all = static_cast<int64_t>(u.tiles) * u.row_tiles * a.kv_heads;
  return u;
}

__device__ __forceinline__ int64_t warp_inclusive(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int64_t n = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Two channels of a row of out: those of m-tile i of O^T, which lane group g holds (codes
// 2 (i & 1) .. of its word of the block).
template <typename QT, int D>
__device__ __forceinline__ void store_pair(const PagedArgs& a, const Seq& sq, int kvh, int row, int i, int g, float y0,
                                           float y1) {
  const bool odd = i & 2;
  int c = 64 * (i / 4) + (odd ? 32 : 2) + 4 * g + 2 * (i & 1);
  if (!odd && g == 7 && (i & 1)) c -= 32;   // the word made of a row's first and ninth words
  const int tok = row / a.group;
  QT* op = static_cast<QT*>(a.out) + ((sq.q0 + tok) * a.heads + kvh * a.group + row - tok * a.group) * D + c;
  if (std::is_same<QT, __half>::value) {
    *reinterpret_cast<uint32_t*>(op) = pack_half2(y0, y1);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(y0, y1);
    *reinterpret_cast<uint32_t*>(op) = *reinterpret_cast<const uint32_t*>(&v);
  }
}

// kDirect: a CTA per unit, its tiles dealt to the eight warps, nothing left to join.
template <typename QT, int D, int NT, bool kDirect>
__global__ void __launch_bounds__(kThreads, 2)
paged_few_kernel(const PagedArgs a) {
  using Sh = Shape<D, NT>;
  using Pt = Part<D, NT>;
  constexpr int kStages = Sh::STAGES;
  constexpr int S = Sh::S, KT = Sh::KT, RW = Sh::RW, P = Sh::P, R = Pt::R, NREG = Pt::NREG;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[kWarps * kStages];
  __shared__ __align__(16) float v_ups[kWarps][D / 32];
  __shared__ int64_t sums[kDirect ? 1 : kWarps], found[kDirect ? 1 : kWarps][2];
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  if (lane == 0)
    for (int s = 0; s < kStages; ++s) mbar_init(smem_u32(&bars[warp * kStages + s]), 1);
  fence_mbar_init();
  pdl_wait();

  // ---- this warp's share of all key tiles: [pos, end) of the tiles laid end to end
  int64_t total, share, gw, pos0, pos, end, cta_end, base = 0;
  int b;
  bool inner;   // one unit holds all of the CTA's tiles
  int32_t* desc = nullptr;
  float* parts = a.part + kMaxWarps * kDescInts;
  if (kDirect) {
    // tiles of this unit alone; a sequence has one row tile
    b = blockIdx.x / a.kv_heads;
    const auto un = units_of<D, NT>(a, read_seq(a, b));
    if (un.row_tiles == 0) return;   // uniform
    total = cta_end = un.tiles;
    share = (un.tiles + kWarps - 1) / kWarps;
    gw = pos0 = 0;
    pos = warp * share;
    end = i64min(total, pos + share);
    inner = true;
  } else {
    int64_t mine = 0;
    for (int i = tid; i < a.batch; i += kThreads) mine += units_of<D, NT>(a, read_seq(a, i)).all;
    const int64_t inc = warp_inclusive(mine, lane);
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += sums[w];
    const int64_t shares = static_cast<int64_t>(gridDim.x) * kWarps;
    share = i64max(kMinShare, (total + shares - 1) / shares);
    gw = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    desc = reinterpret_cast<int32_t*>(a.part) + gw * kDescInts;
    if (lane == 0) desc[0] = -1;   // nothing to join at this boundary, until found otherwise
    pos0 = blockIdx.x * (kWarps * share);
    if (pos0 >= total) return;     // uniform over the CTA
    // the sequence that holds each warp's first tile
    for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
      __syncthreads();
      const int b = b0 + tid;
      const int64_t v = b < a.batch ? units_of<D, NT>(a, read_seq(a, b)).all : 0;
      const int64_t i = warp_inclusive(v, lane);
      if (lane == 31) sums[warp] = i;
      __syncthreads();
      int64_t before = base + i - v;
      for (int w = 0; w < warp; ++w) before += sums[w];
      for (int w = 0; w < kWarps; ++w) {
        const int64_t p = pos0 + w * share;
        if (p >= before && p < before + v) {
          found[w][0] = b;
          found[w][1] = before;
        }
      }
      for (int w = 0; w < kWarps; ++w) base += sums[w];
      if (base > pos0 + (kWarps - 1) * share) break;   // uniform: every warp's tile is found
    }
    __syncthreads();
    pos = pos0 + warp * share;
    end = i64min(total, pos + share);
    cta_end = i64min(total, pos0 + kWarps * share);
    {
      const int b0 = static_cast<int>(found[0][0]);
      const int64_t tiles = units_of<D, NT>(a, read_seq(a, b0)).tiles;
      const int64_t last = (cta_end - 1 - pos0) / share;
      inner = found[last][0] == b0 && (pos0 - found[0][1]) / tiles == (cta_end - 1 - found[0][1]) / tiles;
    }
    if (!inner && pos >= end) return;   // no barrier from here on, unless inner
    b = static_cast<int>(found[inner ? 0 : warp][0]);
    base = found[inner ? 0 : warp][1];
  }

  uint8_t* ring = smem + warp * (kStages * Sh::STAGE);
  const uint32_t ring_u = smem_u32(ring), bar_u = smem_u32(&bars[warp * kStages]);
  Waiter waiter{2 * a.timeout_ns, a.status, false};
  uint32_t it = 0;   // tiles this warp has taken: stage and parity of the ring
  const uint32_t sel_k = t == 3 ? 0x7610u : 0x3210u, sel_v = g == 7 ? 0x7610u : 0x3210u;
  // pieces of a tile: one, or (pages of 16, D = 64) two pages' worth
  const int piece_shift = min(a.page_shift, D == 64 ? 5 : 4);
  const int pieces = KT >> piece_shift;
  const uint32_t piece_bytes = static_cast<uint32_t>(RW * 4) << piece_shift;
  const int64_t start = pos;

  while (inner || pos < end) {
    const Seq sq = read_seq(a, b);
    const auto un = units_of<D, NT>(a, sq);
    if (!inner && pos >= base + un.all) {
      base += un.all;
      ++b;
      continue;
    }
    const int64_t unit = ((inner ? pos0 : pos) - base) / un.tiles;
    const int tile0 = static_cast<int>(pos - base - unit * un.tiles);
    const int kvh = kDirect ? static_cast<int>(blockIdx.x % a.kv_heads) : static_cast<int>(unit / un.row_tiles);
    const int rt = kDirect ? 0 : static_cast<int>(unit - static_cast<int64_t>(kvh) * un.row_tiles);
    const int n = static_cast<int>(inner ? i64max(0, end - pos) : i64min(un.tiles - tile0, end - pos));
    const int n_rows = sq.n_q * a.group;

    // ---- copies of this warp's tiles
    const int32_t* table = a.table + b * a.table_stride;
    const int64_t head_off = (static_cast<int64_t>(kvh) << a.page_shift) * (RW * 4);
    auto fetch = [&](int j) -> int {   // page of this lane's piece of tile j
      const int key = (tile0 + j) * KT + (lane << piece_shift);
      return (lane < pieces && j < n && key < sq.kv) ? table[key >> a.page_shift] : 0;
    };
    int issued = 0;
    auto issue = [&](int j, int page) {
      if (j >= n || waiter.bad) return;
      issued = j + 1;
      const uint32_t c = it + j, s = c % kStages;
      const int key0 = (tile0 + j) * KT;
      const int have = max(0, min(pieces, (sq.kv - key0 + (1 << piece_shift) - 1) >> piece_shift));
      if (lane == 0) mbar_arrive_expect_tx(bar_u + 8 * s, 2 * have * piece_bytes);
      __syncwarp();
      if (lane < have) {
        if (page < 0 || page >= a.n_pages) {
          record_index(a.status);
          page = 0;
        }
        const int off = (key0 + (lane << piece_shift)) & ((1 << a.page_shift) - 1);
        const int64_t at = page * a.page_stride + head_off + static_cast<int64_t>(off) * (RW * 4);
        const uint32_t dst = ring_u + s * Sh::STAGE + lane * piece_bytes;
        bulk_load(dst, a.k + at, piece_bytes, bar_u + 8 * s);
        bulk_load(dst + Sh::TILE, a.v + at, piece_bytes, bar_u + 8 * s);
      }
    };
    {
      int pg[kStages];
#pragma unroll
      for (int j = 0; j < kStages; ++j) pg[j] = fetch(j);
#pragma unroll
      for (int j = 0; j < kStages; ++j) issue(j, pg[j]);
    }
    int next_page = fetch(kStages);

    // ---- Q^T fragments: lane (g, t) holds row 8 nt + g, the channels of its words
    uint32_t qf[Sh::QS ? 1 : NT][P][4][2];
    uint2* qs = reinterpret_cast<uint2*>(smem + Sh::RING + warp * Sh::QBYTES) + lane;
    float sl2[NT][2];
    int lim[NT][2];   // keys that the row of column 2 t (+ 1) sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int row = rt * R + 8 * nt + g;
      const int tok = row / a.group;
      const QT* qp = static_cast<const QT*>(a.q) + (sq.q0 + tok) * a.q_stride +
                     static_cast<int64_t>(kvh * a.group + row - tok * a.group) * D;
      float up = 1.0f, down = 1.0f;
      uint32_t raw[P][4][2];
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // first channel of the half word: see the words of a row above
            const int c = st == 0 ? 4 * t + 2 + 2 * h
                          : st == 1 ? (t == 3 && h == 1 ? 0 : 4 * t + 18 + 2 * h)
                                    : 32 + 16 * (st - 2) + 4 * t + 2 * h;
            raw[p][st][h] =
                row < n_rows ? *reinterpret_cast<const uint32_t*>(qp + 64 * p + c) : 0u;
          }
      if (sizeof(QT) == 2 && !std::is_same<QT, __half>::value) {
        uint32_t top = 0;   // largest magnitude, as bits
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int st = 0; st < 4; ++st)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              top = max(top, max(raw[p][st][h] & 0x7FFFu, (raw[p][st][h] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int e = static_cast<int>(top >> 7);   // biased exponent
        const int f = (e == 0 || e == 255) ? 0 : min(141 - e, 100);
        up = __int_as_float((127 + f) << 23);
        down = __int_as_float((127 - f) << 23);
      }
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x = raw[p][st][h];
            if (!std::is_same<QT, __half>::value)
              x = pack_half2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xFFFF0000u) * up);
            qf[Sh::QS ? 0 : nt][p][st][h] = x;
          }
      if (Sh::QS) {   // each lane keeps its own
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int st = 0; st < 4; ++st)
            qs[((p * 4 + st) * NT + nt) * 32] = make_uint2(qf[0][p][st][0], qf[0][p][st][1]);
      }
      const float sc = a.scale_log2 * down;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        sl2[nt][c] = __shfl_sync(kFull, sc, 4 * (2 * t + c));
        const int r = rt * R + 8 * nt + 2 * t + c;
        lim[nt][c] = a.causal ? min(sq.kv, sq.kv - sq.n_q + r / a.group + 1) : sq.kv;
      }
    }
    // keys that every row of the unit sees: tiles below need no mask; keys that some row sees
    const int clear = a.causal ? sq.kv - sq.n_q + rt * R / a.group + 1 : sq.kv;
    const int seen = a.causal ? sq.kv - sq.n_q + (min(rt * R + R, n_rows) - 1) / a.group + 1 : sq.kv;

    float o[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nt][e] = 0.0f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        m[nt][c] = -INFINITY;
        l[nt][c] = 0.0f;
      }
    // V's scales carry a power of two per block of channels (v_ups) that keeps the largest so far
    // below 2^7: its product with a weight stays below 2^15 and keeps fp16's 11 bits down to 2^-20
    // of the largest scale.  Only keys that every row sees count: see `apart`.  One power for all
    // blocks would cost a block its bits where another is 2^20 times larger; in registers the
    // powers cost spills (16 sequences of 32,768 keys, 128 channels, 1 token: 201 us, so 198.5;
    // 193 with one power).
    __syncwarp();
    if (lane < D / 32) v_ups[warp][lane] = kMostUp;
    __syncwarp();

#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const uint32_t c = it + j, st = c % kStages;
      if (j >= issued) break;   // an earlier wait ran out
      waiter.wait(bar_u + 8 * st, (c / kStages) & 1);
      const uint32_t* kw = reinterpret_cast<const uint32_t*>(ring + st * Sh::STAGE);
      const uint32_t* vw = kw + Sh::TILE / 4;
      const int key0 = (tile0 + j) * KT;

      // ---- scores: s[mt][nt][e], key S g + 2 mt (e < 2) or the next, column 2 t + (e & 1)
      float s[S / 2][NT][4];
#pragma unroll
      for (int mt = 0; mt < S / 2; ++mt) {
        const uint32_t* ra = kw + (S * g + 2 * mt) * RW;
        const uint32_t* rb = ra + RW;
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint32_t a0 = ra[17 * p], a8 = ra[17 * p + 8], b0 = rb[17 * p], b8 = rb[17 * p + 8];
          uint32_t f[4][4];   // A fragments of the four steps of 16 channels
          codes_to_half2(ra[17 * p + 1 + t], f[0][0], f[0][2]);
          codes_to_half2(rb[17 * p + 1 + t], f[0][1], f[0][3]);
          codes_to_half2(__byte_perm(ra[17 * p + 5 + t], a0, sel_k), f[1][0], f[1][2]);
          codes_to_half2(__byte_perm(rb[17 * p + 5 + t], b0, sel_k), f[1][1], f[1][3]);
          codes_to_half2(ra[17 * p + 9 + t], f[2][0], f[2][2]);
          codes_to_half2(rb[17 * p + 9 + t], f[2][1], f[2][3]);
          codes_to_half2(ra[17 * p + 13 + t], f[3][0], f[3][2]);
          codes_to_half2(rb[17 * p + 13 + t], f[3][1], f[3][3]);
          const float da0 = half_bits(a0), da1 = half_bits(a8 >> 16);
          const float db0 = half_bits(b0), db1 = half_bits(b8 >> 16);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f}, y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint2 q[4];
#pragma unroll
            for (int st = 0; st < 4; ++st)
              q[st] = Sh::QS ? qs[((p * 4 + st) * NT + nt) * 32]
                             : make_uint2(qf[Sh::QS ? 0 : nt][p][st][0], qf[Sh::QS ? 0 : nt][p][st][1]);
            mma16816(x, f[0], q[0].x, q[0].y);
            mma16816(y, f[2], q[2].x, q[2].y);
            mma16816(x, f[1], q[1].x, q[1].y);
            mma16816(y, f[3], q[3].x, q[3].y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float d0 = e < 2 ? da0 : db0, d1 = e < 2 ? da1 : db1;
              const float z = fmaf(d0, x[e], d1 * y[e]);
              s[mt][nt][e] = p == 0 ? z : s[mt][nt][e] + z;
            }
          }
        }
      }
      // ---- V's scales of keys S g + i
      float dv[S][D / 32];
      float v_up[D / 32];
#pragma unroll
      for (int k = 0; k < D / 32; ++k) v_up[k] = v_ups[warp][k];
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const uint16_t* rv = reinterpret_cast<const uint16_t*>(vw + (S * g + i) * RW);
#pragma unroll
        for (int k = 0; k < D / 32; ++k) dv[i][k] = half_bits(rv[17 * k]) * v_up[k];
      }
#pragma unroll
      for (int mt = 0; mt < S / 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][nt][e] *= sl2[nt][e & 1];
      const bool masked = key0 + KT > clear;
      if (masked) {
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const int key = key0 + S * g + i;
          // rows of the tile that hold no key that any row sees: whatever the page
          // or the ring holds there
          if (key >= seen)
#pragma unroll
            for (int k = 0; k < D / 32; ++k) dv[i][k] = 0.0f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int cc = 0; cc < 2; ++cc)
              if (key >= lim[nt][cc]) s[i / 2][nt][2 * (i & 1) + cc] = -INFINITY;
        }
      }
      {
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int k = 0; k < D / 32; ++k) top = fmaxf(top, fabsf(dv[i][k]));
        if (__any_sync(kFull, top >= 128.0f)) {
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            float mine = 0.0f;
#pragma unroll
            for (int i = 0; i < S; ++i)
              if (key0 + S * g + i < clear) mine = fmaxf(mine, fabsf(dv[i][k]));
            const int e = static_cast<int>(__reduce_max_sync(kFull, __float_as_uint(mine)) >> 23);
            const float f = fmaxf(__int_as_float((127 + 127 + 6 - max(e, 127 + 6)) << 23), kLeastUp / v_up[k]);
            v_up[k] *= f;
            __syncwarp();
            if (lane == 0) v_ups[warp][k] = v_up[k];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < S; ++i) dv[i][k] *= f;
#pragma unroll
            for (int i = 2 * k; i < 2 * k + 2; ++i)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[i][nt][x] *= f;
          }
        }
      }

      // ---- the running reference: moved only when a score exceeds it by more than 2^8
      bool over = false;
#pragma unroll
      for (int mt = 0; mt < S / 2; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) over |= s[mt][nt][e] > m[nt][e & 1] + kLazy;
      if (__any_sync(kFull, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            float top = -INFINITY;
#pragma unroll
            for (int mt = 0; mt < S / 2; ++mt) top = fmaxf(top, fmaxf(s[mt][nt][cc], s[mt][nt][2 + cc]));
#pragma unroll
            for (int x = 4; x < 32; x *= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, x));
            if (top > m[nt][cc] + kLazy) {
              const float al = m[nt][cc] == -INFINITY ? 0.0f : ex2_approx(m[nt][cc] - top);
              m[nt][cc] = top;
              l[nt][cc] *= al;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[i][nt][cc] *= al;
                o[i][nt][2 + cc] *= al;
              }
            }
          }
      }
      // A key that some rows see and others do not (a later token of a burst) may have a far
      // larger scale than all before it, or an infinite one, which must not touch the rows that
      // do not see it: then the tile's keys of that kind are added apart, in fp32.  They are
      // at most a burst's tokens but one, in a sequence's last tiles.
      if (masked) {
        bool apart = false;
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            apart |= key0 + S * g + i >= clear && !(fabsf(dv[i][k]) < 128.0f);   // NaN too
        if (__any_sync(kFull, apart)) {
#pragma unroll 1
          for (int kg = 0; kg < 8; ++kg)
#pragma unroll
            for (int i = 0; i < S; ++i) {
              const int key = key0 + S * kg + i;
              if (key < clear || key >= seen) continue;   // uniform
              const uint32_t* rv = vw + (S * kg + i) * RW;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float w[2];
#pragma unroll
                for (int cc = 0; cc < 2; ++cc)
                  w[cc] = ex2_approx(__shfl_sync(kFull, s[i / 2][nt][2 * (i & 1) + cc], 4 * kg + t) -
                                     (m[nt][cc] == -INFINITY ? 0.0f : m[nt][cc]));
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                  // channels as in the products: m-tile 2 k + h, codes 2 h and 2 h + 1 of the lane's word
                  const int p = k / 2;
                  uint32_t word = rv[17 * p + (k & 1 ? 9 : 1) + g];
                  if ((k & 1) == 0) word = __byte_perm(word, rv[17 * p], sel_v);
                  const float d = half_bits(reinterpret_cast<const uint16_t*>(rv)[17 * k]) * v_ups[warp][k];
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    const float v = d * static_cast<float>(static_cast<int8_t>(word >> (8 * e)));
#pragma unroll
                    for (int cc = 0; cc < 2; ++cc)
                      if (w[cc] != 0.0f) o[2 * k + e / 2][nt][2 * (e & 1) + cc] = fmaf(w[cc], v, o[2 * k + e / 2][nt][2 * (e & 1) + cc]);
                  }
                }
              }
            }
#pragma unroll
          for (int i = 0; i < S; ++i)
            if (key0 + S * g + i >= clear)
#pragma unroll
              for (int k = 0; k < D / 32; ++k) dv[i][k] = 0.0f;
        }
      }
      // ---- weights, per V block times its scale, and their transposition
      uint32_t pb[NT][D / 32][S];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float r0 = m[nt][0] == -INFINITY ? 0.0f : m[nt][0];
        const float r1 = m[nt][1] == -INFINITY ? 0.0f : m[nt][1];
#pragma unroll
        for (int i = 0; i < S; ++i) {
          const float w0 = ex2_approx(s[i / 2][nt][2 * (i & 1)] - r0);
          const float w1 = ex2_approx(s[i / 2][nt][2 * (i & 1) + 1] - r1);
          l[nt][0] += w0;
          l[nt][1] += w1;
#pragma unroll
          for (int k = 0; k < D / 32; ++k) {
            pb[nt][k][i] = transpose8(pack_half2(w0 * dv[i][k], w1 * dv[i][k]));
          }
        }
      }
      // ---- values: channels on the side of 16, keys 2 S t + ...
#pragma unroll
      for (int kk = 0; kk < S / 2; ++kk) {
        const uint32_t* r0 = vw + (2 * S * t + 2 * kk) * RW;   // keys of columns 2 t, 2 t + 8
        const uint32_t* r1 = r0 + S * RW;                      // of columns 2 t + 1, 2 t + 9
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int odd = 0; odd < 2; ++odd) {
            const int w = 17 * p + (odd ? 9 : 1) + g;
            uint32_t w0 = r0[w], w1 = r1[w], w2 = r0[w + RW], w3 = r1[w + RW];
            if (!odd) {
              w0 = __byte_perm(w0, r0[17 * p], sel_v);
              w1 = __byte_perm(w1, r1[17 * p], sel_v);
              w2 = __byte_perm(w2, r0[17 * p + RW], sel_v);
              w3 = __byte_perm(w3, r1[17 * p + RW], sel_v);
            }
            uint32_t f[2][4];
            codes_to_half2(__byte_perm(w0, w1, 0x5140), f[0][0], f[0][1]);
            codes_to_half2(__byte_perm(w2, w3, 0x5140), f[0][2], f[0][3]);
            codes_to_half2(__byte_perm(w0, w1, 0x7362), f[1][0], f[1][1]);
            codes_to_half2(__byte_perm(w2, w3, 0x7362), f[1][2], f[1][3]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816(o[4 * p + 2 * odd + h][nt], f[h], pb[nt][2 * p + odd][2 * kk], pb[nt][2 * p + odd][2 * kk + 1]);
          }
      }
      __syncwarp();
      issue(j + kStages, next_page);
      next_page = fetch(j + kStages + 1);
    }
    it += n;

    // ---- the unit's rows, or this share's part of them
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][nt][e] *= __int_as_float((254 << 23) - __float_as_int(v_ups[warp][i / 2]));   // 1 / v_up
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc)
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[nt][cc] += __shfl_xor_sync(kFull, l[nt][cc], x);
    if (inner) {   // join the warps, in a fixed order
      constexpr int kXch = (NREG + 4 * NT) * 32;
      static_assert(kWarps / 2 * kXch * 4 <= Sh::RING, "the exchange reuses the ring");
      float* xch = reinterpret_cast<float*>(smem);
      __syncthreads();   // every warp's tiles are consumed: the ring is free
#pragma unroll 1
      for (int half = kWarps / 2; half > 0; half /= 2) {
        if (warp >= half && warp < 2 * half) {
          float* dst = xch + (warp - half) * kXch + lane;
#pragma unroll
          for (int i = 0; i < NREG; ++i) dst[32 * i] = o[i / (4 * NT)][i / 4 % NT][i & 3];
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) {
            dst[32 * (NREG + i)] = m[i / 2][i & 1];
            dst[32 * (NREG + 2 * NT + i)] = l[i / 2][i & 1];
          }
        }
        __syncthreads();
        if (warp < half) {
          const float* src = xch + warp * kXch + lane;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float wa[2], wb[2];
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              const float mb = src[32 * (NREG + 2 * nt + cc)], lb = src[32 * (NREG + 2 * NT + 2 * nt + cc)];
              const float top = fmaxf(m[nt][cc], mb);
              wa[cc] = join_weight(m[nt][cc], top);
              wb[cc] = join_weight(mb, top);
              m[nt][cc] = top;
              l[nt][cc] = fmaf(wa[cc], l[nt][cc], wb[cc] * lb);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                o[i][nt][e] = fmaf(wa[e & 1], o[i][nt][e], wb[e & 1] * src[32 * ((i * NT + nt) * 4 + e)]);
          }
        }
        __syncthreads();
      }
      if (warp > 0) return;
    }
    {
      const bool whole = inner ? tile0 == 0 && cta_end - pos0 == un.tiles : n == un.tiles;
      if (kDirect || whole) {   // the whole unit: the rows of out
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const int row = rt * R + 8 * nt + 2 * t + cc;
            if (row >= n_rows) continue;
            const float inv = l[nt][cc] == 0.0f ? 0.0f : 1.0f / l[nt][cc];
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
              store_pair<QT, D>(a, sq, kvh, row, i, g, o[i][nt][cc] * inv, o[i][nt][2 + cc] * inv);
          }
      } else {
        const bool first = pos == start;
        float* part = parts + (2 * gw + (first ? 0 : 1)) * Pt::FLOATS;
#pragma unroll
        for (int i = 0; i < NREG; ++i) part[32 * i + lane] = o[i / (4 * NT)][i / 4 % NT][i & 3];
        if (g == 0) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int cc = 0; cc < 2; ++cc) {
              part[32 * NREG + 8 * nt + 2 * t + cc] = m[nt][cc];
              part[32 * NREG + R + 8 * nt + 2 * t + cc] = l[nt][cc];
            }
        }
        // The first boundary inside a unit names the unit's parts, from share c - 1 on
        // (its first part where the unit starts the share, else its second) to the
        // unit's last share.  An inner CTA is one part, of its first share; the
        // unit's first boundary is its own second share's when the unit starts it.
        const int64_t u0 = pos - tile0;
        const bool starts = inner && tile0 == 0;
        if (lane == 0 && (starts || (first && tile0 > 0 && u0 >= start - share))) {
          int32_t* at = desc + (starts ? kDescInts : 0);
          const int64_t c = gw + (starts ? 1 : 0), u1 = u0 + un.tiles, wide = kWarps * share;
          const int64_t k0 = (u0 + wide - 1) / wide;                                // inner CTAs k0 ..
          const int64_t k1 = u1 == total ? (u1 + wide - 1) / wide : u1 / wide;      // .. k1 - 1
          const int64_t last = (u1 - 1) / share;
          at[1] = kvh;
          at[2] = rt;
          at[3] = u0 == (c - 1) * share ? 0 : 1;
          const int64_t n_a = k0 < k1 ? k0 * kWarps - (c - 1) : last - (c - 1) + 1;  // parts before them
          const int64_t n_b = i64max(0, k1 - k0);
          at[4] = static_cast<int32_t>(n_a + n_b + (n_b ? i64max(0, last - k1 * kWarps + 1) : 0));
          at[5] = static_cast<int32_t>(n_a);
          at[6] = static_cast<int32_t>(n_b);
          at[0] = b;
        }
      }
    }
    if (inner) return;
    pos += n;
  }
}

// Joins the partial states of the units that several shares hold parts of.  Warp w of
// block (x, y) looks at boundary 8 x + w and takes quarter y of its unit's channels: alone
// where the unit has few parts; the parts of one with more are dealt to the block's warps.
constexpr int kJoinY = 4;
constexpr int kAlone = 8;   // parts that one warp joins alone

template <typename QT, int D, int NT>
__global__ void __launch_bounds__(kThreads) paged_few_join_kernel(const PagedArgs a) {
  using Pt = Part<D, NT>;
  constexpr int R = Pt::R, NREG = Pt::NREG, MT = D / 16 / kJoinY;   // m-tiles of a quarter
  __shared__ int32_t big[kWarps][8];
  __shared__ float red[kWarps][4 * MT + 2][32];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const float* parts = a.part + kMaxWarps * kDescInts;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int32_t field = lane < 8 ? reinterpret_cast<const int32_t*>(a.part)[mine * kDescInts + lane] : 0;
  const int b0 = __shfl_sync(kFull, field, 0), n0 = __shfl_sync(kFull, field, 4);
  if (lane < 8) big[warp][lane] = lane == 0 && n0 <= kAlone ? -1 : field;
  if (b0 >= 0 && n0 <= kAlone) {
    const int kvh = __shfl_sync(kFull, field, 1), rt = __shfl_sync(kFull, field, 2);
    const int slot = __shfl_sync(kFull, field, 3), n_a = __shfl_sync(kFull, field, 5), n_b = __shfl_sync(kFull, field, 6);
    const Seq sq = read_seq(a, b0);
    const float* part[kAlone];
#pragma unroll
    for (int p = 0; p < kAlone; ++p) {
      // beyond the last, the first again with weight 0, so that the loads need no branch
      const int q = p < n0 ? p : 0;
      const int s = q < n_a ? q : (q < n_a + n_b ? n_a + kWarps * (q - n_a) : q + (kWarps - 1) * n_b);
      part[p] = parts + (2 * (mine - 1 + s) + (s == 0 ? slot : 0)) * Pt::FLOATS;
    }
#pragma unroll 1
    for (int nt = 0; nt < NT; ++nt) {
      float w[kAlone][2], inv[2];
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int at = 32 * NREG + 8 * nt + 2 * t + cc;
        float top = -INFINITY, l = 0.0f, lp[kAlone];
#pragma unroll
        for (int p = 0; p < kAlone; ++p) {
          w[p][cc] = part[p][at];
          lp[p] = part[p][at + R];
        }
#pragma unroll
        for (int p = 0; p < kAlone; ++p) {
          if (p >= n0) w[p][cc] = -INFINITY;
          top = fmaxf(top, w[p][cc]);
        }
#pragma unroll
        for (int p = 0; p < kAlone; ++p) {
          w[p][cc] = join_weight(w[p][cc], top);
          l = p < n0 ? fmaf(w[p][cc], lp[p], l) : l;
        }
        inv[cc] = l == 0.0f ? 0.0f : 1.0f / l;
      }
      const int row = rt * R + 8 * nt + 2 * t;
      const bool have0 = row < sq.n_q * a.group, have1 = row + 1 < sq.n_q * a.group;
#pragma unroll
      for (int q = 0; q < MT; ++q) {
        const int i = blockIdx.y * MT + q;
        float v[kAlone][4], y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = 0; p < kAlone; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[p][e] = part[p][32 * ((i * NT + nt) * 4 + e) + lane];
#pragma unroll
        for (int p = 0; p < kAlone; ++p)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = p < n0 ? fmaf(w[p][e & 1], v[p][e], y[e]) : y[e];
        if (have0) store_pair<QT, D>(a, sq, kvh, row, i, g, y[0] * inv[0], y[2] * inv[0]);
        if (have1) store_pair<QT, D>(a, sq, kvh, row + 1, i, g, y[1] * inv[1], y[3] * inv[1]);
      }
    }
  }
  __syncthreads();
  for (int j = 0; j < kWarps; ++j) {
    const int b = big[j][0];
    if (b < 0) continue;   // uniform over the block
    const int kvh = big[j][1], rt = big[j][2], slot = big[j][3], n = big[j][4], n_a = big[j][5], n_b = big[j][6];
    const int64_t c1 = static_cast<int64_t>(blockIdx.x) * kWarps + j - 1;
    // part p: share c - 1's, then the first slot of the shares after it, of the
    // inner CTAs' eight shares only the first
    auto part = [&](int p) {
      const int s = p < n_a ? p : (p < n_a + n_b ? n_a + kWarps * (p - n_a) : p + (kWarps - 1) * n_b);
      return parts + (2 * (c1 + s) + (s == 0 ? slot : 0)) * Pt::FLOATS;
    };
    const Seq sq = read_seq(a, b);
#pragma unroll 1
    for (int nt = 0; nt < NT; ++nt) {
      const int at = 32 * NREG + 8 * nt + 2 * t;
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 4
      for (int p = warp; p < n; p += kWarps) {
        top[0] = fmaxf(top[0], part(p)[at]);
        top[1] = fmaxf(top[1], part(p)[at + 1]);
      }
      red[warp][0][lane] = top[0];
      red[warp][1][lane] = top[1];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        top[0] = fmaxf(top[0], red[k][0][lane]);
        top[1] = fmaxf(top[1], red[k][1][lane]);
      }
      __syncthreads();
      float l[2] = {0.0f, 0.0f}, y[MT][4] = {};
#pragma unroll 4
      for (int p = warp; p < n; p += kWarps) {
        const float* s = part(p);
        const float w[2] = {join_weight(s[at], top[0]), join_weight(s[at + 1], top[1])};
        l[0] = fmaf(w[0], s[at + R], l[0]);
        l[1] = fmaf(w[1], s[at + R + 1], l[1]);
#pragma unroll
        for (int q = 0; q < MT; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            y[q][e] = fmaf(w[e & 1], s[32 * (((blockIdx.y * MT + q) * NT + nt) * 4 + e) + lane], y[q][e]);
      }
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) red[warp][4 * q + e][lane] = y[q][e];
      red[warp][4 * MT][lane] = l[0];
      red[warp][4 * MT + 1][lane] = l[1];
      __syncthreads();
      if (warp == 0) {
        float sum[4 * MT + 2];
#pragma unroll
        for (int q = 0; q < 4 * MT + 2; ++q) {
          sum[q] = red[0][q][lane];
#pragma unroll
          for (int k = 1; k < kWarps; ++k) sum[q] += red[k][q][lane];
        }
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          const int row = rt * R + 8 * nt + 2 * t + cc;
          const float inv = sum[4 * MT + cc] == 0.0f ? 0.0f : 1.0f / sum[4 * MT + cc];
          if (row < sq.n_q * a.group)
#pragma unroll
            for (int q = 0; q < MT; ++q)
              store_pair<QT, D>(a, sq, kvh, row, blockIdx.y * MT + q, g, sum[4 * q + cc] * inv,
                                sum[4 * q + 2 + cc] * inv);
        }
      }
      __syncthreads();
    }
  }
}

template <typename QT, int D, int NT, bool kDirect>
cudaError_t launch_few(const PagedArgs& a, int ctas, cudaStream_t stream) {
  auto kernel = paged_few_kernel<QT, D, NT, kDirect>;
  constexpr int smem = Shape<D, NT>::SMEM;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    configured_device = dev;
  }
  e = launch_kernel(kernel, dim3(ctas), dim3(kThreads), smem, stream, a);
  if (e != cudaSuccess || kDirect) return e;
  return launch_kernel(paged_few_join_kernel<QT, D, NT>, dim3(ctas, kJoinY), dim3(kThreads), 0, stream, a);
}

template <typename QT, int D>
cudaError_t launch_few_d(const PagedArgs& a, int64_t rows, bool direct, cudaStream_t stream) {
  // tiles of 8 or 16 rows: 16 cost 16 sequences of 32,768 keys (8 K/V heads) 142 us instead
  // of 106 at 64 channels, 277 instead of 198 at 128
  if (direct) {
    const int ctas = a.batch * a.kv_heads;
    return rows <= 8 ? launch_few<QT, D, 1, true>(a, ctas, stream) : launch_few<QT, D, 2, true>(a, ctas, stream);
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int ctas = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
  return rows <= 8 ? launch_few<QT, D, 1, false>(a, ctas, stream) : launch_few<QT, D, 2, false>(a, ctas, stream);
}

}  // namespace

// Whether every unit is one CTA's: no unit has more than four tiles a warp.  The shares
// and their join would spread so few tiles further, but cost a second launch.
bool paged_few_direct(int64_t batch, int32_t kv_heads, int64_t max_kv, int32_t head_dim) {
  const int64_t tile = head_dim == 64 ? Shape<64, 1>::KT : Shape<128, 1>::KT;
  return max_kv <= 4 * kWarps * tile && batch * kv_heads <= 0x7FFFFFFF;
}

int64_t paged_few_floats(int32_t head_dim, int64_t rows) {
  const int64_t r = rows <= 8 ? 8 : 16;
  return kMaxWarps * (kDescInts + 2 * (r * head_dim + 2 * r));
}

cudaError_t launch_paged_few(const PagedArgs& a, int32_t dtype, int32_t head_dim, int64_t rows, bool direct,
                             cudaStream_t stream) {
  if (dtype == kF16)
    return head_dim == 64 ? launch_few_d<__half, 64>(a, rows, direct, stream)
                          : launch_few_d<__half, 128>(a, rows, direct, stream);
  return head_dim == 64 ? launch_few_d<__nv_bfloat16, 64>(a, rows, direct, stream)
                        : launch_few_d<__nv_bfloat16, 128>(a, rows, direct, stream);
}

}  // namespace q8a
