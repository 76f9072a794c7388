// paged_tiles.cuh -- attention of many query rows per K/V head over a paged Q8_0
// cache: prompts and chunks of prompts.
//
// The function is the one of paged_few.cuh.  With hundreds of rows per key the
// bound is the tensor cores, so the products run on tcgen05 with the
// accumulators in TMEM:
//   S = Q K_hi^T + Q K_lo^T,   O += P V_hi (+ P V_lo),
// where a dequantised key d c (18 significant bits) is split exactly into an fp16
// value and an fp16 residual.  V is split the same way for fp16 outputs; for bf16
// outputs (rounded at 2^-8) V is rounded once to fp16 (2^-11), which saves a third
// of the products at D = 64.  Weights are rounded once to fp16, as everywhere.
//
// One CTA takes two tiles (A, B) of 128 rows of one (sequence, K/V head).  A row is
// a (token, query head of the group) pair, so a dequantised key tile serves 256
// rows whatever the group.  Warps:
//   0-7     softmax of A / B, one thread per row (TMEM lane);
//   12      producer: asynchronous copies of the pages' rows into a raw ring;
//   13, 14  issue the MMAs of S and of O.  One warp for both spends about 1,340 cycles a
//           step at D = 64 on its waits and issues, against 768 of tensor work; apart,
//           neither is the limit (key tiles of 96 keys, 256 rows: 654 -> 701 TFLOP/s).
//   others  dequantisation, a lane per 34-byte block, some warps for K and some for V: a warp's
//           time per key tile is one chain of waits, loads and stores, and with both tensors
//           in every warp that chain was the limit (pairs 290 -> 266 us, whole CTAs up to 6 %).
//           Five and four warps at D = 64 (four and four 384 us, five and three 390, these
//           380); two and two at D = 128, where more of them take shared memory and issue
//           slots from the rest (three and three 705 us, these 638, bf16); in pairs seven
//           and six.
//
// D = 64: key tiles of 96 keys and three score buffers in TMEM, which the steps (A and B
// of each key tile in turn) use one after another, so that the scores of a tile's next key
// tile are ready before its softmax ends.  D = 128: key tiles of 64 keys and two buffers;
// TMEM then has room for both Q tiles.  Q is the A operand in TMEM (stored there by the
// softmax threads, one row each): 64 keys take 32 cycles a k-step so, 48 with Q in
// shared memory, and with B's Q there for a third buffer D = 128 reached 747 TFLOP/s
// instead of 803.  O has no separate columns for the residuals of V.
//
// Pairs (calls of at most 128 rows per K/V head): both tiles hold the same rows and take the
// key tiles in turn, so no half of the CTA idles; dequantisation is the limit then.
//
// Measured without a mask, 9,728 tokens on 16,384 keys, 8 heads: D = 64 854 (fp16) and
// 901 (bf16) TFLOP/s, D = 128 847 and 1,020, of 1,699 sustained for a plain bf16 product;
// K's residuals make S cost twice its nominal work, V's (fp16) O.  What the others wait for
// most is dequantisation (D = 64, bf16, 362 us: without it 311, without exponentials 347, with
// half of S's products and a sixth of O's 359).
//
// Every wait is bounded, as in chunk_step.cu.

#pragma once

#include <cfloat>
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

constexpr int BM = 128;
constexpr int ND = 2;            // dequantised K and V rings
constexpr float kLazy = 8.0f;    // the reference moves when exceeded by more than 2^8
constexpr float kLift = 7.0f;    // weights carry 2^7, so they reach 2^15 and keep fp16's 11 bits down to 2^-21
constexpr uint32_t kFull = 0xFFFFFFFFu;

template <int D, bool kPair>
struct Geo {
  static constexpr int BN = D == 64 ? 96 : 64;          // keys of a tile
  static constexpr int RB = D / 32 * 34;                // bytes of a row
  static constexpr int RAWB = BN * RB;
  static constexpr int ATOMS = D / 64;                  // 64-channel swizzle columns of a tile
  static constexpr int ATOM = BN * 128;                 // bytes of one such column
  static constexpr int TILE = ATOMS * ATOM;             // one fp16 tile
  // Raw ring.  In pairs a key tile serves 128 rows, so the copies' latency counts more: at
  // D = 64 (16 sequences of 32,768 keys, 8 K/V heads, 32 rows) 3 stages 278 us, 4 259, 6 254 (257 since V's scales are clamped);
  // at D = 128 3 stages 446, 4 422.  Otherwise 6 and 4 of them change nothing.
  static constexpr int NR = D == 64 ? (kPair ? 6 : 4) : (kPair ? 4 : 3);
  static constexpr int NS = D == 64 ? 3 : 2;            // score buffers
  static constexpr int kThreads = kPair ? 768 : (D == 64 ? 640 : 512);
  static constexpr int kKDq = kPair ? 7 : D == 64 ? 5 : 2, kVDq = kPair ? 6 : D == 64 ? 4 : 2;   // K's, V's dequantising warps
  static_assert(kKDq + kVDq + 11 <= kThreads / 32, "warps");
  static constexpr int ROWS = kPair ? BM : 2 * BM;      // query rows of a CTA
  // shared memory
  static constexpr int OFF_K = 0;                       // [ND][hi | lo]
  static constexpr int OFF_V = OFF_K + ND * 2 * TILE;   // [ND][hi | lo]
  static constexpr int OFF_RAW = OFF_V + ND * 2 * TILE;
  static constexpr int OFF_BAR = OFF_RAW + NR * 2 * RAWB;
  static constexpr int B_Q = 0, B_RAWFULL = 1, B_RAWEMPTY = B_RAWFULL + NR, B_KFULL = B_RAWEMPTY + NR,
                       B_KEMPTY = B_KFULL + ND, B_VFULL = B_KEMPTY + ND, B_VEMPTY = B_VFULL + ND,
                       B_SFULL = B_VEMPTY + ND, B_PFULL = B_SFULL + NS, B_PV = B_PFULL + NS, B_ODONE = B_PV + NS, B_DRAIN = B_ODONE + 2,
                       NBAR = B_DRAIN + 2;
  static constexpr int OFF_CTL = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_CTL + 64 + 1024;      // + alignment slack
  static_assert(SMEM <= 227 * 1024 && TILE % 1024 == 0 && OFF_RAW % 16 == 0 && RAWB % 16 == 0, "shared memory");
  // TMEM columns
  static constexpr uint32_t T_S = 0, T_O = NS * BN, T_Q = T_O + 2 * D, T_END = T_Q + D;
  static_assert(T_END <= 512, "TMEM");
  // registers of the softmax warpgroups and of the others, out of the launch's REG_L a thread
  static constexpr int REG_S = kPair ? 128 : (D == 64 ? 144 : 136), REG_O = kPair ? 56 : (D == 64 ? 64 : 120),
                       REG_L = kPair ? 80 : (D == 64 ? 96 : 128);
  static_assert(2 * 128 * REG_S + (kThreads - 256) * REG_O <= kThreads * REG_L, "register split");
};

struct Ctl {
  uint32_t tmem;
  uint32_t abort;
  int32_t b;      // sequence of this CTA, or -1
  int32_t unit;   // its row unit
  int32_t kvh;    // K/V head
  int32_t share;  // which share of the key tiles
  int32_t per;    // key tiles of a share
  int32_t first;  // CTA of the unit's first share
  Seq sq;
};

__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, Ctl* ctl, uint64_t budget, uint32_t* status,
                                         bool honour_abort = true) {
  if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
  const long long t0 = clock64();
  while (true) {
    if (__all_sync(kFull, mbar_try_wait_sleep(bar, parity, 100000u))) return true;
    int stop = 0;
    if ((threadIdx.x & 31) == 0) {
      if (honour_abort && *reinterpret_cast<volatile uint32_t*>(&ctl->abort) != 0u) {
        stop = 1;
      } else if (static_cast<uint64_t>(clock64() - t0) > budget) {
        *reinterpret_cast<volatile uint32_t*>(&ctl->abort) = 1u;
        record_timeout(status);
        stop = 1;
      }
    }
    if (__shfl_sync(kFull, stop, 0)) return false;
  }
}

template <uint32_t N>
__device__ __forceinline__ void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <uint32_t N>
__device__ __forceinline__ void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      Q8A_W8(r, 0), Q8A_W8(r, 8)
      : "memory");
}

// Eight words of a thread's own row of Q, O or a partial state.  32 rows are 32 lines of L1
// each time, so 256 bits at once where the rows start 32-byte aligned: a CTA of one key tile
// (64 channels) 7.84 -> 7.48 us, of two (128 channels) 12.1 -> 10.6.
__device__ __forceinline__ void load_row8(const uint4* p, bool wide, uint32_t* v) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "l"(p));
  } else {
    const uint4 x = p[0], y = p[1];
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w, v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
  }
}
__device__ __forceinline__ void store_row8(uint4* p, bool wide, const uint32_t* v) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), Q8A_W8(v, 0) : "memory");
  } else {
    p[0] = make_uint4(v[0], v[1], v[2], v[3]);
    p[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// The work of this CTA: rows r0 .. r0 + 255 of a (sequence, K/V head), key tiles
// t0 .. of its share.
struct Unit {
  Seq sq;
  Span span;  // which keys the tiles are
  int kvh, r0, n_rows;
  int t0;     // first key tile of this CTA's share
  int T[2];   // key tiles of A and B from there
  int per;    // key tiles of a share
};

// kPrefix: the rows of all sequences, on the shared keys.
template <int kMode>
__device__ __forceinline__ Seq seq_at(const PagedArgs& a, int b) {
  if (kMode == kPrefix) return Seq{0, static_cast<int32_t>(a.total_q), prefix_keys(a)};
  return read_seq(a, b);
}

// Keys that row r of a sequence can see end here.
template <int kMode>
__device__ __forceinline__ int end_of(const PagedArgs& a, const Seq& sq, int r) {
  return kMode != kPrefix && a.causal ? min(sq.kv, sq.kv - sq.n_q + r / a.group + 1) : sq.kv;
}

// Key tiles that rows r .. r + 127 of a sequence see.
template <int D, bool kPair, int kMode>
__device__ __forceinline__ int tiles_of(const PagedArgs& a, const Seq& sq, const Span& span, int r, int n_rows) {
  if (r >= n_rows) return 0;
  return span_tiles<kMode, Geo<D, kPair>::BN>(span, end_of<kMode>(a, sq, min(r + BM - 1, n_rows - 1)));
}

// What the tiles of a window can be at most for `rows` rows next to each other: those of the sinks and those of
// window + tokens - 1 keys that start up to 31 keys (a piece of a page) early.
template <int kBN>
__host__ __device__ __forceinline__ int64_t window_bound(int64_t kv, int64_t window, int64_t sinks, int32_t group, int rows) {
  const int64_t tokens = (rows - 1 + group - 1) / group + 1;
  const int64_t all = (kv + kBN - 1) / kBN;
  const int64_t n = ((sinks < kv ? sinks : kv) + kBN - 1) / kBN + (window + tokens - 1 + 31 + kBN - 1) / kBN;
  return all < n ? all : n;
}

template <int D, bool kPair, int kMode>
__device__ __forceinline__ Unit make_unit(const PagedArgs& a, const Ctl* ctl, int split) {
  Unit u;
  u.sq = ctl->sq;
  u.kvh = ctl->kvh;
  u.n_rows = u.sq.n_q * a.group;
  // the unit with the most visible keys first
  u.r0 = ((u.n_rows + Geo<D, kPair>::ROWS - 1) / Geo<D, kPair>::ROWS - 1 - ctl->unit) * Geo<D, kPair>::ROWS;
  u.span = span_of<kMode, Geo<D, kPair>::BN>(a, static_cast<int64_t>(u.sq.kv) - u.sq.n_q + u.r0 / a.group,
                                             end_of<kMode>(a, u.sq, min(u.r0 + Geo<D, kPair>::ROWS, u.n_rows) - 1),
                                             kMode == kOwn ? prefix_keys(a) : 0, min(a.page_shift, 5));
  const int ta = tiles_of<D, kPair, kMode>(a, u.sq, u.span, u.r0, u.n_rows);
  const int tb = kPair ? 0 : tiles_of<D, kPair, kMode>(a, u.sq, u.span, u.r0 + BM, u.n_rows);
  u.per = ctl->per;
  u.t0 = split * u.per;
  u.T[0] = max(0, min(u.per, ta - u.t0));
  u.T[1] = max(0, min(u.per, tb - u.t0));
  if (kPair) {   // the key tiles in turn
    u.T[1] = u.T[0] / 2;
    u.T[0] -= u.T[1];
  }
  return u;
}

// What a sequence brings: row units (0 where the few-row kernel takes it) and key tiles.
struct Load {
  int32_t units, tiles;
};
template <int D, bool kPair, int kMode>
__device__ __forceinline__ Load load_of(const PagedArgs& a, int b) {
  using G = Geo<D, kPair>;
  if (b >= a.batch) return Load{0, 0};
  const Seq sq = seq_at<kMode>(a, b);
  const int64_t rows = static_cast<int64_t>(sq.n_q) * a.group;
  int tiles = (sq.kv + G::BN - 1) / G::BN;
  if (kMode == kOwn) tiles = (max(sq.kv - prefix_keys(a), 0) + G::BN - 1) / G::BN;
  if (kMode == kWindow) tiles = static_cast<int>(window_bound<G::BN>(sq.kv, a.window, a.sinks, a.group, G::ROWS));
  return Load{rows > a.row_limit ? static_cast<int32_t>((rows + G::ROWS - 1) / G::ROWS) : 0, tiles};
}

constexpr int kEnds = 6;    // a CTA's start and end, in key tiles
constexpr int kPlanned = 64;   // most sequences of a call whose shares are planned here

// Key tiles of a share, by one warp: of the longest sequence's tiles cut into 1 .. 32 parts,
// the length that makes waves x (length + a CTA's ends) least.  Lane k - 1 tries k parts.
template <int D, bool kPair, int kMode>
__device__ __forceinline__ int plan_shares(const PagedArgs& a, int lane) {
  if (a.share_tiles > 0) return a.share_tiles;
  if (kMode == kPrefix) {   // one sequence: every unit has the same tiles, cut so that the grid is filled once
    const Load one = load_of<D, kPair, kMode>(a, 0);
    const int parts = static_cast<int>(i64max(1, a.ctas / (static_cast<int64_t>(max(one.units, 1)) * a.kv_heads)));
    return max(4, (one.tiles + parts - 1) / parts);
  }
  Load mine[kPlanned / 32];
  int top = 0;
#pragma unroll
  for (int i = 0; i < kPlanned / 32; ++i) {
    mine[i] = load_of<D, kPair, kMode>(a, 32 * i + lane);
    if (mine[i].units > 0) top = max(top, mine[i].tiles);
  }
  top = max(1, __reduce_max_sync(kFull, top));
  const int len = (top + lane) / (lane + 1);
  int count = 0;
#pragma unroll
  for (int i = 0; i < kPlanned / 32; ++i)
    for (int j = 0; j < min(32, a.batch - 32 * i); ++j) {
      const int units = __shfl_sync(kFull, mine[i].units, j), tiles = __shfl_sync(kFull, mine[i].tiles, j);
      count += units * static_cast<int>(static_cast<unsigned>(tiles + len - 1) / static_cast<unsigned>(len));
    }
  count *= a.kv_heads;
  // the least cost, of equal ones the fewest parts (one part always fits the grid)
  const bool fits = lane == 0 || (len >= 4 && count <= a.ctas);
  const unsigned cost = static_cast<unsigned>((count + kSms - 1) / kSms) * static_cast<unsigned>(len + kEnds);
  const unsigned best = __reduce_min_sync(kFull, fits ? min(cost, 0x03FFFFFFu) * 32u + lane : 0xFFFFFFFFu);
  return __shfl_sync(kFull, len, best & 31u);
}

// Finds, by one warp, what block x of the grid works on: the sequences' (row unit, K/V
// head) pairs laid end to end, each with its shares (kShares), or without (x is the pair).
template <int D, bool kPair, int kMode, bool kShares>
__device__ __forceinline__ void locate(const PagedArgs& a, int64_t x, int per, Ctl* ctl, int lane) {
  int64_t base = 0, ctas = 0;   // of what x counts; CTAs before the sequence
  int found = -1, unit = 0, kvh = 0, share = 0;
  int64_t first = 0;
  for (int b0 = 0; b0 < a.batch && found < 0; b0 += 32) {
    const Load ld = load_of<D, kPair, kMode>(a, b0 + lane);
    const int s = (ld.tiles + per - 1) / per;
    const int64_t pairs = static_cast<int64_t>(ld.units) * a.kv_heads;
    const int64_t n = kShares ? pairs * s : pairs;
    int64_t inc = n, inc_c = pairs * s;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int64_t v = __shfl_up_sync(kFull, inc, o), w = __shfl_up_sync(kFull, inc_c, o);
      if (lane >= o) {
        inc += v;
        inc_c += w;
      }
    }
    const bool here = x >= base + inc - n && x < base + inc;
    const unsigned who = __ballot_sync(kFull, here);
    if (who) {
      const int src = __ffs(who) - 1;
      found = b0 + src;
      const int64_t at = __shfl_sync(kFull, x - (base + inc - n), src);
      const int shares = __shfl_sync(kFull, s, src);
      const int64_t pair = kShares ? at / shares : at;
      share = kShares ? static_cast<int>(at - pair * shares) : 0;
      unit = static_cast<int>(pair / a.kv_heads);
      kvh = static_cast<int>(pair - static_cast<int64_t>(unit) * a.kv_heads);
      first = __shfl_sync(kFull, ctas + inc_c - pairs * s, src) + pair * shares;
    }
    base += __shfl_sync(kFull, inc, 31);
    ctas += __shfl_sync(kFull, inc_c, 31);
  }
  if (lane == 0) {
    ctl->b = found;
    ctl->unit = unit;
    ctl->kvh = kvh;
    ctl->share = share;
    ctl->per = per;
    ctl->first = static_cast<int32_t>(first);
    if (found >= 0) ctl->sq = seq_at<kMode>(a, found);
  }
}

// kPrefix: what pair x of row unit and K/V head is follows from the prefix's length alone, so that every thread of the
// join finds it by itself.  (For the tile kernel itself, where one lane did, the code around it was slower:
// 136 -> 139 us for 100,001 keys of 64 channels.)
template <int D, bool kPair>
__device__ __forceinline__ void locate_prefix(const PagedArgs& a, int64_t x, Ctl* ctl) {
  using G = Geo<D, kPair>;
  const int64_t pairs = (a.total_q * a.group + G::ROWS - 1) / G::ROWS * a.kv_heads;
  const Seq sq = seq_at<kPrefix>(a, 0);
  const int tiles = (sq.kv + G::BN - 1) / G::BN;
  const int parts = static_cast<int>(i64max(1, a.ctas / pairs));   // as plan_shares
  const int per = a.share_tiles > 0 ? a.share_tiles : max(4, (tiles + parts - 1) / parts);
  const int unit = static_cast<int>(x / a.kv_heads);
  ctl->b = x < pairs ? 0 : -1;
  ctl->unit = unit;
  ctl->kvh = static_cast<int>(x - static_cast<int64_t>(unit) * a.kv_heads);
  ctl->share = 0;
  ctl->per = per;
  ctl->first = static_cast<int32_t>(x * ((tiles + per - 1) / per));
  ctl->sq = sq;
}

// Step n <-> (key tile t, tile x), the key tiles counted from t0: A and B in turn, then the
// longer one alone; in pairs, step n is key tile n.  j: tile x's j-th step.
template <bool kPair>
__device__ __forceinline__ int step_of(const Unit& u, int j, int x) {
  const int m = min(u.T[0], u.T[1]);
  return kPair || j < m ? 2 * j + x : m + j;
}
template <bool kPair>
__device__ __forceinline__ int step_key(const Unit& u, int n) {
  const int m = min(u.T[0], u.T[1]);
  return kPair ? n : (n < 2 * m ? n >> 1 : n - m);
}
template <bool kPair>
__device__ __forceinline__ int step_tile(const Unit& u, int n) {
  return kPair || n < 2 * min(u.T[0], u.T[1]) ? n & 1 : (u.T[1] > u.T[0] ? 1 : 0);
}
// Whether tile x's step is the one that reads key tile t last: B's, or A's where B has none.
template <bool kPair>
__device__ __forceinline__ bool last_reader(const Unit& u, int t, int x) {
  return kPair || x == 1 || t >= u.T[1];
}
// Key tiles that go through the CTA.
template <bool kPair>
__device__ __forceinline__ int key_tiles(const Unit& u) {
  return kPair ? u.T[0] + u.T[1] : max(u.T[0], u.T[1]);
}

// ------------------------------------------------------------------ roles --

template <int D, bool kPair, int kMode>
__device__ __forceinline__ void producer(const PagedArgs& a, const Unit& u, int b, uint32_t sbase, Ctl* ctl) {
  using G = Geo<D, kPair>;
  const uint64_t budget = 2 * a.timeout_ns;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
  const int T = key_tiles<kPair>(u);
  const int shift = min(a.page_shift, 5);   // pieces of 32 rows, or of a page of 16
  const int pieces = G::BN >> shift;
  const uint32_t bytes = static_cast<uint32_t>(G::RB) << shift;
  const int32_t* table = a.table + b * a.table_stride;
  const int64_t head_off = (static_cast<int64_t>(u.kvh) << a.page_shift) * G::RB;
  auto fetch = [&](int t) -> int {
    const int key = key_of<kMode, G::BN>(u.span, u.t0 + t) + (lane << shift);
    return (lane < pieces && t < T && key < u.sq.kv) ? table[key >> a.page_shift] : 0;
  };
  int page = fetch(0);
  int t = 0;
  for (; t < T; ++t) {
    const int next = fetch(t + 1);
    const int s = t % G::NR;
    if (!wait_bar(bar(G::B_RAWEMPTY + s), ((t / G::NR) & 1) ^ 1, ctl, budget, a.status)) break;
    const int key0 = key_of<kMode, G::BN>(u.span, u.t0 + t);
    const int have = min(pieces, (u.sq.kv - key0 + (1 << shift) - 1) >> shift);   // > 0: the tile has a visible key
    const bool take = lane < have && piece_needed<kMode>(a, u.span, key0 + (lane << shift));
    const int copies = kMode == kWindow ? __popc(__ballot_sync(kFull, take)) : have;
    if (lane == 0) mbar_arrive_expect_tx(bar(G::B_RAWFULL + s), 2 * copies * bytes);
    __syncwarp();
    if (take) {
      if (page < 0 || page >= a.n_pages) {
        record_index(a.status);
        page = 0;
      }
      const int off = (key0 + (lane << shift)) & ((1 << a.page_shift) - 1);
      const int64_t at = page * a.page_stride + head_off + static_cast<int64_t>(off) * G::RB;
      const uint32_t dst = sbase + G::OFF_RAW + s * 2 * G::RAWB + lane * bytes;
      bulk_load(dst, a.k + at, bytes, bar(G::B_RAWFULL + s));
      bulk_load(dst + G::RAWB, a.v + at, bytes, bar(G::B_RAWFULL + s));
    }
    page = next;
  }
  // never leave with a copy in flight
  for (int i = max(0, t - G::NR); i < t; ++i)
    wait_bar(bar(G::B_RAWFULL + i % G::NR), (i / G::NR) & 1, ctl, budget, a.status, false);
}

// One block of one row (nine-word window w; even blocks start word-aligned, odd ones
// two bytes into the first word) -> 16-byte chunks of the swizzled row.  `odd` is the same for
// a warp: as a branch 672 us, as selections of words 710 (D = 128, bf16).
//
// A weight of 0 does not keep a row from what it does not see: 0 times an infinite or NaN value is NaN.
// So V's scales count as at most 515.5, the largest whose values all fit fp16 (127 x 515.5 =
// 65,468.5), NaN too: no value of V is anything but a number (one instruction a block, no
// time: 799 and 800 us for whole prompts of 64 channels).  For K masked scores are assigned.
// Giving NaN to the rows that see such a key as well, by a note of the first one, took 3 %
// of the time where V's dequantising warps looked, 25 % where the producer did.
template <bool kLo, bool odd, bool kV>
__device__ __forceinline__ void dequant_block(const uint32_t (&w)[9], uint8_t* hi_row, uint8_t* lo_row,
                                              int chunk0, int sw) {
  __half2 d2 = __half2half2(__ushort_as_half(static_cast<unsigned short>(odd ? w[0] >> 16 : w[0] & 0xFFFFu)));
  if (kV) d2 = __hmin2(d2, __half2half2(__ushort_as_half(0x6007)));   // 515.5; of NaN and a number the number
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const uint32_t c0 = odd ? w[1 + 2 * c] : __byte_perm(w[2 * c], w[2 * c + 1], 0x5432);
    const uint32_t c1 = odd ? w[2 + 2 * c] : __byte_perm(w[2 * c + 1], w[2 * c + 2], 0x5432);
    __half2 q0, q1, q2, q3;
    codes_to_half2(c0, q0, q1);
    codes_to_half2(c1, q2, q3);
    const __half2 h0 = __hmul2(q0, d2), h1 = __hmul2(q1, d2), h2 = __hmul2(q2, d2), h3 = __hmul2(q3, d2);
    const int at = ((chunk0 + c) ^ sw) * 16;
    *reinterpret_cast<uint4*>(hi_row + at) = make_uint4(h2u(h0), h2u(h1), h2u(h2), h2u(h3));
    if (kLo) {
      const __half2 l0 = __hfma2(q0, d2, __hneg2(h0)), l1 = __hfma2(q1, d2, __hneg2(h1));
      const __half2 l2 = __hfma2(q2, d2, __hneg2(h2)), l3 = __hfma2(q3, d2, __hneg2(h3));
      *reinterpret_cast<uint4*>(lo_row + at) = make_uint4(h2u(l0), h2u(l1), h2u(l2), h2u(l3));
    }
  }
}

// One (32 rows, block) group of a tile: the lanes read consecutive rows, 17 words apart
// (32 banks; 34 apart at D = 128: two lanes a bank).
template <int D, bool kPair, int kMode, bool kV, bool kLo>
__device__ __forceinline__ void dequant_group(const PagedArgs& a, const Span& span, const uint8_t* raw, uint8_t* tile,
                                              int group, int key0, int kv, int lane) {
  using G = Geo<D, kPair>;
  const int row = (group % (G::BN / 32)) * 32 + lane, blk = group / (G::BN / 32);
  const int shift = min(a.page_shift, 5);
  const bool odd = blk & 1;
  uint8_t* hi = tile + (blk >> 1) * G::ATOM + row * 128;
  uint8_t* lo = hi + G::TILE;
  const int chunk0 = odd ? 4 : 0;
  if (row < kv - key0 && piece_needed<kMode>(a, span, key0 + (row >> shift << shift))) {
    const uint32_t* p = reinterpret_cast<const uint32_t*>(raw + row * G::RB) + 17 * (blk >> 1) + (odd ? 8 : 0);
    uint32_t c[9];
#pragma unroll
    for (int k = 0; k < 9; ++k) c[k] = p[k];
    if (odd)
      dequant_block<kLo, true, kV>(c, hi, lo, chunk0, row & 7);
    else
      dequant_block<kLo, false, kV>(c, hi, lo, chunk0, row & 7);
  } else {   // keys that the sequence does not have, or that were not copied: whatever the buffer holds is not read
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = ((chunk0 + c) ^ (row & 7)) * 16;
      *reinterpret_cast<uint4*>(hi + at) = z;
      if (kLo) *reinterpret_cast<uint4*>(lo + at) = z;
    }
  }
}

// K's or V's tiles, by warps w of G::kKDq or G::kVDq.  The groups go round the warps from tile to
// tile, so any number of warps shares them evenly.
template <int D, bool kPair, int kMode, bool kV, bool kLo>
__device__ __forceinline__ void dequant(const PagedArgs& a, const Unit& u, int w, uint8_t* smem, uint32_t sbase,
                                        Ctl* ctl) {
  using G = Geo<D, kPair>;
  constexpr int kGroups = G::BN / 32 * (D / 32);   // groups of a tile: 6 or 8
  constexpr int kWarps = kV ? G::kVDq : G::kKDq;
  const uint64_t budget = 2 * a.timeout_ns;
  const int lane = threadIdx.x & 31;
  auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
  const int T = key_tiles<kPair>(u);
  int mine = w;   // this warp's next group of the tile
#pragma unroll 1
  for (int t = 0; t < T; ++t) {
    const int s = t % G::NR, sd = t % ND;
    if (!wait_bar(bar(G::B_RAWFULL + s), (t / G::NR) & 1, ctl, budget, a.status)) return;
    if (!wait_bar(bar((kV ? G::B_VEMPTY : G::B_KEMPTY) + sd), ((t / ND) & 1) ^ 1, ctl, budget, a.status)) return;
    const int key0 = key_of<kMode, G::BN>(u.span, u.t0 + t);
#pragma unroll 1
    for (; mine < kGroups; mine += kWarps)
      dequant_group<D, kPair, kMode, kV, kLo>(a, u.span, smem + G::OFF_RAW + (2 * s + kV) * G::RAWB,
                                              smem + (kV ? G::OFF_V : G::OFF_K) + sd * 2 * G::TILE, mine, key0, u.sq.kv,
                                              lane);
    fence_proxy_async_smem();
    mbar_arrive(bar((kV ? G::B_VFULL : G::B_KFULL) + sd));
    mbar_arrive(bar(G::B_RAWEMPTY + s));
    mine -= kGroups;
  }
}

__device__ __forceinline__ bool elect_one() {
  uint32_t pred = 0;
  asm volatile(
      "{\n\t.reg .pred P;\n\t"
      "elect.sync _|P, 0xffffffff;\n\t"
      "selp.b32 %0, 1, 0, P;\n\t}"
      : "=r"(pred));
  return pred != 0;
}

// Scores.  K tiles K-major in 64-channel swizzle columns, a k-step 16 channels (32
// bytes of the swizzled rows); Q's channels 16 k .. in TMEM columns 8 k .. of Q.
template <int D, bool kPair>
__device__ __forceinline__ void score_mma(const PagedArgs& a, const Unit& u, uint32_t sbase, uint32_t tmem, Ctl* ctl) {
  using G = Geo<D, kPair>;
  const uint64_t budget = 2 * a.timeout_ns;
  auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
  constexpr uint32_t kIdesc = idesc_f16_f32(128, G::BN, 0, 0);
  const bool leader = elect_one();
  const uint64_t kdesc = smem_desc(sbase + G::OFF_K, 1024, 1024, kSwizzle128);
  const int N = u.T[0] + u.T[1];
  bool ok = wait_bar(bar(G::B_Q), 0, ctl, budget, a.status);
  for (int n = 0; ok && n < N; ++n) {
    const int t = step_key<kPair>(u, n), x = step_tile<kPair>(u, n), sd = t % ND, buf = n % G::NS;
    if (!wait_bar(bar(G::B_KFULL + sd), (t / ND) & 1, ctl, budget, a.status)) break;
    // the buffer's weights have been used by O's update of step n - G::NS
    if (n >= G::NS && !wait_bar(bar(G::B_PV + buf), (n / G::NS - 1) & 1, ctl, budget, a.status)) break;
    tc_fence_after();
    const uint32_t d = tmem + G::T_S + G::BN * buf;
    const uint64_t kd = kdesc + static_cast<uint64_t>(sd * 2 * (G::TILE >> 4));
    if (leader) {
#pragma unroll
      for (int part = 0; part < 2; ++part)
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t kb = kd + static_cast<uint64_t>((part * G::TILE + (k >> 2) * G::ATOM + (k & 3) * 32) >> 4);
          mma_ts(d, tmem + G::T_Q + (D / 2) * x + 8 * k, kb, kIdesc, (part | k) != 0 ? 1u : 0u);
        }
      mma_commit(bar(G::B_SFULL + buf));
      if (last_reader<kPair>(u, t, x)) mma_commit(bar(G::B_KEMPTY + sd));
    }
    __syncwarp();
  }
  // never leave with an MMA in flight
  if (leader) mma_commit(bar(G::B_DRAIN));
  __syncwarp();
  wait_bar(bar(G::B_DRAIN), 0, ctl, budget, a.status, false);
}

// O's updates.  V tiles MN-major: the 64-channel halves of N one column apart (leading
// offset), a k-step 16 keys = 2 KB.  P of keys 16 k .. sits in columns 8 k .. of its S
// buffer.
template <int D, bool kPair, bool kExactV>
__device__ __forceinline__ void value_mma(const PagedArgs& a, const Unit& u, uint32_t sbase, uint32_t tmem, Ctl* ctl) {
  using G = Geo<D, kPair>;
  const uint64_t budget = 2 * a.timeout_ns;
  auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
  constexpr uint32_t kIdesc = idesc_f16_f32(128, D, 0, 1);
  const bool leader = elect_one();
  const uint64_t vdesc = smem_desc(sbase + G::OFF_V, G::ATOM, 1024, kSwizzle128);
  const int N = u.T[0] + u.T[1];
  for (int n = 0; n < N; ++n) {
    const int t = step_key<kPair>(u, n), x = step_tile<kPair>(u, n), sd = t % ND, buf = n % G::NS;
    if (!wait_bar(bar(G::B_VFULL + sd), (t / ND) & 1, ctl, budget, a.status) ||
        !wait_bar(bar(G::B_PFULL + buf), (n / G::NS) & 1, ctl, budget, a.status))
      break;
    tc_fence_after();
    const uint32_t o = tmem + G::T_O + D * x, p = tmem + G::T_S + G::BN * buf;
    const uint64_t vd = vdesc + static_cast<uint64_t>(sd * 2 * (G::TILE >> 4));
    if (leader) {
#pragma unroll
      for (int part = 0; part < (kExactV ? 2 : 1); ++part)
#pragma unroll
        for (int k = 0; k < G::BN / 16; ++k)
          mma_ts(o, p + 8 * k, vd + static_cast<uint64_t>((part * G::TILE + k * 2048) >> 4), kIdesc, 1u);
      mma_commit(bar(G::B_PV + buf));
      if ((kPair ? n >> 1 : t) == (x ? u.T[1] : u.T[0]) - 1) mma_commit(bar(G::B_ODONE + x));
      if (last_reader<kPair>(u, t, x)) mma_commit(bar(G::B_VEMPTY + sd));
    }
    __syncwarp();
  }
  if (leader) mma_commit(bar(G::B_DRAIN + 1));
  __syncwarp();
  wait_bar(bar(G::B_DRAIN + 1), 0, ctl, budget, a.status, false);
}

// kPrefix: the keys of the prefix that the rows of packed token `tok` see; -1 where no sequence has it.
__device__ __forceinline__ int prefix_end(const PagedArgs& a, int tok, int keys) {
  if (tok < a.cu_q[0] || tok >= a.cu_q[a.seqs]) return -1;
  int lo = 0, hi = a.seqs;   // cu_q[lo] <= tok < cu_q[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.cu_q[mid] <= tok)
      lo = mid;
    else
      hi = mid;
  }
  const int64_t q0 = a.cu_q[lo], q1 = a.cu_q[lo + 1], kv = a.kv_lens[lo];
  return static_cast<int>(i64max(0, i64min(keys, a.causal ? i64min(kv, kv - (q1 - q0) + (tok - q0) + 1) : kv)));
}

template <typename QT, int D, bool kPair, int kMode>
__device__ __forceinline__ void softmax(const PagedArgs& a, const Unit& u, int x, uint32_t (&q)[D / 64][32],
                                        uint32_t sbase, uint32_t tmem, Ctl* ctl) {
  using G = Geo<D, kPair>;
  constexpr int BN = G::BN;
  const uint64_t budget = 2 * a.timeout_ns;
  const int lane_row = threadIdx.x & 127;
  const uint32_t lane_off = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;
  auto bar = [&](int i) { return sbase + G::OFF_BAR + 8u * i; };
  const int row = u.r0 + (kPair ? 0 : x * BM) + lane_row;
  const bool active = row < u.n_rows;
  const int tok = row / a.group;
  const int head = u.kvh * a.group + row - tok * a.group;
  const uint32_t t_o = tmem + lane_off + G::T_O + D * x;
  const int T = x ? u.T[1] : u.T[0];

  // ---- Q's row, as fp16 (bf16 scaled by a power of two), into TMEM
  float sl2 = a.scale_log2;
  {
    if (!std::is_same<QT, __half>::value) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 2; ++i) top = max(top, max(q[i / 32][i % 32] & 0x7FFFu, (q[i / 32][i % 32] >> 16) & 0x7FFFu));
      const int e = static_cast<int>(top >> 7);
      const int f = (e == 0 || e == 255) ? 0 : min(141 - e, 100);
      const float up = __int_as_float((127 + f) << 23);
      // not 0: the mask's -infinity times it has to stay (scores that small are 0 either way)
      sl2 = fmaxf(sl2 * __int_as_float((127 - f) << 23), FLT_MIN);
#pragma unroll
      for (int i = 0; i < D / 2; ++i) {
        const uint32_t v = q[i / 32][i % 32];
        q[i / 32][i % 32] = pack_half2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
      }
    }
#pragma unroll
    for (int h = 0; h < D / 64; ++h) tmem_st32(tmem + lane_off + G::T_Q + (D / 2) * x + 32 * h, q[h]);
#pragma unroll 1
    for (int h = 0; h < D / 32; ++h) {   // O = 0
      uint32_t z[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) z[i] = 0u;
      tmem_st32(t_o + 32 * h, z);
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar(G::B_Q));
  }

  float m_run = -INFINITY, l_run = 0.0f;
  const float2 sl22 = make_float2(sl2, sl2);
  // keys that this row, and that every row of the tile, sees
  int lim, clear;
  if (kMode == kPrefix) {   // each row by its sequence, `clear` of this warp's rows
    lim = active ? prefix_end(a, tok, u.sq.kv) : -1;
    clear = __reduce_min_sync(kFull, lim < 0 ? u.sq.kv : lim);
  } else {
    lim = a.causal ? min(u.sq.kv, u.sq.kv - u.sq.n_q + tok + 1) : u.sq.kv;
    clear = a.causal ? min(u.sq.kv, u.sq.kv - u.sq.n_q + (u.r0 + (kPair ? 0 : x * BM)) / a.group + 1) : u.sq.kv;
  }
  // kWindow: the first key of the window of this row, and of the tile's last
  const int low = max(lim, 0) - a.window;
  const int low_every = max(end_of<kMode>(a, u.sq, min(u.r0 + (kPair ? 0 : x * BM) + BM, u.n_rows) - 1), 0) - a.window;
#pragma unroll 1
  for (int t = 0; t < T; ++t) {
    const int n = step_of<kPair>(u, t, x), buf = n % G::NS;
    const uint32_t t_s = tmem + lane_off + G::T_S + BN * buf;
    if (!wait_bar(bar(G::B_SFULL + buf), (n / G::NS) & 1, ctl, budget, a.status)) return;
    tc_fence_after();
    uint32_t s[BN / 32][32];
#pragma unroll
    for (int i = 0; i < BN / 32; ++i) tmem_ld32(t_s + 32 * i, s[i]);
#pragma unroll
    for (int i = 0; i < BN / 32; ++i) tmem_wait_ld(s[i]);
    const int key0 = key_of<kMode, BN>(u.span, u.t0 + (kPair ? 2 * t + x : t));
    if (__builtin_expect(key0 + BN > clear || (kMode == kWindow && key0 < low_every && key0 + BN > a.sinks), 0)) {
      const int li = lim - key0;
#pragma unroll
      for (int j = 0; j < BN; ++j)
        if (j >= li || (kMode == kWindow && j < low - key0 && j >= a.sinks - key0)) s[j / 32][j % 32] = __float_as_uint(-INFINITY);
    }
    float pm[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) pm[i] = -INFINITY;
#pragma unroll
    for (int p = 0; p < BN / 2; ++p)
      pm[p & 7] = max3(pm[p & 7], __uint_as_float(s[p / 16][2 * p % 32]), __uint_as_float(s[p / 16][2 * p % 32 + 1]));
    const float mx = fmaxf(max3(pm[0], pm[1], pm[2]), max3(pm[3], pm[4], max3(pm[5], pm[6], pm[7]))) * sl2;
    float alpha = 1.0f;
    const bool move = mx > m_run + kLazy;   // the reference moves
    if (move) {
      alpha = m_run == -INFINITY ? 0.0f : ex2_approx(m_run - mx);
      m_run = mx;
    }
    const float ref = m_run == -INFINITY ? 0.0f : m_run - kLift;
    const float2 nm2 = make_float2(-ref, -ref);
    float2 rs[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) rs[i] = make_float2(0.0f, 0.0f);
    uint32_t p[BN / 2];
#pragma unroll
    for (int i = 0; i < BN / 2; ++i) {
      const float2 sv = make_float2(__uint_as_float(s[i / 16][2 * i % 32]), __uint_as_float(s[i / 16][2 * i % 32 + 1]));
      const float2 e = __ffma2_rn(sv, sl22, nm2);
      const float2 w = make_float2(ex2_approx(e.x), ex2_approx(e.y));
      rs[i & 3] = __fadd2_rn(rs[i & 3], w);
      p[i] = pack_half2(w.x, w.y);
    }
    tmem_st32(t_s, *reinterpret_cast<const uint32_t(*)[32]>(&p[0]));
    if (BN == 96) tmem_st16(t_s + 32, &p[BN / 2 - 16]);
    if (t > 0 && __any_sync(kFull, move)) {
      // O is free once this tile's update before, of step p, has completed.  p is n - 2
      // (or n - 1), the buffer's earlier use p - G::NS has completed (scores n were
      // issued behind it) and its next one waits for this step, so the phase is p's.
      const int p = step_of<kPair>(u, t - 1, x);
      if (!wait_bar(bar(G::B_PV + p % G::NS), (p / G::NS) & 1, ctl, budget, a.status)) return;
      tc_fence_after();
#pragma unroll 1
      for (int h = 0; h < D / 32; ++h) {
        uint32_t o[32];
        tmem_ld32(t_o + 32 * h, o);
        tmem_wait_ld(o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
        tmem_st32(t_o + 32 * h, o);
      }
    }
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(bar(G::B_PFULL + buf));
    const float2 r = __fadd2_rn(__fadd2_rn(rs[0], rs[1]), __fadd2_rn(rs[2], rs[3]));
    // the largest weight counts as it was rounded, so that a row dominated by
    // one key divides by exactly that key's weight
    float fix = 0.0f;
    if (mx != -INFINITY) {
      const float w = ex2_approx(mx - ref);
      fix = __half2float(__float2half_rn(w)) - w;
    }
    l_run = fmaf(l_run, alpha, (r.x + r.y) + fix);
  }
  if (T > 0) {
    if (!wait_bar(bar(G::B_ODONE + x), 0, ctl, budget, a.status)) return;
    tc_fence_after();
  }
  if (kPair || kMode == kPrefix || a.shares) {
    // the share's partial state of the tile; one without key tiles is not read
    if (T == 0) return;
    const int64_t at = (static_cast<int64_t>(blockIdx.x) * 2 + x) * BM + lane_row;
    if (active) {
      float2* ml = reinterpret_cast<float2*>(a.part + a.part_ml);
      ml[at] = make_float2(m_run, l_run);
    }
    uint4* dst = reinterpret_cast<uint4*>(a.part + at * D);
    const bool wide = a.wide & kWidePart;
#pragma unroll 1
    for (int h = 0; h < D / 32; ++h) {
      uint32_t o[32];
      tmem_ld32(t_o + 32 * h, o);
      tmem_wait_ld(o);
      if (active)
#pragma unroll
        for (int i = 0; i < 4; ++i) store_row8(dst + 8 * h + 2 * i, wide, o + 8 * i);
    }
    return;
  }
  const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<QT*>(a.out) + ((u.sq.q0 + tok) * a.heads + head) * D);
  const bool wide = a.wide & kWideOut;
#pragma unroll 1
  for (int h = 0; h < D / 32; ++h) {
    uint32_t o[32];
    tmem_ld32(t_o + 32 * h, o);
    tmem_wait_ld(o);
    if (active) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float y0 = __uint_as_float(o[16 * i + 2 * k]) * inv, y1 = __uint_as_float(o[16 * i + 2 * k + 1]) * inv;
          if (std::is_same<QT, __half>::value) {
            y[k] = pack_half2(y0, y1);
          } else {
            const __nv_bfloat162 v = __floats2bfloat162_rn(y0, y1);
            y[k] = *reinterpret_cast<const uint32_t*>(&v);
          }
        }
        store_row8(dst + 4 * h + 2 * i, wide, y);
      }
    }
  }
}

// The whole row of Q of a softmax thread, all loads in flight together, before anything else
// of the CTA's start has to be waited for.
template <typename QT, int D, bool kPair>
__device__ __forceinline__ void load_q(const PagedArgs& a, const Unit& u, int x, uint32_t (&q)[D / 64][32]) {
  const int row = u.r0 + (kPair ? 0 : x * BM) + (threadIdx.x & 127);
  const int tok = row / a.group;
  const uint4* src = reinterpret_cast<const uint4*>(static_cast<const QT*>(a.q) + (u.sq.q0 + tok) * a.q_stride +
                                                    static_cast<int64_t>(u.kvh * a.group + row - tok * a.group) * D);
  const bool wide = a.wide & kWideQ;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t* v = &q[i / 4][8 * i % 32];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0u;
    if (row < u.n_rows) load_row8(src + 2 * i, wide, v);
  }
}

template <typename QT, int D, bool kPair, int kMode>
__global__ void __launch_bounds__(Geo<D, kPair>::kThreads, 1) paged_tiles_kernel(const PagedArgs a) {
  using G = Geo<D, kPair>;
  constexpr bool kExactV = std::is_same<QT, __half>::value;
  extern __shared__ uint8_t smem_raw[];
  pdl_launch_dependents();
  pdl_wait();
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + G::OFF_CTL);
  const int warp = threadIdx.x >> 5, wg = warp >> 2;
  if (warp == 0) {
    const int lane = threadIdx.x & 31;
    if (kPair || kMode == kPrefix || a.shares)
      locate<D, kPair, kMode, true>(a, blockIdx.x, plan_shares<D, kPair, kMode>(a, lane), ctl, lane);
    else
      locate<D, kPair, kMode, false>(a, blockIdx.x, 0x3FFFFFFF, ctl, lane);
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < G::NBAR; ++i) {
      uint32_t count = 1;
      if (i == G::B_Q) count = 256;                                      // softmax threads
      if (i >= G::B_RAWEMPTY && i < G::B_RAWEMPTY + G::NR) count = 32 * (G::kKDq + G::kVDq);   // dequantising threads
      if (i >= G::B_KFULL && i < G::B_KFULL + ND) count = 32 * G::kKDq;
      if (i >= G::B_VFULL && i < G::B_VFULL + ND) count = 32 * G::kVDq;
      if (i >= G::B_PFULL && i < G::B_PFULL + G::NS) count = 128;           // softmax threads of a tile
      mbar_init(sbase + G::OFF_BAR + 8u * i, count);
    }
    ctl->abort = 0u;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(sbase + G::OFF_CTL, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const int b = ctl->b;
  Unit u;
  if (b >= 0) u = make_unit<D, kPair, kMode>(a, ctl, ctl->share);
  // uniform over the CTA: more blocks than work, or an empty share
  if (b < 0 || ((kPair || kMode == kPrefix || a.shares) && u.T[0] + u.T[1] == 0)) {
    if (warp == 13) tmem_dealloc(tmem, 512);
    return;
  }
  if (wg < 2) {
    uint32_t q[D / 64][32];
    load_q<QT, D, kPair>(a, u, wg, q);
    reg_alloc<G::REG_S>();
    softmax<QT, D, kPair, kMode>(a, u, wg, q, sbase, tmem, ctl);
  } else {
    reg_dealloc<G::REG_O>();
    if (warp == 12) {
      producer<D, kPair, kMode>(a, u, b, sbase, ctl);
    } else if (warp == 13) {
      score_mma<D, kPair>(a, u, sbase, tmem, ctl);
    } else if (warp == 14) {
      value_mma<D, kPair, kExactV>(a, u, sbase, tmem, ctl);
    } else {
      const int w = warp < 12 ? warp - 8 : warp - 11;
      if (w < G::kKDq)
        dequant<D, kPair, kMode, false, true>(a, u, w, smem, sbase, ctl);
      else if (w < G::kKDq + G::kVDq)
        dequant<D, kPair, kMode, true, kExactV>(a, u, w - G::kKDq, smem, sbase, ctl);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the shares of a unit's rows, a warp per row, in order; behind a prefix also the row's state over its own keys.
template <typename QT, int D, bool kPair, int kMode>
__global__ void __launch_bounds__(256) paged_tiles_join_kernel(const PagedArgs a) {
  __shared__ Ctl shared_ctl;
  __shared__ float sums[kMode == kPrefix ? 8 : 1][D + 1];
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Ctl own_ctl;   // kPrefix: every thread's, in registers
  Ctl& ctl = kMode == kPrefix ? own_ctl : shared_ctl;
  if (kMode == kPrefix) {
    locate_prefix<D, kPair>(a, blockIdx.x, &ctl);
  } else {
    if (warp == 0) locate<D, kPair, kMode, false>(a, blockIdx.x, plan_shares<D, kPair, kMode>(a, lane), &ctl, lane);
    __syncthreads();
  }
  if (ctl.b < 0) return;
  const Unit u = make_unit<D, kPair, kMode>(a, &ctl, 0);
  // kPrefix with few rows: a block per row, its warps deal the states out among themselves
  const bool one = kMode == kPrefix && a.join_rows == 1;
  const int in_unit = one ? blockIdx.y : blockIdx.y * 8 + warp;
  const int row = u.r0 + in_unit;
  if (row >= u.n_rows) return;
  const int tok = row / a.group;
  const int64_t out_row = (u.sq.q0 + tok) * a.heads + u.kvh * a.group + row - tok * a.group;
  // kPrefix: the row's state over its own keys, on its way before the prefix's length is needed
  float own = 0.0f, own_y[D / 32];
  bool in_seq = true;
  if (kMode == kPrefix) {
    in_seq = tok >= a.cu_q[0] && tok < a.cu_q[a.seqs];
    own = a.state[a.total_q * a.heads * D + out_row];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) own_y[i] = a.state[out_row * D + 32 * i + lane];
  }
  const int tiles = tiles_of<D, kPair, kMode>(a, u.sq, u.span, u.r0 + in_unit / BM * BM, u.n_rows);
  // states of this row's tile: one for each share with key tiles of it (tile in_unit / 128 of
  // the CTA's two); in pairs two, but one for a share of a single key tile
  const int full = (tiles + u.per - 1) / u.per;
  if (static_cast<int64_t>(ctl.first) + full > a.ctas) {   // lengths beyond the call's bounds
    record_index(a.status);
    return;
  }
  const bool two = kPair && u.per > 1;
  const int n = two && full > 0 ? 2 * full - (tiles - (full - 1) * u.per < 2 ? 1 : 0) : full;
  const int64_t step = two ? BM : 2 * BM;
  const int64_t at0 = static_cast<int64_t>(ctl.first) * 2 * BM + in_unit;
  const float2* ml = reinterpret_cast<const float2*>(a.part + a.part_ml);
  float top = -INFINITY;
  float l = 0.0f, y[D / 32] = {};
  if (kMode == kPlain) {
    for (int z = 0; z < n; ++z) top = fmaxf(top, ml[at0 + z * step].x);
#pragma unroll 4
    for (int z = 0; z < n; ++z) {
      const int64_t at = at0 + z * step;
      const float2 v = ml[at];
      const float w = v.x == -INFINITY ? 0.0f : (v.x == top ? 1.0f : ex2_approx(v.x - top));
      l = fmaf(w, v.y, l);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[i] = fmaf(w, a.part[at * D + 32 * i + lane], y[i]);
    }
  } else {
    // the states' references and sums a lane each, then their values, eight in flight
    if (!in_seq) return;   // a row of no sequence stays as it is
#pragma unroll 4
    for (int z = lane; z < n; z += 32) top = fmaxf(top, ml[at0 + z * step].x);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    if (kMode == kPrefix) {
      // the shares' weights carry 2^kLift: their logarithms are that much above the own keys'
      static_assert(kLift == 7.0f, "2^7");
      top = fmaxf(top, own);
      l = one && warp > 0 ? 0.0f : state_weight(own, 1.0f, top) * 128.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[i] = l == 0.0f ? 0.0f : l * own_y[i];
    }
    const int per = one ? (n + 7) / 8 : n, last = one ? min(n, (warp + 1) * per) : n;   // this warp's states
    for (int z0 = one ? warp * per : 0; z0 < last; z0 += 32) {
      const float2 v = z0 + lane < last ? ml[at0 + (z0 + lane) * step] : make_float2(-INFINITY, 0.0f);
      const float w_mine = state_weight(v.x, v.y, top);
      float s = w_mine * v.y;
#pragma unroll
      for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(kFull, s, o);
      l += s;
      const float* part = a.part + (at0 + z0 * step) * D + lane;
      const int here = min(32, last - z0);
#pragma unroll 1
      for (int z = 0; z < here; z += 8) {
        float x[8][D / 32];
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) x[k][i] = z + k < here ? part[(z + k) * step * D + 32 * i] : 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float w = __shfl_sync(kFull, w_mine, (z + k) & 31);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) y[i] = z + k < here ? fmaf(w, x[k][i], y[i]) : y[i];
        }
      }
    }
    if (one) {   // the warps' sums, in order
#pragma unroll
      for (int i = 0; i < D / 32; ++i) sums[warp][32 * i + lane] = y[i];
      if (lane == 0) sums[warp][D] = l;
      __syncthreads();
      if (warp > 0) return;
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        l += sums[k][D];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) y[i] += sums[k][32 * i + lane];
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (kMode == kOwn) {
    if (lane == 0) a.state[a.total_q * a.heads * D + out_row] = state_log(top - kLift, l);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) a.state[out_row * D + 32 * i + lane] = y[i] * inv;
    return;
  }
  QT* dst = static_cast<QT*>(a.out) + out_row * D;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    if (std::is_same<QT, __half>::value)
      reinterpret_cast<__half*>(dst)[32 * i + lane] = __float2half_rn(y[i] * inv);
    else
      reinterpret_cast<__nv_bfloat16*>(dst)[32 * i + lane] = __float2bfloat16_rn(y[i] * inv);
  }
}

template <typename QT, int D, bool kPair, int kMode>
cudaError_t launch_tiles(const PagedArgs& a, const TilesPlan& plan, cudaStream_t stream) {
  using G = Geo<D, kPair>;
  auto kernel = paged_tiles_kernel<QT, D, kPair, kMode>;
  static thread_local int configured_device = -1;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device != dev) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e != cudaSuccess) return e;
    // the register split draws on the launch's allocation: with fewer registers an
    // increase could wait for ever
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * G::kThreads < 2 * 128 * G::REG_S + (G::kThreads - 256) * G::REG_O || fa.maxThreadsPerBlock < G::kThreads)
      return cudaErrorInvalidConfiguration;
    configured_device = dev;
  }
  e = launch_kernel(kernel, dim3(static_cast<unsigned>(plan.ctas)), dim3(G::kThreads), G::SMEM, stream, a);
  if (e != cudaSuccess || !(kPair || kMode == kPrefix || a.shares)) return e;
  const unsigned rows = kMode == kPrefix ? a.join_rows : 8;
  return launch_kernel(paged_tiles_join_kernel<QT, D, kPair, kMode>, dim3(static_cast<unsigned>(plan.slots), G::ROWS / rows), dim3(256), 0, stream, a);
}

template <bool kPair, int kMode>
cudaError_t launch_tiles_mode(const PagedArgs& a, int32_t dtype, int32_t head_dim, const TilesPlan& plan,
                              cudaStream_t stream) {
  if (plan.ctas > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (dtype == kF16)
    return head_dim == 64 ? launch_tiles<__half, 64, kPair, kMode>(a, plan, stream)
                          : launch_tiles<__half, 128, kPair, kMode>(a, plan, stream);
  return head_dim == 64 ? launch_tiles<__nv_bfloat16, 64, kPair, kMode>(a, plan, stream)
                        : launch_tiles<__nv_bfloat16, 128, kPair, kMode>(a, plan, stream);
}

}  // namespace
}  // namespace q8a
