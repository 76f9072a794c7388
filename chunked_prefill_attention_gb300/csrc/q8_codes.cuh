// q8_codes.cuh -- the arithmetic of Q8_0 codes: codes to fp16, for the paged attention, and
// values to codes, for the quantising ones.
// A unit that includes it must not be built with fast-math (IEEE rounding).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

namespace q8a {

__device__ __forceinline__ uint32_t h2u(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) { return h2u(__floats2half2_rn(lo, hi)); }

// Four signed int8 codes -> two half2 (exact): flip the sign bit to get
// u = q + 128 in [0, 255], place u under the fp16 exponent of 1024 (0x64uu is
// 1024 + u exactly) and subtract 1152.
__device__ __forceinline__ void codes_to_half2(uint32_t w, __half2& lo, __half2& hi) {
  const uint32_t u = w ^ 0x80808080u;
  const uint32_t a = __byte_perm(u, 0x64646464u, 0x5140);
  const uint32_t b = __byte_perm(u, 0x64646464u, 0x7362);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));   // 1152
  lo = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  hi = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
}

// Two codes from two values, each as the low byte of a word: q = RN(x / d), rounded half away from
// zero and clamped to [-127, 127], in packed fp32x2.  The quotient is corrected (Markstein, IBM J.
// Res. Dev. 34(1), 1990): y = RN(1 / d) comes in, q0 = RN(x y) is within an ulp of x / d, the residual
// r = x - q0 d is exact as one fma, and RN(q0 + r y) is RN(x / d).  The other steps are exact in fp32:
//   floor(RZ(a + 0.5)) is a rounded half away from zero for 0 <= a < 2^23
//     (a + 0.5 is exact for a >= 0.5; below, round-toward-zero keeps it < 1);
//   clamping t to 127.5 first clamps floor(t) to 127 (and catches a >= 2^23);
//   RZ(t + 2^23) - 2^23 is floor(t) for 0.5 <= t < 2^23;
//   RN(s + 1.5 * 2^23) holds the integer s (|s| <= 127) in its low byte, in
//     two's complement.
// With y = 0 and nd = 0 (scale 0, or +inf in fp16 when amax exceeds
// 65504 * 127, where x / inf = 0) both codes are 0.
__device__ __forceinline__ uint2 code_pair(float2 x, float2 nd2, float2 y2) {
  const float2 q0 = __fmul2_rn(x, y2);
  const float2 r = __ffma2_rn(q0, nd2, x);
  const float2 qq = __ffma2_rn(r, y2, q0);
  float2 t = __fadd2_rz(make_float2(fabsf(qq.x), fabsf(qq.y)), make_float2(0.5f, 0.5f));
  t = make_float2(fminf(t.x, 127.5f), fminf(t.y, 127.5f));
  const float2 m = __fadd2_rz(t, make_float2(8388608.0f, 8388608.0f));
  const float2 f = __fadd2_rn(m, make_float2(-8388608.0f, -8388608.0f));
  const float2 u = __fadd2_rn(make_float2(copysignf(f.x, qq.x), copysignf(f.y, qq.y)),
                              make_float2(12582912.0f, 12582912.0f));
  return make_uint2(__float_as_uint(u.x), __float_as_uint(u.y));
}

// One Q8_0 block from 32 values: the fp16 scale d = fp16(amax / 127) and the
// codes as eight little-endian words.  A zero scale, or one that overflows
// fp16, gives codes 0.
__device__ __forceinline__ uint32_t q8_block(const float (&v)[32], uint32_t (&w)[8]) {
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 32; i += 2) {   // three-input maxima
    float& a = m[i / 2 & 3];
    asm("max.f32 %0, %1, %2, %3;" : "=f"(a) : "f"(a), "f"(fabsf(v[i])), "f"(fabsf(v[i + 1])));
  }
  const float a = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
  const __half d16 = __float2half_rn(__fdiv_rn(a, 127.0f));
  const float d = __half2float(d16);
  const bool finite_nonzero = d > 0.0f && d <= 65504.0f;
  const float y = finite_nonzero ? __frcp_rn(d) : 0.0f;
  const float nd = finite_nonzero ? -d : 0.0f;
  const float2 y2 = make_float2(y, y), nd2 = make_float2(nd, nd);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint2 c01 = code_pair(make_float2(v[4 * k], v[4 * k + 1]), nd2, y2);
    const uint2 c23 = code_pair(make_float2(v[4 * k + 2], v[4 * k + 3]), nd2, y2);
    w[k] = __byte_perm(__byte_perm(c01.x, c01.y, 0x0040), __byte_perm(c23.x, c23.y, 0x0040), 0x5410);
  }
  return __half_as_ushort(d16);
}

// Block `bb` of a head row (d and codes as q8_block gives them) into `row`,
// which is 4-byte aligned: d at 34 * bb, codes behind it.  An even block starts
// 4-byte aligned (codes at 2 mod 4), an odd one 2 mod 4 (codes 4-byte aligned).
__device__ __forceinline__ void q8_put_block(uint8_t* row, int bb, uint32_t d, const uint32_t (&w)[8]) {
  uint8_t* at = row + 34 * bb;
  if ((bb & 1) == 0) {
    uint32_t* p = reinterpret_cast<uint32_t*>(at);
    p[0] = d | (w[0] << 16);
#pragma unroll
    for (int k = 0; k < 7; ++k) p[1 + k] = __funnelshift_r(w[k], w[k + 1], 16);
    *reinterpret_cast<uint16_t*>(at + 32) = static_cast<uint16_t>(w[7] >> 16);
  } else {
    *reinterpret_cast<uint16_t*>(at) = static_cast<uint16_t>(d);
    uint32_t* p = reinterpret_cast<uint32_t*>(at + 2);
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = w[k];
  }
}

}  // namespace q8a
