// rotary.cuh -- the rotation of channel pairs by their positions' angles, and the element types of packed
// tensors, for the kernels that rotate.
//
// Rotary positions.  A pair (a, b) of channels with angle t = position * f is
// turned to (a cos t - b sin t, a sin t + b cos t).  A far position times f
// loses the angle in fp32 (2^20 positions leave 2^-4 rad), so the angle is
// formed in turns, in 64-bit fixed point: F = frac(f / 2 pi) 2^64 from the fp64
// table, position * F modulo 2^64 (integer arithmetic drops the whole turns
// exactly), and the top bits as a fraction of half a turn in [-1, 1) for
// sincospif.  The angle is off by 2^-52 of itself (the division by 2 pi) and
// by 2^-25 half turns from the conversion to fp32.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace q8a {

// Turns per position of f radians, as a fraction of 2^64.
__device__ __forceinline__ uint64_t turn_step(double f) {
  double t = f * 0.15915494309189535;   // 1 / (2 pi)
  t -= floor(t);                        // [0, 1)
  return __double2ull_rn(t * 18446744073709551616.0);
}
// (cos, sin) of position * f radians.
__device__ __forceinline__ float2 rotation(int64_t position, uint64_t step, float mscale, float sign) {
  const int64_t turns = static_cast<int64_t>(static_cast<uint64_t>(position) * step);
  float s, c;
  sincospif(static_cast<float>(turns) * 1.0842021724855044e-19f, &s, &c);   // 2^-63
  return make_float2(c * mscale, s * mscale * sign);
}

// (a cos - b sin, a sin + b cos).  Packed pairs (fma.f32x2) took the appending kernel from
// 64 registers to 102 and from 60 to 91 us.
__device__ __forceinline__ float2 turn_pair(float a, float b, float2 q) {
  return make_float2(fmaf(a, q.x, -b * q.y), fmaf(a, q.y, b * q.x));
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float x) { return x; }
  static __device__ __forceinline__ float put(float x) { return x; }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
  static __device__ __forceinline__ __half put(float x) { return __float2half_rn(x); }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
  static __device__ __forceinline__ __nv_bfloat16 put(float x) { return __float2bfloat16_rn(x); }
};

// N consecutive elements as one access (N * sizeof(T) is 16 bytes, or N = 1).
template <typename T, int N>
struct alignas(N * sizeof(T)) Vec {
  T e[N];
};

}  // namespace q8a
