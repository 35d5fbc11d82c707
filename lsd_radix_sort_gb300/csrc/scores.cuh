// Device helpers shared by the losses: score types, base-2 exponentials,
// warp sums and maxima.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"

namespace lsdrs {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// One score type: its raw word in memory and its conversions.
template <int TYPE>
struct Score;
template <>
struct Score<RS_SCORE_F16> {
  using Raw = uint16_t;
  static __device__ __forceinline__ float load(Raw r) { return __half2float(__ushort_as_half(r)); }
  static __device__ __forceinline__ Raw store(float v) {
    return __half_as_ushort(__float2half_rn(v));
  }
};
template <>
struct Score<RS_SCORE_BF16> {
  using Raw = uint16_t;
  static __device__ __forceinline__ float load(Raw r) {
    return __uint_as_float(static_cast<uint32_t>(r) << 16);
  }
  static __device__ __forceinline__ Raw store(float v) {
    return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
};
template <>
struct Score<RS_SCORE_F32> {
  using Raw = uint32_t;
  static __device__ __forceinline__ float load(Raw r) { return __uint_as_float(r); }
  static __device__ __forceinline__ Raw store(float v) { return __float_as_uint(v); }
};

// A score of a type known at run time (short lists only).
__device__ __forceinline__ float load_score(const void* p, int type, int64_t i) {
  if (type == RS_SCORE_F32) return static_cast<const float*>(p)[i];
  const uint16_t r = static_cast<const uint16_t*>(p)[i];
  return type == RS_SCORE_F16 ? Score<RS_SCORE_F16>::load(r) : Score<RS_SCORE_BF16>::load(r);
}

__device__ __forceinline__ int64_t load_index(const void* p, int bytes, int64_t i) {
  return bytes == 8 ? static_cast<const int64_t*>(p)[i] : static_cast<const int32_t*>(p)[i];
}

// 2^x; 0 for -inf, NaN for NaN.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}

// A softmax in progress: the largest score m and sum = sum exp((x - m) / t).
// Scores of -inf leave it as it is, so m = -inf and sum = 0 until the first
// other one; a NaN or +inf score makes the sum NaN for good.
struct Softmax {
  float m, sum;
};

// The point that exponents are taken from: m, or 0 while there is no score
// (so that -inf - m stays -inf).
__device__ __forceinline__ float origin(float m) { return m == -INFINITY ? 0.0f : m; }

// Both halves of a row: scale2 = log2(e) / temperature.
__device__ __forceinline__ Softmax join(Softmax a, Softmax b, float scale2) {
  const float m = fmaxf(a.m, b.m), o = origin(m);
  return {m, a.sum * exp2_approx((a.m - o) * scale2) + b.sum * exp2_approx((b.m - o) * scale2)};
}

__device__ __forceinline__ Softmax warp_join(Softmax v, float scale2) {
  const float m = warp_max(v.m);
  return {m, warp_sum(v.sum * exp2_approx((v.m - origin(m)) * scale2))};
}

}  // namespace lsdrs
