// qmath.cuh — constants and element arithmetic shared by the attention kernels
// over the paged 4-bit cache.
#pragma once
#include <cuda_runtime.h>
#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

namespace kascade {

#define kNegInf (-CUDART_INF_F)
// Running maximum before the first key: below every score, and finite, so
// that neither exponents nor joins need a case for it.
constexpr float kNoKey = -3.0e38f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPShift = 14;          // weights are held as 2^14 p
// The running maximum is a reference, not the maximum itself: it is raised once
// a score passes it by more than this (weights then reach 2^15.75, within fp16).
constexpr float kSlack = 1.75f;
// kPShift - m for the weights' exponents. From |m| = 2^25 on 14 is less than a few steps
// of m's type, and the difference to the nearest could make the weight at m 2^16, which
// fp16 does not hold; there it is rounded down (weights at m are then 2^0 to 2^14).
__device__ __forceinline__ float below_shift(float m) {
  const float x = kPShift - m;
  return x + m > kPShift + kSlack ? __fsub_rd(static_cast<float>(kPShift), m) : x;
}
constexpr int kQExp = 12;            // q's largest element is scaled to [2^12, 2^13)
// the four bytes of w, each two e2m1 codes, as pairs of fp16 (low half first)
__device__ __forceinline__ void cvt_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t cvt_e4m3x2(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b)));
  return h;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// low nibbles of a, high nibbles of b
__device__ __forceinline__ uint32_t nibbles(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xCA;" : "=r"(d) : "r"(0x0f0f0f0fu), "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// 2^x, to 2^-22; results below 2^-126 are zero
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float f16_rounded(float x) { return __half2float(__float2half_rn(x)); }

// Four output dims of some keys: running maximum (log2 units), sum of the weights
// and of weight * value.
struct Joined {
  float m, l;
  float4 o;
};
// x += the N parts y (their weights do not wait for one another)
template <int N>
__device__ __forceinline__ void join_into(Joined& x, const Joined (&y)[N]) {
  float M = x.m;
#pragma unroll
  for (int k = 0; k < N; ++k) M = fmaxf(M, y[k].m);
  // a part without keys has m = kNoKey and l = o = 0 (or l NaN, which stays)
  const float wx = ex2(x.m - M);
  x.m = M;
  x.l *= wx;
  x.o.x *= wx;
  x.o.y *= wx;
  x.o.z *= wx;
  x.o.w *= wx;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float w = ex2(y[k].m - M);
    x.l = fmaf(w, y[k].l, x.l);
    x.o.x = fmaf(w, y[k].o.x, x.o.x);
    x.o.y = fmaf(w, y[k].o.y, x.o.y);
    x.o.z = fmaf(w, y[k].o.z, x.o.z);
    x.o.w = fmaf(w, y[k].o.w, x.o.w);
  }
}

}  // namespace kascade
