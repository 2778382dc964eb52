// qrows.cuh — rows on their way into the paged 4-bit cache: 16 elements become
// one scale and 16 codes (number format: see qcache_store.cu).
#pragma once
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

namespace kascade {

__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
__device__ __forceinline__ float e4m3_value(uint32_t b) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(b & 0xffu)));
  float f;
  asm("{.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.f32.f16 %0, lo;}" : "=f"(f) : "r"(h));
  return f;
}
// eight e2m1 codes, the first in the lowest four bits
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// x / s such that rounding it to the 1 to 4 bits of e2m1 or e4m3 is rounding
// the exact quotient. One Newton correction of x * (1/s) makes q the quotient
// to its last bit, and exact where the quotient has few bits, as every tie
// has. A bf16 x (8 bits) over an s of at most 4 bits is otherwise at least 2^-13
// away from a tie, so that is all it needs (EXACT false). The quotient of an
// fp32 x may lie within a last place of a tie: where the division leaves a
// remainder, q is rounded to odd (cut towards zero, its last bit set), which keeps
// it on the exact quotient's side of every number of fewer bits.
template <bool EXACT>
__device__ __forceinline__ float round_quotient(float x, float s, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, s, x), inv, q);
  if (EXACT) {
    const float r = fmaf(-q, s, x);
    // a quotient that passed the exact one: r and q differ in sign
    const int u = __float_as_int(q), cut = (__float_as_int(r) ^ u) >> 31;
    if (r != 0.f) q = __int_as_float((u + cut) | 1);
  }
  return q;
}

// 16 elements as stored: raw words, the largest magnitude (NaN if there is one).
template <typename T>
struct Row16;
template <>
struct Row16<float> {
  float x[16];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = __ldg(static_cast<const float4*>(p) + i);
      x[4 * i] = f.x;
      x[4 * i + 1] = f.y;
      x[4 * i + 2] = f.z;
      x[4 * i + 3] = f.w;
    }
  }
  __device__ __forceinline__ float amax() const {
    uint32_t m = 0u;   // magnitudes order as their bits do, NaNs above infinity
#pragma unroll
    for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
    return __uint_as_float(m);
  }
  __device__ __forceinline__ float get(int i) const { return x[i]; }
};
template <>
struct Row16<__nv_bfloat16> {
  uint32_t w[8];
  __device__ __forceinline__ void load(const void* p) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = __ldg(static_cast<const uint4*>(p) + i);
      w[4 * i] = u.x;
      w[4 * i + 1] = u.y;
      w[4 * i + 2] = u.z;
      w[4 * i + 3] = u.w;
    }
  }
  __device__ __forceinline__ float amax() const {
    uint32_t m = w[0] & 0x7fff7fffu;   // two magnitudes side by side
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    return __uint_as_float(max(m << 16, m & 0xffff0000u));
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float((i & 1) ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
};
// Quantises one piece into its codes and scale byte; unit: 1 / the cache's scale.
template <typename T>
__device__ __forceinline__ void put16(const Row16<T>& x, float unit, uint8_t* codes_at,
                                      uint8_t* scale_at) {
  constexpr bool kExact = sizeof(T) == 4;
  // the cache's own scale is a power of two: it goes into the block's scale
  float amax = x.amax();
  const bool nan = amax != amax;
  amax = fminf(amax * unit, 2688.f);   // what is above saturates, infinities among it
  const uint32_t sb = nan ? 0x7fu : e4m3_of(round_quotient<kExact>(amax, 6.f, 1.f / 6.f));
  uint32_t w[2] = {0u, 0u};
  if ((sb & 0x7fu) != 0u && !nan) {   // scale 0: the block's elements all round to 0
    const float s = e4m3_value(sb) / unit, inv = 1.f / s;
    auto codes = [&](auto element) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = round_quotient<kExact>(element(8 * h + e), s, inv);
        w[h] = e2m1x8(y);
      }
    };
    if (amax < 2688.f) {
      codes([&](int i) { return x.get(i); });
    } else {   // an infinity's quotient is NaN: what passes 6 s is cut first
      const float most = 8.f * s;
      codes([&](int i) { return fminf(fmaxf(x.get(i), -most), most); });
    }
  }
  *reinterpret_cast<uint2*>(codes_at) = make_uint2(w[0], w[1]);
  *scale_at = static_cast<uint8_t>(sb);
}

}  // namespace kascade
