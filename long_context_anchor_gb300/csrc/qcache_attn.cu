// qcache_attn.cu — decode attention over the paged 4-bit key/value cache
// (layout in qcache.h): one query per sequence, ragged lengths.
//
//   k_qdecode_dense   all cached keys of every sequence (and the scaled logits
//                     an anchor layer ranks)
//   k_qdecode_reuse   only the saved sets' keys
//
// Both run the G query heads of a KV head together, 16 keys at a time, on
// mma.sync m16n8k16 with fp16 operands and fp32 sums. A stored element is
// code * scale with 2 + 4 significant bits, at most 2688 and a multiple of
// 2^-10, so it is exact in fp16. q is scaled by a power of two per head so that
// its largest element lies in [2^12, 2^13): a bf16 q is then exact in fp16
// down to 2^-26 of that element, an fp32 q is the sum of two fp16 terms (22 bits). The softmax weights
// are kept as 2^14 p, so that a weight down to 2^-38 of the row's largest one
// still counts; for fp32 outputs they too are a sum of two fp16 terms.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "common.cuh"
#include "qcache.h"

namespace kascade {
namespace {

#define kNegInf (-CUDART_INF_F)
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPShift = 14;          // weights are held as 2^14 p
constexpr int kQExp = 12;            // q's largest element is scaled to [2^12, 2^13)
constexpr int kNW = 8;               // warps per CTA (and at most 8 heads per KV head)

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
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

// Running state of one warp over the keys of one (sequence, KV head). Thread
// (gid = lane/4, c4 = lane%4) owns heads 2 c4, 2 c4 + 1 and output dims
// gid * D/8 .. + D/8 of both: o[i] = (dim 2i, head 2c4), (2i, 2c4+1),
// (2i + 1, 2c4), (2i + 1, 2c4 + 1).
// mu = m - 14 (what the exponents subtract), finite while m is still -inf.
template <int D>
struct QState {
  float m[2], mu[2], l[2];
  float o[D / 16][4];
};

template <int D>
__device__ __forceinline__ void qstate_init(QState<D>& st) {
  st.m[0] = st.m[1] = kNegInf;
  st.mu[0] = st.mu[1] = -kPShift;
  st.l[0] = st.l[1] = 0.f;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) st.o[i][0] = st.o[i][1] = st.o[i][2] = st.o[i][3] = 0.f;
}

// The query fragments (B operand) of head gid of the group: lane c4 holds dims
// c4 * D/4 .. + D/4, four of them per MMA, so that a key row's codes are the A
// operand in stored order. mult[i]: what turns the raw product of head
// 2 c4 + i into the scaled logit.
template <int D, int TERMS>
struct QFrag {
  uint32_t f[TERMS][D / 16][2];
  float mult[2];
};

// Head gid's dims c4 * D/4 .. + D/4 as they are in memory (zeros for no head).
template <int D, int TERMS>
__device__ __forceinline__ void load_q(const QDecodeArgs& a, int b, int g, float (&x)[D / 4]) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
  const bool ok = gid < a.G;
  const size_t row = ok ? static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + gid] : 0;
  if (TERMS == 2) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + row * D +
                                                      c4 * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const float4 v = ok ? __ldg(p + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[4 * i] = v.x;
      x[4 * i + 1] = v.y;
      x[4 * i + 2] = v.z;
      x[4 * i + 3] = v.w;
    }
  } else {
    const uint2* p = reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.q) +
                                                    row * D + c4 * (D / 4));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint2 v = ok ? __ldg(p + i) : make_uint2(0u, 0u);
      x[4 * i] = __uint_as_float(v.x << 16);
      x[4 * i + 1] = __uint_as_float(v.x & 0xffff0000u);
      x[4 * i + 2] = __uint_as_float(v.y << 16);
      x[4 * i + 3] = __uint_as_float(v.y & 0xffff0000u);
    }
  }
}

template <int D, int TERMS>
__device__ __forceinline__ void make_q(const QDecodeArgs& a, const float (&x)[D / 4],
                                       QFrag<D, TERMS>& qf) {
  const int c4 = threadIdx.x & 3;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < D / 4; ++i) amax = fmaxf(amax, fabsf(x[i]));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  // exponent of the largest element (an infinite or zero one leaves q as it is)
  int e = kQExp;
  if (amax > 0.f && amax < CUDART_INF_F) e = max(ilogbf(amax), -100);
  const float up = ldexpf(1.f, kQExp - e);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float lo = x[4 * i + 2 * j] * up, hi = x[4 * i + 2 * j + 1] * up;
      qf.f[0][i][j] = pack_f16(lo, hi);
      if (TERMS == 2) qf.f[TERMS - 1][i][j] = pack_f16(lo - f16_rounded(lo), hi - f16_rounded(hi));
    }
  }
  // positive even where it underflows: masked scores are -inf times it
  const float down = fmaxf(a.scale * ldexpf(1.f, e - kQExp), 1e-37f);
  qf.mult[0] = __shfl_sync(0xffffffffu, down, 8 * c4);
  qf.mult[1] = __shfl_sync(0xffffffffu, down, 8 * c4 + 4);
}

// One slice of 16 keys in registers: the K rows of score rows gid and gid + 8
// (this lane's D/4 elements of each), the V rows of score rows 2 c4, 2 c4 + 1,
// 2 c4 + 8, 2 c4 + 9 (elements gid * D/8 .. of each), and their scales.
template <int D>
struct QSlice {
  uint32_t k[2][D / 32];
  uint32_t ks[2];        // e4m3 bytes: two at d = 128, one at d = 64
  uint32_t v[4][D / 64];
  uint32_t vs[4];
};

// raw[0] = (score row gid, head 2c4), raw[1] = (gid, 2c4+1), raw[2], raw[3]: gid + 8
template <int D, int TERMS>
__device__ __forceinline__ void slice_logits(const QSlice<D>& s, const QFrag<D, TERMS>& qf,
                                             float (&raw)[4]) {
  raw[0] = raw[1] = raw[2] = raw[3] = 0.f;
  uint32_t sc[2][D / 64];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t h = cvt_e4m3x2(s.ks[r]);
    sc[r][0] = __byte_perm(h, h, 0x1010);
    if (D == 128) sc[r][D / 64 - 1] = __byte_perm(h, h, 0x3232);
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {   // 8 elements of each row: two MMAs
    uint32_t x[4], y[4];
    cvt_e2m1x8(s.k[0][w], x);
    cvt_e2m1x8(s.k[1][w], y);
    const int blk = D == 128 ? w / 2 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = hmul2(x[i], sc[0][blk]);
      y[i] = hmul2(y[i], sc[1][blk]);
    }
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      mma_f16_16816(raw, x[0], y[0], x[1], y[1], qf.f[t][2 * w][0], qf.f[t][2 * w][1]);
      mma_f16_16816(raw, x[2], y[2], x[3], y[3], qf.f[t][2 * w + 1][0], qf.f[t][2 * w + 1][1]);
    }
  }
}

// Moves the running maxima up to those of NS slices' log2-domain scores x. The
// maximum changes rarely (one vote finds out), so the common slice rescales
// nothing.
template <int D, int NS>
__device__ __forceinline__ void raise_max(QState<D>& st, const float (&x)[NS][4]) {
  float mx0 = fmaxf(x[0][0], x[0][2]), mx1 = fmaxf(x[0][1], x[0][3]);
#pragma unroll
  for (int i = 1; i < NS; ++i) {
    mx0 = fmax3(mx0, x[i][0], x[i][2]);
    mx1 = fmax3(mx1, x[i][1], x[i][3]);
  }
  if (!__any_sync(0xffffffffu, mx0 > st.m[0] || mx1 > st.m[1])) return;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
    mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
  }
  const float mn0 = fmaxf(st.m[0], mx0), mn1 = fmaxf(st.m[1], mx1);
  const float al0 = st.m[0] == kNegInf ? 0.f : fast_exp2(st.m[0] - mn0);
  const float al1 = st.m[1] == kNegInf ? 0.f : fast_exp2(st.m[1] - mn1);
  st.m[0] = mn0;
  st.m[1] = mn1;
  st.mu[0] = (mn0 == kNegInf ? 0.f : mn0) - kPShift;
  st.mu[1] = (mn1 == kNegInf ? 0.f : mn1) - kPShift;
  st.l[0] *= al0;
  st.l[1] *= al1;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    st.o[i][0] *= al0;
    st.o[i][1] *= al1;
    st.o[i][2] *= al0;
    st.o[i][3] *= al1;
  }
}

// O^T += V^T P^T with one slice's weights p. Masked keys' V scales must be zero
// in `s` (what lies there may be anything).
template <int D, int TERMS>
__device__ __forceinline__ void slice_pv(float (&o)[D / 16][4], const float (&p)[4],
                                         const QSlice<D>& s) {
  uint32_t b[TERMS][2];
  b[0][0] = movmatrix_t(pack_f16(p[0], p[1]));
  b[0][1] = movmatrix_t(pack_f16(p[2], p[3]));
  if (TERMS == 2) {
    b[TERMS - 1][0] = movmatrix_t(pack_f16(p[0] - f16_rounded(p[0]), p[1] - f16_rounded(p[1])));
    b[TERMS - 1][1] = movmatrix_t(pack_f16(p[2] - f16_rounded(p[2]), p[3] - f16_rounded(p[3])));
  }
  const uint32_t s01 = cvt_e4m3x2(__byte_perm(s.vs[0], s.vs[1], 0x0040));
  const uint32_t s23 = cvt_e4m3x2(__byte_perm(s.vs[2], s.vs[3], 0x0040));
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    // codes of one element of two keys side by side: even elements, odd ones
    const uint32_t e01 = (s.v[0][w] & 0x0f0f0f0fu) | ((s.v[1][w] << 4) & 0xf0f0f0f0u);
    const uint32_t d01 = ((s.v[0][w] >> 4) & 0x0f0f0f0fu) | (s.v[1][w] & 0xf0f0f0f0u);
    const uint32_t e23 = (s.v[2][w] & 0x0f0f0f0fu) | ((s.v[3][w] << 4) & 0xf0f0f0f0u);
    const uint32_t d23 = ((s.v[2][w] >> 4) & 0x0f0f0f0fu) | (s.v[3][w] & 0xf0f0f0f0u);
    uint32_t ea[4], da[4], eb[4], db[4];
    cvt_e2m1x8(e01, ea);
    cvt_e2m1x8(d01, da);
    cvt_e2m1x8(e23, eb);
    cvt_e2m1x8(d23, db);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a0 = hmul2(ea[i], s01), a1 = hmul2(da[i], s01);
      const uint32_t a2 = hmul2(eb[i], s23), a3 = hmul2(db[i], s23);
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
        mma_f16_16816(o[4 * w + i], a0, a1, a2, a3, b[t][0], b[t][1]);
    }
  }
}

// ------------------------------------------------------------------ joining --
// A piece is one warp's (or CTA's) state over part of a (sequence, KV head):
// m[G], l[G] (log2-domain maximum; sum of 2^14 p), and at qpart_head(G) o[G][D].
template <int D>
__device__ __forceinline__ void piece_store(float* p, QState<D>& st, int G) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    st.l[0] += __shfl_xor_sync(0xffffffffu, st.l[0], off);
    st.l[1] += __shfl_xor_sync(0xffffffffu, st.l[1], off);
  }
  const int h = 2 * c4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (h + i >= G) continue;
    if (gid == 0) {
      p[h + i] = st.m[i];
      p[G + h + i] = st.l[i];
    }
    float* o = p + qpart_head(G) + (h + i) * D + gid * (D / 8);
#pragma unroll
    for (int j = 0; j < D / 16; j += 2)
      *reinterpret_cast<float4*>(o + 2 * j) =
          make_float4(st.o[j][i], st.o[j][2 + i], st.o[j + 1][i], st.o[j + 1][2 + i]);
  }
}

template <bool F32>
__device__ __forceinline__ void out_store4(const QDecodeArgs& a, size_t at, float4 y) {
  if (F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
  } else {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  }
}

__device__ __forceinline__ void write_row_stat(const QDecodeArgs& a, size_t row, float m, float l) {
  if (a.row_stat != nullptr)   // in logit units, without the 2^14
    a.row_stat[row] = make_float2(m * kLn2, l == 0.f ? 0.f : ldexpf(1.f / l, kPShift));
}

// Four dims e (float4 index within [G][D / 4]) of head h over pieces s0 .. s1-1,
// the i-th at piece(i): running maximum, sum and output, with the loads of
// several pieces in flight together.
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
  // a part without keys has m = -inf and l = o = 0 (or l NaN, which stays)
  const float wx = x.m == kNegInf ? 1.f : ex2(x.m - M);
  x.m = M;
  x.l *= wx;
  x.o.x *= wx;
  x.o.y *= wx;
  x.o.z *= wx;
  x.o.w *= wx;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float w = y[k].m == kNegInf ? 1.f : ex2(y[k].m - M);
    x.l = fmaf(w, y[k].l, x.l);
    x.o.x = fmaf(w, y[k].o.x, x.o.x);
    x.o.y = fmaf(w, y[k].o.y, x.o.y);
    x.o.z = fmaf(w, y[k].o.z, x.o.z);
    x.o.w = fmaf(w, y[k].o.w, x.o.w);
  }
}
template <bool GLOBAL, typename Piece>
__device__ __forceinline__ Joined join_some(Piece piece, int s0, int s1, int G, int h, int e) {
  constexpr int kBatch = GLOBAL ? 8 : 4;   // loads of L2 lines take longer
  Joined x = {kNegInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s = s0; s < s1; s += kBatch) {
    Joined y[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      y[k] = {kNegInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      if (s + k < s1) {
        const float* p = piece(s + k);
        const float4* o = reinterpret_cast<const float4*>(p + qpart_head(G)) + e;
        y[k].m = GLOBAL ? __ldcg(p + h) : p[h];
        y[k].l = GLOBAL ? __ldcg(p + G + h) : p[G + h];
        y[k].o = GLOBAL ? __ldcg(o) : *o;
      }
    }
    join_into(x, y);
  }
  return x;
}

// The output (b, g, head slot h, dims 4 e4 ..) of a joined whole.
template <int D, bool F32>
__device__ __forceinline__ void joined_output(const QDecodeArgs& a, const Joined& x, int b, int g,
                                              int h, int e4) {
  const size_t row = static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + h];
  const float inv = x.l == 0.f ? 0.f : a.v_scale / x.l;   // 0: no key at all
  out_store4<F32>(a, row * D + 4 * e4,
                  make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv));
  if (e4 == 0) write_row_stat(a, row, x.m, x.l);
}

// A unit shared by n CTAs: its first CTA's piece, and the others' from `rest` on.
struct SharedUnit {
  int unit, b, g, n;
  const float* first;
  const float* rest;
  size_t step;
};

// This CTA's pieces of up to two such units are in their places. Count them,
// and where this CTA is the last to arrive join all of the unit's pieces into
// the output: equal shares of the pieces per group of threads, added in order,
// so the result does not depend on timing. `scratch`: blockDim.x Joined.
template <int D, bool F32>
__device__ void arrive_and_join(const QDecodeArgs& a, int n_units, const SharedUnit (&units)[2],
                                Joined* scratch) {
  __shared__ unsigned int s_last;
  const int tid = threadIdx.x, G = a.G;
  __syncthreads();   // every piece of this CTA is written
  if (tid == 0) {
    __threadfence();
    unsigned int last = 0u;
#pragma unroll
    for (int k = 0; k < 2; ++k)
      if (k < n_units && atomicAdd(&a.counters[units[k].unit], 1u) ==
                             static_cast<unsigned int>(units[k].n - 1)) {
        a.counters[units[k].unit] = 0u;   // ready for the next launch
        last |= 1u << k;
      }
    __threadfence();
    s_last = last;
  }
  __syncthreads();
  const unsigned int last = s_last;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!((last >> k) & 1u)) continue;
    const SharedUnit& u = units[k];
    const int n = u.n;
    const int elems = G * (D / 4);                 // 16 .. 256
    int shares = static_cast<int>(blockDim.x) / elems;
    if (shares > (n + 3) / 4) shares = (n + 3) / 4;
    const int e = tid % elems, share = tid / elems, h = e / (D / 4), e4 = e & (D / 4 - 1);
    const int per = (n + shares - 1) / shares;
    auto mine = [&](int i) -> const float* { return i == 0 ? u.first : u.rest + (i - 1) * u.step; };
    Joined x = {kNegInf, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (share < shares) x = join_some<true>(mine, share * per, min(n, (share + 1) * per), G, h, e);
    if (shares > 1) {
      if (share > 0 && share < shares) scratch[tid] = x;
      __syncthreads();
      if (share == 0)
        for (int i = 1; i < shares; ++i) {
          const Joined y[1] = {scratch[i * elems + e]};
          join_into(x, y);
        }
      __syncthreads();
    }
    if (share == 0) joined_output<D, F32>(a, x, u.b, u.g, h, e4);
  }
}

// A whole unit held by one warp: straight from its registers to the output.
template <int D, bool F32>
__device__ __forceinline__ void warp_output(const QDecodeArgs& a, QState<D>& st, int b, int g) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) st.l[i] += __shfl_xor_sync(0xffffffffu, st.l[i], off);
    if (2 * c4 + i >= a.G) continue;
    const size_t row = static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + 2 * c4 + i];
    const float inv = st.l[i] == 0.f ? 0.f : a.v_scale / st.l[i];
#pragma unroll
    for (int j = 0; j < D / 16; j += 2)
      out_store4<F32>(a, row * D + gid * (D / 8) + 2 * j,
                      make_float4(st.o[j][i] * inv, st.o[j][2 + i] * inv, st.o[j + 1][i] * inv,
                                  st.o[j + 1][2 + i] * inv));
    if (gid == 0) write_row_stat(a, row, st.m[i], st.l[i]);
  }
}

// ------------------------------------------------------------------- slices --
// A sequence's cached tokens; one outside what the call and its block table
// hold is reported and cut to it.
__device__ __forceinline__ int len_of(const QDecodeArgs& a, int b, bool report) {
  const int cap = static_cast<int>(
      min(static_cast<long long>(a.N), static_cast<long long>(a.max_blocks) << a.bs_shift));
  const int n = a.lens[b];
  if (n >= 0 && n <= cap) return n;
  if (report) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x521);
  return n < 0 ? 0 : cap;
}

// The group that holds keys 16 s .. 16 s + 15 of a sequence, for KV head g;
// null (and reported) if the table's entry is no block of the cache.
template <int D>
__device__ __forceinline__ const uint8_t* group_at(const QDecodeArgs& a, const int32_t* table_row,
                                                   int g, int s) {
  const int sh = a.bs_shift - 4;
  const int block = __ldg(table_row + (s >> sh));
  if (block < 0 || block >= a.num_blocks) {
    report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x522);
    return nullptr;
  }
  return a.cache + (((static_cast<size_t>(block) * a.Hkv + g) << sh) + (s & ((1 << sh) - 1))) *
                       qgroup_bytes(D);
}

// Row r of a slice's score tile is its key row_key(r): within each four rows
// the second pair is swapped, so that the four V rows that lanes c4 = 0 .. 3
// load together (rows 2 c4 of the tile) alternate between even and odd keys.
// In shared memory at d = 128 (64-byte rows) that halves their bank conflicts.
__device__ __forceinline__ int row_key(int r) { return r ^ ((r >> 1) & 1); }
// key of a slice that V register i of this lane belongs to
__device__ __forceinline__ int v_key(int i) {
  return row_key(2 * (threadIdx.x & 3) + (i & 1)) + 8 * (i >> 1);
}

// Loads from global memory (through the read-only path) or from shared memory.
template <bool SHARED, typename T>
__device__ __forceinline__ T load_as(const uint8_t* p) {
  const T* q = reinterpret_cast<const T*>(p);
  return SHARED ? *q : __ldg(q);
}
template <bool SHARED, int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one vector load");
  if (N == 4) {
    const uint4 v = load_as<SHARED, uint4>(p);
    w[0] = v.x;
    w[N / 4] = v.y;
    w[N / 2] = v.z;
    w[N - 1] = v.w;
  } else if (N == 2) {
    const uint2 v = load_as<SHARED, uint2>(p);
    w[0] = v.x;
    w[N - 1] = v.y;
  } else {
    w[0] = load_as<SHARED, uint32_t>(p);
  }
}

// This lane's part of the K row (grp, r) and of the V row (grp, r).
template <int D, bool SHARED>
__device__ __forceinline__ void load_k_row(QSlice<D>& s, int i, const uint8_t* grp, int r) {
  const int c4 = threadIdx.x & 3;
  load_words<SHARED>(grp + r * (D / 2) + c4 * (D / 8), s.k[i]);
  const uint8_t* sc = grp + 8 * D + r * (D / 16) + c4 * (D / 64);
  s.ks[i] = D == 128 ? static_cast<uint32_t>(load_as<SHARED, uint16_t>(sc))
                     : static_cast<uint32_t>(load_as<SHARED, uint8_t>(sc));
}
template <int D, bool SHARED>
__device__ __forceinline__ void load_v_row(QSlice<D>& s, int i, const uint8_t* grp, int r) {
  const int gid = (threadIdx.x & 31) >> 2;
  load_words<SHARED>(grp + 9 * D + r * (D / 2) + gid * (D / 16), s.v[i]);
  s.vs[i] = load_as<SHARED, uint8_t>(grp + 17 * D + r * (D / 16) + gid * D / 128);
}

// -------------------------------------------------------------------- dense --
// The steps of all units (unit = sequence * Hkv + KV head; a step is 16 *
// kStep keys, and a sequence of n keys has ceil(n / (16 kStep)) per head) form one
// line, and every warp of the grid takes an equal run of it, so that ragged
// batches balance. A run may span units: the warp's pieces of units it does
// not hold alone go to shared memory, the CTA joins those of its warps after
// one barrier, and a unit that several CTAs share is joined by the last of
// them to arrive.
//
// Every warp feeds itself: a ring of kDenseStages stages of one step, each
// filled by one bulk copy per block that the step touches (groups of a block
// are contiguous), which the first lanes issue as soon as the warp has left
// the stage; no warp waits for another one before the end.
constexpr int kMinRun = 2;        // steps per warp at least
constexpr int kDenseStages = 2;
template <int D>
constexpr int kStepOf = 256 / D;  // slices per step: 4608 bytes either way

// Where a warp is in the line of steps.
struct Cursor {
  int f;           // its run's first step of this unit
  int b, g, n;     // unit, cached tokens
  int ns;          // steps of the unit
  int s0, s, s1;   // this run's part of them: [s0, s1), next one s
};
__device__ __forceinline__ void cursor_enter(Cursor& c, const QDecodeArgs& a, const int* pref,
                                             int f, int end) {
  int lo = 0, hi = a.B;   // the sequence: pref[lo] * Hkv <= f < pref[lo + 1] * Hkv
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] * a.Hkv <= f) lo = mid;
    else hi = mid;
  }
  c.f = f;
  c.b = lo;
  c.n = len_of(a, lo, false);
  c.ns = pref[lo + 1] - pref[lo];
  const int in = f - pref[lo] * a.Hkv;
  c.g = in / c.ns;
  c.s0 = c.s = in - c.g * c.ns;
  c.s1 = min(c.ns, c.s0 + end - f);
}

template <int D, int TERMS, bool SCORES>
__global__ void __launch_bounds__(kNW * 32, 2)
    k_qdecode_dense(const __grid_constant__ QDecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr bool F32 = TERMS == 2;
  constexpr int kStep = kStepOf<D>, kKeys = 16 * kStep;
  constexpr int kGroupBytes = qgroup_bytes(D), kStageBytes = kStep * kGroupBytes;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t s_full[kNW][kDenseStages];
  __shared__ int s_tot[kNW];
  __shared__ int s_unit[2 * kNW], s_list[2 * kNW], s_nlist;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c4 = lane & 3;
  const int pf = static_cast<int>(qpart_floats(a.G, D));
  // a ring per warp, which at the end holds the warp's last piece; a place for
  // its first piece; steps before every sequence, per head
  uint8_t* ring = smem + warp * kDenseStages * kStageBytes;
  float* firsts = reinterpret_cast<float*>(smem + kNW * kDenseStages * kStageBytes);   // [kNW][pf]
  int* pref = reinterpret_cast<int*>(firsts + kNW * pf);                               // [B + 1]
  auto slot_at = [&](int i) -> float* {   // slot 2w: warp w's first piece, 2w + 1: its last
    return (i & 1) ? reinterpret_cast<float*>(smem + (i >> 1) * kDenseStages * kStageBytes)
                   : firsts + (i >> 1) * pf;
  };

  if (lane == 0)
    for (int i = 0; i < kDenseStages; ++i) mbar_init(&s_full[warp][i], 1);
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kNW * 32) {
    const int b = b0 + tid;
    const int n = b < a.B ? (len_of(a, b, blockIdx.x == 0) + kKeys - 1) / kKeys : 0;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += o;
    }
    if (lane == 31) s_tot[warp] = incl;
    __syncthreads();
    int base = carry;
    for (int w = 0; w < kNW; ++w) {
      if (w < warp) base += s_tot[w];
      carry += s_tot[w];
    }
    if (b < a.B) pref[b] = base + incl - n;
    __syncthreads();
  }
  if (tid == 0) pref[a.B] = carry;
  if (tid < 2 * kNW) s_unit[tid] = -1;
  fence_barrier_init();
  __syncthreads();
  const int total = carry * a.Hkv;
  const int nwarps = static_cast<int>(gridDim.x) * kNW;
  const int per = max(kMinRun, (total + nwarps - 1) / nwarps);
  const int w0 = min(total, (static_cast<int>(blockIdx.x) * kNW + warp) * per);
  const int w1 = min(total, w0 + per);

  // ---- copies: `in` runs ahead of the arithmetic by kDenseStages steps. Lane i
  // < ncopy issues the step's i-th copy of copy_slices slices; its block id is
  // loaded when `in` gets to the step, one step before it is used.
  const int copy_sh = min(a.bs_shift, D == 128 ? 5 : 6);   // log2 of a copy's keys
  const int ncopy = kKeys >> copy_sh;
  const uint32_t copy_bytes = static_cast<uint32_t>(kGroupBytes) << (copy_sh - 4);
  const int gmask = (1 << (a.bs_shift - 4)) - 1;
  Cursor in = {}, at = {};
  int id = -1;
  bool more = w0 < w1;            // `in` stands at a step of this run
  int in_stage = 0;
  unsigned int have = 0u;         // byte i: the copies that stage i got
  int pending = 0;                // steps issued and not taken
  bool alive = true;
  auto fetch_id = [&]() {
    const int key = in.s * kKeys + (lane << copy_sh);
    id = 0;                       // nothing to copy: neither read nor reported
    if (lane < ncopy && key < in.n)
      id = __ldg(a.table + static_cast<size_t>(in.b) * a.max_blocks + (key >> a.bs_shift));
  };
  auto issue = [&]() {            // all lanes, `more` holds
    const int key = in.s * kKeys + (lane << copy_sh);
    const bool want = lane < ncopy && key < in.n;
    const bool ok = want && static_cast<unsigned int>(id) < static_cast<unsigned int>(a.num_blocks);
    if (want && !ok) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x522);
    const unsigned int got = __ballot_sync(0xffffffffu, ok);
    uint64_t* bar = &s_full[warp][in_stage];
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(got) * copy_bytes);
    __syncwarp();
    if (ok) {
      const size_t grp = ((static_cast<size_t>(id) * a.Hkv + in.g) << (a.bs_shift - 4)) +
                         ((key >> 4) & gmask);
      bulk_load(ring + in_stage * kStageBytes + lane * copy_bytes, a.cache + grp * kGroupBytes,
                copy_bytes, bar);
    }
    have = (have & ~(0xffu << (8 * in_stage))) | (got << (8 * in_stage));
    in_stage ^= 1;
    ++pending;
    if (++in.s == in.s1) {
      const int next = in.f + in.s1 - in.s0;
      more = next < w1;
      if (more) cursor_enter(in, a, pref, next, w1);
    }
    if (more) fetch_id();
  };
  static_assert(kDenseStages == 2, "stages alternate");
  float qx[D / 4];   // the query of the unit that comes next
  if (more) {
    cursor_enter(in, a, pref, w0, w1);
    fetch_id();
    at = in;
    load_q<D, TERMS>(a, at.b, at.g, qx);
    issue();
    if (more) issue();
  }

  // ---- arithmetic
  const int row0 = row_key(gid);   // keys row0 and row0 + 8 of a slice
  int stage = 0;
  uint32_t phase = 0;
  for (int f = w0; f < w1;) {
    if (f != w0) {
      cursor_enter(at, a, pref, f, w1);
      load_q<D, TERMS>(a, at.b, at.g, qx);
    }
    const int n = at.n;
    QFrag<D, TERMS> qf;
    make_q(a, qx, qf);
    float* sp[2] = {nullptr, nullptr};
    if (SCORES)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (2 * c4 + i < a.G)
          sp[i] = a.scores +
                  (static_cast<size_t>(at.b) * a.Hq + a.heads[at.g * a.G + 2 * c4 + i]) * a.N;
    const uint64_t ml = f2_pack(qf.mult[0] * kLog2e, qf.mult[1] * kLog2e);
    // m: running maxima (log2 units); nmu = 14 - m, +inf before the first key
    float m0 = kNegInf, m1 = kNegInf;
    uint64_t nmu = f2_pack(-kNegInf, -kNegInf), l = f2_pack(0.f, 0.f);
    float o[D / 16][4];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    for (; at.s < at.s1 && alive; ++at.s) {
      if (!mbar_wait_warp(&s_full[warp][stage], phase, a.err, 0x531)) {
        // a wait that gave up (reported): leave no copy in flight, and pass over
        // the rest of the run so that every unit still gets its arrivals
        for (; pending > 0; --pending) {
          mbar_wait_warp(&s_full[warp][stage], phase, a.err, 0x532);
          stage ^= 1;
          phase ^= stage == 0 ? 1u : 0u;
        }
        alive = false;
        break;
      }
      const uint8_t* buf = ring + stage * kStageBytes;
      const unsigned int got = (have >> (8 * stage)) & 0xffu;
      if (got != 0u || SCORES) {
        uint64_t t[kStep][2];   // scores of (row0; row0 + 8) for both heads: raw, then exponents
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
          QSlice<D> sl;
          load_k_row<D, true>(sl, 0, buf + i * kGroupBytes, row0);
          load_k_row<D, true>(sl, 1, buf + i * kGroupBytes, row0 + 8);
          float raw[4];
          slice_logits(sl, qf, raw);
          t[i][0] = f2_pack(raw[0], raw[1]);
          t[i][1] = f2_pack(raw[2], raw[3]);
        }
        // keys that do not count: behind the sequence's end, or in a block the
        // table does not name
        const int key0 = at.s * kKeys + row0;
        const bool full = got == (1u << ncopy) - 1u && (at.s + 1) * kKeys <= n;
        auto counts = [&](int i, int key) {
          return ((got >> ((16 * i) >> copy_sh)) & 1u) != 0u && key < n;
        };
        if (!full) {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              // -inf through any multiplier's sign: the multiplier is positive
              if (!counts(i, key0 + 16 * i + 8 * r)) t[i][r] = f2_pack(kNegInf, kNegInf);
        }
        if (SCORES) {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int key = key0 + 16 * i + 8 * r;
              float v0, v1;
              f2_unpack(t[i][r], v0, v1);
              if (full || key < n) {
                if (sp[0] != nullptr) sp[0][key] = v0 * qf.mult[0];
                if (sp[1] != nullptr) sp[1][key] = v1 * qf.mult[1];
              }
            }
        }
        if (got != 0u) {
          auto exponents = [&](float& top0, float& top1, uint64_t (&y)[kStep][2]) {
            top0 = top1 = kNegInf;
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
              float a0, a1, b0, b1;
              // product and sum rounded apart, as the maximum was: a fused one
              // would leave the product's rounding, large for a huge score
              y[i][0] = f2_add(f2_mul(t[i][0], ml), nmu);
              y[i][1] = f2_add(f2_mul(t[i][1], ml), nmu);
              f2_unpack(y[i][0], a0, a1);
              f2_unpack(y[i][1], b0, b1);
              top0 = fmax3(top0, a0, b0);
              top1 = fmax3(top1, a1, b1);
            }
          };
          uint64_t y[kStep][2];
          float top0, top1;
          exponents(top0, top1, y);
          if (__any_sync(0xffffffffu, fmaxf(top0, top1) > static_cast<float>(kPShift))) {
            // a score above the running maximum: raise it and rescale
            float x0 = kNegInf, x1 = kNegInf, ml0, ml1;
            f2_unpack(ml, ml0, ml1);
#pragma unroll
            for (int i = 0; i < kStep; ++i) {
              float a0, a1, b0, b1;
              f2_unpack(t[i][0], a0, a1);
              f2_unpack(t[i][1], b0, b1);
              x0 = fmax3(x0, a0 * ml0, b0 * ml0);
              x1 = fmax3(x1, a1 * ml1, b1 * ml1);
            }
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) {
              x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
              x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
            }
            x0 = fmaxf(x0, m0);
            x1 = fmaxf(x1, m1);
            const float al0 = m0 == kNegInf ? 0.f : fast_exp2(m0 - x0);
            const float al1 = m1 == kNegInf ? 0.f : fast_exp2(m1 - x1);
            m0 = x0;
            m1 = x1;
            nmu = f2_pack(kPShift - m0, kPShift - m1);
            l = f2_mul(l, f2_pack(al0, al1));
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              o[i][0] *= al0;
              o[i][1] *= al1;
              o[i][2] *= al0;
              o[i][3] *= al1;
            }
            exponents(top0, top1, y);
          }
#pragma unroll
          for (int i = 0; i < kStep; ++i) {
            QSlice<D> sl;
#pragma unroll
            for (int j = 0; j < 4; ++j) load_v_row<D, true>(sl, j, buf + i * kGroupBytes, v_key(j));
            if (!full) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (!counts(i, at.s * kKeys + 16 * i + v_key(j))) sl.vs[j] = 0u;
            }
            float p[4];
            f2_unpack(y[i][0], p[0], p[1]);
            f2_unpack(y[i][1], p[2], p[3]);
#pragma unroll
            for (int j = 0; j < 4; ++j) p[j] = ex2(p[j]);
            l = f2_add(l, f2_add(f2_pack(p[0], p[1]), f2_pack(p[2], p[3])));
            slice_pv<D, TERMS>(o, p, sl);
          }
        }
      }
      stage ^= 1;
      phase ^= stage == 0 ? 1u : 0u;
      --pending;
      // the stage is refilled through the async proxy: this warp's reads first
      fence_proxy_async_smem();
      __syncwarp();
      if (more) issue();
    }
    f += at.s1 - at.s0;
    QState<D> st;
    st.m[0] = m0;
    st.m[1] = m1;
    f2_unpack(l, st.l[0], st.l[1]);
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[i][j] = o[i][j];
    if (at.s0 == 0 && at.s1 == at.ns) {
      warp_output<D, F32>(a, st, at.b, at.g);
    } else {
      // in part: a run's first unit or its last (whose ring is free by then)
      const int slot = 2 * warp + (at.f == w0 ? 0 : 1);
      piece_store<D>(slot_at(slot), st, a.G);
      if (lane == 0) s_unit[slot] = at.b * a.Hkv + at.g;
    }
  }
  __syncthreads();
  if (tid == 0) {
    int m = 0;
    for (int i = 0; i < 2 * kNW; ++i)
      if (s_unit[i] >= 0) s_list[m++] = i;
    s_nlist = m;
  }
  __syncthreads();
  const int nlist = s_nlist;
  const int per_cta = per * kNW, c0 = static_cast<int>(blockIdx.x) * per_cta;
  // This CTA's pieces, in order of their units: a unit is joined here if the
  // CTA holds all of it, else its piece goes to CTA c's place 2c + 1 (a unit
  // that starts inside c's run) or 2c (one that started before it, or with it).
  const size_t stride = qpart_floats(a.G, D);
  SharedUnit shared[2] = {};   // at most the first and the last unit of the run
  int n_shared = 0;
  const int elems = a.G * (D / 4);
  for (int i = 0, first_elem = 0; i < nlist;) {
    const int unit = s_unit[s_list[i]];
    int j = i;
    while (j < nlist && s_unit[s_list[j]] == unit) ++j;
    const int b = unit / a.Hkv, g = unit % a.Hkv, nb = pref[b + 1] - pref[b];
    const int u0 = pref[b] * a.Hkv + g * nb, u1 = u0 + nb;   // the unit's steps
    float* dst = nullptr;
    if (u0 < c0 || u1 > c0 + per_cta) {
      dst = a.part + (2 * static_cast<size_t>(blockIdx.x) + (u0 > c0 ? 1 : 0)) * stride;
      const int first = u0 / per_cta;
      const SharedUnit u = {unit, b, g, (u1 - 1) / per_cta - first + 1,
                            a.part + (2 * static_cast<size_t>(first) +
                                      (u0 > first * per_cta ? 1 : 0)) * stride,
                            a.part + 2 * (static_cast<size_t>(first) + 1) * stride, 2 * stride};
      if (n_shared == 0) shared[0] = u;
      else shared[1] = u;
      ++n_shared;
    }
    // the next unit's elements go to the threads that this one leaves free
    const int e = (tid - first_elem) & (kNW * 32 - 1);
    if (e < elems) {
      const int h = e / (D / 4), e4 = e & (D / 4 - 1);
      const Joined x = join_some<false>(
          [&](int s) -> const float* { return slot_at(s_list[i + s]); }, 0, j - i, a.G, h, e);
      if (dst != nullptr) {
        reinterpret_cast<float4*>(dst + qpart_head(a.G))[e] = x.o;
        if (e4 == 0) {
          dst[h] = x.m;
          dst[a.G + h] = x.l;
        }
      } else {
        joined_output<D, F32>(a, x, b, g, h, e4);
      }
    }
    first_elem += elems;
    i = j;
  }
  if (n_shared > 0)
    arrive_and_join<D, F32>(a, n_shared, shared, reinterpret_cast<Joined*>(smem));
  // sequences without keys: zeros; scores behind the last key
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (pref[b + 1] != pref[b]) continue;
    const size_t base = static_cast<size_t>(b) * a.Hq * D;
    for (int e = 4 * tid; e < a.Hq * D; e += 4 * kNW * 32)
      out_store4<F32>(a, base + e, make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = tid; h < a.Hq; h += kNW * 32)
      write_row_stat(a, static_cast<size_t>(b) * a.Hq + h, kNegInf, 0.f);
  }
  if (SCORES && a.fill_tail)
    for (int r = blockIdx.x; r < a.B * a.Hq; r += gridDim.x)
      for (int j = len_of(a, r / a.Hq, false) + tid; j < a.N; j += blockDim.x)
        a.scores[static_cast<size_t>(r) * a.N + j] = kNegInf;
}

__global__ void __launch_bounds__(256) k_qfill_tail(float* __restrict__ rows,
                                                    const int32_t* __restrict__ lens, int H,
                                                    int N) {
  pdl_wait();
  pdl_trigger();
  const int n = max(0, lens[blockIdx.x / H]);
  for (int j = n + threadIdx.x; j < N; j += 256)
    rows[static_cast<size_t>(blockIdx.x) * N + j] = kNegInf;
}

// -------------------------------------------------------------------- reuse --
// One (sequence, KV head) per blockIdx.y; its 16-entry slices, numbered across
// the chunks of its union plan (per query head sets: key | head mask << 24,
// ascending) or across its set (pooled), are split into S equal runs, one per
// CTA, and a run's slices go to the CTA's warps in turn. Rows are gathered
// through the block table straight into the MMA fragments: a K row is read by
// four lanes, a V row by eight, whole 32-byte sectors either way.
template <int D, int TERMS, bool POOLED>
__global__ void __launch_bounds__(kNW * 32, 2)
    k_qdecode_reuse(const __grid_constant__ QDecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr bool F32 = TERMS == 2;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int s_pref[kMaxSplits + 1], s_cnt[kMaxSplits];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c4 = lane & 3;
  const int pf = static_cast<int>(qpart_floats(a.G, D));
  float* slots = reinterpret_cast<float*>(smem);   // [kNW][pf]
  const int unit = blockIdx.y, b = unit / a.Hkv, g = unit % a.Hkv;
  const int n = len_of(a, b, blockIdx.x == 0 && g == 0);
  const int nch = POOLED ? 0 : a.plan_chunks;
  if (!POOLED && warp == 0) {
    int carry = 0;
    for (int cb = 0; cb < nch; cb += 32) {
      const int c = cb + lane;
      const int cnt = c < nch ? min(kPlanCapEntries, a.plan_count[unit * nch + c]) : 0;
      const int sl = (cnt + 15) / 16;
      int incl = sl;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += o;
      }
      if (c < nch) {
        s_cnt[c] = cnt;
        s_pref[c] = carry + incl - sl;
      }
      carry += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) s_pref[nch] = carry;
  }
  __syncthreads();
  const int total = POOLED ? (a.topk + 15) / 16 : s_pref[nch];
  const int per = (total + a.S - 1) / a.S;
  const int g0 = min(total, static_cast<int>(blockIdx.x) * per), g1 = min(total, g0 + per);
  const int32_t* set = POOLED ? a.idx + static_cast<size_t>(unit) * a.topk : nullptr;
  const int32_t* trow = a.table + static_cast<size_t>(b) * a.max_blocks;
  const uint32_t every = (1u << a.G) - 1u;

  QState<D> st;
  qstate_init(st);
  QFrag<D, TERMS> qf;
  {
    float x[D / 4];
    load_q<D, TERMS>(a, b, g, x);
    make_q(a, x, qf);
  }
  int fc = 0;
  for (int sl = g0 + warp; sl < g1; sl += kNW) {
    // entry i of the slice in lanes i and i + 16: its key's group and row, and
    // the heads that attend to it (none: padding, not read)
    uint32_t mask = 0u;
    int key = 0;
    if (POOLED) {
      const int e = sl * 16 + (lane & 15);
      if (e < a.topk) {
        key = __ldg(set + e);
        const int before = e > 0 ? __ldg(set + e - 1) : -1;
        if (key >= n || (key >= 0 && (key <= before || (before < 0 && e > 0)))) {
          report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x523);
        } else if (key >= 0) {
          mask = every;
        } else if (key != -1) {
          report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x524);
        }
      }
    } else {
      while (fc + 1 < nch && s_pref[fc + 1] <= sl) ++fc;
      const int e = (sl - s_pref[fc]) * 16 + (lane & 15);
      if (e < s_cnt[fc]) {
        const uint32_t ent =
            __ldg(a.plan + (static_cast<size_t>(unit) * nch + fc) * kPlanCapEntries + e);
        key = static_cast<int>(ent & 0xffffffu);
        mask = key < n ? ent >> 24 : 0u;
      }
    }
    const uint8_t* grp = nullptr;
    if (mask != 0u) grp = group_at<D>(a, trow, g, key >> 4);
    if (grp == nullptr) mask = 0u;
    const unsigned long long base = reinterpret_cast<unsigned long long>(grp);
    QSlice<D> s;
    float x[1][4];
    uint32_t mk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = row_key(gid) + 8 * i;
      const uint8_t* p =
          reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, base, src));
      const int r = __shfl_sync(0xffffffffu, key, src) & 15;
      mk[i] = __shfl_sync(0xffffffffu, mask, src);
      if (mk[i] != 0u) {
        load_k_row<D, false>(s, i, p, r);
      } else {
#pragma unroll
        for (int w = 0; w < D / 32; ++w) s.k[i][w] = 0u;
        s.ks[i] = 0u;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int src = v_key(i);
      const uint8_t* p =
          reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, base, src));
      const int r = __shfl_sync(0xffffffffu, key, src) & 15;
      if (p != nullptr) {
        load_v_row<D, false>(s, i, p, r);
      } else {
#pragma unroll
        for (int w = 0; w < D / 64; ++w) s.v[i][w] = 0u;
        s.vs[i] = 0u;
      }
    }
    slice_logits(s, qf, x[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = (mk[i >> 1] >> (2 * c4 + (i & 1))) & 1u;
      x[0][i] = in ? x[0][i] * (qf.mult[i & 1] * kLog2e) : kNegInf;
    }
    // A V block that holds a NaN (scale 0x7f or 0xff) would reach every head of
    // the group through 0 * NaN in the product: it is taken out of the slice,
    // and only the heads whose set holds the key get the NaN.
    uint32_t nan_heads = 0u;
    if (!POOLED) {
      const uint32_t vs4 = s.vs[0] | (s.vs[1] << 8) | (s.vs[2] << 16) | (s.vs[3] << 24);
      const uint32_t bad = __vcmpeq4(vs4 & 0x7f7f7f7fu, 0x7f7f7f7fu);
      if (__any_sync(0xffffffffu, bad != 0u)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t km = __shfl_sync(0xffffffffu, mask, v_key(i));
          if ((bad >> (8 * i)) & 1u) {
            s.vs[i] = 0u;
            nan_heads |= km;
          }
        }
        // the four lanes that share these dims hold other keys and other heads
        nan_heads |= __shfl_xor_sync(0xffffffffu, nan_heads, 1);
        nan_heads |= __shfl_xor_sync(0xffffffffu, nan_heads, 2);
        nan_heads >>= 2 * c4;
      }
    }
    raise_max<D, 1>(st, x);
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] = ex2(x[0][i] - st.mu[i & 1]);
      st.l[i & 1] += p[i];
    }
    slice_pv<D, TERMS>(st.o, p, s);
    if (!POOLED && (nan_heads & 3u) != 0u) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((nan_heads >> (i & 1)) & 1u) st.o[j][i] = CUDART_NAN_F;
    }
  }
  piece_store<D>(slots + warp * pf, st, a.G);
  __syncthreads();
  float* part = a.part + static_cast<size_t>(unit) * a.S * pf;
  float* dst = part + static_cast<size_t>(blockIdx.x) * pf;
  const int elems = a.G * (D / 4);
  for (int e = tid; e < elems; e += kNW * 32) {
    const int h = e / (D / 4), e4 = e & (D / 4 - 1);
    const Joined x = join_some<false>([&](int w) -> const float* { return slots + w * pf; }, 0,
                                      kNW, a.G, h, e);
    if (a.S == 1) {
      joined_output<D, F32>(a, x, b, g, h, e4);
    } else {
      reinterpret_cast<float4*>(dst + qpart_head(a.G))[e] = x.o;
      if (e4 == 0) {
        dst[h] = x.m;
        dst[a.G + h] = x.l;
      }
    }
  }
  if (a.S == 1) return;
  const SharedUnit units[2] = {{unit, b, g, a.S, part, part + pf, static_cast<size_t>(pf)}, {}};
  arrive_and_join<D, F32>(a, 1, units, reinterpret_cast<Joined*>(slots));
}

// CTAs of a kernel that the current device holds at once (asked once per host
// thread, device and shared memory size). The kernel may use all the shared
// memory there is: the same value whatever the call, so that threads calling
// with different sizes do not undo one another's setting.
template <void (*kern)(const QDecodeArgs)>   // by value: each kernel has its own record
cudaError_t resident_ctas(size_t smem, int& ctas) {
  thread_local int dev_of = -1, slots = 0;
  thread_local size_t smem_of = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev != dev_of || smem != smem_of) {
    int sms = 0, per_sm = 0, most = 0;
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) !=
        cudaSuccess)
      return e;
    most -= static_cast<int>(fa.sharedSizeBytes);
    if (smem > static_cast<size_t>(most)) return cudaErrorNotSupported;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most)) !=
        cudaSuccess)
      return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, kNW * 32, smem)) !=
        cudaSuccess)
      return e;
    slots = sms * per_sm;
    dev_of = dev;
    smem_of = smem;
  }
  if (slots < 1) return cudaErrorNotSupported;
  ctas = slots < kQMaxCtas ? slots : kQMaxCtas;
  return cudaSuccess;
}

template <int D, int TERMS, bool SCORES>
cudaError_t launch_dense_t(const QDecodeArgs& a, cudaStream_t st) {
  // rings (at the end the scratch of the join between CTAs), first pieces, prefix
  constexpr size_t kRing = kDenseStages * kStepOf<D> * qgroup_bytes(D), kRings = kNW * kRing;
  static_assert(kRings >= kNW * 32 * sizeof(Joined), "scratch of the join between CTAs");
  static_assert(kRing >= qpart_floats(8, D) * sizeof(float), "a warp's last piece in its ring");
  const size_t smem = kRings + kNW * qpart_floats(a.G, D) * sizeof(float) +
                      qalign16((static_cast<size_t>(a.B) + 1) * sizeof(int));
  constexpr auto kern = k_qdecode_dense<D, TERMS, SCORES>;
  int ctas = 0;
  const cudaError_t e = resident_ctas<kern>(smem, ctas);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kNW * 32), smem, st, a);
}

template <int D, int TERMS>
cudaError_t launch_dense_s(const QDecodeArgs& a, cudaStream_t st) {
  return a.scores != nullptr ? launch_dense_t<D, TERMS, true>(a, st)
                             : launch_dense_t<D, TERMS, false>(a, st);
}

template <int D, int TERMS, bool POOLED>
cudaError_t launch_reuse_t(const QDecodeArgs& a, cudaStream_t st) {
  size_t smem = kNW * qpart_floats(a.G, D) * sizeof(float);
  if (smem < kNW * 32 * sizeof(Joined)) smem = kNW * 32 * sizeof(Joined);
  constexpr auto kern = k_qdecode_reuse<D, TERMS, POOLED>;
  int ctas = 0;
  const cudaError_t e = resident_ctas<kern>(smem, ctas);
  if (e != cudaSuccess) return e;
  QDecodeArgs u = a;
  const int units = a.B * a.Hkv;
  // at least one slice per warp where the sets are long enough
  const int most = POOLED ? (a.topk + 16 * kNW - 1) / (16 * kNW)
                          : (a.G * a.topk + 16 * kNW - 1) / (16 * kNW);
  int s = ctas / units;
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;   // the last CTA joins that many pieces
  u.S = s < 1 ? 1 : s;
  return launch_pdl(kern, dim3(u.S, units), dim3(kNW * 32), smem, st, u);
}

}  // namespace

cudaError_t launch_qdecode_dense(const QDecodeArgs& a, int d, int dtype, cudaStream_t st) {
  if (dtype == KASCADE_F32)
    return d == 128 ? launch_dense_s<128, 2>(a, st) : launch_dense_s<64, 2>(a, st);
  return d == 128 ? launch_dense_s<128, 1>(a, st) : launch_dense_s<64, 1>(a, st);
}

cudaError_t launch_qdecode_reuse(const QDecodeArgs& a, int d, int dtype, cudaStream_t st) {
  const bool pooled = a.idx != nullptr;
  if (dtype == KASCADE_F32) {
    if (pooled)
      return d == 128 ? launch_reuse_t<128, 2, true>(a, st) : launch_reuse_t<64, 2, true>(a, st);
    return d == 128 ? launch_reuse_t<128, 2, false>(a, st) : launch_reuse_t<64, 2, false>(a, st);
  }
  if (pooled)
    return d == 128 ? launch_reuse_t<128, 1, true>(a, st) : launch_reuse_t<64, 1, true>(a, st);
  return d == 128 ? launch_reuse_t<128, 1, false>(a, st) : launch_reuse_t<64, 1, false>(a, st);
}

cudaError_t launch_qfill_tail(float* rows, const int32_t* lens, int B, int H, int N,
                              cudaStream_t st) {
  return launch_pdl(k_qfill_tail, dim3(B * H), dim3(256), 0, st, rows, lens, H, N);
}

}  // namespace kascade
