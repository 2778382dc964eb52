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
// down to 2^-26 of that element, an fp32 q is the sum of two fp16 terms (22
// bits). The softmax weights are kept as 2^14 p, so that a weight down to 2^-38
// of the row's largest one still counts in the product with V; smaller ones count
// in the sum of the weights alone, which is taken in fp32 before the rounding. For
// bf16 outputs a weight is one fp16 term, whose half step of 2^-11 is an eighth of
// the output's own 2^-8 (distance from 64-bit results on 8 x 32768 keys: 1.7e-3
// of the output's norm, 1.6e-3 with weights in 32 bits). For fp32 outputs it too
// is a sum of two fp16 terms.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "common.cuh"
#include "qcache.h"
#include "qmath.cuh"
#include "qprefix.cuh"

namespace kascade {
namespace {

// Slices of 16 keys per step: a step is 4608 bytes at either head size.
template <int D>
constexpr int kStepOf = 256 / D;

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with a zero addend
__device__ __forceinline__ void mma_f16_16816_first(float (&d)[4], uint32_t a0, uint32_t a1,
                                                    uint32_t a2, uint32_t a3, uint32_t b0,
                                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// -------------------------------------------------------------------- query --
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
struct QRaw {
  uint4 v[TERMS * D / 32];
};
template <int D, int TERMS>
__device__ __forceinline__ void load_q(const QDecodeArgs& a, int b, int g, QRaw<D, TERMS>& x) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
  const bool ok = gid < a.G;
  const size_t row = ok ? static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + gid] : 0;
  const uint4* p = static_cast<const uint4*>(a.q) + (row * D + c4 * (D / 4)) * TERMS / 8;
#pragma unroll
  for (int i = 0; i < TERMS * D / 32; ++i) x.v[i] = ok ? __ldg(p + i) : make_uint4(0u, 0u, 0u, 0u);
}

template <int D, int TERMS>
__device__ __forceinline__ void make_q(const QDecodeArgs& a, const QRaw<D, TERMS>& raw,
                                       QFrag<D, TERMS>& qf) {
  const int c4 = threadIdx.x & 3;
  float x[D / 4];
#pragma unroll
  for (int i = 0; i < TERMS * D / 32; ++i) {
    const uint32_t w[4] = {raw.v[i].x, raw.v[i].y, raw.v[i].z, raw.v[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (TERMS == 2) {
        x[4 * i + j] = __uint_as_float(w[j]);
      } else {   // two bf16
        x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
        x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
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

// --------------------------------------------------------------------- step --
// A step's kStepOf<D> slices lie in shared memory, each laid out as a group of
// the cache. Row r of a slice's score tile is its key row_key(r): within each
// four rows the second pair is swapped, so that the four V rows that lanes c4
// = 0 .. 3 load together (rows 2 c4 of the tile) alternate between even and odd
// keys, which halves their bank conflicts at d = 128 (64-byte rows).
__device__ __forceinline__ int row_key(int r) { return r ^ ((r >> 1) & 1); }
// key of a slice that V row i (0 .. 3) of this lane belongs to
__device__ __forceinline__ int v_key(int i) {
  return row_key(2 * (threadIdx.x & 3) + (i & 1)) + 8 * (i >> 1);
}

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one vector load");
  if (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[N / 4] = v.y;
    w[N / 2] = v.z;
    w[N - 1] = v.w;
  } else if (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[N - 1] = v.y;
  } else {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// This lane's places in a group: its D/4 elements of the K row of score row
// gid (score row gid + 8 lies 8 rows on), its elements gid * D/8 .. of the V
// rows of score rows 2 c4 and 2 c4 + 1 (and 8 rows on), and their scales.
template <int D>
struct LanePlaces {
  int k, ks, v[2], vs[2];
  __device__ __forceinline__ LanePlaces() {
    const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
    k = row_key(gid) * (D / 2) + c4 * (D / 8);
    ks = 8 * D + row_key(gid) * (D / 16) + c4 * (D / 64);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[i] = 9 * D + v_key(i) * (D / 2) + gid * (D / 16);
      vs[i] = 17 * D + v_key(i) * (D / 16) + gid * D / 128;
    }
  }
};

// Raw products of one slice: raw[0] = (score row gid, head 2 c4), raw[1] =
// (gid, 2 c4 + 1), raw[2], raw[3]: score row gid + 8.
template <int D, int TERMS>
__device__ __forceinline__ void slice_products(const uint8_t* grp, const LanePlaces<D>& at,
                                               const QFrag<D, TERMS>& qf, float (&raw)[4]) {
  uint32_t k[2][D / 32], sc[2][D / 64];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    load_words(grp + at.k + 8 * r * (D / 2), k[r]);
    const uint8_t* p = grp + at.ks + 8 * r * (D / 16);
    const uint32_t h =
        cvt_e4m3x2(D == 128 ? static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p))
                            : static_cast<uint32_t>(*p));
    sc[r][0] = __byte_perm(h, h, 0x1010);
    if (D == 128) sc[r][D / 64 - 1] = __byte_perm(h, h, 0x3232);
  }
#pragma unroll
  for (int w = 0; w < D / 32; ++w) {   // 8 elements of each row: two MMAs
    uint32_t x[4], y[4];
    cvt_e2m1x8(k[0][w], x);
    cvt_e2m1x8(k[1][w], y);
    const int blk = D == 128 ? w / 2 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = hmul2(x[i], sc[0][blk]);
      y[i] = hmul2(y[i], sc[1][blk]);
    }
#pragma unroll
    for (int t = 0; t < TERMS; ++t) {
      if (w == 0 && t == 0)
        mma_f16_16816_first(raw, x[0], y[0], x[1], y[1], qf.f[t][2 * w][0], qf.f[t][2 * w][1]);
      else
        mma_f16_16816(raw, x[0], y[0], x[1], y[1], qf.f[t][2 * w][0], qf.f[t][2 * w][1]);
      mma_f16_16816(raw, x[2], y[2], x[3], y[3], qf.f[t][2 * w + 1][0], qf.f[t][2 * w + 1][1]);
    }
  }
}

// Running state of one warp over keys of one (sequence, KV head). Thread
// (gid = lane/4, c4 = lane%4) owns heads 2 c4, 2 c4 + 1 and output dims
// gid * D/8 .. + D/8 of both: o[i] = (dim 2i, head 2c4), (2i, 2c4+1),
// (2i + 1, 2c4), (2i + 1, 2c4 + 1). m: running maxima (log2 units, within kSlack);
// nmu = 14 - m; l: this lane's sums of 2^14 p. nmu and l hold both heads, packed.
template <int D>
struct QState {
  float m[2];
  uint64_t nmu, l;
  float o[D / 16][4];
  __device__ __forceinline__ void clear() {
    m[0] = m[1] = kNoKey;
    nmu = f2_pack(kPShift - kNoKey, kPShift - kNoKey);
    l = f2_pack(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }
};

// O^T += V^T P^T of one slice with weights p and scales vs of this lane's V rows.
template <int D, int TERMS>
__device__ __forceinline__ void slice_values(float (&o)[D / 16][4], const float (&p)[4],
                                             const uint8_t* grp, const LanePlaces<D>& at,
                                             const uint32_t (&vs)[4]) {
  uint32_t v[4][D / 64];
#pragma unroll
  for (int i = 0; i < 4; ++i) load_words(grp + at.v[i & 1] + (i >> 1) * 8 * (D / 2), v[i]);
  uint32_t b[TERMS][2];
  b[0][0] = movmatrix_t(pack_f16(p[0], p[1]));
  b[0][1] = movmatrix_t(pack_f16(p[2], p[3]));
  if (TERMS == 2) {
    b[TERMS - 1][0] = movmatrix_t(pack_f16(p[0] - f16_rounded(p[0]), p[1] - f16_rounded(p[1])));
    b[TERMS - 1][1] = movmatrix_t(pack_f16(p[2] - f16_rounded(p[2]), p[3] - f16_rounded(p[3])));
  }
  const uint32_t s01 = cvt_e4m3x2(__byte_perm(vs[0], vs[1], 0x0040));
  const uint32_t s23 = cvt_e4m3x2(__byte_perm(vs[2], vs[3], 0x0040));
#pragma unroll
  for (int w = 0; w < D / 64; ++w) {
    // codes of one element of two keys side by side: even elements, odd ones
    uint32_t ea[4], da[4], eb[4], db[4];
    cvt_e2m1x8(nibbles(v[0][w], v[1][w] << 4), ea);
    cvt_e2m1x8(nibbles(v[0][w] >> 4, v[1][w]), da);
    cvt_e2m1x8(nibbles(v[2][w], v[3][w] << 4), eb);
    cvt_e2m1x8(nibbles(v[2][w] >> 4, v[3][w]), db);
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

// One step: t[i][r] holds the raw products of slice i, score row gid + 8 r, for
// both heads (masked: -inf), ml the heads' factors to log2 units. The running
// maximum moves only when a score passes it by kSlack (one vote), so the common
// step rescales nothing. fix(i, vs) may change the V scales of slice i (a masked
// key's must become 0: what lies there may be anything) and returns the heads
// of this lane (bits 0, 1) whose outputs become NaN.
template <int D, int TERMS, typename Fix>
__device__ __forceinline__ void attend(QState<D>& st, const uint64_t (&t)[kStepOf<D>][2],
                                       uint64_t ml, const uint8_t* buf, const LanePlaces<D>& at,
                                       Fix fix) {
  constexpr int kStep = kStepOf<D>;
  uint64_t y[kStep][2];
  auto exponents = [&]() {   // 14 + score - maximum; their largest over both heads
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < kStep; ++i)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // product and sum rounded apart, as the maximum was: a fused one would
        // leave the product's rounding, large for a huge score
        y[i][r] = f2_add(f2_mul(t[i][r], ml), st.nmu);
        float y0, y1;
        f2_unpack(y[i][r], y0, y1);
        top = fmax3(top, y0, y1);
      }
    return top;
  };
  if (__any_sync(0xffffffffu, exponents() > kPShift + kSlack)) {
    float x0 = kNoKey, x1 = kNoKey;
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      float a0, a1, b0, b1;
      f2_unpack(f2_mul(t[i][0], ml), a0, a1);
      f2_unpack(f2_mul(t[i][1], ml), b0, b1);
      x0 = fmax3(x0, a0, b0);
      x1 = fmax3(x1, a1, b1);
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, off));
      x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, off));
    }
    x0 = fmaxf(x0, st.m[0]);
    x1 = fmaxf(x1, st.m[1]);
    const float al0 = ex2(st.m[0] - x0), al1 = ex2(st.m[1] - x1);
    st.m[0] = x0;
    st.m[1] = x1;
    st.nmu = f2_pack(below_shift(x0), below_shift(x1));
    st.l = f2_mul(st.l, f2_pack(al0, al1));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      st.o[i][0] *= al0;
      st.o[i][1] *= al1;
      st.o[i][2] *= al0;
      st.o[i][3] *= al1;
    }
    exponents();
  }
#pragma unroll
  for (int i = 0; i < kStep; ++i) {
    const uint8_t* grp = buf + i * qgroup_bytes(D);
    uint32_t vs[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) vs[j] = grp[at.vs[j & 1] + (j >> 1) * 8 * (D / 16)];
    const uint32_t nan_heads = fix(i, vs);
    float p[4];
    f2_unpack(y[i][0], p[0], p[1]);
    f2_unpack(y[i][1], p[2], p[3]);
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = ex2(p[j]);
    st.l = f2_add(st.l, f2_add(f2_pack(p[0], p[1]), f2_pack(p[2], p[3])));
    slice_values<D, TERMS>(st.o, p, grp, at, vs);
    if ((nan_heads & 3u) != 0u) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if ((nan_heads >> (e & 1)) & 1u) st.o[j][e] = CUDART_NAN_F;
    }
  }
}

// ------------------------------------------------------------------ joining --
// A piece is one warp's (or CTA's) state over part of a (sequence, KV head):
// m[G], l[G] (log2-domain maximum; sum of 2^14 p), and at qpart_head(G) o[G][D].
template <int D>
__device__ __forceinline__ void lane_sums(const QState<D>& st, float (&l)[2]) {
  f2_unpack(st.l, l[0], l[1]);
#pragma unroll
  for (int off = 4; off < 32; off <<= 1) {
    l[0] += __shfl_xor_sync(0xffffffffu, l[0], off);
    l[1] += __shfl_xor_sync(0xffffffffu, l[1], off);
  }
}

template <int D>
__device__ __forceinline__ void piece_store(float* p, const QState<D>& st, int G) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
  float l[2];
  lane_sums(st, l);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int h = 2 * c4 + i;
    if (h >= G) continue;
    if (gid == 0) {
      p[h] = st.m[i];
      p[G + h] = l[i];
    }
    float* o = p + qpart_head(G) + h * D + gid * (D / 8);
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
// the i-th at piece(i), with the loads of several pieces in flight together.
template <bool GLOBAL, typename Piece>
__device__ __forceinline__ Joined join_some(Piece piece, int s0, int s1, int G, int h, int e) {
  constexpr int kBatch = GLOBAL ? 8 : 4;   // loads of L2 lines take longer
  Joined x = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s = s0; s < s1; s += kBatch) {
    Joined y[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      y[k] = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
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

// With a shared prefix: the token that sequence b's own part starts at.
template <bool PREFIX>
__device__ __forceinline__ int start_of(const QDecodeArgs& a, int b) {
  return PREFIX ? pfx_start(a.lens, b, a.P, a.N, a.max_blocks, a.bs_shift) : 0;
}

// The output (b, g, head slot h, dims 4 e4 ..) of a joined whole; behind a shared
// prefix its state.
template <int D, bool F32, bool PREFIX = false>
__device__ __forceinline__ void joined_output(const QDecodeArgs& a, const Joined& x, int b, int g,
                                              int h, int e4) {
  if (PREFIX) {
    const size_t at = (static_cast<size_t>(b) * a.Hkv + g) * a.G + h;
    a.state_o[at * (D / 4) + e4] = x.o;
    if (e4 == 0) a.state_ml[at] = make_float2(x.m, x.l);
    return;
  }
  const size_t row = static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + h];
  const float inv = x.l == 0.f ? 0.f : a.v_scale / x.l;   // 0: no key at all
  out_store4<F32>(a, row * D + 4 * e4,
                  make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv));
  if (e4 == 0) write_row_stat(a, row, x.m, x.l);
}

// Adds 1: what the CTA wrote before its last barrier is seen by whoever arrives
// later.
__device__ __forceinline__ unsigned int arrive_acq_rel(unsigned int* counter) {
  unsigned int old;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;"
               : "=r"(old) : "l"(counter) : "memory");
  return old;
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
template <int D, bool F32, bool PREFIX = false>
__device__ void arrive_and_join(const QDecodeArgs& a, int n_units, const SharedUnit (&units)[2],
                                Joined* scratch) {
  __shared__ unsigned int s_last;
  const int tid = threadIdx.x, G = a.G;
  __syncthreads();   // every piece of this CTA is written
  if (tid < 32) {    // a lane per unit
    bool mine = false;
    if (tid < n_units) {
      const int unit = tid == 0 ? units[0].unit : units[1].unit;
      const int n = tid == 0 ? units[0].n : units[1].n;
      mine = arrive_acq_rel(&a.counters[unit]) == static_cast<unsigned int>(n - 1);
      if (mine) a.counters[unit] = 0u;   // ready for the next launch
    }
    const unsigned int last = __ballot_sync(0xffffffffu, mine);
    if (tid == 0) s_last = last;
  }
  __syncthreads();
  const unsigned int last = s_last;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!((last >> k) & 1u)) continue;
    const SharedUnit& u = units[k];
    const int n = u.n;
    auto mine = [&](int i) -> const float* { return i == 0 ? u.first : u.rest + (i - 1) * u.step; };
    const int elems = G * (D / 4), threads = static_cast<int>(blockDim.x);   // 16 .. 256
    int shares = threads / elems;
    if (shares > (n + 3) / 4) shares = (n + 3) / 4;
    if (shares <= 1) {
      for (int e = tid; e < elems; e += threads) {
        const int h = e / (D / 4);
        joined_output<D, F32, PREFIX>(a, join_some<true>(mine, 0, n, G, h, e), u.b, u.g, h,
                                      e & (D / 4 - 1));
      }
      continue;
    }
    const int e = tid % elems, share = tid / elems, h = e / (D / 4), e4 = e & (D / 4 - 1);
    const int per = (n + shares - 1) / shares;
    Joined x = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (share < shares) x = join_some<true>(mine, share * per, min(n, (share + 1) * per), G, h, e);
    if (share > 0 && share < shares) scratch[tid] = x;
    __syncthreads();
    if (share == 0) {
      for (int i = 1; i < shares; ++i) {
        const Joined y[1] = {scratch[i * elems + e]};
        join_into(x, y);
      }
      joined_output<D, F32, PREFIX>(a, x, u.b, u.g, h, e4);
    }
    __syncthreads();
  }
}

// A whole unit held by one warp: straight from its registers to the output.
template <int D, bool F32, bool PREFIX>
__device__ __forceinline__ void warp_output(const QDecodeArgs& a, const QState<D>& st, int b,
                                            int g) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
  float l[2];
  lane_sums(st, l);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (2 * c4 + i >= a.G) continue;
    if (PREFIX) {
#pragma unroll
      for (int j = 0; j < D / 16; j += 2)
        joined_output<D, F32, true>(
            a, {st.m[i], l[i], make_float4(st.o[j][i], st.o[j][2 + i], st.o[j + 1][i], st.o[j + 1][2 + i])},
            b, g, 2 * c4 + i, gid * (D / 32) + j / 2);
      continue;
    }
    const size_t row = static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + 2 * c4 + i];
    const float inv = l[i] == 0.f ? 0.f : a.v_scale / l[i];
#pragma unroll
    for (int j = 0; j < D / 16; j += 2)
      out_store4<F32>(a, row * D + gid * (D / 8) + 2 * j,
                      make_float4(st.o[j][i] * inv, st.o[j][2 + i] * inv, st.o[j + 1][i] * inv,
                                  st.o[j + 1][2 + i] * inv));
    if (gid == 0) write_row_stat(a, row, st.m[i], l[i]);
  }
}

// -------------------------------------------------------------------- dense --
// The steps of all units (unit = sequence * Hkv + KV head; a step is 16 *
// kStep keys, and a sequence of n keys has ceil(n / (16 kStep)) per head) form one
// line, and every warp of the grid takes an equal run of it, so that ragged
// batches balance. A unit starts with kUnitCost places without a step: what
// its query, its first loads and its output cost a warp, so that runs of many
// short units do not come last (48 sequences of 0 to 16001 keys: 82 us without,
// 72 with one place, 66 with two, 67 with four; 63.5 after later steps). A run
// may span units: the warp's pieces of units it does not hold alone go to shared
// memory, the CTA joins those of its warps after one barrier, and a unit that
// several CTAs share is joined by the last of them to arrive.
//
// Every warp feeds itself: a ring of kDenseStages stages of one step, each
// filled by one bulk copy per block that the step touches (groups of a block
// are contiguous), which the first lanes issue as soon as the warp has left
// the stage; no warp waits for another one before the end.
// One CTA of 16 warps per SM: on a GB300 the 8B shape took 65.5 us so, 67.3 as
// two CTAs of 8 and 69.2 as four of 4 (the joins get longer); five of 4, with
// 102 registers per thread, 95; three stages per ring changed nothing.
// What bounds it: 8 sequences of 32768 keys, 8 KV heads of 4 query heads, d 128,
// are 302 MB in 61.1 us = 4.9 TB/s (0.73 of the copy rate). Time stamps of that
// launch: every warp has its places after 1.7 us and its first step after 7.7 (all
// rings fill at once), the warps' loops end between 55.6 and 58.1 (the SMs' means
// within 0.5 of one another, a CTA's warps 3.4 apart), the CTAs' joins take 1.1 us
// and those between CTAs 2.2. A copy of the kernel that moved the bytes and
// computed nothing took 57.7 us before the joins were shortened by 1.5; the
// arithmetic issues 331 instructions per 16 keys (16 HMMA of 8 cycles, 64
// conversions of code pairs on the half-rate ALU) and keeps the issue slots 60%
// busy meanwhile.
constexpr int kNW = 16, kDenseCtasPerSm = 1;
constexpr int kMinRun = 2;        // steps per warp at least
constexpr int kDenseStages = 2;

constexpr int kUnitCost = 2;

// The pages are read once, so their L2 lines are the first to go (62.6 us
// against 63.5 on the 8B shape). With logits that leaves room for them until the
// Top-k has read them, as long as they fit: an anchor layer with 34 MB of them takes
// 104 us against 107, with 98 MB 120 against 126; 134 MB pass the cache's 129 MB
// and are best written out at once: 158 us against 154.
constexpr size_t kL2Logits = size_t(100) << 20;

// The part of a run that lies in the unit at place f of the line: steps [s0, s1)
// of its ns (none, if the run has only the unit's first place), and the place
// behind it.
struct Part {
  int b, g, n;     // sequence, KV head, cached tokens
  int ns, s0, s1;
  int next;
};
template <bool PREFIX>
__device__ __forceinline__ Part part_at(const QDecodeArgs& a, const int* pref, int f, int end) {
  int lo = 0, hi = a.B;   // the sequence: pref[lo] * Hkv <= f < pref[lo + 1] * Hkv
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] * a.Hkv <= f) lo = mid;
    else hi = mid;
  }
  Part p;
  p.b = lo;
  p.n = len_of(a, lo, false) - start_of<PREFIX>(a, lo);
  const int places = pref[lo + 1] - pref[lo];
  const int in = f - pref[lo] * a.Hkv;
  p.g = in / places;
  const int at = in - p.g * places;
  p.ns = places - kUnitCost;
  p.next = min(end, f + places - at);
  p.s0 = max(0, at - kUnitCost);
  p.s1 = max(0, at - kUnitCost + p.next - f);
  return p;
}

template <int D, int TERMS, bool SCORES, bool PREFIX>
__global__ void __launch_bounds__(kNW * 32, kDenseCtasPerSm)
    k_qdecode_dense(const __grid_constant__ QDecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr bool F32 = TERMS == 2;
  constexpr int kStep = kStepOf<D>, kKeys = 16 * kStep;
  constexpr int kGroupBytes = qgroup_bytes(D), kStageBytes = kStep * kGroupBytes;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ __align__(8) uint64_t s_full[kNW][kDenseStages];
  __shared__ int s_tot[kNW];
  __shared__ int s_unit[2 * kNW], s_list[2 * kNW], s_start[2 * kNW + 1], s_nunits;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c4 = lane & 3;
  const int pf = static_cast<int>(qpart_floats(a.G, D));
  // a ring per warp, which at the end holds the warp's last piece; places before
  // every sequence in the line, per head; room for the warps' first pieces (in
  // global memory, behind the CTAs' pieces, where a batch's places take it)
  uint8_t* ring = smem + warp * kDenseStages * kStageBytes;
  int* pref = reinterpret_cast<int*>(smem + kNW * kDenseStages * kStageBytes);   // [B + 1]
  float* firsts = a.firsts_global
                      ? a.part + (2 * static_cast<size_t>(gridDim.x) + blockIdx.x * kNW) * pf
                      : reinterpret_cast<float*>(reinterpret_cast<unsigned char*>(pref) +
                                                 qalign16((static_cast<size_t>(a.B) + 1) * 4));
  auto slot_at = [&](int i) -> float* {   // slot 2w: warp w's first piece, 2w + 1: its last
    return (i & 1) ? reinterpret_cast<float*>(smem + (i >> 1) * kDenseStages * kStageBytes)
                   : firsts + static_cast<size_t>(i >> 1) * pf;
  };

  if (lane == 0)
    for (int i = 0; i < kDenseStages; ++i) mbar_init(&s_full[warp][i], 1);
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kNW * 32) {
    const int b = b0 + tid;
    int n = b < a.B ? (len_of(a, b, blockIdx.x == 0) - start_of<PREFIX>(a, b) + kKeys - 1) / kKeys : 0;
    if (n > 0) n += kUnitCost;
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

  // ---- copies, kDenseStages steps ahead of the arithmetic. Lane i < ncopy
  // issues the step's i-th copy; its block id is loaded when the step before
  // is issued.
  const int copy_sh = min(a.bs_shift, D == 128 ? 5 : 6);   // log2 of a copy's keys
  const int ncopy = kKeys >> copy_sh;
  const uint32_t copy_bytes = static_cast<uint32_t>(kGroupBytes) << (copy_sh - 4);
  const uint32_t gmask = (1u << (a.bs_shift - 4)) - 1u;
  const uint32_t head_bytes = static_cast<uint32_t>(kGroupBytes) << (a.bs_shift - 4);
  const uint32_t block_bytes = head_bytes * static_cast<uint32_t>(a.Hkv);
  int in_next = w0;               // place of the unit after the one being issued
  int in_left = 0;                // steps of the run left to issue in this unit
  int in_key = 0, in_n = 0;       // this lane's copy: first key, tokens of the sequence
  const int32_t* in_row = a.table;     // the sequence's row of the block table
  const uint8_t* in_base = a.cache;    // the KV head's place in block 0
  int id = 0;                     // this lane's block
  int in_stage = 0;
  unsigned int have = 0u;         // byte i: the copies that stage i got
  int pending = 0;                // steps issued and not taken
  bool alive = true;
  auto enter = [&](const Part& p) {
    in_next = p.next;
    in_left = p.s1 - p.s0;
    in_key = lane < ncopy ? p.s0 * kKeys + (lane << copy_sh) : p.n;   // other lanes copy nothing
    in_n = p.n;
    in_row = a.table + static_cast<size_t>(p.b) * a.max_blocks +
             (start_of<PREFIX>(a, p.b) >> a.bs_shift);
    in_base = a.cache + static_cast<size_t>(p.g) * head_bytes;
  };
  auto fetch_id = [&]() {
    id = 0;
    if (in_key < in_n) id = __ldg(in_row + (in_key >> a.bs_shift));
  };
  auto issue = [&]() {            // all lanes; in_left > 0 holds
    const bool want = in_key < in_n;
    const bool ok = want && static_cast<uint32_t>(id) < static_cast<uint32_t>(a.num_blocks);
    const unsigned int got = __ballot_sync(0xffffffffu, ok);
    uint64_t* bar = &s_full[warp][in_stage];
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(got) * copy_bytes);
    __syncwarp();
    if (ok) {
      uint8_t* dst = ring + in_stage * kStageBytes + lane * copy_bytes;
      const uint8_t* src = in_base +
                           static_cast<uint64_t>(static_cast<uint32_t>(id)) * block_bytes +
                           ((static_cast<uint32_t>(in_key) >> 4) & gmask) * kGroupBytes;
      if (SCORES && !a.pages_once) bulk_load(dst, src, copy_bytes, bar);
      else bulk_load_once(dst, src, copy_bytes, bar);
    } else if (want) {
      report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x522);
    }
    have = __byte_perm(have, got, in_stage == 0 ? 0x3214 : 0x3240);
    in_stage ^= 1;
    ++pending;
    in_key += kKeys;
    if (lane >= ncopy) in_key = in_n;
    if (--in_left == 0) {
      while (in_left == 0 && in_next < w1) enter(part_at<PREFIX>(a, pref, in_next, w1));
    }
    if (in_left > 0) fetch_id();
  };
  static_assert(kDenseStages == 2, "stages alternate");
  Part at = {};
  QRaw<D, TERMS> qx;   // the query of the unit that comes next
  at.next = w0;
  while (at.s0 == at.s1 && at.next < w1) at = part_at<PREFIX>(a, pref, at.next, w1);
  if (at.s0 < at.s1) {
    enter(at);
    fetch_id();
    load_q<D, TERMS>(a, at.b, at.g, qx);
    issue();
    if (in_left > 0) issue();
  }

  // ---- arithmetic
  const LanePlaces<D> places;
  const int row0 = row_key(gid);   // keys row0 and row0 + 8 of a slice
  int stage = 0;
  uint32_t phase = 0;
  for (bool first_unit = true; at.s0 < at.s1; first_unit = false) {
    const int n = at.n, steps = at.s1 - at.s0;
    int first = at.s0 * kKeys;   // first key of the step
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
    QState<D> st;
    st.clear();
    for (int left = steps; left > 0 && alive; --left, first += kKeys) {
      if (!__all_sync(0xffffffffu, mbar_try_wait(&s_full[warp][stage], phase)) &&
          !mbar_wait_warp(&s_full[warp][stage], phase, a.err, 0x531)) {
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
        uint64_t t[kStep][2];
#pragma unroll
        for (int i = 0; i < kStep; ++i) {
          float raw[4];
          slice_products(buf + i * kGroupBytes, places, qf, raw);
          t[i][0] = f2_pack(raw[0], raw[1]);
          t[i][1] = f2_pack(raw[2], raw[3]);
        }
        // keys that do not count: behind the sequence's end, or in a block the
        // table does not name
        const bool full = got == (1u << ncopy) - 1u && first + kKeys <= n;
        if (!full) {
          // rare, and kept apart by its loop: as selects in every step it cost
          // 30 instructions a slice. What lies in these keys' V rows may be
          // anything: their scales become 0 in the stage.
          auto counts = [&](int key) {
            return ((got >> (key >> copy_sh)) & 1u) != 0u && first + key < n;
          };
          for (int r = lane; r < kKeys; r += 32)
            if (!counts(r)) {
              uint8_t* sc = ring + stage * kStageBytes + (r >> 4) * kGroupBytes + 17 * D +
                            (r & 15) * (D / 16);
#pragma unroll
              for (int i = 0; i < D / 64; ++i) reinterpret_cast<uint32_t*>(sc)[i] = 0u;
            }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kStep; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (!counts(16 * i + row0 + 8 * r)) t[i][r] = f2_pack(kNegInf, kNegInf);
        }
        if (SCORES) {
#pragma unroll
          for (int i = 0; i < kStep; ++i)
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const int key = first + row0 + 16 * i + 8 * r;
              float v0, v1;
              f2_unpack(t[i][r], v0, v1);
              if (full || key < n) {
                if (sp[0] != nullptr) sp[0][key] = v0 * qf.mult[0];
                if (sp[1] != nullptr) sp[1][key] = v1 * qf.mult[1];
              }
            }
        }
        if (got != 0u)
          attend<D, TERMS>(st, t, ml, buf, places, [](int, uint32_t (&)[4]) { return 0u; });
      }
      stage ^= 1;
      phase ^= stage == 0 ? 1u : 0u;
      --pending;
      // the stage is refilled through the async proxy: this warp's reads first
      fence_proxy_async_smem();
      __syncwarp();
      if (in_left > 0) issue();
    }
    if (steps == at.ns) {
      warp_output<D, F32, PREFIX>(a, st, at.b, at.g);
    } else {
      // in part: a run's first unit or its last (whose ring is free by then)
      const int slot = 2 * warp + (first_unit ? 0 : 1);
      piece_store<D>(slot_at(slot), st, a.G);
      if (lane == 0) s_unit[slot] = at.b * a.Hkv + at.g;
    }
    // the run's next unit
    int next = at.next;
    at.s0 = at.s1 = 0;
    while (at.s0 == at.s1 && next < w1) {
      at = part_at<PREFIX>(a, pref, next, w1);
      next = at.next;
    }
    if (at.s0 < at.s1) load_q<D, TERMS>(a, at.b, at.g, qx);
  }
  __syncthreads();
  static_assert(2 * kNW == 32 && kNW + 2 <= kQPieces / kQMaxCtas,
                "a lane per slot, pieces per CTA");
  if (warp == 0) {   // the slots in use, in order, and where each unit's begin
    const int unit = s_unit[lane];
    const unsigned int m = __ballot_sync(0xffffffffu, unit >= 0), below = (1u << lane) - 1u;
    const int before = __shfl_sync(0xffffffffu, unit, (31 - __clz(m & below)) & 31);
    const bool first = unit >= 0 && ((m & below) == 0u || before != unit);
    const unsigned int f = __ballot_sync(0xffffffffu, first);
    if (unit >= 0) s_list[__popc(m & below)] = lane;
    if (first) s_start[__popc(f & below)] = __popc(m & below);
    if (lane == 0) {
      s_nunits = __popc(f);
      s_start[__popc(f)] = __popc(m);
    }
  }
  __syncthreads();
  const int nunits = s_nunits;
  const int per_cta = per * kNW, c0 = static_cast<int>(blockIdx.x) * per_cta;
  // This CTA's pieces, in order of their units: a unit is joined here if the
  // CTA holds all of it, else its piece goes to CTA c's place 2c + 1 (a unit
  // that starts inside c's run) or 2c (one that started before it, or with it).
  const size_t stride = qpart_floats(a.G, D);
  SharedUnit shared[2] = {};   // at most the first and the last unit of the run
  int n_shared = 0;
  const int elems = a.G * (D / 4);
  for (int k = 0, first_elem = 0; k < nunits; ++k, first_elem += elems) {
    const int i = s_start[k], j = s_start[k + 1], unit = s_unit[s_list[i]];
    const int b = unit / a.Hkv, g = unit % a.Hkv, nb = pref[b + 1] - pref[b];
    const int u1 = pref[b] * a.Hkv + (g + 1) * nb, u0 = u1 - nb + kUnitCost;   // its steps' places
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
    for (int e = (tid - first_elem) & (kNW * 32 - 1); e < elems; e += kNW * 32) {
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
        joined_output<D, F32, PREFIX>(a, x, b, g, h, e4);
      }
    }
  }
  if (n_shared > 0)
    arrive_and_join<D, F32, PREFIX>(a, n_shared, shared, reinterpret_cast<Joined*>(smem));
  // sequences without keys: zeros; scores behind the last key
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    if (pref[b + 1] != pref[b]) continue;
    if (PREFIX) {
      for (int e = tid; e < a.Hq * (D / 4); e += kNW * 32)
        joined_output<D, F32, true>(a, {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)}, b,
                                    e / elems, e % elems / (D / 4), e & (D / 4 - 1));
      continue;
    }
    const size_t base = static_cast<size_t>(b) * a.Hq * D;
    for (int e = 4 * tid; e < a.Hq * D; e += 4 * kNW * 32)
      out_store4<F32>(a, base + e, make_float4(0.f, 0.f, 0.f, 0.f));
    for (int h = tid; h < a.Hq; h += kNW * 32)
      write_row_stat(a, static_cast<size_t>(b) * a.Hq + h, kNoKey, 0.f);
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
// One (sequence, KV head) per blockIdx.y. Its gather list (per query head sets:
// the union plan's entries key | head mask << 24, in 16-entry slices per plan
// chunk; pooled: the set itself) is numbered in steps of kStepOf<D> slices, and
// the steps are split into S equal runs, one per CTA, whose steps go to the
// CTA's warps in turn. A warp gathers each step's rows through the block table
// into the group layout of one of its two stages (16-byte cp.async for codes,
// one 8- or 4-byte one per row for scales; rows of no use are zero-filled, not
// read), so that the arithmetic is the dense kernel's. Entries are loaded two
// steps before their copies and block ids one step before, so that no copy
// waits for either.
// Four CTAs per SM, 128 registers per thread, took 52.0 us on the 8B shape (with
// the plan), three 49.3; one or two larger CTAs per SM 56.8 and 55.6.
// What bounds it: scattered rows. DRAM delivers 64 bytes for each 64-byte row of
// codes and as many for its 8 bytes of scales: 8B shape, 4096 of 32768 keys per
// head, 37.6 us from cold caches for 127 MB of useful bytes (3.4 TB/s), of which
// 29 between the first step and the last at 5.1 TB/s of DRAM traffic. Three or four
// stages per ring change nothing.
constexpr int kReuseNW = 4, kReuseStages = 2, kReuseCtasPerSm = 3;
// A row in one word: the group's number in the cache and the row in it.
constexpr uint32_t kNoRow = 0xffffffffu;

template <int D, int TERMS, bool POOLED>
__global__ void __launch_bounds__(kReuseNW * 32, kReuseCtasPerSm)
    k_qdecode_reuse(const __grid_constant__ QDecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr bool F32 = TERMS == 2;
  constexpr int kStep = kStepOf<D>, kRows = 16 * kStep, kPer = kRows / 32;   // rows per lane
  constexpr int kGroupBytes = qgroup_bytes(D), kStageBytes = kStep * kGroupBytes;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int s_pref[kMaxSplits + 1], s_cnt[kMaxSplits];
  __shared__ unsigned char s_mask[kReuseNW][kReuseStages][kRows];   // heads per gathered row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c4 = lane & 3;
  const int pf = static_cast<int>(qpart_floats(a.G, D));
  uint8_t* ring = smem + warp * kReuseStages * kStageBytes;   // at the end: the warp's piece
  const int unit = blockIdx.y, b = unit / a.Hkv, g = unit % a.Hkv;
  QRaw<D, TERMS> qx;
  load_q<D, TERMS>(a, b, g, qx);
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
  if (!POOLED) __syncthreads();
  const int slices = POOLED ? (a.topk + 15) / 16 : s_pref[nch];
  const int total = (slices + kStep - 1) / kStep;
  const int per = (total + a.S - 1) / a.S;
  const int g0 = min(total, static_cast<int>(blockIdx.x) * per), g1 = min(total, g0 + per);
  const int32_t* set = POOLED ? a.idx + static_cast<size_t>(unit) * a.topk : nullptr;
  const int32_t* trow = a.table + static_cast<size_t>(b) * a.max_blocks;
  const int sh = a.bs_shift - 4, gmask = (1 << sh) - 1;

  // ---- gather: row j of lane l is row l + 32 j of a step
  int fc[kPer] = {};        // plan chunk cursors: rows only move forward
  int2 raw[kPer];           // entries of the step after the next to be copied (pooled: and
                            // the entry before each)
  int key[kPer], blk[kPer]; // rows of the next step to be copied
  uint32_t mask[kPer];
  auto fetch = [&](int step) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      raw[j] = POOLED ? make_int2(-1, -1) : make_int2(0, 0);
      if (step >= g1) continue;
      const int row = lane + 32 * j;
      if (POOLED) {
        const int e = step * kRows + row;
        if (e < a.topk) raw[j] = make_int2(__ldg(set + e), e > 0 ? __ldg(set + e - 1) : -2);
      } else {
        const int sl = step * kStep + (row >> 4);
        if (sl >= slices) continue;
        while (fc[j] + 1 < nch && s_pref[fc[j] + 1] <= sl) ++fc[j];
        const int e = (sl - s_pref[fc[j]]) * 16 + (row & 15);
        if (e < s_cnt[fc[j]])
          raw[j].x = static_cast<int>(
              __ldg(a.plan + (static_cast<size_t>(unit) * nch + fc[j]) * kPlanCapEntries + e));
      }
    }
  };
  auto resolve = [&]() {    // the fetched entries become rows; their block ids are requested
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      mask[j] = 0u;
      key[j] = blk[j] = 0;
      if (POOLED) {
        const int k = raw[j].x, before = raw[j].y;   // -2 before the first entry
        const bool ok = k >= 0 && k < n && k > before && before != -1;
        if (ok) {
          key[j] = k;
          mask[j] = (1u << a.G) - 1u;
        } else if (k != -1) {
          report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x523);
        }
      } else {
        const int k = raw[j].x & 0xffffff;
        if (k < n) {
          key[j] = k;
          mask[j] = static_cast<uint32_t>(raw[j].x) >> 24;
        }
      }
      if (mask[j] != 0u) blk[j] = __ldg(trow + (key[j] >> a.bs_shift));
    }
  };
  auto copy = [&](int stage) {
    uint8_t* dst = ring + stage * kStageBytes;
    uint32_t place[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      place[j] = kNoRow;
      if (mask[j] != 0u) {
        if (static_cast<unsigned int>(blk[j]) < static_cast<unsigned int>(a.num_blocks)) {
          const uint32_t grp = ((static_cast<uint32_t>(blk[j]) * a.Hkv + g) << sh) |
                               ((key[j] >> 4) & gmask);
          place[j] = (grp << 4) | (key[j] & 15);
        } else {
          report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x522);
        }
      }
      const bool ok = place[j] != kNoRow;
      const int row = lane + 32 * j;
      s_mask[warp][stage][row] = static_cast<unsigned char>(ok ? mask[j] : 0u);
      // this lane's own rows' scales
      const uint8_t* src = a.cache + static_cast<size_t>(ok ? place[j] >> 4 : 0u) * kGroupBytes +
                           8 * D + (ok ? place[j] & 15u : 0u) * (D / 16);
      uint8_t* to = dst + (row >> 4) * kGroupBytes + 8 * D + (row & 15) * (D / 16);
      cp_async_scattered<D / 16>(to, src, ok);
      cp_async_scattered<D / 16>(to + 9 * D, src + 9 * D, ok);
    }
    constexpr int kChunks = D / 32;               // 16-byte pieces of a row's codes
    constexpr int kTurns = kRows * kChunks / 32;
    const int ch = lane % kChunks;
#pragma unroll
    for (int i = 0; i < kTurns; ++i) {
      const int row = lane / kChunks + i * (32 / kChunks);
      const uint32_t pl = __shfl_sync(0xffffffffu, place[(i * (32 / kChunks)) / 32], row & 31);
      const bool ok = pl != kNoRow;
      const uint8_t* src = a.cache + static_cast<size_t>(ok ? pl >> 4 : 0u) * kGroupBytes +
                           (ok ? pl & 15u : 0u) * (D / 2) + ch * 16;
      uint8_t* to = dst + (row >> 4) * kGroupBytes + (row & 15) * (D / 2) + ch * 16;
      cp_async_scattered<16>(to, src, ok);
      cp_async_scattered<16>(to + 9 * D, src + 9 * D, ok);
    }
  };
  int next = g0 + warp;           // step that is copied next
  fetch(next);
  resolve();
  fetch(next + kReuseNW);
#pragma unroll
  for (int i = 0; i < kReuseStages; ++i) {
    if (next < g1) copy(i);
    cp_async_commit();
    next += kReuseNW;
    resolve();
    fetch(next + kReuseNW);
  }

  // ---- arithmetic
  QFrag<D, TERMS> qf;
  make_q(a, qx, qf);
  const uint64_t ml = f2_pack(qf.mult[0] * kLog2e, qf.mult[1] * kLog2e);
  const LanePlaces<D> places;
  const int row0 = row_key(gid);
  QState<D> st;
  st.clear();
  int stage = 0;
  for (int s = g0 + warp; s < g1; s += kReuseNW) {
    cp_async_wait<kReuseStages - 1>();
    __syncwarp();
    const uint8_t* buf = ring + stage * kStageBytes;
    const unsigned char* masks = s_mask[warp][stage];
    uint64_t t[kStep][2];
#pragma unroll
    for (int i = 0; i < kStep; ++i) {
      float r[4];
      slice_products(buf + i * kGroupBytes, places, qf, r);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t m = masks[16 * i + row0 + 8 * e] >> (2 * c4);
        t[i][e] = f2_pack((m & 1u) ? r[2 * e] : kNegInf, (m & 2u) ? r[2 * e + 1] : kNegInf);
      }
    }
    attend<D, TERMS>(st, t, ml, buf, places, [&](int i, uint32_t (&vs)[4]) -> uint32_t {
      if (POOLED) return 0u;
      // A V block that holds a NaN (scale 0x7f or 0xff) would reach every head of
      // the group through 0 * NaN in the product: it is taken out of the
      // slice, and only the heads whose set holds the key get the NaN.
      const uint32_t vs4 = __byte_perm(__byte_perm(vs[0], vs[1], 0x0040),
                                       __byte_perm(vs[2], vs[3], 0x0040), 0x5410);
      const uint32_t bad = __vcmpeq4(vs4 & 0x7f7f7f7fu, 0x7f7f7f7fu);
      if (!__any_sync(0xffffffffu, bad != 0u)) return 0u;
      uint32_t heads = 0u;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if ((bad >> (8 * j)) & 1u) {
          vs[j] = 0u;
          heads |= masks[16 * i + v_key(j)];
        }
      // the four lanes that share these dims hold other keys and other heads
      heads |= __shfl_xor_sync(0xffffffffu, heads, 1);
      heads |= __shfl_xor_sync(0xffffffffu, heads, 2);
      return heads >> (2 * c4);
    });
    __syncwarp();   // the stage is free
    if (next < g1) copy(stage);
    cp_async_commit();
    next += kReuseNW;
    resolve();
    fetch(next + kReuseNW);
    stage ^= 1;
  }
  static_assert(kReuseStages == 2, "stages alternate");
  cp_async_wait<0>();
  __syncwarp();
  auto slot = [&](int w) { return reinterpret_cast<float*>(smem + w * kReuseStages * kStageBytes); };
  piece_store<D>(slot(warp), st, a.G);
  __syncthreads();
  float* part = a.part + static_cast<size_t>(unit) * a.S * pf;
  float* dst = part + static_cast<size_t>(blockIdx.x) * pf;
  const int elems = a.G * (D / 4);
  for (int e = tid; e < elems; e += kReuseNW * 32) {
    const int h = e / (D / 4), e4 = e & (D / 4 - 1);
    const Joined x = join_some<false>([&](int w) -> const float* { return slot(w); }, 0, kReuseNW,
                                      a.G, h, e);
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
  arrive_and_join<D, F32>(a, 1, units, reinterpret_cast<Joined*>(smem));
}

// CTAs of a kernel that the current device holds at once (asked once per host
// thread, device and shared memory size). The kernel may use all the shared
// memory there is: the same value whatever the call, so that threads calling
// with different sizes do not undo one another's setting.
template <void (*kern)(const QDecodeArgs)>   // by value: each kernel has its own record
cudaError_t resident_ctas(size_t smem, int threads, int& ctas) {
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
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem)) !=
        cudaSuccess)
      return e;
    slots = sms * per_sm;
    dev_of = dev;
    smem_of = smem;
  }
  if (slots < 1) return cudaErrorNotSupported;
  ctas = slots;
  return cudaSuccess;
}

template <int D, int TERMS, bool SCORES, bool PREFIX>
cudaError_t launch_dense_t(const QDecodeArgs& a, cudaStream_t st) {
  // rings (at the end the scratch of the join between CTAs), places, first
  // pieces; the latter only up to what fits beside them at every batch size
  // (16384 sequences: 64 KB of places)
  constexpr size_t kRing = kDenseStages * kStepOf<D> * qgroup_bytes(D), kRings = kNW * kRing;
  static_assert(kRings >= kNW * 32 * sizeof(Joined), "scratch of the join between CTAs");
  static_assert(kRing >= qpart_floats(8, D) * sizeof(float), "a warp's last piece in its ring");
  size_t smem = kRings + qalign16((static_cast<size_t>(a.B) + 1) * sizeof(int));
  const size_t firsts = kNW * qpart_floats(a.G, D) * sizeof(float);
  QDecodeArgs u = a;
  u.firsts_global = smem + firsts > 224 * 1024 ? 1 : 0;
  u.pages_once = static_cast<size_t>(a.B) * a.Hq * a.N * 4 <= kL2Logits ? 1 : 0;
  if (!u.firsts_global) smem += firsts;
  constexpr auto kern = k_qdecode_dense<D, TERMS, SCORES, PREFIX>;
  int ctas = 0;
  const cudaError_t e = resident_ctas<kern>(smem, kNW * 32, ctas);
  if (e != cudaSuccess) return e;
  if (ctas > kQMaxCtas) ctas = kQMaxCtas;
  if (a.max_ctas > 0) {
    // beside another kernel: both SMs of a TPC or none (clusters of two), since a CTA of
    // each kernel on one TPC slows both down (10 to 40%)
    if (ctas > a.max_ctas) ctas = a.max_ctas;
    if (ctas > 1)
      return launch_pdl_clusters(2, kern, dim3(ctas & ~1), dim3(kNW * 32), smem, st, u);
  }
  return launch_pdl(kern, dim3(ctas), dim3(kNW * 32), smem, st, u);
}

template <int D, int TERMS>
cudaError_t launch_dense_s(const QDecodeArgs& a, cudaStream_t st) {
  if (a.P > 0) return launch_dense_t<D, TERMS, false, true>(a, st);
  return a.scores != nullptr ? launch_dense_t<D, TERMS, true, false>(a, st)
                             : launch_dense_t<D, TERMS, false, false>(a, st);
}

template <int D, int TERMS, bool POOLED>
cudaError_t launch_reuse_t(const QDecodeArgs& a, cudaStream_t st) {
  constexpr size_t kRing = kReuseStages * kStepOf<D> * qgroup_bytes(D), smem = kReuseNW * kRing;
  static_assert(smem >= kReuseNW * 32 * sizeof(Joined), "scratch of the join between CTAs");
  static_assert(kRing >= qpart_floats(8, D) * sizeof(float), "a warp's piece in its ring");
  constexpr auto kern = k_qdecode_reuse<D, TERMS, POOLED>;
  int ctas = 0;
  const cudaError_t e = resident_ctas<kern>(smem, kReuseNW * 32, ctas);
  if (e != cudaSuccess) return e;
  if (ctas > kQPieces) ctas = kQPieces;   // a place per CTA, as S * units <= ctas or S = 1
  QDecodeArgs u = a;
  const int units = a.B * a.Hkv;
  // as many CTAs per unit as fill one wave, and at least one step per warp
  // where the sets are long enough
  const int rows = (POOLED ? 1 : a.G) * a.topk, cta_rows = 16 * kStepOf<D> * kReuseNW;
  const int most = (rows + cta_rows - 1) / cta_rows;
  int s = ctas / units;
  if (s > most) s = most;
  if (s > kMaxSplits) s = kMaxSplits;   // the last CTA joins that many pieces
  u.S = s < 1 ? 1 : s;
  return launch_pdl(kern, dim3(u.S, units), dim3(kReuseNW * 32), smem, st, u);
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
