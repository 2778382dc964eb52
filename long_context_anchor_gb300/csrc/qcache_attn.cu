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
constexpr int kNW = 8;               // warps per CTA

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
__device__ __forceinline__ float f16_rounded(float x) { return __half2float(__float2half_rn(x)); }

// Running state of one warp over the keys of one (sequence, KV head). Thread
// (gid = lane/4, c4 = lane%4) owns heads 2 c4, 2 c4 + 1 and output dims
// gid * D/8 .. + D/8 of both: o[i] = (dim 2i, head 2c4), (2i, 2c4+1),
// (2i + 1, 2c4), (2i + 1, 2c4 + 1).
template <int D>
struct QState {
  float m[2], l[2];
  float o[D / 16][4];
};

template <int D>
__device__ __forceinline__ void qstate_init(QState<D>& st) {
  st.m[0] = st.m[1] = kNegInf;
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

template <int D, int TERMS>
__device__ void load_q(const QDecodeArgs& a, int b, int g, QFrag<D, TERMS>& qf) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, c4 = lane & 3;
  float x[D / 4];
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
  const float down = a.scale * ldexpf(1.f, e - kQExp);
  qf.mult[0] = __shfl_sync(0xffffffffu, down, 8 * c4);
  qf.mult[1] = __shfl_sync(0xffffffffu, down, 8 * c4 + 4);
}

// One slice of 16 keys in registers: the K rows of keys gid and gid + 8 (this
// lane's D/4 elements of each), the V rows of keys 2 c4, 2 c4 + 1, 2 c4 + 8,
// 2 c4 + 9 (elements gid * D/8 .. of each), and their scales.
template <int D>
struct QSlice {
  uint32_t k[2][D / 32];
  uint32_t ks[2];        // e4m3 bytes: two at d = 128, one at d = 64
  uint32_t v[4][D / 64];
  uint32_t vs[4];
};

// raw[0] = (key gid, head 2c4), raw[1] = (gid, 2c4+1), raw[2], raw[3]: gid + 8
template <int D, int TERMS>
__device__ __forceinline__ void slice_logits(const QSlice<D>& s, const QFrag<D, TERMS>& qf,
                                             float (&raw)[4]) {
  float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
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
      mma_f16_16816(acc[0], x[0], y[0], x[1], y[1], qf.f[t][2 * w][0], qf.f[t][2 * w][1]);
      mma_f16_16816(acc[1], x[2], y[2], x[3], y[3], qf.f[t][2 * w + 1][0], qf.f[t][2 * w + 1][1]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) raw[i] = acc[0][i] + acc[1][i];
}

// Online softmax on the log2-domain scores x (masked entries -inf) and
// O^T += V^T P^T. The running maximum moves only when a score exceeds it
// (one vote), so the common slice rescales nothing. Masked keys' V scales
// must be zero in `s` (what lies there may be anything).
template <int D, int TERMS>
__device__ __forceinline__ void slice_softmax_pv(QState<D>& st, const float (&x)[4],
                                                 const QSlice<D>& s) {
  if (__any_sync(0xffffffffu, fmaxf(x[0], x[2]) > st.m[0] || fmaxf(x[1], x[3]) > st.m[1])) {
    float mx0 = fmaxf(x[0], x[2]), mx1 = fmaxf(x[1], x[3]);
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
  const float mu0 = (st.m[0] == kNegInf ? 0.f : st.m[0]) - kPShift;
  const float mu1 = (st.m[1] == kNegInf ? 0.f : st.m[1]) - kPShift;
  const float p0 = fast_exp2(x[0] - mu0), p1 = fast_exp2(x[1] - mu1);
  const float p2 = fast_exp2(x[2] - mu0), p3 = fast_exp2(x[3] - mu1);
  st.l[0] += p0 + p2;
  st.l[1] += p1 + p3;
  uint32_t b[TERMS][2];
  b[0][0] = movmatrix_t(pack_f16(p0, p1));
  b[0][1] = movmatrix_t(pack_f16(p2, p3));
  if (TERMS == 2) {
    b[TERMS - 1][0] = movmatrix_t(pack_f16(p0 - f16_rounded(p0), p1 - f16_rounded(p1)));
    b[TERMS - 1][1] = movmatrix_t(pack_f16(p2 - f16_rounded(p2), p3 - f16_rounded(p3)));
  }
  const uint32_t s01 = cvt_e4m3x2(s.vs[0] | (s.vs[1] << 8));
  const uint32_t s23 = cvt_e4m3x2(s.vs[2] | (s.vs[3] << 8));
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
        mma_f16_16816(st.o[4 * w + i], a0, a1, a2, a3, b[t][0], b[t][1]);
    }
  }
}

// ------------------------------------------------------------------ joining --
// A piece is one warp's (or CTA's) state over part of a (sequence, KV head):
// m[G], l[G] (log2-domain maximum; sum of 2^14 p), o[G][D].
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
    float* o = p + 2 * G + (h + i) * D + gid * (D / 8);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      *reinterpret_cast<float2*>(o + 2 * j) = make_float2(st.o[j][i], st.o[j][2 + i]);
  }
}

// Join n pieces, the i-th at piece(i), with all threads of the CTA. When `dst`
// is null the result is the output of (b, g), else the joined piece goes to
// dst. Pieces are added in order, so the result does not depend on timing.
template <int D, bool F32, typename Piece>
__device__ void join_pieces(const QDecodeArgs& a, Piece piece, int n, int b, int g, float* dst) {
  const int G = a.G;
  for (int e = threadIdx.x; e < G * D; e += blockDim.x) {
    const int h = e / D, dd = e % D;
    float M = kNegInf;
    for (int s = 0; s < n; ++s) M = fmaxf(M, piece(s)[h]);
    float L = 0.f, acc = 0.f;
    for (int s = 0; s < n; ++s) {
      const float* p = piece(s);
      // a piece without keys has m = -inf and l = o = 0
      const float w = p[h] == kNegInf ? 1.f : fast_exp2(p[h] - M);
      L = fmaf(w, p[G + h], L);
      acc = fmaf(w, p[2 * G + e], acc);
    }
    if (dst != nullptr) {
      dst[2 * G + e] = acc;
      if (dd == 0) {
        dst[h] = M;
        dst[G + h] = L;
      }
    } else {
      const size_t row = static_cast<size_t>(b) * a.Hq + a.heads[g * G + h];
      const float y = L == 0.f ? 0.f : acc / L * a.v_scale;   // L == 0: no key at all
      if (F32) static_cast<float*>(a.out)[row * D + dd] = y;
      else static_cast<__nv_bfloat16*>(a.out)[row * D + dd] = __float2bfloat16_rn(y);
      if (dd == 0 && a.row_stat != nullptr)   // in logit units, without the 2^14
        a.row_stat[row] = make_float2(M * kLn2, L == 0.f ? 0.f : ldexpf(1.f / L, kPShift));
    }
  }
}

// This CTA's piece of a unit shared by n CTAs is in its place: count it, and
// let the last CTA to arrive join all of them into the output.
template <int D, bool F32, typename Piece>
__device__ void arrive_and_join(const QDecodeArgs& a, int unit, Piece piece, int n, int b, int g) {
  __shared__ unsigned int s_last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0)
    s_last = atomicAdd(&a.counters[unit], 1u) == static_cast<unsigned int>(n - 1) ? 1u : 0u;
  __syncthreads();
  if (s_last != 0u) {
    __threadfence();
    join_pieces<D, F32>(a, piece, n, b, g, nullptr);
    if (threadIdx.x == 0) a.counters[unit] = 0u;   // ready for the next launch
  }
  __syncthreads();
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

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "one vector load");
  if (N == 4) {
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x;
    w[N / 4] = v.y;
    w[N / 2] = v.z;
    w[N - 1] = v.w;
  } else if (N == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = v.x;
    w[N - 1] = v.y;
  } else {
    w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

// This lane's part of the K row (grp, r) and of the V row (grp, r).
template <int D>
__device__ __forceinline__ void load_k_row(QSlice<D>& s, int i, const uint8_t* grp, int r) {
  const int c4 = threadIdx.x & 3;
  load_words(grp + r * (D / 2) + c4 * (D / 8), s.k[i]);
  const uint8_t* sc = grp + 8 * D + r * (D / 16);
  s.ks[i] = D == 128 ? __ldg(reinterpret_cast<const uint16_t*>(sc) + c4)
                     : static_cast<uint32_t>(__ldg(sc + c4));
}
template <int D>
__device__ __forceinline__ void load_v_row(QSlice<D>& s, int i, const uint8_t* grp, int r) {
  const int gid = (threadIdx.x & 31) >> 2;
  load_words(grp + 9 * D + r * (D / 2) + gid * (D / 16), s.v[i]);
  s.vs[i] = __ldg(grp + 17 * D + r * (D / 16) + gid * D / 128);
}
// key of a slice that V register i of this lane belongs to
__device__ __forceinline__ int v_key(int i) {
  return 2 * (threadIdx.x & 3) + (i & 1) + 8 * (i >> 1);
}

// -------------------------------------------------------------------- dense --
// The slices of all units (unit = sequence * Hkv + KV head; a sequence of n
// keys has ceil(n / 16) per head) form one line, and every warp of the grid
// takes an equal run of it, so that ragged batches balance. A run may span
// units: the warp's pieces of units it does not hold alone go to shared
// memory, the CTA joins those of its warps after one barrier, and a unit that
// several CTAs share is joined by the last of them to arrive.
constexpr int kMinRun = 4;   // slices per warp at least

template <int D, int TERMS>
__global__ void __launch_bounds__(kNW * 32, 2)
    k_qdecode_dense(const __grid_constant__ QDecodeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr bool F32 = TERMS == 2;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int s_tot[kNW];
  __shared__ int s_unit[2 * kNW], s_list[2 * kNW], s_nlist;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, c4 = lane & 3;
  const int pf = static_cast<int>(qpart_floats(a.G, D));
  float* slots = reinterpret_cast<float*>(smem);                 // [2 kNW][pf]
  int* pref = reinterpret_cast<int*>(slots + 2 * kNW * pf);      // [B + 1] slices before b, per head

  // slices before every sequence
  int carry = 0;
  for (int b0 = 0; b0 < a.B; b0 += kNW * 32) {
    const int b = b0 + tid;
    const int n = b < a.B ? (len_of(a, b, blockIdx.x == 0) + 15) >> 4 : 0;
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
  __syncthreads();
  const int total = carry * a.Hkv;
  const int nwarps = static_cast<int>(gridDim.x) * kNW;
  const int per = max(kMinRun, (total + nwarps - 1) / nwarps);
  const int w0 = min(total, (static_cast<int>(blockIdx.x) * kNW + warp) * per);
  const int w1 = min(total, w0 + per);

  QState<D> st;
  for (int f = w0; f < w1;) {
    int lo = 0, hi = a.B;   // the sequence: pref[lo] * Hkv <= f < pref[lo + 1] * Hkv
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] * a.Hkv <= f) lo = mid;
      else hi = mid;
    }
    const int b = lo, nb = pref[b + 1] - pref[b];
    const int g = (f - pref[b] * a.Hkv) / nb;
    const int s0 = f - pref[b] * a.Hkv - g * nb;
    const int s1 = min(nb, s0 + w1 - f);
    const int n = len_of(a, b, false);
    const int32_t* trow = a.table + static_cast<size_t>(b) * a.max_blocks;
    QFrag<D, TERMS> qf;
    load_q(a, b, g, qf);
    qstate_init(st);
    float* sp[2] = {nullptr, nullptr};
    if (a.scores != nullptr)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (2 * c4 + i < a.G)
          sp[i] = a.scores + (static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + 2 * c4 + i]) * a.N;
    for (int s = s0; s < s1; ++s) {
      const uint8_t* grp = group_at<D>(a, trow, g, s);
      const int key0 = 16 * s + gid;
      float lg[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
      QSlice<D> sl;
      if (grp != nullptr) {
        load_k_row(sl, 0, grp, gid);
        load_k_row(sl, 1, grp, gid + 8);
#pragma unroll
        for (int i = 0; i < 4; ++i) load_v_row(sl, i, grp, v_key(i));
        slice_logits(sl, qf, lg);
#pragma unroll
        for (int i = 0; i < 4; ++i) lg[i] *= qf.mult[i & 1];
        if (16 * s + 16 > n) {   // the sequence ends inside this slice
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (key0 + 8 * (i >> 1) >= n) lg[i] = kNegInf;
            if (16 * s + v_key(i) >= n) sl.vs[i] = 0u;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (sp[i & 1] != nullptr && key0 + 8 * (i >> 1) < n) sp[i & 1][key0 + 8 * (i >> 1)] = lg[i];
      if (grp == nullptr) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) lg[i] *= kLog2e;
      slice_softmax_pv<D, TERMS>(st, lg, sl);
    }
    // a warp's run holds at most its first and its last unit in part
    const int slot = 2 * warp + (f == w0 ? 0 : 1);
    const bool whole = s0 == 0 && s1 == nb;
    piece_store<D>(slots + slot * pf, st, a.G);
    if (!whole) {
      if (lane == 0) s_unit[slot] = b * a.Hkv + g;
    } else {
      __syncwarp();
      const float* p = slots + slot * pf;
      for (int e = lane; e < a.G * D; e += 32) {
        const int h = e / D;
        const size_t row = static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + h];
        const float L = p[a.G + h];
        const float y = L == 0.f ? 0.f : p[2 * a.G + e] / L * a.v_scale;
        if (F32) static_cast<float*>(a.out)[row * D + e % D] = y;
        else static_cast<__nv_bfloat16*>(a.out)[row * D + e % D] = __float2bfloat16_rn(y);
        if (e % D == 0 && a.row_stat != nullptr)
          a.row_stat[row] = make_float2(p[h] * kLn2, L == 0.f ? 0.f : ldexpf(1.f / L, kPShift));
      }
      __syncwarp();   // the slot is used again
    }
    f += s1 - s0;
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
  for (int i = 0; i < nlist;) {
    const int unit = s_unit[s_list[i]];
    int j = i;
    while (j < nlist && s_unit[s_list[j]] == unit) ++j;
    const int b = unit / a.Hkv, g = unit % a.Hkv, nb = pref[b + 1] - pref[b];
    const int u0 = pref[b] * a.Hkv + g * nb, u1 = u0 + nb;   // the unit's slices
    auto mine = [&](int s) -> const float* { return slots + s_list[i + s] * pf; };
    const int first = u0 / per_cta, ncta = (u1 - 1) / per_cta - first + 1;
    if (ncta == 1) {
      join_pieces<D, F32>(a, mine, j - i, b, g, nullptr);
    } else {
      // CTA c keeps the piece of a unit that starts inside its run at 2c + 1,
      // of one that started before it (or with it) at 2c
      float* part = a.part;
      const size_t stride = qpart_floats(a.G, D);
      join_pieces<D, F32>(a, mine, j - i, b, g,
                          part + (2 * static_cast<size_t>(blockIdx.x) + (u0 > c0 ? 1 : 0)) * stride);
      const int odd = u0 > first * per_cta ? 1 : 0;
      auto all = [=](int s) -> const float* {
        return part + (2 * static_cast<size_t>(first + s) + (s == 0 ? odd : 0)) * stride;
      };
      arrive_and_join<D, F32>(a, unit, all, ncta, b, g);
    }
    i = j;
  }
  // sequences without keys: zeros; scores behind the last key
  for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
    const int n = len_of(a, b, false);
    if (n == 0) {
      const size_t base = static_cast<size_t>(b) * a.Hq * D;
      for (int e = tid; e < a.Hq * D; e += blockDim.x) {
        if (F32) static_cast<float*>(a.out)[base + e] = 0.f;
        else static_cast<__nv_bfloat16*>(a.out)[base + e] = __float2bfloat16_rn(0.f);
      }
      if (a.row_stat != nullptr)
        for (int h = tid; h < a.Hq; h += blockDim.x)
          a.row_stat[static_cast<size_t>(b) * a.Hq + h] = make_float2(kNegInf, 0.f);
    }
  }
  if (a.scores != nullptr && a.fill_tail)
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
  load_q(a, b, g, qf);
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
    float lg[4];
    uint32_t mk[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int src = gid + 8 * i;
      const uint8_t* p =
          reinterpret_cast<const uint8_t*>(__shfl_sync(0xffffffffu, base, src));
      const int r = __shfl_sync(0xffffffffu, key, src) & 15;
      mk[i] = __shfl_sync(0xffffffffu, mask, src);
      if (mk[i] != 0u) {
        load_k_row(s, i, p, r);
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
        load_v_row(s, i, p, r);
      } else {
#pragma unroll
        for (int w = 0; w < D / 64; ++w) s.v[i][w] = 0u;
        s.vs[i] = 0u;
      }
    }
    slice_logits(s, qf, lg);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = (mk[i >> 1] >> (2 * c4 + (i & 1))) & 1u;
      lg[i] = in ? lg[i] * qf.mult[i & 1] * kLog2e : kNegInf;
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
    slice_softmax_pv<D, TERMS>(st, lg, s);
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
  auto mine = [&](int w) -> const float* { return slots + w * pf; };
  if (a.S == 1) {
    join_pieces<D, F32>(a, mine, kNW, b, g, nullptr);
    return;
  }
  float* part = a.part + static_cast<size_t>(unit) * a.S * pf;
  join_pieces<D, F32>(a, mine, kNW, b, g, part + static_cast<size_t>(blockIdx.x) * pf);
  auto all = [=](int w) -> const float* { return part + static_cast<size_t>(w) * pf; };
  arrive_and_join<D, F32>(a, unit, all, a.S, b, g);
}

// CTAs of a kernel that the current device holds at once (asked once per host
// thread, device and shared memory size).
template <typename K>
cudaError_t resident_ctas(K kern, size_t smem, int& ctas) {
  thread_local int dev_of = -1, slots = 0;
  thread_local size_t smem_of = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if (dev != dev_of || smem != smem_of) {
    int sms = 0, per_sm = 0;
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

template <int D, int TERMS>
cudaError_t launch_dense_t(const QDecodeArgs& a, cudaStream_t st) {
  const size_t smem = 2 * kNW * qpart_floats(a.G, D) * sizeof(float) +
                      (static_cast<size_t>(a.B) + 1) * sizeof(int);
  auto kern = k_qdecode_dense<D, TERMS>;
  int ctas = 0;
  const cudaError_t e = resident_ctas(kern, smem, ctas);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(ctas), dim3(kNW * 32), smem, st, a);
}

template <int D, int TERMS, bool POOLED>
cudaError_t launch_reuse_t(const QDecodeArgs& a, cudaStream_t st) {
  const size_t smem = kNW * qpart_floats(a.G, D) * sizeof(float);
  auto kern = k_qdecode_reuse<D, TERMS, POOLED>;
  int ctas = 0;
  const cudaError_t e = resident_ctas(kern, smem, ctas);
  if (e != cudaSuccess) return e;
  QDecodeArgs u = a;
  const int units = a.B * a.Hkv;
  // at least one slice per warp where the sets are long enough
  const int most = POOLED ? (a.topk + 16 * kNW - 1) / (16 * kNW)
                          : (a.G * a.topk + 16 * kNW - 1) / (16 * kNW);
  int s = ctas / units;
  if (s > most) s = most;
  u.S = s < 1 ? 1 : s;
  return launch_pdl(kern, dim3(u.S, units), dim3(kNW * 32), smem, st, u);
}

}  // namespace

cudaError_t launch_qdecode_dense(const QDecodeArgs& a, int d, int dtype, cudaStream_t st) {
  if (dtype == KASCADE_F32)
    return d == 128 ? launch_dense_t<128, 2>(a, st) : launch_dense_t<64, 2>(a, st);
  return d == 128 ? launch_dense_t<128, 1>(a, st) : launch_dense_t<64, 1>(a, st);
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
