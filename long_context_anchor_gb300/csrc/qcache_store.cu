// qcache_store.cu — the paged 4-bit key/value cache's bookkeeping and rows:
//
//   k_qplan    block tables, the stack of free blocks and the slots of new
//              tokens from request lengths
//   k_qappend  rows quantised into their slots
//   k_qread    rows read back from their slots
//
// Number format: 16 consecutive elements of a row share one scale. With
// x' = x / {k,v}_scale (a power of two, so exact), amax = max |x'|:
//   s    = amax / 6 rounded to e4m3 (nearest, ties to even, at most 448)
//   code = x' / s rounded to e2m1 {0, .5, 1, 1.5, 2, 3, 4, 6} (same, at most 6)
// and the stored element is code * s * {k,v}_scale. Both quotients are
// rounded once, from their exact value: see round_quotient.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "qcache.h"

namespace kascade {
namespace {

// ---------------------------------------------------------------- planner --
// A sequence of L tokens that changes by n tokens ends with L' = max(0, L + n)
// of them and holds ceil(L' / block_size) blocks. Blocks given back are pushed
// on the stack in (sequence, column) order, then blocks taken are popped in
// the same order, so the outcome does not depend on timing: with c blocks on
// the stack and G given back, the j-th block taken is the one at c + G - 1 - j,
// which is the (G - 1 - j)-th given back or an old entry of the stack. No
// entry that is read is written in the same step, so after the checks every
// move and every slot is made on its own.
//
// Everything is checked before anything is written: a step that cannot be
// served changes nothing, leaves every slot -1 and records bad input. Small
// steps run in one CTA and one launch; larger ones in two launches of many
// CTAs, checks first, each CTA scanning the lengths for itself.
constexpr int kPlanThreads = 1024;
// One launch up to this many blocks and new tokens (one round of the CTA's
// threads or two): 1.1 us of 8 requests' step are saved by the second launch
// not made, while 32768 moved blocks take one CTA 150 us and two launches of
// 152 CTAs 14 us.
constexpr int kPlanOneCta = 2048;

struct PlanScan {
  int gives, takes;      // blocks given back and taken by all sequences
  int c;                 // valid entries of the stack
  bool bad;              // the same in every thread
};

// Inclusive scan over the block, three values at once; totals in tot.
__device__ __forceinline__ void block_scan3(int (&v)[3], int3* warp_tot, int (&tot)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto scan = [&](int (&x)[3]) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const unsigned int o = __shfl_up_sync(0xffffffffu, x[i], off);
        if (lane >= off) x[i] = static_cast<int>(x[i] + o);
      }
    }
  };
  scan(v);
  if (lane == 31) warp_tot[warp] = make_int3(v[0], v[1], v[2]);
  __syncthreads();
  if (warp == 0) {
    const int3 t = warp_tot[lane];
    int w[3] = {t.x, t.y, t.z};
    scan(w);
    warp_tot[lane] = make_int3(w[0], w[1], w[2]);
  }
  __syncthreads();
  if (warp > 0) {
    const int3 t = warp_tot[warp - 1];
    v[0] += t.x;
    v[1] += t.y;
    v[2] += t.z;
  }
  const int3 t = warp_tot[31];
  tot[0] = t.x;
  tot[1] = t.y;
  tot[2] = t.z;
  __syncthreads();
}

// Largest b in [0, B) with pre[b] <= i (pre ascending, pre[0] = 0 <= i).
__device__ __forceinline__ int owner_of(const int* pre, int B, int i) {
  int lo = 0, hi = B;   // pre[lo] <= i, and pre[hi] > i or hi == B
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A sequence's tokens before and after; false (both 0) if out of range.
__device__ __forceinline__ bool plan_len(const QPlanArgs& a, int b, int& L, int& to) {
  const long long cap = static_cast<long long>(a.max_blocks) << a.bs_shift;
  L = a.kv_lens[b];
  const long long t = static_cast<long long>(L) + a.new_lens[b];
  const bool ok = L >= 0 && L <= cap && t <= cap;
  to = t < 0 ? 0 : static_cast<int>(t);
  if (!ok) L = to = 0;
  return ok;
}
__device__ __forceinline__ int plan_blocks(const QPlanArgs& a, int tokens) {
  return (tokens + (1 << a.bs_shift) - 1) >> a.bs_shift;
}

// pre[0..2]: what sequences before b give back, take and add, [B + 1] each.
__device__ PlanScan plan_scan(const QPlanArgs& a, int* const (&pre)[3]) {
  __shared__ int3 warp_tot[32];
  const int tid = threadIdx.x;
  PlanScan r;
  r.c = *a.free_count;
  __shared__ long long s_tokens[32];
  int carry[3] = {0, 0, 0};
  long long tokens = 0;
  bool bad = false;
  for (int b0 = 0; b0 < a.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int v[3] = {0, 0, 0}, own[3], tot[3];
    if (b < a.B) {
      int L, to;
      bad |= !plan_len(a, b, L, to);
      const int have = plan_blocks(a, L), need = plan_blocks(a, to);
      v[0] = max(0, have - need);
      v[1] = max(0, need - have);
      v[2] = max(0, to - L);   // may add up to more than 32 bits: refused below
      tokens += v[2];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) own[i] = v[i];
    block_scan3(v, warp_tot, tot);
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (b < a.B) pre[i][b] = carry[i] + v[i] - own[i];
#pragma unroll
    for (int i = 0; i < 3; ++i)
      carry[i] = static_cast<int>(static_cast<unsigned int>(carry[i]) + tot[i]);
  }
  auto warp_sum = [](long long x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    return x;
  };
  tokens = warp_sum(tokens);
  if ((tid & 31) == 0) s_tokens[tid >> 5] = tokens;
  r.gives = carry[0];
  r.takes = carry[1];
  if (tid == 0) {
    pre[0][a.B] = r.gives;
    pre[1][a.B] = r.takes;
    pre[2][a.B] = carry[2];
  }
  const long long top = static_cast<long long>(r.c) + r.gives;
  bad |= r.c < 0 || r.c > a.num_blocks || top > a.num_blocks || r.takes > top;
  __syncthreads();
  if (tid < 32) bad |= warp_sum(s_tokens[tid]) > a.max_new;
  r.bad = __syncthreads_or(bad) != 0;
  return r;
}

// The i-th block given back.
__device__ __forceinline__ int plan_given(const QPlanArgs& a, const int* give, int i) {
  const int b = owner_of(give, a.B, i);
  int L, to;
  plan_len(a, b, L, to);
  return a.table[static_cast<size_t>(b) * a.max_blocks + plan_blocks(a, to) + i - give[b]];
}
// The j-th block taken.
__device__ __forceinline__ int plan_taken(const QPlanArgs& a, const PlanScan& r, const int* give,
                                          int j) {
  return j < r.gives ? plan_given(a, give, r.gives - 1 - j) : a.free_blocks[r.c + r.gives - 1 - j];
}

// Ids that move: those given back, and the old part of the stack that is taken.
__device__ bool plan_bad_ids(const QPlanArgs& a, const PlanScan& r, const int* give, int t0,
                             int step) {
  bool bad = false;
  auto check = [&](int id) { bad |= id < 0 || id >= a.num_blocks; };
  for (int i = t0; i < r.gives; i += step) check(plan_given(a, give, i));
  for (int j = r.gives + t0; j < r.takes; j += step) check(plan_taken(a, r, give, j));
  return bad;
}

// Thread t0 of `step`: its share of the moves and of the slots.
__device__ void plan_apply(const QPlanArgs& a, const PlanScan& r, int* const (&pre)[3], bool bad,
                           int t0, int step) {
  const int sh = a.bs_shift;
  if (!bad) {
    for (int i = t0; i < r.gives; i += step) a.free_blocks[r.c + i] = plan_given(a, pre[0], i);
    for (int j = t0; j < r.takes; j += step) {
      const int b = owner_of(pre[1], a.B, j);
      int L, to;
      plan_len(a, b, L, to);
      a.table[static_cast<size_t>(b) * a.max_blocks + plan_blocks(a, L) + j - pre[1][b]] =
          plan_taken(a, r, pre[0], j);
    }
  }
  const int total = bad ? 0 : pre[2][a.B];
  for (int i = t0; i < a.max_new; i += step) {
    int slot = -1;
    if (i < total) {
      const int b = owner_of(pre[2], a.B, i);
      int L, to;
      plan_len(a, b, L, to);
      const int p = L + i - pre[2][b], col = p >> sh, have = plan_blocks(a, L);
      // the block that the sequence's last token is in, or one taken now
      const int id = col < have ? a.table[static_cast<size_t>(b) * a.max_blocks + col]
                                : plan_taken(a, r, pre[0], pre[1][b] + col - have);
      if (id >= 0 && id < a.num_blocks) slot = (id << sh) | (p & ((1 << sh) - 1));
      else report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x502);
    }
    a.slot_map[i] = slot;
  }
}

// Lengths, running numbers of new tokens and the stack's count, by one CTA
// once nothing reads the old ones (they may be the same arrays).
__device__ void plan_finish(const QPlanArgs& a, const PlanScan& r, const int* add, bool bad) {
  for (int b = threadIdx.x; b < a.B; b += kPlanThreads) {
    int L, to;
    const int keep = a.kv_lens[b];
    plan_len(a, b, L, to);
    a.kv_lens_out[b] = bad ? keep : to;
    a.cu_new[b + 1] = bad ? 0 : add[b + 1];
  }
  if (threadIdx.x == 0) {
    a.cu_new[0] = 0;
    *a.free_count_out = bad ? r.c : r.c + r.gives - r.takes;
    if (bad) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x501);
  }
}

// CHECK: bad ids are noted in the workspace header's word `flag`. APPLY: the
// step itself; the last CTA to finish writes the lengths and clears the
// header's words again. Both: the whole step in one CTA. Bound by latency: a
// few dependent rounds of loads and block scans.
template <bool CHECK, bool APPLY>
__global__ void __launch_bounds__(kPlanThreads) k_qplan(const __grid_constant__ QPlanArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* const pre[3] = {sm, sm + a.B + 1, sm + 2 * (a.B + 1)};
  const PlanScan r = plan_scan(a, pre);
  const int t0 = blockIdx.x * kPlanThreads + threadIdx.x, step = gridDim.x * kPlanThreads;
  bool bad = r.bad;
  if (CHECK && !bad) {
    bad = plan_bad_ids(a, r, pre[0], t0, step);
    if (APPLY) bad = __syncthreads_or(bad) != 0;
    else if (bad) atomicOr(a.flag, 1u);
  }
  if (!APPLY) return;
  if (!CHECK) bad |= *a.flag != 0u;
  plan_apply(a, r, pre, bad, t0, step);
  __syncthreads();
  if (CHECK) {
    plan_finish(a, r, pre[2], bad);
    return;
  }
  __shared__ bool s_last;
  if (threadIdx.x == 0) s_last = atomicAdd(a.flag + 1, 1u) == gridDim.x - 1;
  __syncthreads();
  if (!s_last) return;
  plan_finish(a, r, pre[2], bad);
  if (threadIdx.x == 0) a.flag[0] = a.flag[1] = 0u;
}

// -------------------------------------------------------------------- rows --
constexpr int kRowThreads = 256;

// x / s rounded so that the rounding to a few bits that follows is the
// rounding of the exact quotient: q is x / s to the last bit (one Newton
// correction of x * (1/s)), and where the division leaves a remainder q is
// moved one last place towards it, so that a q that sits on a tie only by
// its own rounding falls on the right side. Rounding q to 2 to 4 bits cannot
// be changed by that step otherwise.
__device__ __forceinline__ float round_quotient(float x, float s, float inv) {
  float q = x * inv;
  q = fmaf(fmaf(-q, s, x), inv, q);
  const float r = fmaf(-q, s, x);
  if (r != 0.f && q != 0.f) {
    const int step = ((r > 0.f) == (q > 0.f)) ? 1 : -1;
    q = __int_as_float(__float_as_int(q) + step);
  }
  return q;
}

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
// two e2m1 codes, `lo` in the low half of the byte
__device__ __forceinline__ uint32_t e2m1_pair(float lo, float hi) {
  uint32_t r;
  asm("{.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;}"
      : "=r"(r)
      : "f"(hi), "f"(lo));
  return r;
}

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&x)[16]);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
    x[4 * i] = f.x;
    x[4 * i + 1] = f.y;
    x[4 * i + 2] = f.z;
    x[4 * i + 3] = f.w;
  }
}
template <>
__device__ __forceinline__ void load16<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  }
}
__device__ __forceinline__ void store16(float* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(p)[i] =
        make_uint4(pack_bf16(x[8 * i], x[8 * i + 1]), pack_bf16(x[8 * i + 2], x[8 * i + 3]),
                   pack_bf16(x[8 * i + 4], x[8 * i + 5]), pack_bf16(x[8 * i + 6], x[8 * i + 7]));
}

// Byte address of (slot, head)'s row of codes of K (which = 0) or V (1), and
// of its scales.
struct RowAddr {
  uint8_t* codes;
  uint8_t* scales;
};
__device__ __forceinline__ RowAddr row_addr(const QRowArgs& a, int which, int slot, int head) {
  const int sh = a.bs_shift, gpb = 1 << (sh - 4);
  const size_t block = static_cast<size_t>(slot >> sh);
  const int in = slot & ((1 << sh) - 1);
  uint8_t* grp = a.cache + ((block * a.Hkv + head) * gpb + (in >> 4)) * (18 * a.d) +
                 which * (9 * a.d);
  const int r = in & 15;
  return {grp + r * (a.d / 2), grp + 8 * a.d + r * (a.d / 16)};
}

// One thread per 16 elements; consecutive threads take a row's blocks, then
// the next token of the same head, so that a warp writes neighbouring rows of
// one group. Bound by DRAM: each element is read once and its 4.5 bits are
// written once.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_qappend(const __grid_constant__ QRowArgs a) {
  pdl_wait();
  pdl_trigger();
  const int per_row = a.d / 16, which = blockIdx.y;
  const long long n = static_cast<long long>(a.T) * a.Hkv * per_row;
  const long long i = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= n) return;
  const int blk = static_cast<int>(i % per_row);
  const long long row = i / per_row;
  const int tok = static_cast<int>(row % a.T), head = static_cast<int>(row / a.T);
  const int slot = a.slot_map[tok];
  if (slot < 0) return;   // padding
  if (slot >= (a.num_blocks << a.bs_shift)) {
    report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x511);
    return;
  }
  float x[16];
  load16(static_cast<const T*>(a.src[which]) + tok * a.tok_stride[which] +
             head * a.head_stride[which] + blk * 16, x);
  float amax = 0.f;
  bool nan = false;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    x[e] *= a.scale[which];
    nan |= x[e] != x[e];
    // what saturates does so here already, infinities among it
    x[e] = fminf(fmaxf(x[e], -2688.f), 2688.f);
    amax = fmaxf(amax, fabsf(x[e]));
  }
  const uint32_t sb = nan ? 0x7fu : e4m3_of(round_quotient(amax, 6.f, 1.f / 6.f));
  const float s = e4m3_value(sb);
  uint32_t w[2] = {0u, 0u};
  if (s > 0.f) {   // a block of zeros, or one that rounds to them, has scale 0 (and NaN none)
    const float inv = 1.f / s;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      w[e >> 2] |= e2m1_pair(round_quotient(x[2 * e], s, inv), round_quotient(x[2 * e + 1], s, inv))
                   << (8 * (e & 3));
  }
  const RowAddr ra = row_addr(a, which, slot, head);
  reinterpret_cast<uint2*>(ra.codes)[blk] = make_uint2(w[0], w[1]);
  ra.scales[blk] = static_cast<uint8_t>(sb);
}

// The same threads, the other way; a padding slot's row is zero.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) k_qread(const __grid_constant__ QRowArgs a) {
  pdl_wait();
  pdl_trigger();
  const int per_row = a.d / 16, which = blockIdx.y;
  const long long n = static_cast<long long>(a.T) * a.Hkv * per_row;
  const long long i = static_cast<long long>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i >= n) return;
  const int blk = static_cast<int>(i % per_row);
  const long long row = i / per_row;
  const int tok = static_cast<int>(row % a.T), head = static_cast<int>(row / a.T);
  const int slot = a.slot_map[tok];
  float x[16];
  if (slot >= 0 && slot < (a.num_blocks << a.bs_shift)) {
    const RowAddr ra = row_addr(a, which, slot, head);
    const uint2 c = *(reinterpret_cast<const uint2*>(ra.codes) + blk);
    const float s = e4m3_value(ra.scales[blk]) * a.scale[which];
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t h;
      asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;}" : "=r"(h) : "r"(w[e >> 2] >> (8 * (e & 3))));
      float lo, hi;
      asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
          : "=f"(lo), "=f"(hi) : "r"(h));
      x[2 * e] = lo * s;
      x[2 * e + 1] = hi * s;
    }
  } else {
    if (slot >= 0) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x512);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = 0.f;
  }
  store16(static_cast<T*>(a.dst[which]) + tok * a.tok_stride[which] +
              head * a.head_stride[which] + blk * 16, x);
}

template <typename K>
cudaError_t launch_rows(K kern, const QRowArgs& a, cudaStream_t st) {
  const long long n = static_cast<long long>(a.T) * a.Hkv * (a.d / 16);
  if (n == 0) return cudaSuccess;
  const long long blocks = (n + kRowThreads - 1) / kRowThreads;
  if (blocks > 0x7fffffffll) return cudaErrorNotSupported;
  return launch_pdl(kern, dim3(static_cast<unsigned int>(blocks), 2), dim3(kRowThreads), 0, st, a);
}

}  // namespace

namespace {
template <bool CHECK, bool APPLY>
cudaError_t launch_plan(const QPlanArgs& a, int ctas, cudaStream_t st) {
  const size_t smem = 3 * (static_cast<size_t>(a.B) + 1) * sizeof(int);
  auto kern = k_qplan<CHECK, APPLY>;
  if (smem > 48 * 1024) {   // up to 192 KB, the same setting whatever the call
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * (kMaxCounterUnits + 1) * static_cast<int>(sizeof(int)));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, dim3(ctas), dim3(kPlanThreads), smem, st, a);
}
}  // namespace

cudaError_t launch_qplan(const QPlanArgs& a, cudaStream_t st) {
  const int most = a.num_blocks > a.max_new ? a.num_blocks : a.max_new;   // ids or slots to write
  if (a.B <= kPlanThreads && most <= kPlanOneCta) return launch_plan<true, true>(a, 1, st);
  int ctas = (most + kPlanThreads - 1) / kPlanThreads;
  if (ctas > 152) ctas = 152;
  const cudaError_t e = launch_plan<true, false>(a, ctas, st);
  return e != cudaSuccess ? e : launch_plan<false, true>(a, ctas, st);
}

cudaError_t launch_qappend(const QRowArgs& a, int dtype, cudaStream_t st) {
  return dtype == KASCADE_F32 ? launch_rows(k_qappend<float>, a, st)
                              : launch_rows(k_qappend<__nv_bfloat16>, a, st);
}

cudaError_t launch_qread(const QRowArgs& a, int dtype, cudaStream_t st) {
  return dtype == KASCADE_F32 ? launch_rows(k_qread<float>, a, st)
                              : launch_rows(k_qread<__nv_bfloat16>, a, st);
}

}  // namespace kascade
