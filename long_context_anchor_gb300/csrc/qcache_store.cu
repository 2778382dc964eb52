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
// rounded as their exact values would be: see round_quotient.
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
// served changes nothing, leaves every slot -1 and records bad input. Steps over
// a small pool with few new tokens run in one CTA and one launch; others in two
// launches of many CTAs, checks first, each CTA scanning the lengths for itself.
constexpr int kPlanThreads = 1024;
// One launch up to this many blocks of the pool (any of which a step may move: the
// host does not know the lengths) and new tokens. A step of 64 sequences, half of
// them ending and half starting, blocks of 16, a pool that holds both halves, calls
// back to back in a graph on a GB300 (one CTA / two launches): 512 new tokens 5.3 /
// 7.9 us, 2048 7.1 / 8.6, 4096 9.5 / 8.7, 32768 47 / 10. A step that moves
// little over a large pool pays for the second launch: eight sequences that add a
// token each take 3.3 us over 100 blocks and 6.1 over 4200.
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

// Ids that the step uses: those given back, the old part of the stack that is
// taken, and the partly filled block that a growing sequence's first new tokens go to.
__device__ bool plan_bad_ids(const QPlanArgs& a, const PlanScan& r, const int* give, int t0,
                             int step) {
  bool bad = false;
  auto check = [&](int id) { bad |= id < 0 || id >= a.num_blocks; };
  for (int i = t0; i < r.gives; i += step) check(plan_given(a, give, i));
  for (int j = r.gives + t0; j < r.takes; j += step) check(plan_taken(a, r, give, j));
  for (int b = t0; b < a.B; b += step) {
    int L, to;
    plan_len(a, b, L, to);
    if (to > L && (L & ((1 << a.bs_shift) - 1)) != 0)
      check(a.table[static_cast<size_t>(b) * a.max_blocks + (L >> a.bs_shift)]);
  }
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
      // the block that the sequence's last token is in, or one taken now: checked
      const int id = col < have ? a.table[static_cast<size_t>(b) * a.max_blocks + col]
                                : plan_taken(a, r, pre[0], pre[1][b] + col - have);
      slot = (id << sh) | (p & ((1 << sh) - 1));
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
// Every element is read once and its 4.5 bits written once (or the other way):
// bound by DRAM. A thread has one piece of a token's K row of a head and the same
// piece of its V row, so that a warp works on neighbouring rows of one group of
// the cache, two rows wait for one slot, and their loads are in flight
// together (K and V by different CTAs: 18.6 us to write, 18.7 to read 16384
// tokens x 8 heads x 128 in bf16, 86 MB). Reading takes pieces of 8 elements, whose
// stores join into whole sectors (14.6 us, 18.4 with 16); writing takes whole
// blocks of 16, which find their scale alone (15.6 us, 21.7 with two threads per
// block). 5.5 and 5.9 TB/s, 0.81 and 0.87 of the copy rate. The same rows in fp32,
// 153 MB: 25.8 us to write (5.9 TB/s), 35.1 to read (4.4 TB/s, 0.64).
constexpr int kRowThreads = 256;
constexpr int kAppendPiece = 16, kReadPiece = 8;   // elements per thread

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
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(p)[i] =
        make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                            pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// What one thread works on, and where its codes and scales are (V's lie 9 D
// bytes behind K's).
struct RowPlace {
  int tok, head, at;        // at: first element of the row
  int slot;                 // negative: padding
  uint8_t* codes;
  uint8_t* scale;
};
template <int D, int PIECE>
__device__ __forceinline__ bool row_place(const QRowArgs& a, RowPlace& p) {
  constexpr int kPieces = D / PIECE;
  p.head = blockIdx.y;
  p.tok = blockIdx.x * (kRowThreads / kPieces) + threadIdx.x / kPieces;
  p.at = threadIdx.x % kPieces * PIECE;
  if (p.tok >= a.T) return false;
  p.slot = a.slot_map[p.tok];
  if (p.slot < 0) return true;
  const int sh = a.bs_shift;
  if ((p.slot >> sh) >= a.num_blocks) {
    report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x511);
    p.slot = -1;
    return true;
  }
  const size_t grp = ((static_cast<size_t>(p.slot >> sh) * a.Hkv + p.head) << (sh - 4)) +
                     ((p.slot & ((1 << sh) - 1)) >> 4);
  uint8_t* grp_at = a.cache + grp * (18 * D);
  const int r = p.slot & 15;
  p.codes = grp_at + r * (D / 2) + p.at / 2;
  p.scale = grp_at + 8 * D + r * (D / 16) + p.at / 16;
  return true;
}

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

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) k_qappend(const __grid_constant__ QRowArgs a) {
  pdl_wait();
  pdl_trigger();
  RowPlace p;
  if (!row_place<D, kAppendPiece>(a, p) || p.slot < 0) return;
  Row16<T> x[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    x[i].load(static_cast<const T*>(a.src[i]) + p.tok * a.tok_stride[i] +
              p.head * a.head_stride[i] + p.at);
#pragma unroll
  for (int i = 0; i < 2; ++i) put16(x[i], a.scale[i], p.codes + i * 9 * D, p.scale + i * 9 * D);
}

// The other way; a padding slot's row is zero.
template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads) k_qread(const __grid_constant__ QRowArgs a) {
  pdl_wait();
  pdl_trigger();
  RowPlace p;
  if (!row_place<D, kReadPiece>(a, p)) return;
  uint32_t c[2] = {}, sb[2] = {};
  if (p.slot >= 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i] = *reinterpret_cast<const uint32_t*>(p.codes + i * 9 * D);
      sb[i] = p.scale[i * 9 * D];
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float s = e4m3_value(sb[i]) * a.scale[i];
    float x[kReadPiece];
#pragma unroll
    for (int e = 0; e < kReadPiece / 2; ++e) {
      uint32_t h;
      asm("{.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\t"
          "cvt.rn.f16x2.e2m1x2 %0, b0;}" : "=r"(h) : "r"(c[i] >> (8 * e)));
      float lo, hi;
      asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}"
          : "=f"(lo), "=f"(hi) : "r"(h));
      x[2 * e] = lo * s;
      x[2 * e + 1] = hi * s;
    }
    store8(static_cast<T*>(a.dst[i]) + p.tok * a.tok_stride[i] + p.head * a.head_stride[i] + p.at,
           x);
  }
}

template <int PIECE, typename K>
cudaError_t launch_rows(K kern, const QRowArgs& a, cudaStream_t st) {
  if (a.T == 0) return cudaSuccess;
  const int per_cta = kRowThreads / (a.d / PIECE);   // tokens
  return launch_pdl(kern, dim3((a.T + per_cta - 1) / per_cta, a.Hkv), dim3(kRowThreads), 0, st,
                    a);
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
  if (dtype == KASCADE_F32)
    return a.d == 128 ? launch_rows<kAppendPiece>(k_qappend<float, 128>, a, st)
                      : launch_rows<kAppendPiece>(k_qappend<float, 64>, a, st);
  return a.d == 128 ? launch_rows<kAppendPiece>(k_qappend<__nv_bfloat16, 128>, a, st)
                    : launch_rows<kAppendPiece>(k_qappend<__nv_bfloat16, 64>, a, st);
}

cudaError_t launch_qread(const QRowArgs& a, int dtype, cudaStream_t st) {
  if (dtype == KASCADE_F32)
    return a.d == 128 ? launch_rows<kReadPiece>(k_qread<float, 128>, a, st)
                      : launch_rows<kReadPiece>(k_qread<float, 64>, a, st);
  return a.d == 128 ? launch_rows<kReadPiece>(k_qread<__nv_bfloat16, 128>, a, st)
                    : launch_rows<kReadPiece>(k_qread<__nv_bfloat16, 64>, a, st);
}

}  // namespace kascade
