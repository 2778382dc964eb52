// qcache_store.cu — the paged 4-bit key/value cache's bookkeeping and rows:
//
//   k_qplan    block tables and the stack of free blocks from request lengths
//   k_qslots   the slot of every new token
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
constexpr int kPlanThreads = 1024;

// Inclusive scan over the block, two values at once.
__device__ __forceinline__ void block_scan2(int& x, int& y, int2* warp_tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int ox = __shfl_up_sync(0xffffffffu, x, off);
    const int oy = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) {
      x += ox;
      y += oy;
    }
  }
  if (lane == 31) warp_tot[warp] = make_int2(x, y);
  __syncthreads();
  if (warp == 0) {
    int2 t = warp_tot[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int ox = __shfl_up_sync(0xffffffffu, t.x, off);
      const int oy = __shfl_up_sync(0xffffffffu, t.y, off);
      if (lane >= off) {
        t.x += ox;
        t.y += oy;
      }
    }
    warp_tot[lane] = t;
  }
  __syncthreads();
  if (warp > 0) {
    x += warp_tot[warp - 1].x;
    y += warp_tot[warp - 1].y;
  }
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

// One CTA. A sequence of L tokens that changes by n tokens ends with
// L' = max(0, L + n) of them and holds ceil(L' / block_size) blocks. Blocks
// given back are pushed on the stack in (sequence, column) order, then blocks
// taken are popped in the same order, so the outcome does not depend on
// timing. Everything is checked before anything is written: a step that
// cannot be served (not enough free blocks, a table row too short, more new
// tokens than slots, an id or a length out of range) changes nothing, leaves
// every slot -1 and records bad input. Bound by latency: a few dependent
// rounds of loads and block scans.
__global__ void __launch_bounds__(kPlanThreads) k_qplan(const __grid_constant__ QPlanArgs a) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ int sm[];
  int* pre_give = sm;                 // [B + 1] blocks given back before sequence b
  int* pre_take = sm + a.B + 1;       // [B + 1] blocks taken before sequence b
  __shared__ int2 warp_tot[32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, B = a.B, sh = a.bs_shift;
  const int bs = 1 << sh;
  const long long cap = static_cast<long long>(a.max_blocks) << sh;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  auto read_len = [&](int b, int& L, int& to) -> bool {
    L = a.kv_lens[b];
    const long long t = static_cast<long long>(L) + a.new_lens[b];
    const bool ok = L >= 0 && L <= cap && t <= cap;
    to = t < 0 ? 0 : static_cast<int>(t);
    if (!ok) L = to = 0;
    return ok;
  };
  int carry_g = 0, carry_t = 0;
  long long tokens = 0;
  bool bad = false;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int give = 0, take = 0;
    if (b < B) {
      int L, to;
      bad |= !read_len(b, L, to);
      const int have = (L + bs - 1) >> sh, need = (to + bs - 1) >> sh;
      give = max(0, have - need);
      take = max(0, need - have);
      tokens += max(0, to - L);
    }
    int ig = give, it = take;
    block_scan2(ig, it, warp_tot);
    if (b < B) {
      pre_give[b] = carry_g + ig - give;
      pre_take[b] = carry_t + it - take;
    }
    carry_g += warp_tot[31].x;   // totals of this round (the scan ends with a barrier)
    carry_t += warp_tot[31].y;
    __syncthreads();
  }
  const int gives = carry_g, takes = carry_t;
  if (tid == 0) {
    pre_give[B] = gives;
    pre_take[B] = takes;
  }
  const int c = *a.free_count;
  const long long top = static_cast<long long>(c) + gives;
  bad |= c < 0 || c > a.num_blocks || top > a.num_blocks || takes > top;
  // new tokens of all sequences
  __shared__ unsigned long long s_tokens;
  if (tid == 0) s_tokens = 0;
  __syncthreads();
  if (tokens) atomicAdd(&s_tokens, static_cast<unsigned long long>(tokens));
  if (bad) s_bad = 1;
  __syncthreads();
  if (static_cast<long long>(s_tokens) > a.max_new && tid == 0) s_bad = 1;
  __syncthreads();
  // ids that move: those given back, and the old part of the stack that is taken
  if (!s_bad) {
    for (int i = tid; i < gives; i += kPlanThreads) {
      const int b = owner_of(pre_give, B, i);
      int L, to;
      read_len(b, L, to);
      const int id = a.table[static_cast<size_t>(b) * a.max_blocks + ((to + bs - 1) >> sh) + i -
                             pre_give[b]];
      if (id < 0 || id >= a.num_blocks) s_bad = 1;
    }
    for (int i = max(0, takes - gives) - 1 - tid; i >= 0; i -= kPlanThreads) {
      const int id = a.free_blocks[c - 1 - i];
      if (id < 0 || id >= a.num_blocks) s_bad = 1;
    }
  }
  __syncthreads();
  bad = s_bad != 0;
  if (bad && tid == 0) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x501);
  if (!bad) {
    for (int i = tid; i < gives; i += kPlanThreads) {
      const int b = owner_of(pre_give, B, i);
      int L, to;
      read_len(b, L, to);
      a.free_blocks[c + i] = a.table[static_cast<size_t>(b) * a.max_blocks +
                                     ((to + bs - 1) >> sh) + i - pre_give[b]];
    }
    __syncthreads();   // the blocks given back are on the stack before any is taken
    for (int i = tid; i < takes; i += kPlanThreads) {
      const int b = owner_of(pre_take, B, i);
      int L, to;
      read_len(b, L, to);
      a.table[static_cast<size_t>(b) * a.max_blocks + ((L + bs - 1) >> sh) + i - pre_take[b]] =
          a.free_blocks[static_cast<int>(top) - 1 - i];
    }
  }
  __syncthreads();
  // lengths (kv_lens_out may be kv_lens: each is read and written by one thread) and
  // the running number of new tokens
  int carry = 0;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int add = 0, zero = 0;
    if (b < B) {
      int L, to;
      const bool ok = read_len(b, L, to);
      const int keep = a.kv_lens[b];
      add = bad ? 0 : max(0, to - L);
      a.kv_lens_out[b] = bad || !ok ? keep : to;
    }
    int incl = add;
    block_scan2(incl, zero, warp_tot);
    if (b < B) a.cu_new[b + 1] = carry + incl;
    carry += warp_tot[31].x;
    __syncthreads();
  }
  if (tid == 0) {
    a.cu_new[0] = 0;
    *a.free_count_out = bad ? c : static_cast<int>(top) - takes;
  }
}

// Slots of the new tokens, in sequence order; -1 behind the last one. The
// position follows from the new length, so kv_lens_out may be kv_lens.
__global__ void __launch_bounds__(256) k_qslots(const __grid_constant__ QPlanArgs a) {
  pdl_wait();
  pdl_trigger();
  const int sh = a.bs_shift, mask = (1 << sh) - 1;
  const int total = a.cu_new[a.B];
  for (int i = blockIdx.x * 256 + threadIdx.x; i < a.max_new; i += gridDim.x * 256) {
    int slot = -1;
    if (i < total) {
      int lo = 0, hi = a.B;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.cu_new[mid] <= i) lo = mid;
        else hi = mid;
      }
      const int p = a.kv_lens_out[lo] - a.cu_new[lo + 1] + i;
      const int id = a.table[static_cast<size_t>(lo) * a.max_blocks + (p >> sh)];
      if (id >= 0 && id < a.num_blocks) slot = (id << sh) | (p & mask);
      else report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x502);   // the old last block's id
    }
    a.slot_map[i] = slot;
  }
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

cudaError_t launch_qplan(const QPlanArgs& a, cudaStream_t st) {
  const size_t smem = 2 * (static_cast<size_t>(a.B) + 1) * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(k_qplan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  if ((e = launch_pdl(k_qplan, dim3(1), dim3(kPlanThreads), smem, st, a)) != cudaSuccess) return e;
  if (a.max_new == 0) return cudaSuccess;
  const int blocks = (a.max_new + 255) / 256;
  return launch_pdl(k_qslots, dim3(blocks < 608 ? blocks : 608), dim3(256), 0, st, a);
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
