// rope.cu — queries and keys on their way into attention: each head's row is
// divided by its root mean square (where there is a weight) and its pairs are
// turned by the token's position, in one pass.
//
//   k_qk_rope       q and k into the layouts the attention calls take
//   k_qappend_rope  k and v of new tokens into the paged 4-bit cache, and the
//                   step's queries
//
//   y = x * rsqrt(mean(x^2) + eps) * w
//   (a, b) -> (a c - b s, b c + a s),  (c, s) = table[pos[axis of the pair]][pair]
// in fp32, rounded once at the end. The two products of an element are rounded
// apart (no fused multiply-add), so that an element has one value whatever a
// compiler or a plain program makes of it: the 4-bit codes behind it depend on
// every bit. The pages describe no rotation; a Kascade layer's q and k are
// the rotated ones.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "qcache.h"
#include "qrows.cuh"
#include "rope.h"

namespace kascade {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// A thread has 32 elements of a row, two blocks of 16 that hold whole pairs:
// blocks (t, t + n_pairs / 16) where pair i is (i, i + n_pairs), neighbouring
// ones where it is (2 i, 2 i + 1) or where nothing is turned. D / 32 threads
// share a row, and the pairs of thread t are 16 t .. 16 t + 15.
template <int D>
struct Lane {
  static constexpr int kPerRow = D / 32, kSlots = 32 / kPerRow;   // threads, rows of a warp
  int t, slot, at[2];   // thread of the row, row of the warp, first element of the blocks
  bool turns;
  __device__ __forceinline__ Lane(const RopeSpec& r) {
    const int lane = threadIdx.x & 31, groups = r.n_pairs >> 4;
    t = lane % kPerRow;
    slot = lane / kPerRow;
    turns = t < groups;
    const bool far = turns && !r.interleaved;
    at[0] = far ? 16 * t : 32 * t;
    at[1] = far ? 16 * (t + groups) : 32 * t + 16;
  }
};

// 32 elements as they are in memory.
template <typename T>
struct Raw {
  static constexpr int kVec = sizeof(T);   // 16-byte pieces of a block
  uint4 v[2][kVec];
  __device__ __forceinline__ void load(const T* row, const int (&at)[2], bool ok) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < kVec; ++i)
        v[b][i] = ok ? *(reinterpret_cast<const uint4*>(row + at[b]) + i) : make_uint4(0u, 0u, 0u, 0u);
  }
  __device__ __forceinline__ void get(float (&x)[32]) const {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const uint32_t w[4] = {v[b][i].x, v[b][i].y, v[b][i].z, v[b][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (sizeof(T) == 4) {
            x[16 * b + 4 * i + j] = __uint_as_float(w[j]);
          } else {
            x[16 * b + 8 * i + 2 * j] = __uint_as_float(w[j] << 16);
            x[16 * b + 8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
        }
      }
  }
};

__device__ __forceinline__ void store_row(float* row, const int (&at)[2], const float (&x)[32]) {
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* p = x + 16 * b + 4 * i;
      *(reinterpret_cast<float4*>(row + at[b]) + i) = make_float4(p[0], p[1], p[2], p[3]);
    }
}
__device__ __forceinline__ void store_row(__nv_bfloat16* row, const int (&at)[2],
                                          const float (&x)[32]) {
#pragma unroll
  for (int b = 0; b < 2; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float* p = x + 16 * b + 8 * i;
      *(reinterpret_cast<uint4*>(row + at[b]) + i) =
          make_uint4(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]),
                     pack_bf16(p[6], p[7]));
    }
}

// Cosines and sines of this thread's pairs. pos(axis) gives the token's position.
struct Turn {
  float c[16], s[16];
};
template <bool MIXED, int D, typename Pos>
__device__ __forceinline__ void load_turn(const RopeSpec& r, const Lane<D>& l, Pos pos,
                                          unsigned int* err, Turn& u) {
  if (!l.turns) return;
  const size_t width = 2 * static_cast<size_t>(r.n_pairs);
  auto row = [&](int axis) -> const float* {   // null: a position outside the table
    const int p = pos(axis);
    if (p < 0 || p >= r.n_pos) {
      report_error(err, KASCADE_ERR_BAD_INPUT, 0x541);
      return nullptr;
    }
    return r.table + p * width + 16 * l.t;
  };
  if (MIXED) {
    const float* rows[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[i] = i < r.n_axes ? row(i) : nullptr;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int axis = r.axis[16 * l.t + i];
      const float* p = axis == 0 ? rows[0] : axis == 1 ? rows[1] : axis == 2 ? rows[2] : rows[3];
      u.c[i] = p != nullptr ? __ldg(p + i) : 1.f;
      u.s[i] = p != nullptr ? __ldg(p + r.n_pairs + i) : 0.f;
    }
  } else {
    const float* p = row(r.axis[0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 c = p != nullptr ? __ldg(reinterpret_cast<const float4*>(p) + i)
                                    : make_float4(1.f, 1.f, 1.f, 1.f);
      const float4 s = p != nullptr ? __ldg(reinterpret_cast<const float4*>(p + r.n_pairs) + i)
                                    : make_float4(0.f, 0.f, 0.f, 0.f);
      u.c[4 * i] = c.x, u.c[4 * i + 1] = c.y, u.c[4 * i + 2] = c.z, u.c[4 * i + 3] = c.w;
      u.s[4 * i] = s.x, u.s[4 * i + 1] = s.y, u.s[4 * i + 2] = s.z, u.s[4 * i + 3] = s.w;
    }
  }
}

// x / rms(row) * w; all lanes of the warp.
template <typename T, int D>
__device__ __forceinline__ void normalise(float (&x)[32], const T* w, const Lane<D>& l, float eps) {
  float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 32; ++i) part[i & 3] = fmaf(x[i], x[i], part[i & 3]);
  float ss = (part[0] + part[1]) + (part[2] + part[3]);
#pragma unroll
  for (int off = 1; off < Lane<D>::kPerRow; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
  const float r = rsqrtf(ss * (1.f / D) + eps);
  Raw<T> raw;
  raw.load(w, l.at, true);
  float g[32];
  raw.get(g);
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = x[i] * r * g[i];
}

template <bool INTER, int D>
__device__ __forceinline__ void turn(float (&x)[32], const Turn& u, const Lane<D>& l) {
  if (!l.turns) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    constexpr int kA = INTER ? 2 : 1, kB = INTER ? 1 : 16;
    float& xa = x[kA * i];
    float& xb = x[kA * i + kB];
    const float a = xa, b = xb;
    xa = __fsub_rn(__fmul_rn(a, u.c[i]), __fmul_rn(b, u.s[i]));
    xb = __fadd_rn(__fmul_rn(b, u.c[i]), __fmul_rn(a, u.s[i]));
  }
}

// ------------------------------------------------------------- q and k rows --
// A warp has one token and `per` heads of its list of q and k heads, kSlots of
// them at a time.
template <typename T, int D, bool INTER, bool MIXED>
__global__ void __launch_bounds__(kThreads) k_qk_rope(const __grid_constant__ RopeRowArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t token = unit / a.splits;
  if (token >= static_cast<int64_t>(a.B) * a.N) return;
  const int part = static_cast<int>(unit - token * a.splits);
  const int b = static_cast<int>(token / a.N), n = static_cast<int>(token - static_cast<int64_t>(b) * a.N);
  const Lane<D> l(a.rope);
  const int total = a.H[0] + a.H[1], h1 = min(total, (part + 1) * a.per);
  const int64_t plane = static_cast<int64_t>(a.B) * a.N;
  Turn u;
  Raw<T> raw;
  auto load = [&](int h) {
    const int which = h >= a.H[0] ? 1 : 0;
    const int64_t* st = a.src_stride[which];
    const T* row = static_cast<const T*>(a.src[which]) + b * st[0] + n * st[1] +
                   (h - (which ? a.H[0] : 0)) * st[2];
    raw.load(row, l.at, h < h1);
  };
  int h = part * a.per + l.slot;
  load(h);
  load_turn<MIXED>(a.rope, l, [&](int axis) { return __ldg(a.positions + axis * plane + token); },
                   a.err, u);
  for (int h0 = part * a.per; h0 < h1; h0 += Lane<D>::kSlots, h += Lane<D>::kSlots) {
    float x[32];
    raw.get(x);
    if (h0 + Lane<D>::kSlots < h1) load(h + Lane<D>::kSlots);
    const int which = h >= a.H[0] ? 1 : 0;
    const T* w = static_cast<const T*>(a.weight[which]);
    if (a.weight[0] != nullptr || a.weight[1] != nullptr) {
      float y[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) y[i] = x[i];
      normalise<T, D>(y, w != nullptr ? w : static_cast<const T*>(a.weight[1 - which]), l,
                      a.rope.eps);
      if (w != nullptr)
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = y[i];
    }
    turn<INTER, D>(x, u, l);
    if (h < h1) {
      const int64_t* st = a.dst_stride[which];
      store_row(static_cast<T*>(a.dst[which]) + b * st[0] + n * st[1] +
                    (h - (which ? a.H[0] : 0)) * st[2],
                l.at, x);
    }
  }
}

// ------------------------------------------------------------ cache appends --
// The sequence whose new tokens hold row t: the largest b with cu[b] <= t, by 32
// tests at a time (all lanes).
__device__ __forceinline__ int owner_of_row(const int32_t* cu, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seqs;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lane * step;
    const bool below = at < n && __ldg(cu + lo + at) <= t;
    const unsigned int m = __ballot_sync(0xffffffffu, below) | 1u;
    const int last = 31 - __clz(m);
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

template <typename T, int D, bool INTER, bool MIXED>
__global__ void __launch_bounds__(kThreads)
    k_qappend_rope(const __grid_constant__ RopeAppendArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int kSlots = Lane<D>::kSlots;
  int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t q_units = static_cast<int64_t>(a.Tq) * a.q_splits;
  const Lane<D> l(a.rope);
  Turn u;
  if (unit < q_units) {   // queries
    const int row = static_cast<int>(unit / a.q_splits), part = static_cast<int>(unit % a.q_splits);
    const int h1 = min(a.Hq, (part + 1) * a.q_per);
    const T* src = static_cast<const T*>(a.q) + row * a.q_stride[0];
    T* dst = static_cast<T*>(a.q_out) + row * a.out_stride[0];
    int h = part * a.q_per + l.slot;
    Raw<T> raw;
    raw.load(src + h * a.q_stride[1], l.at, h < h1);
    load_turn<MIXED>(
        a.rope, l,
        [&](int axis) {
          return a.positions != nullptr ? __ldg(a.positions + static_cast<int64_t>(axis) * a.T + row)
                                        : max(0, __ldg(a.kv_lens + row) - 1);
        },
        a.err, u);
    for (int h0 = part * a.q_per; h0 < h1; h0 += kSlots, h += kSlots) {
      float x[32];
      raw.get(x);
      if (h0 + kSlots < h1) raw.load(src + (h + kSlots) * a.q_stride[1], l.at, h + kSlots < h1);
      if (a.weight[0] != nullptr)
        normalise<T, D>(x, static_cast<const T*>(a.weight[0]), l, a.rope.eps);
      turn<INTER, D>(x, u, l);
      if (h < h1) store_row(dst + h * a.out_stride[1], l.at, x);
    }
    return;
  }
  unit -= q_units;
  const int64_t token = unit / a.kv_splits;
  if (token >= a.T) return;
  const int t = static_cast<int>(token), part = static_cast<int>(unit - token * a.kv_splits);
  const int slot = a.slot_map[t];
  if (slot < 0) return;
  const int sh = a.bs_shift;
  if ((slot >> sh) >= a.num_blocks) {
    report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x511);
    return;
  }
  const int h1 = min(2 * a.Hkv, (part + 1) * a.kv_per);   // K heads, then V heads
  const T* src[2] = {static_cast<const T*>(a.k) + t * a.k_stride[0],
                     static_cast<const T*>(a.v) + t * a.v_stride[0]};
  Raw<T> raw;
  auto load = [&](int h) {
    const int which = h >= a.Hkv ? 1 : 0;
    raw.load(src[which] + (which ? (h - a.Hkv) * a.v_stride[1] : h * a.k_stride[1]), l.at, h < h1);
  };
  int h = part * a.kv_per + l.slot;
  load(h);
  if (part * a.kv_per < a.Hkv) {
    int from_plan = 0;
    if (a.positions == nullptr) {
      const int b = owner_of_row(a.cu_new, a.n_seqs, t);
      from_plan = __ldg(a.kv_lens + b) - __ldg(a.cu_new + b + 1) + t;
    }
    load_turn<MIXED>(
        a.rope, l,
        [&](int axis) {
          return a.positions != nullptr ? __ldg(a.positions + static_cast<int64_t>(axis) * a.T + t)
                                        : from_plan;
        },
        a.err, u);
  }
  const int r = slot & 15;
  const size_t first = (static_cast<size_t>(slot >> sh) * a.Hkv << (sh - 4)) +
                       ((slot & ((1 << sh) - 1)) >> 4);
  for (int h0 = part * a.kv_per; h0 < h1; h0 += kSlots, h += kSlots) {
    float x[32];
    raw.get(x);
    const bool key = h < a.Hkv;
    if (h0 + kSlots < h1) load(h + kSlots);
    if (a.weight[1] != nullptr && h0 < a.Hkv) {
      float y[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) y[i] = x[i];
      normalise<T, D>(y, static_cast<const T*>(a.weight[1]), l, a.rope.eps);
      if (key)
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = y[i];
    }
    if (key) turn<INTER, D>(x, u, l);
    if (h >= h1) continue;
    const int head = key ? h : h - a.Hkv;
    uint8_t* grp = a.cache + (first + (static_cast<size_t>(head) << (sh - 4))) * (18 * D) +
                   (key ? 0 : 9 * D);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      Row16<float> y;
#pragma unroll
      for (int i = 0; i < 16; ++i) y.x[i] = x[16 * b + i];
      put16(y, a.unit[key ? 0 : 1], grp + r * (D / 2) + l.at[b] / 2,
            grp + 8 * D + r * (D / 16) + l.at[b] / 16);
    }
  }
}

// Heads of a warp: all of a token's, where there are enough tokens to fill the
// GPU with `want` warps, else fewer.
void split_heads(int64_t tokens, int heads, int slots, int& splits, int& per) {
  constexpr int64_t want = 152 * 16;
  const int chunks = (heads + slots - 1) / slots;
  int64_t n = tokens > 0 ? (want + tokens - 1) / tokens : 1;
  if (n > chunks) n = chunks;
  const int each = (chunks + static_cast<int>(n) - 1) / static_cast<int>(n);
  per = each * slots;
  splits = (chunks + each - 1) / each;
}

template <typename T, int D>
cudaError_t launch_qk(const RopeRowArgs& a, cudaStream_t st) {
  RopeRowArgs u = a;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  split_heads(tokens, a.H[0] + a.H[1], Lane<D>::kSlots, u.splits, u.per);
  const int64_t ctas = (tokens * u.splits + kWarps - 1) / kWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned int>(ctas));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kThreads), 0, st, u); };
  if (a.rope.interleaved)
    return a.rope.mixed ? go(k_qk_rope<T, D, true, true>) : go(k_qk_rope<T, D, true, false>);
  return a.rope.mixed ? go(k_qk_rope<T, D, false, true>) : go(k_qk_rope<T, D, false, false>);
}

template <typename T, int D>
cudaError_t launch_append(const RopeAppendArgs& a, cudaStream_t st) {
  RopeAppendArgs u = a;
  split_heads(a.Tq, a.Hq, Lane<D>::kSlots, u.q_splits, u.q_per);
  split_heads(a.T, 2 * a.Hkv, Lane<D>::kSlots, u.kv_splits, u.kv_per);
  const int64_t warps = static_cast<int64_t>(a.Tq) * u.q_splits + static_cast<int64_t>(a.T) * u.kv_splits;
  const int64_t ctas = (warps + kWarps - 1) / kWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned int>(ctas));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kThreads), 0, st, u); };
  if (a.rope.interleaved)
    return a.rope.mixed ? go(k_qappend_rope<T, D, true, true>)
                        : go(k_qappend_rope<T, D, true, false>);
  return a.rope.mixed ? go(k_qappend_rope<T, D, false, true>)
                      : go(k_qappend_rope<T, D, false, false>);
}

inline bool aligned(const void* p, uintptr_t n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

}  // namespace

cudaError_t launch_qk_rope(const RopeRowArgs& a, int d, int dtype, cudaStream_t st) {
  if (a.B == 0 || a.N == 0) return cudaSuccess;
  if (dtype == KASCADE_F32) return d == 128 ? launch_qk<float, 128>(a, st) : launch_qk<float, 64>(a, st);
  return d == 128 ? launch_qk<__nv_bfloat16, 128>(a, st) : launch_qk<__nv_bfloat16, 64>(a, st);
}

cudaError_t launch_qappend_rope(const RopeAppendArgs& a, int d, int dtype, cudaStream_t st) {
  if (a.T == 0 && a.Tq == 0) return cudaSuccess;
  if (dtype == KASCADE_F32)
    return d == 128 ? launch_append<float, 128>(a, st) : launch_append<float, 64>(a, st);
  return d == 128 ? launch_append<__nv_bfloat16, 128>(a, st)
                  : launch_append<__nv_bfloat16, 64>(a, st);
}

kascade_status check_rope(const kascade_rope* rope, int head_dim, float eps, RopeSpec& s) {
  memset(&s, 0, sizeof(s));
  if (!(eps >= 0.f) || eps > 1e30f) return KASCADE_ERR_INVALID_ARG;
  s.eps = eps;
  s.n_axes = 1;
  if (head_dim != 64 && head_dim != 128) return KASCADE_ERR_UNSUPPORTED;
  if (rope == nullptr) return KASCADE_OK;
  if (!aligned(rope->table, 16) || rope->n_positions < 1 || rope->n_pairs < 1 ||
      2 * static_cast<int64_t>(rope->n_pairs) > head_dim || rope->n_axes < 1 || rope->n_axes > 4)
    return KASCADE_ERR_INVALID_ARG;
  if (rope->n_pairs % 16 != 0) return KASCADE_ERR_UNSUPPORTED;
  s.table = rope->table;
  s.n_pos = rope->n_positions;
  s.n_pairs = rope->n_pairs;
  s.n_axes = rope->n_axes;
  s.interleaved = rope->interleaved != 0;
  for (int i = 0; rope->axes != nullptr && i < rope->n_pairs; ++i) {
    if (rope->axes[i] < 0 || rope->axes[i] >= rope->n_axes) return KASCADE_ERR_INVALID_ARG;
    s.axis[i] = static_cast<uint8_t>(rope->axes[i]);
    if (s.axis[i] != s.axis[0]) s.mixed = 1;
  }
  return KASCADE_OK;
}

}  // namespace kascade

using namespace kascade;

extern "C" kascade_status kascade_qk_norm_rope(
    const kascade_rope* rope, int32_t batch, int32_t n_tokens, int32_t n_q_heads,
    int32_t n_kv_heads, int32_t head_dim, int32_t dtype, const void* q, const void* k,
    const void* q_weight, const void* k_weight, float eps, const int32_t* positions, void* q_out,
    void* k_out, const int64_t* strides, void* ws, size_t ws_bytes, void* stream) {
  RopeRowArgs a{};
  const kascade_status r = check_rope(rope, head_dim, eps, a.rope);
  if (r != KASCADE_OK) return r;
  if (dtype != KASCADE_F32 && dtype != KASCADE_BF16) return KASCADE_ERR_INVALID_ARG;
  if (batch < 0 || n_tokens < 0 || n_q_heads < 0 || n_kv_heads < 0 || n_q_heads > kMaxQHeads ||
      n_kv_heads > kMaxQHeads || n_q_heads + n_kv_heads < 1 || strides == nullptr)
    return KASCADE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * n_tokens >= (int64_t(1) << 28)) return KASCADE_ERR_UNSUPPORTED;
  if (!aligned(ws, 256) || ws_bytes < sizeof(WsHeader)) return KASCADE_ERR_WORKSPACE;
  if (batch == 0 || n_tokens == 0) return KASCADE_OK;
  const void* src[2] = {q, k};
  void* dst[2] = {q_out, k_out};
  const void* weight[2] = {q_weight, k_weight};
  const int heads[2] = {n_q_heads, n_kv_heads};
  const int64_t unit = dtype == KASCADE_F32 ? 4 : 8;   // rows start on 16-byte boundaries
  for (int i = 0; i < 2; ++i) {
    a.H[i] = heads[i];
    if (heads[i] == 0) continue;
    if (!aligned(src[i], 16) || !aligned(dst[i], 16) ||
        (weight[i] != nullptr && !aligned(weight[i], 16)))
      return KASCADE_ERR_INVALID_ARG;
    a.src[i] = src[i];
    a.dst[i] = dst[i];
    a.weight[i] = weight[i];
    for (int j = 0; j < 3; ++j) {
      a.src_stride[i][j] = strides[3 * i + j];
      a.dst_stride[i][j] = strides[6 + 3 * i + j];
      if (a.src_stride[i][j] < 0 || a.src_stride[i][j] % unit != 0 || a.dst_stride[i][j] < 0 ||
          a.dst_stride[i][j] % unit != 0)
        return KASCADE_ERR_INVALID_ARG;
    }
  }
  if (a.rope.table != nullptr && !aligned(positions, 4)) return KASCADE_ERR_INVALID_ARG;
  a.positions = positions;
  a.err = static_cast<unsigned int*>(ws);
  a.B = batch;
  a.N = n_tokens;
  const cudaError_t e = launch_qk_rope(a, head_dim, dtype, static_cast<cudaStream_t>(stream));
  if (e == cudaErrorNotSupported) return KASCADE_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KASCADE_OK : KASCADE_ERR_CUDA;
}
