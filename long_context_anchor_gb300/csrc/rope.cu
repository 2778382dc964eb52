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
//
// Both are bound by memory where they are large. Rows of 16384 tokens, 32 + 8 heads of
// 128, bf16 with norm: 60.2 us, 5.7 TB/s (issue slots 70% full); 131072 tokens, 64 + 8
// heads of 64, half turned: 399 us, 6.1 TB/s; 2 x 5003 tokens, 16 + 4 heads of 64 in fp32
// on three axes: 23.8 us, 4.4 TB/s: its 1251 CTAs are 2.06 rounds of the 608 that run at once
// (9728 tokens, 2.00 rounds, take 20.4). Into the cache with queries, 16384 tokens, 32 + 8
// heads: 71 us, 5.0 TB/s (issue 54%, loads waited for 7 issues each: a warp has few rows in
// flight in 64 registers), 74 with norms. A step's few rows take 2.3 and 3.4 us (3.8 with
// norms), a launch's latency; a row's way into the cache is a chain of slot, owner, lengths
// and the table's row, in front of its first elements.
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
constexpr int kCtasPerSm = 4;   // 64 registers a thread

// ------------------------------------------------------------- q and k rows --
// A thread has two 16-byte pieces of a row that hold whole pairs: pieces (t, t +
// n_pairs / kVec) where pair i is (i, i + n_pairs), neighbouring ones where it is
// (2 i, 2 i + 1) or where nothing is turned; the pairs of thread t are kVec t .. . So
// the loads and the stores of neighbouring threads fill whole sectors, and a token's
// cosines and sines stay in 4 kVec registers while a warp goes through its heads.
template <typename T, int D>
struct Lane {
  static constexpr int kVec = 16 / sizeof(T), kPerRow = D / (2 * kVec), kSlots = 32 / kPerRow;
  int t, slot, at[2];   // thread of the row, row of the warp, first element of the pieces
  bool turns;
  __device__ __forceinline__ Lane(const RopeSpec& r) {
    const int lane = threadIdx.x & 31, groups = r.n_pairs / kVec;
    t = lane % kPerRow;
    slot = lane / kPerRow;
    turns = t < groups;
    const bool far = turns && !r.interleaved;
    at[0] = far ? kVec * t : 2 * kVec * t;
    at[1] = far ? kVec * (t + groups) : 2 * kVec * t + kVec;
  }
};

__device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
  x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
  x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = __uint_as_float(w[j] << 16);
    x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ uint4 packed(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                    __float_as_uint(x[3]));
}
__device__ __forceinline__ uint4 packed(const float (&x)[8]) {
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                    pack_bf16(x[6], x[7]));
}
// Rows may be turned in place, so they are no read-only data.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* p) { return *reinterpret_cast<const uint4*>(p); }

// Row `pos` of the table (null: outside it, reported).
__device__ __forceinline__ const float* table_row(const RopeSpec& r, int pos, unsigned int* err) {
  if (pos < 0 || pos >= r.n_pos) {
    report_error(err, KASCADE_ERR_BAD_INPUT, 0x541);
    return nullptr;
  }
  return r.table + pos * (2 * static_cast<size_t>(r.n_pairs));
}

// Four pairs' cosines and sines from pair `first` on (a multiple of 4) at rows[axis].
template <bool MIXED>
__device__ __forceinline__ void load_turn4(const RopeSpec& r, const float* const (&rows)[4], int first,
                                           float* c, float* s) {
  auto row_of = [&](int axis) {
    return axis == 0 ? rows[0] : axis == 1 ? rows[1] : axis == 2 ? rows[2] : rows[3];
  };
  if (MIXED && !r.quads) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float* p = row_of(r.axis[first + i]);
      c[i] = p != nullptr ? __ldg(p + first + i) : 1.f;
      s[i] = p != nullptr ? __ldg(p + r.n_pairs + first + i) : 0.f;
    }
    return;
  }
  const float* p = MIXED ? row_of(r.axis[first]) : rows[0];
  float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p != nullptr) {
    a = __ldg(reinterpret_cast<const float4*>(p + first));
    b = __ldg(reinterpret_cast<const float4*>(p + r.n_pairs + first));
  }
  c[0] = a.x, c[1] = a.y, c[2] = a.z, c[3] = a.w;
  s[0] = b.x, s[1] = b.y, s[2] = b.z, s[3] = b.w;
}
// The rows of the axes that pairs follow; pos(axis) gives a token's positions.
template <bool MIXED, typename Pos>
__device__ __forceinline__ void table_rows(const RopeSpec& r, Pos pos, unsigned int* err,
                                           const float* (&rows)[4]) {
  if (MIXED) {
#pragma unroll
    for (int i = 0; i < 4; ++i) rows[i] = (r.used >> i) & 1 ? table_row(r, pos(i), err) : nullptr;
  } else {
    rows[0] = table_row(r, pos(r.axis[0]), err);
    rows[1] = rows[2] = rows[3] = nullptr;
  }
}

__device__ __forceinline__ void turn_pair(float& xa, float& xb, float c, float s) {
  const float a = xa, b = xb;
  xa = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  xb = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}

// What a warp does of one token's rows: heads h0 .. h1 - 1 of a list, kSlots at a time,
// the next ones loaded while these are computed. src(h), dst(h): rows, weight(h): the
// norm's weights or null (any: whether some head has them).
template <typename T, int D, bool INTER, bool MIXED, typename Src, typename Dst, typename Weight,
          typename Pos>
__device__ __forceinline__ void turn_rows(const RopeSpec& r, int h0, int h1, Src src, Dst dst,
                                          Weight weight, bool any, Pos pos, unsigned int* err) {
  using L = Lane<T, D>;
  constexpr int V = L::kVec;
  const L l(r);
  uint4 raw[2];
  int h = h0 + l.slot;
  auto load = [&](int at) {
    raw[0] = raw[1] = make_uint4(0u, 0u, 0u, 0u);
    if (at < h1) {
      const T* row = src(at);
      raw[0] = load16(row + l.at[0]);
      raw[1] = load16(row + l.at[1]);
    }
  };
  load(h);
  float c[V], s[V];
  if (l.turns) {
    const float* rows[4];
    table_rows<MIXED>(r, pos, err, rows);
#pragma unroll
    for (int i = 0; i < V; i += 4) load_turn4<MIXED>(r, rows, V * l.t + i, c + i, s + i);
  }
  for (int first = h0; first < h1; first += L::kSlots, h += L::kSlots) {
    float x[2][V];
    unpack(raw[0], x[0]);
    unpack(raw[1], x[1]);
    if (first + L::kSlots < h1) load(h + L::kSlots);
    if (any) {
      const T* w = weight(min(h, h1 - 1));
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x[0][i], x[0][i], ss);
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x[1][i], x[1][i], ss);
#pragma unroll
      for (int off = 1; off < L::kPerRow; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (w != nullptr) {
        const float n = rsqrtf(ss * (1.f / D) + r.eps);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float g[V];
          unpack(__ldg(reinterpret_cast<const uint4*>(w + l.at[b])), g);
#pragma unroll
          for (int i = 0; i < V; ++i) x[b][i] = x[b][i] * n * g[i];
        }
      }
    }
    if (l.turns) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (INTER) turn_pair(x[2 * i / V][2 * i % V], x[2 * i / V][2 * i % V + 1], c[i], s[i]);
        else turn_pair(x[0][i], x[1][i], c[i], s[i]);
      }
    }
    if (h < h1) {
      T* row = dst(h);
      *reinterpret_cast<uint4*>(row + l.at[0]) = packed(x[0]);
      *reinterpret_cast<uint4*>(row + l.at[1]) = packed(x[1]);
    }
  }
}

template <typename T, int D, bool INTER, bool MIXED>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    k_qk_rope(const __grid_constant__ RopeRowArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t token = unit / a.splits;
  if (token >= static_cast<int64_t>(a.B) * a.N) return;
  const int part = static_cast<int>(unit - token * a.splits);
  const int b = static_cast<int>(token / a.N), n = static_cast<int>(token - static_cast<int64_t>(b) * a.N);
  const int64_t plane = static_cast<int64_t>(a.B) * a.N;
  // q's head 0, and what would be k's if its heads were counted from q's first one
  const T* q = static_cast<const T*>(a.src[0]) + b * a.src_stride[0][0] + n * a.src_stride[0][1];
  const T* k = static_cast<const T*>(a.src[1]) + b * a.src_stride[1][0] + n * a.src_stride[1][1] -
               a.H[0] * a.src_stride[1][2];
  T* q_to = static_cast<T*>(a.dst[0]) + b * a.dst_stride[0][0] + n * a.dst_stride[0][1];
  T* k_to = static_cast<T*>(a.dst[1]) + b * a.dst_stride[1][0] + n * a.dst_stride[1][1] -
            a.H[0] * a.dst_stride[1][2];
  const int h0 = part * a.per;
  turn_rows<T, D, INTER, MIXED>(
      a.rope, h0, min(a.H[0] + a.H[1], h0 + a.per),
      [&](int h) { return h < a.H[0] ? q + h * a.src_stride[0][2] : k + h * a.src_stride[1][2]; },
      [&](int h) { return h < a.H[0] ? q_to + h * a.dst_stride[0][2] : k_to + h * a.dst_stride[1][2]; },
      [&](int h) { return static_cast<const T*>(h < a.H[0] ? a.weight[0] : a.weight[1]); },
      a.weight[0] != nullptr || a.weight[1] != nullptr,
      [&](int axis) { return __ldg(a.positions + axis * plane + token); }, a.err);
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

// New keys and values: a thread has 32 elements of a row, two blocks of 16 that find
// their scales alone (blocks as the pieces above: (t, t + n_pairs / 16) or neighbouring
// ones). Few heads share a token's cosines and sines, which are loaded where they are
// used instead of held.
template <typename T>
__device__ __forceinline__ void load_block(const T* p, float (&x)[16]) {
  constexpr int V = 16 / sizeof(T);
#pragma unroll
  for (int i = 0; i < 16; i += V) {
    float y[V];
    unpack(load16(p + i), y);
#pragma unroll
    for (int j = 0; j < V; ++j) x[i + j] = y[j];
  }
}

template <typename T, int D, bool INTER, bool MIXED>
__device__ __forceinline__ void append_rows(const RopeAppendArgs& a, int t, int h0, int h1) {
  constexpr int kPerRow = D / 32, kSlots = 32 / kPerRow;
  const int slot = a.slot_map[t];
  if (slot < 0) return;
  const int sh = a.bs_shift;
  if ((slot >> sh) >= a.num_blocks) {
    report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x511);
    return;
  }
  const int lane = threadIdx.x & 31, part = lane % kPerRow, groups = a.rope.n_pairs / 16;
  const bool turns = part < groups, far = turns && !INTER;
  const int at[2] = {far ? 16 * part : 32 * part, far ? 16 * (part + groups) : 32 * part + 16};
  const float* rows[4] = {};
  if (h0 < a.Hkv && a.rope.table != nullptr) {   // without a table there may be no positions
    int from_plan = 0;
    if (a.positions == nullptr) {
      const int b = owner_of_row(a.cu_new, a.n_seqs, t);
      from_plan = __ldg(a.kv_lens + b) - __ldg(a.cu_new + b + 1) + t;
    }
    if (turns)
      table_rows<MIXED>(
          a.rope,
          [&](int axis) {
            return a.positions != nullptr ? __ldg(a.positions + static_cast<int64_t>(axis) * a.T + t)
                                          : from_plan;
          },
          a.err, rows);
  }
  const int r = slot & 15;
  const size_t first = (static_cast<size_t>(slot >> sh) * a.Hkv << (sh - 4)) +
                       ((slot & ((1 << sh) - 1)) >> 4);
  for (int g0 = h0; g0 < h1; g0 += kSlots) {
    const int h = g0 + lane / kPerRow;   // K heads, then V heads
    const bool key = h < a.Hkv;
    const int head = key ? h : h - a.Hkv;
    Row16<float> x[2] = {};
    if (h < h1) {
      const T* row = key ? static_cast<const T*>(a.k) + t * a.k_stride[0] + head * a.k_stride[1]
                         : static_cast<const T*>(a.v) + t * a.v_stride[0] + head * a.v_stride[1];
      load_block(row + at[0], x[0].x);
      load_block(row + at[1], x[1].x);
    }
    if (a.weight[1] != nullptr && g0 < a.Hkv) {
      float ss = 0.f;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(x[b].x[i], x[b].x[i], ss);
#pragma unroll
      for (int off = 1; off < kPerRow; off <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      if (key) {
        const float n = rsqrtf(ss * (1.f / D) + a.rope.eps);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          float g[16];
          load_block(static_cast<const T*>(a.weight[1]) + at[b], g);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[b].x[i] = x[b].x[i] * n * g[i];
        }
      }
    }
    if (key && turns) {
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        float c[4], s[4];
        load_turn4<MIXED>(a.rope, rows, 16 * part + i, c, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = i + j;
          if (INTER) turn_pair(x[k / 8].x[2 * k % 16], x[k / 8].x[2 * k % 16 + 1], c[j], s[j]);
          else turn_pair(x[0].x[k], x[1].x[k], c[j], s[j]);
        }
      }
    }
    if (h >= h1) continue;
    uint8_t* grp = a.cache + (first + (static_cast<size_t>(head) << (sh - 4))) * (18 * D) +
                   (key ? 0 : 9 * D);
#pragma unroll
    for (int b = 0; b < 2; ++b)
      put16(x[b], a.unit[key ? 0 : 1], grp + r * (D / 2) + at[b] / 2,
            grp + 8 * D + r * (D / 16) + at[b] / 16);
  }
}

template <typename T, int D, bool INTER, bool MIXED, int CTAS_PER_SM>
__global__ void __launch_bounds__(kThreads, CTAS_PER_SM)
    k_qappend_rope(const __grid_constant__ RopeAppendArgs a) {
  pdl_wait();
  pdl_trigger();
  int64_t unit = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t q_units = static_cast<int64_t>(a.Tq) * a.q_splits;
  if (unit < q_units) {   // queries
    const int row = static_cast<int>(unit / a.q_splits), part = static_cast<int>(unit % a.q_splits);
    const T* src = static_cast<const T*>(a.q) + row * a.q_stride[0];
    T* dst = static_cast<T*>(a.q_out) + row * a.out_stride[0];
    const int h0 = part * a.q_per;
    turn_rows<T, D, INTER, MIXED>(
        a.rope, h0, min(a.Hq, h0 + a.q_per), [&](int h) { return src + h * a.q_stride[1]; },
        [&](int h) { return dst + h * a.out_stride[1]; },
        [&](int) { return static_cast<const T*>(a.weight[0]); }, a.weight[0] != nullptr,
        [&](int axis) {
          return a.positions != nullptr ? __ldg(a.positions + static_cast<int64_t>(axis) * a.T + row)
                                        : max(0, __ldg(a.kv_lens + row) - 1);
        },
        a.err);
    return;
  }
  unit -= q_units;
  const int64_t token = unit / a.kv_splits;
  if (token >= a.T) return;
  const int h0 = static_cast<int>(unit - token * a.kv_splits) * a.kv_per;
  append_rows<T, D, INTER, MIXED>(a, static_cast<int>(token), h0, min(2 * a.Hkv, h0 + a.kv_per));
}

// Heads of a warp: all of a token's, where there are enough tokens to fill the
// GPU with `want` warps, else fewer. No tokens or heads (an append without queries): none.
void split_heads(int64_t tokens, int heads, int slots, int& splits, int& per) {
  constexpr int64_t want = 152 * 32;
  splits = per = 0;
  if (tokens < 1 || heads < 1) return;
  const int chunks = (heads + slots - 1) / slots;
  int64_t n = (want + tokens - 1) / tokens;
  if (n > chunks) n = chunks;
  const int each = (chunks + static_cast<int>(n) - 1) / static_cast<int>(n);
  per = each * slots;
  splits = (chunks + each - 1) / each;
}

template <typename T, int D>
cudaError_t launch_qk(const RopeRowArgs& a, cudaStream_t st) {
  RopeRowArgs u = a;
  const int64_t tokens = static_cast<int64_t>(a.B) * a.N;
  split_heads(tokens, a.H[0] + a.H[1], Lane<T, D>::kSlots, u.splits, u.per);
  const int64_t ctas = (tokens * u.splits + kWarps - 1) / kWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned int>(ctas));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kThreads), 0, st, u); };
  if (a.rope.interleaved)
    return a.rope.mixed ? go(k_qk_rope<T, D, true, true>) : go(k_qk_rope<T, D, true, false>);
  return a.rope.mixed ? go(k_qk_rope<T, D, false, true>) : go(k_qk_rope<T, D, false, false>);
}

// From this many tokens (those with keys plus those with queries) on, four CTAs of 64
// registers a thread share an SM, below it three of 80, whose cache rows have more loads
// in flight. 32 and 8 heads of 128, as many queries as keys: 16384 tokens of each take
// 70.1 us with four CTAs and 76.3 with three, 4096 take 19.9 and 21.6, 2048 take 10.7 and
// 11.1, 1024 take 7.1 and 6.5, 512 take 6.3 and 5.1.
constexpr int64_t kAppendMany = 4096;

template <typename T, int D>
cudaError_t launch_append(const RopeAppendArgs& a, cudaStream_t st) {
  RopeAppendArgs u = a;
  split_heads(a.Tq, a.Hq, Lane<T, D>::kSlots, u.q_splits, u.q_per);
  split_heads(a.T, 2 * a.Hkv, 32 / (D / 32), u.kv_splits, u.kv_per);
  const int64_t warps = static_cast<int64_t>(a.Tq) * u.q_splits + static_cast<int64_t>(a.T) * u.kv_splits;
  const int64_t ctas = (warps + kWarps - 1) / kWarps;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorNotSupported;
  const dim3 grid(static_cast<unsigned int>(ctas));
  auto go = [&](auto kern) { return launch_pdl(kern, grid, dim3(kThreads), 0, st, u); };
  const bool many = static_cast<int64_t>(a.T) + a.Tq >= kAppendMany;
  if (a.rope.interleaved) {
    if (a.rope.mixed)
      return many ? go(k_qappend_rope<T, D, true, true, 4>) : go(k_qappend_rope<T, D, true, true, 3>);
    return many ? go(k_qappend_rope<T, D, true, false, 4>) : go(k_qappend_rope<T, D, true, false, 3>);
  }
  if (a.rope.mixed)
    return many ? go(k_qappend_rope<T, D, false, true, 4>) : go(k_qappend_rope<T, D, false, true, 3>);
  return many ? go(k_qappend_rope<T, D, false, false, 4>) : go(k_qappend_rope<T, D, false, false, 3>);
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
  if (head_dim != 64 && head_dim != 128) return KASCADE_ERR_UNSUPPORTED;
  if (rope == nullptr) return KASCADE_OK;
  if (!aligned(rope->table, 16) || rope->n_positions < 1 || rope->n_pairs < 1 ||
      2 * static_cast<int64_t>(rope->n_pairs) > head_dim || rope->n_axes < 1 || rope->n_axes > 4)
    return KASCADE_ERR_INVALID_ARG;
  if (rope->n_pairs % 16 != 0) return KASCADE_ERR_UNSUPPORTED;
  s.table = rope->table;
  s.n_pos = rope->n_positions;
  s.n_pairs = rope->n_pairs;
  s.interleaved = rope->interleaved != 0;
  for (int i = 0; rope->axes != nullptr && i < rope->n_pairs; ++i) {
    if (rope->axes[i] < 0 || rope->axes[i] >= rope->n_axes) return KASCADE_ERR_INVALID_ARG;
    s.axis[i] = static_cast<uint8_t>(rope->axes[i]);
    if (s.axis[i] != s.axis[0]) s.mixed = 1;
  }
  s.quads = 1;
  for (int i = 0; i < rope->n_pairs; ++i) {
    if (s.axis[i] != s.axis[i & ~3]) s.quads = 0;
    s.used |= 1 << s.axis[i];
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
