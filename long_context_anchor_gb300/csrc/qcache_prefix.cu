// qcache_prefix.cu — decode attention of a batch over a prefix that its
// sequences share in the paged 4-bit cache (layout in qcache.h): the keys of the
// prefix for all queries of a KV head together, as a matrix product.
//
// A KV head has B * G queries, G per sequence: rows of tiles of 128. The
// prefix comes in chunks of 64 keys, each turned from 4 bits into fp16 once in
// shared memory for up to two tiles: S = Q K^T and O += P V on tcgen05 with fp16
// operands and fp32 sums. As in the dense kernel a stored element is exact in
// fp16, a row of q is scaled by a power of two (an fp32 q is two fp16 terms), weights
// are 2^kShift p against a reference that is raised to the running maximum when a
// chunk's weights add up to more than fp16 holds, rounded to fp16 (fp32 outputs: two
// terms) for the product and summed unrounded. So the reference moves in a
// part's first chunk and then rarely: raising it for any row of a warp rescales
// 32 rows of O in TMEM, and looking for the maximum costs a fifth of a chunk's
// arithmetic. The weights' fp16 steps are 2^-24, so 2^-28 (bf16) or 2^-32 (fp32) of a
// reference's weight.
//
//   k_qdecode_dense  (qcache_attn.cu) leaves each sequence's state over its own keys
//   k_qprefix        beside it on other SMs: the prefix, a run of chunks per CTA
//   k_qprefix_join   both, and the tables' check
//
// or, where that is not reckoned to help (prefix_geo), the dense call's kernel and
//   k_qprefix_check  the tables' check alone
//
// Measured (bf16, one launch sequence in a graph): 16 sequences x 64 heads over 131072
// keys at d = 64 56.8 us (605 TFLOP/s of the products, 1.4 TB/s of pages), 128 x 32 heads
// over 32768 at d = 128 77.9 us (881 TFLOP/s), 32 x 32 heads over 8192 with 1024 own keys
// each 25.5 us; one by one, as the dense call does it, 218, 810 and 66.5 us. A chunk takes
// an SM 740 cycles at d = 64, two tiles of one 1700 at d = 128. What bounds it is a chunk's
// way round with two score buffers: 1500 cycles of softmax (830 of arithmetic beside the
// other warps', 400 of a TMEM load) and as many from the weights to the next scores in
// their place (product, its wait, scores, five waits of 100 cycles); the issue slots are
// 50 to 60% full, tensor cores busy 30% (d = 64) and 50% (d = 128, where the scores read Q
// from shared memory, as TMEM is full). About 6 us of a launch are its start (4: lengths,
// queries, first chunk) and end. Slower, 16 x 131072 keys and 128 x 32768: against 57.8 and
// 86.8 us, when those were the times, two warps per 32 rows with half of the keys each (61.5,
// 91), the next chunk's load begun before this one's end (63, 91), scores and products issued
// by warps of their own (65, 103), one arrival per warp for the weights (58.7, 87.9); against
// 56.8 and 77.9, queries loaded before the barriers are set up (59.6, 81).
// fp32 queries have two terms, and so have their weights: twice the products, a tile per CTA.
// 128 x 8192 keys, 32 heads, d = 128 64.8 us (bf16 41), 16 x 131072, 64 heads, d = 64 77.6
// (57), 32 x 8192 with 1024 own keys each 34.6 (25.5); one by one 278, 285 and 84.
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

#include "common.cuh"
#include "qcache.h"
#include "qmath.cuh"
#include "qprefix.cuh"
#include "tc.cuh"

namespace kascade {
namespace {

// Weights are 2^kShift p. Larger ones of a wide spread raise the reference less often
// with a small shift (bf16: 12 bits of room), and small ones keep more bits with a
// large one (fp32).
template <int TERMS>
constexpr float kShift = TERMS == 2 ? 8.f : 4.f;

// Two streams, each with its scores, its running state and its O, run through
// the same code: a unit of two row tiles gives each stream one of them and every
// chunk; a unit of one tile gives both streams that tile and every other chunk
// (their states are two pieces of the same rows). While one stream's softmax
// runs, the tensor cores work for the other.
//
// Roles: warps 4s .. 4s+3 are stream s's softmax, a thread per row; then
// kDeqWarps warps that turn codes into fp16; a warp per stream that issues its
// MMAs; one that copies the blocks in.
// The widening warps work in teams, each on chunks of its own: a chunk costs a
// warp two waits and two arrivals whatever its share of it (all eight warps on every
// chunk: 1130 cycles a chunk at d = 64, half of them work).
constexpr int kDeqWarps = 8;
template <int D>
constexpr int kTeamWarps = D == 128 ? 4 : 2;
constexpr int kMmaWarp = 8 + kDeqWarps, kLoadWarp = kMmaWarp + 2;
constexpr int kThreads = 32 * (kLoadWarp + 2);   // a whole number of warpgroups
// Registers: 640 threads are launched with 96 each; the warpgroups give back what
// they do not need before the softmax takes more.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 136, kDeqRegs = 64, kIssueRegs = 80;
static_assert(kThreads == 640 && 256 * kSoftmaxRegs + 256 * kDeqRegs + 128 * kIssueRegs <=
                                     kThreads * kLaunchRegs, "shares of what was launched");
template <int N>
__device__ __forceinline__ void more_regs() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_regs() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// mbar_wait_warp with the test that usually succeeds in front.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, unsigned int* err,
                                          unsigned int where) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || mbar_wait_warp(bar, parity, err, where);
}

template <int D, int TERMS>
struct Shapes {
  // TMEM columns, 512 in all: O of each stream, two buffers of scores for each (a
  // chunk's weights, both terms for fp32, lie over its scores: the next chunk's scores
  // go into the other buffer meanwhile), and at d = 64 Q (fp16 pairs; a tile per
  // stream, or the two terms of one tile). At d = 128 Q is in shared memory.
  static constexpr bool QSMEM = D == 128;
  static constexpr int Q_COLS = QSMEM ? 0 : 32;
  static constexpr int S0 = 2 * Q_COLS, O0 = S0 + 256, O_COLS = D;
  static_assert(O0 + 2 * O_COLS <= 512, "TMEM columns");

  static constexpr int HALF = kPfxKeys * 128;           // 64 dims of a chunk's K or V in fp16
  static constexpr int TILE = HALF * (D / 64);          // a chunk's K, or its V
  // Rings: K in fp16 (a stage is free once its scores are in), V in fp16, chunks as
  // stored. A stage is always the same team's and, where each stream has its own
  // chunks, the same stream's: who waits for a phase of its barriers has seen the
  // phase before.
  static constexpr int KST = D == 128 ? 2 : 8, VST = D == 128 ? 4 : 8, NR = D == 128 ? 6 : 12;
  static constexpr int kTeams = kDeqWarps / kTeamWarps<D>;
  static_assert(KST % kTeams == 0 && VST % kTeams == 0 && NR % kTeams == 0 && kTeams % 2 == 0,
                "stages belong to one team and one stream");
  // what the softmax reads of chunk k is written with its K: by then the scores of
  // chunk k - KST are in, and so the softmax of the chunk 16 before is done
  static constexpr int kValid = 16;
  static_assert(KST + 6 <= kValid, "two scores of a stream, every other chunk, behind K's ring");
  static constexpr int RAW = (kPfxKeys / kQGroup) * qgroup_bytes(D);
  static constexpr int Q_TILE = kPfxRows * 2 * D;   // d = 64: on its way to TMEM
  static constexpr int V0 = KST * TILE, QS = V0 + VST * TILE;
  static constexpr int RAW0 = QS + 2 * Q_TILE;
  static constexpr int BAR = RAW0 + NR * RAW;
  static constexpr int NBAR = 2 * (NR + KST + VST) + 14;
  static constexpr int VALID = BAR + NBAR * 8;          // int [NR + kValid]: bit per 16 keys
  static constexpr int TMEM = VALID + (NR + kValid) * 4;
  static constexpr int BYTES = TMEM + 8;
  static constexpr size_t SMEM = BYTES + 1024;          // slack for 1024-byte alignment
  static_assert(SMEM <= 232448 - 64, "fits in shared memory");
};

// Matrix descriptors: of a chunk's K (16 dims of 64 keys a step), V (16 keys of
// all dims a step) and the upper half of a Q tile; a step adds to the address.
__device__ __forceinline__ uint64_t kq_desc(uint32_t tile) { return sw128_desc(tile, 16, 1024); }
__device__ __forceinline__ uint64_t v_desc(uint32_t tile) {
  return sw128_desc(tile, kPfxKeys * 128, 1024);
}
__device__ __forceinline__ constexpr uint64_t k_step(int kk) {
  return static_cast<uint64_t>(((kk >> 2) * (kPfxKeys * 128) + (kk & 3) * 32) >> 4);
}
__device__ __forceinline__ constexpr uint64_t q_step(int kk) {
  return static_cast<uint64_t>(((kk >> 2) * (kPfxRows * 128) + (kk & 3) * 32) >> 4);
}
__device__ __forceinline__ constexpr uint64_t v_step(int kk) {
  return static_cast<uint64_t>((kk * 2048) >> 4);
}
// fp16 x fp16 -> fp32
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N, int b_mn_major) {
  return (1u << 4) | (static_cast<uint32_t>(b_mn_major) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// What a CTA does: chunks c0 .. c1 - 1 of one unit, for one or two row tiles.
struct Part {
  int g, tile0, tiles, c0, c1;
  // With one tile stream s has the chunks whose number in the run is even (s = 0) or odd.
  __device__ __forceinline__ int chunks(int stream) const {   // of one stream
    return tiles == 2 ? c1 - c0 : (c1 - c0 - stream + 1) / 2;
  }
  __device__ __forceinline__ uint32_t chunk(int stream, int t) const {   // its t-th
    return tiles == 2 ? t : 2 * t + stream;
  }
};
__device__ __forceinline__ Part part_of(const QPrefixGeo& geo, int Hkv, int cta) {
  Part p;
  const int base = Hkv * geo.pairs * geo.pair_runs;
  int run, len;
  if (cta < base) {
    const int unit = cta / geo.pair_runs;
    run = cta - unit * geo.pair_runs;
    len = geo.pair_len;
    p.g = unit / geo.pairs;
    p.tile0 = 2 * (unit - p.g * geo.pairs);
    p.tiles = 2;
  } else {
    const int unit = (cta - base) / geo.single_runs;
    run = cta - base - unit * geo.single_runs;
    len = geo.single_len;
    p.g = unit / geo.singles;
    p.tile0 = 2 * geo.pairs + unit - p.g * geo.singles;
    p.tiles = 1;
  }
  p.c0 = min(geo.nch, run * len);
  p.c1 = min(geo.nch, p.c0 + len);
  return p;
}

// A widening thread's 32 elements of a row: 16 bytes of codes and two scales become
// four 16-byte pieces of the swizzled tile. The rows a thread takes are a multiple
// of 8 apart, so its places in a row are the same in all of them. At d = 128 the
// pieces of parts 2 and 3 go in another order (their second half first): eight lanes
// with two rows of four parts each then store to all banks.
template <int D>
struct Widen {
  static constexpr int kParts = D / 32;
  int codes[2], scales;         // of the first row: its two halves in the order they go, its scales
  uint32_t to[4];               // places of the pieces
  uint32_t pick[2];             // which scale the halves have
  __device__ __forceinline__ Widen(int row, int part) {
    const int flip = D == 128 ? part & 2 : 0, r = row & 15;
    codes[0] = (row >> 4) * qgroup_bytes(D) + r * (D / 2) + part * 16 + (flip ? 8 : 0);
    codes[1] = (row >> 4) * qgroup_bytes(D) + r * (D / 2) + part * 16 + (flip ? 0 : 8);
    scales = (row >> 4) * qgroup_bytes(D) + r * (D / 16) + part * 2;
    pick[0] = flip ? 0x3232u : 0x1010u;
    pick[1] = flip ? 0x1010u : 0x3232u;
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = sw128_offset(kPfxKeys, row, 4 * part + (i ^ flip));
  }
  // The row `rows` (a constant) behind the first; raw: K's codes of the chunk, or V's.
  template <int ROWS>
  __device__ __forceinline__ void row(const uint8_t* raw, uint32_t tile, bool valid) const {
    static_assert(ROWS % 16 == 0, "whole groups");
    const uint8_t* p = raw + (ROWS / 16) * qgroup_bytes(D);
    uint2 half[2] = {};
    uint32_t h = 0u;
    if (valid) {   // what lies there otherwise may be anything
      half[0] = *reinterpret_cast<const uint2*>(p + codes[0]);
      half[1] = *reinterpret_cast<const uint2*>(p + codes[1]);
      h = cvt_e4m3x2(*reinterpret_cast<const uint16_t*>(p + 8 * D + scales));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t s = __byte_perm(h, h, pick[i >> 1]);
      uint32_t x[4];
      cvt_e2m1x8((i & 1) ? half[i >> 1].y : half[i >> 1].x, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = hmul2(x[j], s);
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(tile + to[i] + ROWS * 128),
                   "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                   : "memory");
    }
  }
};

// A query row's largest element is scaled to [2^kQExp, 2^(kQExp + 1)), one below 2^-100 as if it
// were that. Zero and infinity are left.
__device__ __forceinline__ int q_exponent(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;   // denormals: -127
  return amax > 0.f && e < 128 ? max(e, -100) : kQExp;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// The lowest sequence that holds the whole prefix, whose table names its blocks, into
// src (a.B before; shared memory; all threads).
__device__ __forceinline__ void first_holder(const QPrefixArgs& a, int& src) {
  for (int b = threadIdx.x; b < a.B; b += blockDim.x)
    if (pfx_start(a.lens, b, a.P, a.N, a.max_blocks, a.bs_shift) > 0) {
      atomicMin(&src, b);
      break;
    }
  __syncthreads();
}

// The float4 e4 of row r in a piece: eight rows side by side, so that both the rows'
// threads and the join's fill whole lines (a row after the other, the stores of a
// piece took 5 us).
template <int D>
__device__ __forceinline__ int pfx_piece_at(int r, int e4) { return ((r >> 3) * (D / 4) + e4) * 8 + (r & 7); }

template <int D, int TERMS>
__global__ void __launch_bounds__(kThreads, 1) k_qprefix(const __grid_constant__ QPrefixArgs a) {
  using SM = Shapes<D, TERMS>;
  constexpr int KST = SM::KST, VST = SM::VST, NR = SM::NR;
  // The kernel before this one is the own parts' (launch_qdecode_dense), of which
  // nothing is used here: a CTA starts where one of its CTAs has ended. All of those
  // had waited for what came before them by then; the end of the kernel is waited
  // for at this one's end, for the sake of the kernel behind it.
  pdl_trigger();
  extern __shared__ unsigned char smem_raw[];
  __shared__ int s_src;
  unsigned char* sm = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SM::BAR);
  uint64_t* raw_full = bars;            // [NR] a chunk's copies have landed
  uint64_t* raw_free = bars + NR;       // [NR] ... and were read
  uint64_t* k_free = bars + 2 * NR;     // [KST] a chunk's K was used by both streams
  uint64_t* k_ready = k_free + KST;     // [KST] K widened
  uint64_t* v_free = k_ready + KST;     // [VST] the same for V
  uint64_t* v_ready = v_free + VST;
  uint64_t* q_ready = v_ready + VST;    // [2] by stream: Q written
  // by stream and buffer (2 * stream + buffer):
  uint64_t* s_full = q_ready + 2;       // [4] scores of a chunk
  uint64_t* p_full = q_ready + 6;       // [4] its weights written
  uint64_t* pv_done = q_ready + 10;     // [4] their product with V
  int* raw_valid = reinterpret_cast<int*>(sm + SM::VALID);
  int* kv_valid = raw_valid + NR;
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(sm + SM::TMEM);

  const Part p = part_of(a.geo, a.Hkv, static_cast<int>(blockIdx.x));
  // a softmax thread's row of the KV head's queries, and whether it takes part
  const int gr = (p.tile0 + (p.tiles == 2 ? (tid >> 7) & 1 : 0)) * 128 + (tid & 127);
  const bool live = tid < 256 && gr < a.B * a.G &&
                    pfx_start(a.lens, gr / a.G, a.P, a.N, a.max_blocks, a.bs_shift) > 0;
  if (tid == 0) s_src = a.B;
  if (tid < SM::NBAR) {
    const int i = tid, j = i - 2 * NR, l = j - 2 * KST, k = l - 2 * VST;   // k: from q_ready on
    const int count = i < NR ? 1 : i < 2 * NR ? kTeamWarps<D>
                      : j < KST ? 2 : j < 2 * KST ? kTeamWarps<D>   // both streams, or one twice
                      : l < VST ? 2 : l < 2 * VST ? kTeamWarps<D>
                      : k < 2 ? 128 : k < 6 ? 1 : k < 10 ? 128 : 1;
    mbar_init(bars + i, count);
    fence_barrier_init();
  }
  if (warp == kMmaWarp) tmem_alloc(s_tmem, 512);   // one CTA per SM
  tc_fence_before();
  __syncthreads();
  first_holder(a, s_src);
  tc_fence_after();
  const uint32_t tmem = warp_uniform(*s_tmem);
  const int src = s_src;
  if (src >= a.B) {   // nobody has it: no piece is read either
    if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
    if (tid == 0) pdl_wait();
    return;
  }
  const int32_t* ids = a.table + static_cast<size_t>(src) * a.max_blocks;

  if (warp >= kMmaWarp) {
    fewer_regs<kIssueRegs>();
    if (warp == kLoadWarp) {
      // ------------------------------------------------------------- copies
      // kAhead chunks at a time, four lanes each: one chunk at a time took 1050 cycles
      constexpr int kAhead = D == 128 ? 2 : 4;
      const int copy_sh = min(a.bs_shift, 6), ncopy = kPfxKeys >> copy_sh;   // copies of a chunk
      const uint32_t copy_bytes = static_cast<uint32_t>(qgroup_bytes(D)) << (copy_sh - 4);
      const uint32_t head_bytes = static_cast<uint32_t>(qgroup_bytes(D)) << (a.bs_shift - 4);
      const uint64_t block_bytes = static_cast<uint64_t>(head_bytes) * a.Hkv;
      const int gmask = (1 << (a.bs_shift - 4)) - 1;
      const unsigned int groups = (1u << (1 << (copy_sh - 4))) - 1u;   // a copy's bits
      const int sub = lane >> 2, cp = lane & 3;
      const uint8_t* head = a.cache + static_cast<size_t>(p.g) * head_bytes;
      // this lane's copy of chunks c + sub; ids are loaded a turn ahead
      auto key_of = [&](int c) { return (c + sub) * kPfxKeys + (cp << copy_sh); };
      auto wanted = [&](int c) {
        return sub < kAhead && cp < ncopy && c + sub < p.c1 && key_of(c) < a.P;
      };
      auto fetch = [&](int c) { return wanted(c) ? __ldg(ids + (key_of(c) >> a.bs_shift)) : 0; };
      int next = fetch(p.c0);
      uint32_t issued = 0;
      for (int c = p.c0; c < p.c1; c += kAhead) {
        const int id = next, key = key_of(c);
        next = fetch(c + kAhead);
        const bool here = sub < kAhead && c + sub < p.c1, want = wanted(c);
        const bool take = want && static_cast<unsigned int>(id) < static_cast<unsigned int>(a.num_blocks);
        if (want && !take) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x552);
        const unsigned int got = (__ballot_sync(0xffffffffu, take) >> (lane & 28)) & 0xfu;
        const uint32_t k = c - p.c0 + sub, st = k % NR;
        if (!__all_sync(0xffffffffu,
                        !here || mbar_wait(raw_free + st, ((k / NR) & 1) ^ 1, a.err, 0x561)))
          break;
        if (here && cp == 0) {
          unsigned int bits = 0u;
  #pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((got >> i) & 1u) bits |= groups << (i << (copy_sh - 4));
          raw_valid[st] = static_cast<int>(bits);
          mbar_arrive_expect_tx(raw_full + st, __popc(got) * copy_bytes);
        }
        __syncwarp();
        if (take)
          bulk_load(sm + SM::RAW0 + st * SM::RAW + cp * copy_bytes,
                    head + static_cast<uint64_t>(id) * block_bytes +
                        static_cast<uint32_t>((key >> 4) & gmask) * qgroup_bytes(D),
                    copy_bytes, raw_full + st);
        issued += min(kAhead, p.c1 - c);
      }
      // leave no copy in flight
      for (uint32_t k = issued > NR ? issued - NR : 0; k < issued; ++k)
        mbar_wait(raw_full + k % NR, (k / NR) & 1, a.err, 0x562);
    } else if (warp < kLoadWarp) {
      // --------------------------------------------------------- tensor cores
      constexpr uint32_t idq = idesc_f16_f32(128, kPfxKeys, 0), idv = idesc_f16_f32(128, D, 1);
      const int s = static_cast<int>(warp_uniform(static_cast<uint32_t>(warp - kMmaWarp)));
      const uint32_t kv0 = smem_u32(sm);
      const uint32_t q0 = smem_u32(sm + SM::QS);
      const uint32_t tS0 = tmem + SM::S0 + 128 * s, tO = tmem + SM::O0 + SM::O_COLS * s;
      const int n = p.chunks(s);
      // S = Q K^T of the stream's t-th chunk
      auto issue_s = [&](int t) {
        const uint32_t k = p.chunk(s, t), ks = k % KST, buf = t & 1;
        if (!wait_warp(k_ready + ks, (k / KST) & 1, a.err, 0x571)) return false;
        tc_fence_after();
        const uint64_t kd = warp_uniform(kq_desc(kv0 + ks * SM::TILE));
        const uint32_t tS = tS0 + 64 * buf;
  #pragma unroll
        for (int term = 0; term < TERMS; ++term) {
          const int tile = TERMS == 2 ? term : s;
          const uint64_t qd = warp_uniform(kq_desc(q0 + tile * SM::Q_TILE));
  #pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t acc = term > 0 || kk > 0 ? 1u : 0u;
            if (SM::QSMEM)
              tc_mma(tS, qd + q_step(kk), kd + k_step(kk), idq, acc);
            else
              tc_mma_ts(tS, tmem + SM::Q_COLS * tile + kk * 8, kd + k_step(kk), idq, acc);
          }
        }
        tc_commit(s_full + 2 * s + buf);
        tc_commit(k_free + ks);
        if (p.tiles == 1) tc_commit(k_free + ks);   // for the stream that does not use it
        return true;
      };
      // O += P V; the first product overwrites O
      auto issue_pv = [&](int t) {
        const uint32_t k = p.chunk(s, t), st = k % VST, buf = t & 1;
        if (!wait_warp(v_ready + st, (k / VST) & 1, a.err, 0x576) ||
            !wait_warp(p_full + 2 * s + buf, (t >> 1) & 1, a.err, 0x572))
          return false;
        tc_fence_after();
        const uint64_t vd = warp_uniform(v_desc(kv0 + SM::V0 + st * SM::TILE));
        const uint32_t tP = tS0 + 64 * buf;
  #pragma unroll
        for (int term = 0; term < TERMS; ++term)
  #pragma unroll
          for (int kk = 0; kk < kPfxKeys / 16; ++kk)
            tc_mma_ts(tO, tP + 32 * term + kk * 8, vd + v_step(kk), idv,
                      t > 0 || term > 0 || kk > 0 ? 1u : 0u);
        tc_commit(pv_done + 2 * s + buf);
        tc_commit(v_free + st);
        if (p.tiles == 1) tc_commit(v_free + st);
        return true;
      };
      bool ok = wait_warp(q_ready + s, 0, a.err, 0x573);
      if (TERMS == 2 && ok) ok = wait_warp(q_ready + 1 - s, 0, a.err, 0x573);
      tc_fence_after();
      for (int t = 0; ok && t < n && t < 2; ++t) ok = issue_s(t);
      for (int t = 0; ok && t < n; ++t) {
        ok = issue_pv(t);
        if (ok && t + 2 < n)   // over this chunk's weights
          ok = wait_warp(pv_done + 2 * s + (t & 1), (t >> 1) & 1, a.err, 0x574) && issue_s(t + 2);
      }
    }
  } else if (warp >= 8) {
    fewer_regs<kDeqRegs>();
    // ------------------------------------------------------- codes to fp16
    constexpr int kTeam = kTeamWarps<D>, kTeams = SM::kTeams, kParts = Widen<D>::kParts;
    constexpr int kRows = 32 * kTeam / kParts;   // rows of K (and V) at a time
    static_assert(kRows == 32 && kPfxKeys == 64, "two rows per thread, whole groups apart");
    const int team = (warp - 8) / kTeam, t = tid - 256 - team * 32 * kTeam;
    const Widen<D> w(t / kParts, t % kParts);
    const int group0 = t / kParts / 16;
    for (int k = team; k < p.c1 - p.c0; k += kTeams) {
      const int rs = k % NR, st = k % VST, ks = k % KST;
      if (!wait_warp(raw_full + rs, (k / NR) & 1, a.err, 0x581) ||
          !wait_warp(k_free + ks, ((k / KST) & 1) ^ 1, a.err, 0x582))
        break;
      const int bits = raw_valid[rs];
      const uint8_t* raw = sm + SM::RAW0 + rs * SM::RAW;
      auto both_rows = [&](int at, uint32_t tile) {
        if (bits == 0xf) {
          w.template row<0>(raw + at, tile, true);
          w.template row<32>(raw + at, tile, true);
        } else {
          w.template row<0>(raw + at, tile, (bits >> group0) & 1);
          w.template row<32>(raw + at, tile, (bits >> (group0 + 2)) & 1);
        }
        fence_proxy_async_smem();
        __syncwarp();
      };
      both_rows(0, smem_u32(sm) + ks * SM::TILE);
      if (t == 0) kv_valid[k % SM::kValid] = bits;
      __syncwarp();
      if (lane == 0) mbar_arrive(k_ready + ks);
      if (!wait_warp(v_free + st, ((k / VST) & 1) ^ 1, a.err, 0x583)) break;
      both_rows(9 * D, smem_u32(sm) + SM::V0 + st * SM::TILE);
      if (lane == 0) {
        mbar_arrive(v_ready + st);
        mbar_arrive(raw_free + rs);
      }
    }
  } else {
    more_regs<kSoftmaxRegs>();
    // ------------------------------------------------------------- softmax
    const int s = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS0 = tmem + SM::S0 + 128 * s + lane_base;
    const uint32_t tO = tmem + SM::O0 + SM::O_COLS * s + lane_base;
    const uint32_t sQ = smem_u32(sm + SM::QS) + s * SM::Q_TILE;
    bool ok = true;
    const uint32_t alive = __ballot_sync(0xffffffffu, live);
    const bool idle = alive == 0u;
    // ---- these 32 rows of Q: neighbouring lanes load neighbouring pieces (a row per
    // thread, as the softmax has them, took 3 us of loads of 32 lines each), scale them
    // and put them into the tile
    constexpr int kPerRow = D * (TERMS == 2 ? 4 : 2) / 16, kRowsAt = 32 / kPerRow;   // lanes per row
    constexpr int kLoads = 32 / kRowsAt, kBatch = kLoads < 16 ? kLoads : 16;
    const int piece = lane % kPerRow;
    const int q_row = live ? (gr / a.G) * a.Hq + a.heads[p.g * a.G + gr % a.G] : 0;   // of row r
    float amax = 0.f;                                                                // of row r
#pragma unroll
    for (int i0 = 0; i0 < kLoads; i0 += kBatch) {
      uint4 raw[kBatch];
      float m[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int j = (i0 + i) * kRowsAt + lane / kPerRow;
        const int from = __shfl_sync(0xffffffffu, q_row, j);
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if ((alive >> j) & 1u)
          raw[i] = __ldg(reinterpret_cast<const uint4*>(a.q) + static_cast<size_t>(from) * kPerRow + piece);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        m[i] = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (TERMS == 2) {
            m[i] = fmaxf(m[i], fabsf(__uint_as_float(w[j])));
          } else {
            m[i] = fmaxf(m[i], fabsf(__uint_as_float(w[j] << 16)));
            m[i] = fmaxf(m[i], fabsf(__uint_as_float(w[j] & 0xffff0000u)));
          }
        }
      }
#pragma unroll
      for (int off = 1; off < kPerRow; off <<= 1)   // all rows' steps in flight together
#pragma unroll
        for (int i = 0; i < kBatch; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float own = __shfl_sync(0xffffffffu, m[i], (lane % kRowsAt) * kPerRow);
        if (lane / kRowsAt == i0 + i) amax = own;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        const float up = pow2(kQExp - q_exponent(m[i]));
        const int to = (warp & 3) * 32 + (i0 + i) * kRowsAt + lane / kPerRow;
        if (TERMS == 2) {
          uint32_t x[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float lo = __uint_as_float(w[2 * j]) * up, hi = __uint_as_float(w[2 * j + 1]) * up;
            if (s == 1) {
              lo -= f16_rounded(lo);
              hi -= f16_rounded(hi);
            }
            x[j] = pack_f16(lo, hi);
          }
          asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(
                           sQ + sw128_offset(kPfxRows, to, piece >> 1) + 8 * (piece & 1)),
                       "r"(x[0]), "r"(x[1])
                       : "memory");
        } else {
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[j] = pack_f16(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
          asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(sQ + sw128_offset(kPfxRows, to, piece)),
                       "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3])
                       : "memory");
        }
      }
    }
    const float ml = fmaxf(a.scale * pow2(q_exponent(amax) - kQExp), 1e-37f) * kLog2e;
    if constexpr (SM::QSMEM) {
      fence_proxy_async_smem();
    } else {   // a row per thread from here on
      __syncwarp();
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                     : "r"(sQ + sw128_offset(kPfxRows, r, i))
                     : "memory");
      tmem_st32(tmem + SM::Q_COLS * s + lane_base, w);
      tmem_wait_st();
    }
    tc_fence_before();
    mbar_arrive(q_ready + s);
    // ---- its chunks
    // weights are 2^(product * ml + c), c = kShift - ref * ml: the reference is a raw
    // product. c's rounding is common to a row's weights; where it would be felt, or
    // would overflow them, `careful` chunks have the reference taken off their products
    // first (c = kShift then).
    float ref = kNoKey, l = 0.f, c = 0.f;
    bool careful = false;
    const int n = p.chunks(s);
    for (int t = 0; ok && t < n; ++t) {
      const uint32_t buf = t & 1, tS = tS0 + 64 * buf;
      ok = wait_warp(s_full + 2 * s + buf, (t >> 1) & 1, a.err, 0x591);
      if (!ok) break;
      tc_fence_after();
      if (!idle) {
        // (written before k_ready, which the MMAs waited for)
        const int bits = kv_valid[p.chunk(s, t) % SM::kValid];
        if (bits != 0xf) {   // rare: the products of keys that do not count
          uint32_t none[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) none[i] = __float_as_uint(kNegInf);
#pragma unroll 1
          for (int i = 0; i < 4; ++i)
            if (!((bits >> i) & 1)) tmem_st16(tS + 16 * i, none);
          tmem_wait_st();
        }
        // A chunk's weights are taken with the reference as it is; only where their sum
        // shows that one may have passed fp16 the reference goes up to the chunk's
        // largest product (all lanes), and the weights are taken again. The weights lie
        // over the products, so they are kept until then.
        uint32_t hi[32], lo[TERMS == 2 ? 32 : 1];
        float sum;
        for (bool raise = t == 0 || careful;; raise = true) {
          if (raise) {
            float up_to = ref;
#pragma unroll 1
            for (int cc = 0; cc < 64; cc += 32) {
              uint32_t v[32];
              tmem_ld32(tS + cc, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 2)
                up_to = fmax3(up_to, __uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            }
            const float al = ex2((ref - up_to) * ml);
            const bool moved = __any_sync(0xffffffffu, up_to > ref);
            ref = up_to;
            l *= al;
            if (moved && t > 0) {
              const int before = t - 1;   // O is still once its product is in
              ok = wait_warp(pv_done + 2 * s + (before & 1), (before >> 1) & 1, a.err, 0x593);
              if (!ok) break;
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < D; cc += 16) {
                uint32_t o[16];
                tmem_ld16(tO + cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * al);
                tmem_st16(tO + cc, o);
              }
            }
            c = fmaf(-ref, ml, kShift<TERMS>);
            careful = __any_sync(0xffffffffu, !(fabsf(c) < 1024.f));
            if (careful) {
              c = kShift<TERMS>;
#pragma unroll 1
              for (int cc = 0; cc < 64; cc += 16) {
                uint32_t v[16];
                tmem_ld16(tS + cc, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) - ref);
                tmem_st16(tS + cc, v);
              }
            }
            tmem_wait_st();
          }
          uint32_t v[2][32];
          tmem_ld32(tS, v[0]);
          tmem_ld32(tS + 32, v[1]);
          tmem_wait_ld();
          const uint64_t ml2 = f2_pack(ml, ml), c2 = f2_pack(c, c);
          uint64_t part_sum[2] = {0ull, 0ull};
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint32_t(&x)[32] = v[i >> 4];
            const int at = 2 * (i & 15);
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[at]), __uint_as_float(x[at + 1])), ml2, c2), p0, p1);
            p0 = ex2(p0);
            p1 = ex2(p1);
            part_sum[i & 1] = f2_add(part_sum[i & 1], f2_pack(p0, p1));
            hi[i] = pack_f16(p0, p1);
            if (TERMS == 2) lo[i] = pack_f16(p0 - f16_rounded(p0), p1 - f16_rounded(p1));
          }
          float s0, s1;
          f2_unpack(f2_add(part_sum[0], part_sum[1]), s0, s1);
          sum = s0 + s1;
          if (raise || !__any_sync(0xffffffffu, !(sum < 65000.f))) break;
        }
        if (!ok) break;
        tmem_st32(tS, hi);
        if constexpr (TERMS == 2) tmem_st32(tS + 32, lo);
        l += sum;
        tmem_wait_st();
      }
      tc_fence_before();
      mbar_arrive(p_full + 2 * s + buf);
    }
    // ---- the piece
    if (ok && n > 0) {
      ok = wait_warp(pv_done + 2 * s + ((n - 1) & 1), ((n - 1) >> 1) & 1, a.err, 0x594);
    }
    tc_fence_after();
    if (!idle) {
      float* piece = a.part + pfx_piece_floats(D) * (2 * static_cast<size_t>(blockIdx.x) + s);
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t o[32];
        tmem_ld32(tO + 32 * cc, o);
        tmem_wait_ld();
        float4* dst = reinterpret_cast<float4*>(piece) + pfx_piece_at<D>(r, 8 * cc);
        if (live)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[8 * i] = n > 0 ? make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                         __uint_as_float(o[4 * i + 2]),
                                         __uint_as_float(o[4 * i + 3]))
                           : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (live) {
        // (as the reference of weights held as 2^14 p)
        piece[kPfxRows * D + r] = ref == kNoKey ? kNoKey
                                  : careful ? ref * ml + (kPShift - kShift<TERMS>) : kPShift - c;
        piece[kPfxRows * (D + 1) + r] = l;
      }
    }
    tc_fence_before();
  }
  if (warp == kLoadWarp) pdl_wait();
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

constexpr int kJoinThreads = 256;

// Sequences whose tables name other blocks than the lowest one's; this CTA's share of
// `ctas`: a warp has kCheck entries of one sequence at a time (all threads).
constexpr int kCheck = 256;
__device__ __forceinline__ void check_tables(const QPrefixArgs& a, int& s_src, int cta, int ctas) {
  if (threadIdx.x == 0) s_src = a.B;
  __syncthreads();
  first_holder(a, s_src);
  const int src = s_src, front = a.P >> a.bs_shift, pieces = (front + kCheck - 1) / kCheck;
  const int32_t* ids = a.table + static_cast<size_t>(src) * a.max_blocks;
  const int64_t units = static_cast<int64_t>(a.B - src - 1) * pieces;   // none: -1
  for (int64_t u = static_cast<int64_t>(cta) * (kJoinThreads / 32) + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(ctas) * (kJoinThreads / 32)) {
    const int b = src + 1 + static_cast<int>(u / pieces), j0 = static_cast<int>(u % pieces) * kCheck;
    if (pfx_start(a.lens, b, a.P, a.N, a.max_blocks, a.bs_shift) == 0) continue;
    bool other = false;
#pragma unroll
    for (int i = 0; i < kCheck; i += 32) {
      const int j = j0 + i + static_cast<int>(threadIdx.x & 31);
      if (j < front) other |= a.table[static_cast<size_t>(b) * a.max_blocks + j] != ids[j];
    }
    if (other) report_error(a.err, KASCADE_ERR_BAD_INPUT, 0x551);
  }
}

// The check alone, beside the dense call's kernel (what it reads that kernel has waited
// for; its end is waited for here for the sake of what comes behind).
__global__ void __launch_bounds__(kJoinThreads) k_qprefix_check(const __grid_constant__ QPrefixArgs a) {
  __shared__ int s_src;
  pdl_trigger();
  check_tables(a, s_src, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
  pdl_wait();
}

// Every row's pieces and its own part's state joined into the output: a thread has four
// dims of a row, or every WORKERS-th of its pieces, which are then joined in order. A CTA has
// kRows rows of a KV head and kLanes of their float4s (kParts CTAs have a row); those behind the
// last head check the tables.
template <int D, int WORKERS>
struct JoinShape {
  static constexpr int kLanes = WORKERS * (D / 4) > 32 ? 32 / WORKERS : D / 4;
  static constexpr int kRows = kJoinThreads / (kLanes * WORKERS), kParts = D / 4 / kLanes;
};

template <int D, bool F32, int WORKERS>
__global__ void __launch_bounds__(kJoinThreads) k_qprefix_join(const __grid_constant__ QPrefixArgs a) {
  pdl_wait();
  pdl_trigger();
  using J = JoinShape<D, WORKERS>;
  constexpr int kBatch = 8;
  __shared__ Joined scratch[kJoinThreads];
  __shared__ int s_src;
  const int g = static_cast<int>(blockIdx.y);
  if (g == a.Hkv) {
    check_tables(a, s_src, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x));
    return;
  }
  // neighbouring lanes have neighbouring rows, which lie side by side in a piece
  const int e4 = static_cast<int>(blockIdx.x) % J::kParts * J::kLanes + threadIdx.x / J::kRows % J::kLanes;
  const int worker = threadIdx.x / (J::kRows * J::kLanes);
  const int kv_row = static_cast<int>(blockIdx.x) / J::kParts * J::kRows + threadIdx.x % J::kRows;
  const int b = kv_row >> (31 - __clz(a.G)), slot = kv_row & (a.G - 1);   // G: a power of two
  const bool here = b < a.B;
  Joined x = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (here && worker == 0) {
    const int64_t at = (static_cast<int64_t>(b) * a.Hkv + g) * a.G + slot;
    const float2 ml = __ldcg(a.own_ml + at);
    x = {ml.x, ml.y, __ldcg(a.own_o + at * (D / 4) + e4)};
  }
  if (here && pfx_start(a.lens, b, a.P, a.N, a.max_blocks, a.bs_shift) > 0) {
    const QPrefixGeo& geo = a.geo;
    const int tile = kv_row / kPfxRows, r = kv_row % kPfxRows;
    const bool pair = tile < 2 * geo.pairs;
    const int cta = pair ? (g * geo.pairs + tile / 2) * geo.pair_runs
                         : a.Hkv * geo.pairs * geo.pair_runs +
                               (g * geo.singles + tile - 2 * geo.pairs) * geo.single_runs;
    // pair: the tile's piece of every CTA; else both pieces of each
    const int n = pair ? geo.pair_runs : 2 * geo.single_runs;
    const size_t stride = (pair ? 2 : 1) * pfx_piece_floats(D);
    const float* p = a.part + pfx_piece_floats(D) * (2 * static_cast<size_t>(cta) +
                                                     (pair ? tile & 1 : 0));
    for (int s = worker; s < n; s += kBatch * WORKERS) {
      Joined y[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        y[k] = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        if (s + k * WORKERS < n) {
          const float* at = p + (s + k * WORKERS) * stride;
          y[k].m = __ldcg(at + kPfxRows * D + r);
          y[k].l = __ldcg(at + kPfxRows * (D + 1) + r);
          y[k].o = __ldcg(reinterpret_cast<const float4*>(at) + pfx_piece_at<D>(r, e4));
        }
      }
      join_into(x, y);
    }
  }
  if (WORKERS > 1) {
    scratch[threadIdx.x] = x;
    __syncthreads();
    if (worker > 0) return;
    for (int w = 1; w < WORKERS; ++w) {
      const Joined y[1] = {scratch[threadIdx.x + w * J::kRows * J::kLanes]};
      join_into(x, y);
    }
  }
  if (!here) return;
  const float inv = x.l == 0.f ? 0.f : a.v_scale / x.l;   // 0: no key at all
  const float4 y = make_float4(x.o.x * inv, x.o.y * inv, x.o.z * inv, x.o.w * inv);
  const size_t at = (static_cast<size_t>(b) * a.Hq + a.heads[g * a.G + slot]) * D + 4 * e4;
  if (F32)
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = y;
  else
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
        make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
}

// CTAs that check the tables.
int checkers_of(const QPrefixArgs& a) {
  const int front = a.P >> a.bs_shift, pieces = (front + kCheck - 1) / kCheck;
  const int64_t ctas = (static_cast<int64_t>(a.B) * pieces + kJoinThreads / 32 - 1) / (kJoinThreads / 32);
  return ctas < 256 ? static_cast<int>(ctas) : 256;
}

template <int D, bool F32, int WORKERS>
cudaError_t launch_join_w(const QPrefixArgs& a, cudaStream_t st) {
  using J = JoinShape<D, WORKERS>;
  // (a few rows' CTAs would be too few for a long table)
  const int blocks = max((a.B * a.G + J::kRows - 1) / J::kRows * J::kParts, checkers_of(a));
  return launch_pdl(k_qprefix_join<D, F32, WORKERS>,
                    dim3(static_cast<unsigned int>(blocks), static_cast<unsigned int>(a.Hkv) + 1),
                    dim3(kJoinThreads), 0, st, a);
}

template <int D, bool F32>
cudaError_t launch_join_t(const QPrefixArgs& a, cudaStream_t st) {
  // pieces of a row at most, eight of them per worker
  const int pieces = max(a.geo.pairs > 0 ? a.geo.pair_runs : 0,
                         a.geo.singles > 0 ? 2 * a.geo.single_runs : 0);
  return pieces > 32   ? launch_join_w<D, F32, 8>(a, st)
         : pieces > 16 ? launch_join_w<D, F32, 4>(a, st)
         : pieces > 8  ? launch_join_w<D, F32, 2>(a, st)
                       : launch_join_w<D, F32, 1>(a, st);
}

template <int D, int TERMS>
cudaError_t launch_prefix_t(const QPrefixArgs& a, cudaStream_t st) {
  constexpr size_t smem = Shapes<D, TERMS>::SMEM;
  constexpr auto kern = k_qprefix<D, TERMS>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(a.geo.ctas), dim3(kThreads), smem, st, a);
}

}  // namespace

// A unit's runs are as many as finish first together with the sequences' own parts, whose
// kernel runs beside this one on the SMs that are left (own_sms): one CTA per SM, and
// a CTA has one run of one unit (a second one would cost its start, its queries
// and its pieces again, 10 us); units that are more than the SMs have one run and come CTA
// after CTA. Measured: a chunk takes an SM `pair` ns with two tiles of queries and `single`
// with one, the own parts' kernel reads 33 bytes a ns on an SM and spends 350 ns on a
// sequence and KV head; 6.5 and 9 us to start and end. Half of the `own` tokens that a
// sequence may have are assumed, since the lengths are not known here.
//
// `alone`: every sequence on its own (the dense call's kernel), unless sharing is reckoned
// to be a tenth quicker (a third, where CTAs come after CTAs): 13 us for that kernel's start
// and end and 36 bytes a ns and SM; 8 us for the join. Measured, 32 heads on 8, d = 128, bf16
// (shared, alone): 32 sequences of 512 + up to 500 tokens 18.5 us, 16.2; of 2048 + 500 19.0,
// 26.0; 8 of 1024 + 8000 21.3, 17.0; 128 of 1024 + 4000 74.5, 86.9; 2048 of 1024 + 512 251,
// 544; one of 131072 (64 heads, d = 64) 53, 25.
QPrefixGeo prefix_geo(int B, int G, int Hkv, int P, int own, int d, int dtype, int sms) {
  const double pair = d == 128 ? 900 : 780;
  const double single = (d == 128 ? 640 : 400) * (dtype == KASCADE_F32 ? 2 : 1);
  const double token = static_cast<double>(B) * Hkv * (9 * d / 8), start = 9000;
  const double rest = 0.5 * token * own / 33, units = 350.0 * B * Hkv;
  QPrefixGeo g{};
  const int tiles = static_cast<int>((static_cast<int64_t>(B) * G + kPfxRows - 1) / kPfxRows);
  g.nch = (P + kPfxKeys - 1) / kPfxKeys;
  g.pairs = dtype == KASCADE_F32 ? 0 : tiles / 2;
  g.singles = tiles - 2 * g.pairs;
  const int least = sms < 32 ? 2 : sms / 16 & ~1, most_runs = (g.nch + kPfxMinRun - 1) / kPfxMinRun;
  double best = 0;
  bool best_fits = false;
  // runs of the larger kind of unit; the smaller kind's take as long at most
  for (int r = 1; r <= most_runs; ++r) {
    const int len = (g.nch + r - 1) / r;
    int single_len = g.pairs > 0 ? static_cast<int>(len * pair / single) : len;
    if (single_len < kPfxMinRun) single_len = kPfxMinRun;
    const int single_runs = (g.nch + single_len - 1) / single_len;
    const int64_t ctas = static_cast<int64_t>(Hkv) * (static_cast<int64_t>(g.pairs) * r +
                                                      static_cast<int64_t>(g.singles) * single_runs);
    if (r > 1 && ctas > sms - least) break;
    const double run = 6500 + len * (g.pairs > 0 ? pair : single);
    // SMs for the own parts: whole TPCs, what the runs leave or, with one run, more
    const int first = ctas <= sms - least ? (sms - static_cast<int>(ctas)) & ~1 : least;
    for (int o = first; o < sms && (o == first || r == 1); o += 2) {
      const double t_prefix = run * static_cast<double>((ctas + sms - o - 1) / (sms - o));
      const double t_own = start + (rest + units) / o, t = t_prefix > t_own ? t_prefix : t_own;
      // (CTA after CTA only where it gains much: 16 units and 4000 own tokens take 79 us with
      // an SM for each unit, 107 with half as many)
      if (g.own_sms == 0 || t < (ctas > sms - o && best_fits ? 0.75 : 1) * best) {
        best = t;
        best_fits = ctas <= sms - o;
        g.alone = 13000 + (token * (P + 0.5 * own) / 36 + units) / sms <
                  (best_fits ? 1.1 : 1.35) * (8000 + t);
        g.pair_runs = g.pairs > 0 ? r : 1;
        g.single_runs = single_runs;
        g.ctas = static_cast<int>(ctas);
        g.own_sms = o;
      }
    }
  }
  g.pair_len = (g.nch + g.pair_runs - 1) / g.pair_runs;
  g.single_len = (g.nch + g.single_runs - 1) / g.single_runs;
  return g;
}

cudaError_t launch_qprefix_check(const QPrefixArgs& a, cudaStream_t st) {
  if (a.B < 2) return cudaSuccess;
  return launch_pdl(k_qprefix_check, dim3(static_cast<unsigned int>(checkers_of(a))),
                    dim3(kJoinThreads), 0, st, a);
}

cudaError_t launch_qprefix(const QPrefixArgs& a, int d, int dtype, cudaStream_t st) {
  cudaError_t e;
  if (dtype == KASCADE_F32)
    e = d == 128 ? launch_prefix_t<128, 2>(a, st) : launch_prefix_t<64, 2>(a, st);
  else
    e = d == 128 ? launch_prefix_t<128, 1>(a, st) : launch_prefix_t<64, 1>(a, st);
  if (e != cudaSuccess) return e;
  if (dtype == KASCADE_F32)
    return d == 128 ? launch_join_t<128, true>(a, st) : launch_join_t<64, true>(a, st);
  return d == 128 ? launch_join_t<128, false>(a, st) : launch_join_t<64, false>(a, st);
}

}  // namespace kascade
