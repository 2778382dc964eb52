// qcache.h — launch interfaces of the paged 4-bit key/value cache: its layout,
// the block planner, the row writer and reader, and decode attention over it.
#pragma once
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace kascade {

// A block holds block_size tokens of every KV head, in groups of kQGroup
// tokens: [num_blocks][Hkv][block_size / 16][group], and a group is
//   16 rows of K codes   (d / 2 bytes each, element 2i in the low half of byte i)
//   16 rows of K scales  (d / 16 e4m3 bytes each, one per 16 elements)
//   16 rows of V codes, 16 rows of V scales (as K's)
// = 18 d bytes: 2304 at d = 128, 1152 at d = 64, so a group is one contiguous
// 16-byte aligned piece whatever the block size.
constexpr int kQGroup = 16;
constexpr int qgroup_bytes(int d) { return 18 * d; }

// Geometry of one cache, checked on the host.
struct QCacheShape {
  int block_size, bs_shift;   // 16 .. 256, a power of two
  int num_blocks, max_blocks;
  float k_scale, v_scale;     // powers of two
};

// A shared prefix (qcache_prefix.cu): its keys in nch chunks, the B * G queries of a KV
// head in row tiles. A unit is two row tiles of a KV head (`pairs` per head) or one
// (`singles`), cut into runs of pair_len or single_len chunks, one per CTA: first
// the pairs' CTAs, then the singles'. CTA c leaves pieces 2 c and 2 c + 1: of the two
// tiles, or both of the one tile.
constexpr int kPfxKeys = 64, kPfxRows = 128;
constexpr int kPfxMinRun = 4;             // chunks of a run at least
struct QPrefixGeo {
  int nch, pairs, singles, pair_runs, single_runs, pair_len, single_len, ctas;
  int own_sms;   // for the sequences' own parts, which run beside the prefix
  bool alone;    // not worth it: every sequence on its own
};
QPrefixGeo prefix_geo(int B, int G, int Hkv, int P, int own, int d, int dtype, int sms);
// A piece: o [rows/8][d/4][8] of float4, m [rows], l [rows].
constexpr size_t pfx_piece_floats(int d) { return static_cast<size_t>(kPfxRows) * (d + 2); }
// Pieces at most, on a GPU of up to `sms` SMs.
inline size_t pfx_pieces(const QPrefixGeo& g, int Hkv, int sms) {
  const size_t units = static_cast<size_t>(Hkv) * (g.pairs + g.singles);
  return 2 * (units > static_cast<size_t>(sms) ? units : sms);
}

struct QPrefixArgs {
  const void* q;              // [B,Hq,d] bf16 or fp32
  const uint8_t* cache;
  const int32_t* table;       // [B,max_blocks]
  const int32_t* lens;        // [B]
  float* part;                // pieces
  const float4* own_o;        // the sequences' own parts (QDecodeArgs::state_o, state_ml)
  const float2* own_ml;
  void* out;                  // [B,Hq,d], q's type
  float v_scale;
  unsigned int* err;
  int B, Hq, Hkv, G, N, P;    // P: tokens of the prefix, > 0
  int bs_shift, num_blocks, max_blocks;
  float scale;                // sigma * k_scale
  QPrefixGeo geo;
  int16_t heads[kMaxQHeads];
};
cudaError_t launch_qprefix(const QPrefixArgs& a, int head_dim, int dtype, cudaStream_t st);
cudaError_t launch_qprefix_check(const QPrefixArgs& a, cudaStream_t st);   // of the tables alone

struct QDecodeArgs {
  const void* q;              // [B,Hq,d] bf16 or fp32
  const uint8_t* cache;
  const int32_t* table;       // [B,max_blocks]
  const int32_t* lens;        // [B] cached tokens
  void* out;                  // [B,Hq,d], q's type
  float* scores;              // [B,Hq,N] scaled logits, or null
  float2* row_stat;           // [B*Hq] (reference, 1 / sum exp(logit - reference)), or null;
                              // the reference is the largest logit or up to 1.75 ln 2 below it
  float* part;                // split partials
  unsigned int* counters;     // [B*Hkv] split arrival counters (self-resetting)
  unsigned int* err;
  int firsts_global;          // dense: where a warp's first piece waits (see there)
  int pages_once;             // with logits: the pages' L2 lines are the first to go
  int fill_tail;              // scores behind a sequence's last key become -inf
  int B, Hq, Hkv, G, N;
  int bs_shift, num_blocks, max_blocks;
  float scale;                // sigma * k_scale
  float v_scale;
  // reuse: the sets and, per query head, their union plan (decode.cu)
  const int32_t* idx;         // [B,Hkv,topk] (pooled), null otherwise
  const uint32_t* plan;       // [B*Hkv][chunks][kPlanCapEntries]: key | mask << 24
  const int32_t* plan_count;  // [B*Hkv][chunks]
  int plan_chunks, topk;
  int S;                      // splits per (sequence, KV head) of the reuse kernel
  // dense behind a shared prefix of P tokens (0: none): a sequence with at least as many
  // starts there, and instead of an output every row, numbered (sequence * Hkv + KV head)
  // * G + slot, leaves its state: sums of weight * value [d / 4], and (reference, sum)
  float4* state_o;
  float2* state_ml;
  int P;
  int max_ctas;               // dense: CTAs at most (0: as many as fit)
  int16_t heads[kMaxQHeads];  // heads[g*G + slot]
};

// Floats of one split partial: per query head of the group m and l, then (on a
// 16-byte boundary) d outputs each.
constexpr int qpart_head(int G) { return (2 * G + 3) & ~3; }
constexpr size_t qpart_floats(int G, int d) { return qpart_head(G) + static_cast<size_t>(G) * d; }
constexpr size_t qalign16(size_t x) { return (x + 15) & ~size_t(15); }
constexpr int kQMaxCtas = 256;   // CTAs of one dense launch at most (one per SM)
// Pieces that QDecodeArgs::part holds: two per dense CTA and one per warp of it,
// or one per reuse CTA.
constexpr int kQPieces = kQMaxCtas * (2 + 16);

cudaError_t launch_qdecode_dense(const QDecodeArgs& a, int head_dim, int dtype, cudaStream_t st);
cudaError_t launch_qdecode_reuse(const QDecodeArgs& a, int head_dim, int dtype, cudaStream_t st);
// rows [B*H][N]: -inf at positions >= lens[b] (H rows per sequence)
cudaError_t launch_qfill_tail(float* rows, const int32_t* lens, int B, int H, int N,
                              cudaStream_t st);

struct QPlanArgs {
  const int32_t* kv_lens;     // [B]
  const int32_t* new_lens;    // [B]
  int32_t* table;             // [B,max_blocks]
  int32_t* free_blocks;       // [num_blocks] stack
  const int32_t* free_count;  // [1]
  int32_t* kv_lens_out;       // [B]
  int32_t* free_count_out;    // [1]
  int32_t* cu_new;            // [B + 1]
  int32_t* slot_map;          // [max_new]
  unsigned int* err;
  unsigned int* flag;         // two words of the workspace header, zero between calls
  int B, bs_shift, num_blocks, max_blocks, max_new;
};
cudaError_t launch_qplan(const QPlanArgs& a, cudaStream_t st);

struct QRowArgs {
  const void* src[2];         // append: K rows, V rows
  void* dst[2];               // read: K rows, V rows
  int64_t tok_stride[2];      // elements between tokens / heads of K and of V
  int64_t head_stride[2];
  const int32_t* slot_map;    // [T]
  uint8_t* cache;
  unsigned int* err;
  int T, Hkv, d, bs_shift, num_blocks;
  float scale[2];             // append: 1 / k_scale, 1 / v_scale; read: k_scale, v_scale
};
cudaError_t launch_qappend(const QRowArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_qread(const QRowArgs& a, int dtype, cudaStream_t st);

}  // namespace kascade
