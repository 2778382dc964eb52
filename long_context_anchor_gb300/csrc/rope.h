// rope.h — launch interfaces of the rotation of queries and keys (rope.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace kascade {

// A checked kascade_rope, and the norm in front of it.
struct RopeSpec {
  const float* table;     // [n_pos][2][n_pairs], or null: nothing is turned
  int n_pos, n_pairs, interleaved;
  int used;               // bit per axis that some pair follows
  int mixed;              // pairs of one head follow different axes
  int quads;              // ... but four neighbouring ones the same
  float eps;
  uint8_t axis[64];
};

// Queries and keys as they are attended to.
struct RopeRowArgs {
  const void* src[2];           // q, k
  void* dst[2];
  const void* weight[2];        // [d], the rows' type, or null: no norm
  int64_t src_stride[2][3];     // elements between sequences, tokens, heads
  int64_t dst_stride[2][3];
  const int32_t* positions;     // [n_axes][B][N]
  unsigned int* err;
  int B, N, H[2];               // heads of q and of k
  int splits, per;              // parts of a token's heads, heads of a part
  RopeSpec rope;
};
cudaError_t launch_qk_rope(const RopeRowArgs& a, int head_dim, int dtype, cudaStream_t st);

// Rows of new tokens into the cache, and the step's queries.
struct RopeAppendArgs {
  const void* k;
  const void* v;
  const void* q;                // or null
  void* q_out;
  const void* weight[2];        // q's, k's, or null
  int64_t k_stride[2], v_stride[2], q_stride[2], out_stride[2];   // tokens, heads
  const int32_t* slot_map;      // [T]
  const int32_t* positions;     // [n_axes][T], or null: from the two below
  const int32_t* cu_new;        // [n_seqs + 1]
  const int32_t* kv_lens;       // [n_seqs]
  uint8_t* cache;
  unsigned int* err;
  int T, Tq, n_seqs, Hq, Hkv;   // rows of k and v, rows of q
  int bs_shift, num_blocks;
  float unit[2];                // 1 / k_scale, 1 / v_scale
  int q_splits, q_per, kv_splits, kv_per;
  RopeSpec rope;
};
cudaError_t launch_qappend_rope(const RopeAppendArgs& a, int head_dim, int dtype,
                                cudaStream_t st);

// Checks a rotation for heads of head_dim elements (null: none); rope.cu.
kascade_status check_rope(const kascade_rope* rope, int head_dim, float eps, RopeSpec& s);

}  // namespace kascade
