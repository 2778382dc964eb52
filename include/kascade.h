/*
 * kascade.h — C ABI of libkascade: head-aware Top-k sparse attention with
 * cross-layer index reuse (Kascade) on one GB300 GPU (sm_103a).
 *
 * Method (Kascade: A Practical Sparse Attention Method for Long-Context LLM
 * Inference; euno.news summary, sections Key Contributions and Methodology;
 * opentrain.ai page, Abstract):
 *   - anchor layers compute attention exactly and take an exact Top-k of key
 *     indices per head (Methodology 2, 5);
 *   - reuse layers recompute attention with their own q, K, V, the softmax
 *     restricted to the saved indices (Methodology 3);
 *   - prefill works per query tile (Abstract, "tile-level operations"): one
 *     index set per (head, 128-row tile), ranked by the tile's summed
 *     post-softmax weights, capped at the tile's causal prefix;
 *   - anchors are chosen offline by a DP that maximises cross-layer Top-k
 *     overlap (Key Contributions, Methodology 4).
 *
 * Conventions for every entry point
 *   - Device pointers are plain CUDA device addresses; the caller owns every
 *     buffer. The library never allocates or frees device memory.
 *   - Tensors are dense, row-major ("C-contiguous"), and their base addresses
 *     are 16-byte aligned. Element type is given by kascade_desc.dtype for q,
 *     k, v and out (bf16 or fp32); indices are int32; scores are fp32.
 *   - Layouts (B batch, Hq query heads, Hkv KV heads, N length, d head_dim):
 *       decode : q [B,Hq,d]   k,v [B,Hkv,N,d]   out [B,Hq,d]
 *                idx [B,Hq,topk]            ascending key positions
 *       prefill: q [B,Hq,N,d] k,v [B,Hkv,N,d]   out [B,Hq,N,d]
 *                idx [B,Hq,nT,topk], nT = ceil(N/128); row t holds
 *                k_t = min(topk, min(N,128(t+1))) ascending positions, then
 *                -1 padding.
 *   - Top-k rule: larger score first, lower index wins a tie, -0 == +0.
 *     Decode ranks the scaled logits sigma*q.k (the same set as ranking the
 *     softmax weights); prefill ranks the tile weights
 *     w_j = sum_{i in tile, i >= j} softmax_i(j).
 *   - `ws` is a caller-owned device workspace of at least
 *     kascade_workspace_size() bytes, 256-byte aligned. It must be zeroed
 *     once (kascade_workspace_init) before first use; afterwards the library
 *     leaves it in a reusable state: its first 65,792 bytes (error word and
 *     split counters) stay zero between calls of any shape or entry point,
 *     and must not be written by the caller. Calls sharing one workspace must
 *     be ordered (same stream, or synchronised).
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream). Argument errors are returned before anything is
 *     launched; launch failures return KASCADE_ERR_CUDA. Faults found on the
 *     device (NaN scores, an out-of-range index, an expired bounded wait) are
 *     recorded in the workspace and read by kascade_device_error().
 *   - No entry point throws, blocks on the device (except
 *     kascade_device_error) or keeps pointers after it returns.
 */
#ifndef KASCADE_H
#define KASCADE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  KASCADE_OK = 0,
  KASCADE_ERR_INVALID_ARG = 1,  /* bad shape, pointer, alignment, k, schedule */
  KASCADE_ERR_UNSUPPORTED = 2,  /* valid but not built: head_dim, dtype, group size */
  KASCADE_ERR_WORKSPACE = 3,    /* workspace missing or too small */
  KASCADE_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed */
  KASCADE_ERR_BAD_INPUT = 5,    /* device-detected: NaN score or index out of range */
  KASCADE_ERR_TIMEOUT = 6       /* device-detected: a bounded wait expired */
} kascade_status;

typedef enum { KASCADE_F32 = 0, KASCADE_BF16 = 1 } kascade_dtype;
typedef enum { KASCADE_DECODE = 0, KASCADE_PREFILL = 1 } kascade_mode;

/* Granularity of the index sets. The pages give every attention head its own
 * Top-k list (euno.news summary, Methodology 5); for GQA models the library
 * also offers one list per KV head ("pooled"): key j's score is the sum over
 * the group's query heads h of their softmax weights p_hj (decode) or tile
 * weights w_{t,h,j} (prefill), and every head of the group attends over the
 * group's set. Index layouts then use Hkv in place of Hq:
 *   decode idx [B,Hkv,topk], prefill idx [B,Hkv,nT,topk]. */
typedef enum { KASCADE_IDX_PER_QHEAD = 0, KASCADE_IDX_PER_KVHEAD = 1 } kascade_index_mode;

/* Shape and numerics of one attention layer. */
typedef struct {
  int32_t batch;        /* B >= 1 */
  int32_t n_q_heads;    /* Hq, a multiple of n_kv_heads, <= 256 */
  int32_t n_kv_heads;   /* Hkv >= 1 */
  int32_t head_dim;     /* d: 64 or 128 */
  int32_t kv_len;       /* N: cached keys (decode) or sequence length (prefill) */
  int32_t dtype;        /* kascade_dtype of q, k, v, out; prefill needs BF16 */
  float scale;          /* sigma; <= 0 selects 1/sqrt(head_dim) */
  /* Host array [n_q_heads]: KV head read by each query head (GQA), or NULL
   * for h / (Hq/Hkv). Every KV head must serve exactly Hq/Hkv query heads;
   * group sizes 1, 2, 4 and 8 are built. Read only during the call. */
  const int32_t* group_map;
  int32_t index_mode;   /* kascade_index_mode; 0 (zero-initialised) = per query head */
} kascade_desc;
/* Size limits (KASCADE_ERR_UNSUPPORTED beyond them): N < 2^24;
 * B*Hkv*N < 2^31; B*Hkv <= 16384; prefill also B*Hq*N < 2^31. Bf16 reuse
 * decode also needs N <= 262144 (at most 128 key-range chunks of 2048). */

/* Human-readable name of a status code (static storage). */
const char* kascade_status_string(kascade_status s);

/* Bytes of workspace the calls below need for this shape, Top-k size and
 * mode (covers every decode or prefill entry point and kascade_run_stack).
 * Returns 0 for an invalid descriptor. */
size_t kascade_workspace_size(const kascade_desc* desc, int32_t topk, int32_t mode);

/* Zero a workspace (cudaMemsetAsync on `stream`). */
kascade_status kascade_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Synchronise `stream`, then read and clear the device error word of `ws`:
 * KASCADE_OK, KASCADE_ERR_BAD_INPUT or KASCADE_ERR_TIMEOUT. */
kascade_status kascade_device_error(void* ws, void* stream);

/* Failure path of the bounded device waits, for tests: launches one wait on
 * an mbarrier that nothing completes. After the library's wait limit (about
 * two seconds) the device records KASCADE_ERR_TIMEOUT in the workspace's
 * error word (read it with kascade_device_error) and the kernel returns; the
 * context stays usable. Uses only the workspace header (>= 256 bytes). */
kascade_status kascade_check_wait_timeout(void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- decode -- */

/* Exact attention for one query per sequence over all N cached keys (the
 * library's own dense baseline; also the anchor layer's output).
 * out[b,h] = sum_j softmax_j(sigma q[b,h].k[b,g(h),j]) v[b,g(h),j]. */
kascade_status kascade_dense_decode(const kascade_desc* desc, const void* q, const void* k,
                                    const void* v, void* out, void* ws, size_t ws_bytes,
                                    void* stream);

/* Anchor layer (Methodology 2): exact output as kascade_dense_decode, and the
 * exact Top-k (1 <= topk <= N) of the scaled logits of every (sequence,
 * query head) in idx_out [B,Hq,topk], ascending. When scores_out is not NULL
 * the fp32 logits sigma*q.k are also written there, [B,Hq,N].
 * Pooled index mode: idx_out [B,Hkv,topk] is the Top-k of the pooled weights
 * w[b,g,j] = sum_{h: g(h)=g} softmax_j(sigma q[b,h].k[b,g,j]), and
 * scores_out (when not NULL) receives those fp32 weights, [B,Hkv,N]. */
kascade_status kascade_anchor_decode(const kascade_desc* desc, const void* q, const void* k,
                                     const void* v, int32_t topk, void* out, int32_t* idx_out,
                                     float* scores_out, void* ws, size_t ws_bytes, void* stream);

/* The anchor layer of kascade_anchor_decode (bf16, per query head sets; other
 * modes return KASCADE_ERR_UNSUPPORTED) with the Top-k fused into the
 * attention kernel (the logit spill fused with a threshold pass; euno.news
 * summary, Methodology 2: the anchor's exact attention and its Top-k):
 * a first kernel brackets each row's k-th logit from an evenly spaced sample
 * of its keys; the attention kernel then files every logit at or above the
 * bracket's lower end, as (key, position), in per-(row, split, warp) lists
 * while it spills, and the selection is made from those lists, re-reading a
 * row's logits only when its bracket missed (all logits equal, heavy ties, an
 * unrepresentative sample). Outputs and the index sets are identical to
 * kascade_anchor_decode's (the same fp32 logits under the same rule); on
 * GB300 the two-kernel kascade_anchor_decode is as fast or faster at the
 * measured shapes, and kascade_run_stack uses it. Same arguments and
 * workspace as kascade_anchor_decode. */
kascade_status kascade_anchor_decode_fused(const kascade_desc* desc, const void* q,
                                           const void* k, const void* v, int32_t topk, void* out,
                                           int32_t* idx_out, float* scores_out, void* ws,
                                           size_t ws_bytes, void* stream);

/* Reuse layer (Methodology 3): out[b,h] = softmax restricted to the saved set
 * S = idx[b,h,:] (topk ascending, distinct positions in [0,N)), computed with
 * this layer's q, k, v. Rows of k and v outside the sets are not read. Query
 * heads of one KV head share one pass over the union of their sets.
 * Pooled index mode: S = idx[b,g(h),:], one set per KV head. */
kascade_status kascade_reuse_decode(const kascade_desc* desc, const void* q, const void* k,
                                    const void* v, int32_t topk, const int32_t* idx, void* out,
                                    void* ws, size_t ws_bytes, void* stream);

/* Exact Top-k of fp32 rows: scores [rows, n] (row stride n) -> idx [rows,k]
 * ascending, 1 <= k <= n. A NaN anywhere sets KASCADE_ERR_BAD_INPUT on the
 * device. This is the selection the anchor calls use. Needs no workspace
 * beyond the error word (ws may be any workspace, >= 256 bytes). */
kascade_status kascade_topk(const float* scores, int32_t rows, int32_t n, int32_t k,
                            int32_t* idx_out, void* ws, size_t ws_bytes, void* stream);

/* Dense decode (as kascade_dense_decode, bf16 only) for callers that cannot
 * allocate device memory and so cannot supply a workspace: code whose device
 * memory is all owned by another allocator, or that runs where cudaMalloc is
 * not allowed. The paper has no counterpart to this entry point. Its scratch
 * (split partials, counters, error word) is a fixed 8 MiB device array inside
 * the library, held by every GPU that loads it until the process exits;
 * shapes needing more return KASCADE_ERR_WORKSPACE (the descriptor limits
 * above apply as for every entry point). The first call on a device looks
 * up the array's device address, so make it before any stream capture, and
 * do not use the library across a cudaDeviceReset. All calls share the
 * array: calls that overlap on the GPU race and must be serialised by the
 * caller. Allocates nothing. Faults found on the device (an expired bounded
 * wait) are recorded in the array's error word; kascade_noalloc_device_error
 * is the only way to read them. */
kascade_status kascade_dense_decode_noalloc(const kascade_desc* desc, const void* q,
                                            const void* k, const void* v, void* out,
                                            void* stream);

/* Synchronise `stream`, then read and clear the error word of the
 * no-allocation scratch array on the current device: KASCADE_OK,
 * KASCADE_ERR_BAD_INPUT or KASCADE_ERR_TIMEOUT. Faults of every
 * kascade_dense_decode_noalloc call since the last read accumulate there.
 * The paper has no counterpart to this entry point. Allocates nothing. */
kascade_status kascade_noalloc_device_error(void* stream);

/* ------------------------------------------ sequence-sharded anchor decode -- */
/* Context-parallel form of the anchor decode layer (Methodology 2: exact
 * attention, then an exact per-head Top-k), for a KV cache split along the
 * key axis into S contiguous shards in key order (the pages run on one
 * device and do not shard a sequence). Each shard runs
 * kascade_anchor_decode_shard on its own keys; one exchange of its partials
 * (an all-gather across the devices holding the shards) and
 * kascade_merge_decode_shards give the exact layer output and the exact
 * global Top-k: every key of the global Top-k is among its own shard's
 * Top-k, and the merge applies the same rule (larger logit first, lower
 * global position on ties) to the union. Per query head sets only
 * (index_mode 0); pooled mode returns KASCADE_ERR_UNSUPPORTED. */

/* One shard: desc->kv_len = N_s, this shard's keys; k, v [B,Hkv,N_s,d] hold
 * global positions key_offset .. key_offset + N_s - 1 (key_offset >= 0,
 * key_offset + N_s < 2^31); 1 <= topk <= N_s. Writes
 *   out         [B,Hq,d] (desc dtype): attention over the shard's keys only;
 *   lse_out     [B,Hq] fp32: log sum_j exp(s_j) over the shard, s_j = sigma q.k_j;
 *   cand_idx    [B,Hq,topk] int32: the shard's Top-k as global positions,
 *               ascending;
 *   cand_scores [B,Hq,topk] fp32: the logits s_j at those positions (the same
 *               fp32 values the unsharded anchor layer ranks).
 * ws: kascade_workspace_size(desc, topk, KASCADE_DECODE) bytes, as for
 * kascade_anchor_decode. */
kascade_status kascade_anchor_decode_shard(const kascade_desc* desc, const void* q,
                                           const void* k, const void* v, int32_t key_offset,
                                           int32_t topk, void* out, float* lse_out,
                                           int32_t* cand_idx, float* cand_scores, void* ws,
                                           size_t ws_bytes, void* stream);

/* Bytes of workspace kascade_merge_decode_shards needs (0 for an invalid
 * descriptor or sizes). */
size_t kascade_merge_workspace_size(const kascade_desc* desc, int32_t n_shards, int32_t topk);

/* Merge of n_shards (1..1024) shards' partials, shard s holding keys before
 * those of shard s + 1: desc describes the whole layer (kv_len = N, the
 * total keys; B, Hq, head_dim, dtype as the shards'). Inputs, device,
 * stacked over shards in key order: outs [S,B,Hq,d] (desc dtype), lses
 * [S,B,Hq] fp32, cand_idx [S,B,Hq,topk] int32, cand_scores [S,B,Hq,topk]
 * fp32, as kascade_anchor_decode_shard wrote them (S*topk < 2^24). Writes
 *   out     [B,Hq,d]: sum_s exp(lse_s - LSE) o_s, LSE = log sum_s exp(lse_s);
 *   idx_out [B,Hq,topk]: the global Top-k, ascending positions.
 * Candidates out of [0, N) or not ascending across the shards (shards out of
 * order), and NaN logits, set KASCADE_ERR_BAD_INPUT on the device (read with
 * kascade_device_error). */
kascade_status kascade_merge_decode_shards(const kascade_desc* desc, int32_t n_shards,
                                           const void* outs, const float* lses,
                                           const int32_t* cand_idx, const float* cand_scores,
                                           int32_t topk, void* out, int32_t* idx_out, void* ws,
                                           size_t ws_bytes, void* stream);

/* --------------------------------------------------------------- prefill -- */

/* Causal exact attention (the library's own dense baseline), bf16 only. */
kascade_status kascade_dense_prefill(const kascade_desc* desc, const void* q, const void* k,
                                     const void* v, void* out, void* ws, size_t ws_bytes,
                                     void* stream);

/* Anchor layer, prefill: exact causal output, then per (sequence, query
 * head, 128-row tile t) the Top-k_t of the tile weights w_j, k_t =
 * min(topk, L_t), L_t = min(N, 128(t+1)), into idx_out [B,Hq,nT,topk]
 * (ascending, -1 padded). Pooled index mode: per (sequence, KV head g,
 * tile) the Top-k_t of sum_{h: g(h)=g} w_{t,h,j}, idx_out [B,Hkv,nT,topk].
 * When weights_out is not NULL (16-byte aligned) the fp32 tile weights the
 * selection ranked are also written there, packed per (sequence, head):
 * [B, H, P] with P = 64*(nT-1)*nT + N (the sum of the L_t), tile t's L_t
 * weights w_0..w_{L_t-1} starting at offset 64*t*(t+1) of its (b, h) row;
 * H = Hq, or Hkv in pooled index mode (then the group sums). Feeding one
 * packed row to kascade_topk's rule reproduces idx_out exactly. */
kascade_status kascade_anchor_prefill(const kascade_desc* desc, const void* q, const void* k,
                                      const void* v, int32_t topk, void* out, int32_t* idx_out,
                                      float* weights_out, void* ws, size_t ws_bytes,
                                      void* stream);

/* Reuse layer, prefill: row i of tile t attends to S_i = {j in idx[b,h,t,:],
 * j >= 0, j <= i}; a row whose S_i is empty outputs zeros. Pooled index
 * mode: the set is idx[b,g(h),t,:]. */
kascade_status kascade_reuse_prefill(const kascade_desc* desc, const void* q, const void* k,
                                     const void* v, int32_t topk, const int32_t* idx, void* out,
                                     void* ws, size_t ws_bytes, void* stream);

/* ----------------------------------------------------------------- stack -- */

/* Run n_layers layers of one mode. q[l], k[l], v[l], out[l] are host arrays
 * of device pointers (layouts as above). anchors: host array, strictly
 * ascending layer numbers in [0, n_layers). Layer l is an anchor when listed;
 * otherwise it reuses the sets of the most recent anchor <= l, or runs dense
 * when no anchor precedes it. idx_buf (device, the decode or prefill idx
 * layout of the descriptor's index mode) holds the current sets; on return
 * it holds the last anchor's. The sets never leave the device. */
kascade_status kascade_run_stack(const kascade_desc* desc, int32_t mode, int32_t n_layers,
                                 const void* const* q, const void* const* k,
                                 const void* const* v, int32_t topk, const int32_t* anchors,
                                 int32_t n_anchors, void* const* out, int32_t* idx_buf,
                                 void* ws, size_t ws_bytes, void* stream);

/* kascade_run_stack, additionally recording layer_events[l] (a cudaEvent_t,
 * or NULL to skip) on `stream` after the launches of layer l; for per-layer
 * timing. layer_events: host array [n_layers] or NULL. */
kascade_status kascade_run_stack_profiled(const kascade_desc* desc, int32_t mode,
                                          int32_t n_layers, const void* const* q,
                                          const void* const* k, const void* const* v,
                                          int32_t topk, const int32_t* anchors,
                                          int32_t n_anchors, void* const* out, int32_t* idx_buf,
                                          void* ws, size_t ws_bytes, void* stream,
                                          void* const* layer_events);

/* ------------------------------------------------------------- rotation -- */
/* Attention takes queries and keys that are turned by their positions (the
 * pages say nothing about that; their layers' q and k are the turned ones). */

/* A rotation. Pair i of a head's row is elements (i, i + n_pairs), or
 * (2i, 2i + 1) where interleaved; elements from 2*n_pairs on stay as they are. A
 * token at position p turns pair i by table[p][0][i] (cosine) and
 * table[p][1][i] (sine): (a, b) -> (a c - b s, b c + a s), every product and
 * sum rounded to fp32. With several axes (a video's time, height and width) a token
 * has a position on each, and axes[i] names the one that pair i follows. */
typedef struct {
  const float* table;    /* device [n_positions][2][n_pairs], 16-byte aligned */
  int32_t n_positions;
  int32_t n_pairs;       /* a multiple of 16, 2*n_pairs <= head_dim */
  int32_t interleaved;
  int32_t n_axes;        /* 1 .. 4 */
  const int32_t* axes;   /* host [n_pairs], read during the call; NULL: axis 0 */
} kascade_rope;

/* Queries and keys for the attention calls, in one pass: a head's row x
 * becomes x * rsqrt(mean(x^2) + eps) * weight (weights [head_dim] of the rows'
 * type; NULL: left out), then is turned (rope NULL: not turned, positions
 * unused), in fp32, rounded once. q and k: row (b, t, h) of head_dim contiguous
 * elements at q + b*strides[0] + t*strides[1] + h*strides[2], k likewise with
 * strides[3..5], q_out and k_out with strides[6..8] and [9..11] (host array,
 * elements, multiples of 16 bytes). q_out and k_out may be q and k with the same
 * strides; other overlaps are not allowed. n_q_heads or n_kv_heads may be 0.
 * positions [n_axes][batch][n_tokens] int32; one outside the table sets
 * KASCADE_ERR_BAD_INPUT on the device, and its axis' pairs are turned by no angle
 * (cosine 1, sine 0). Positions on an axis that no pair follows are not looked at.
 * batch*n_tokens < 2^28. ws: the workspace header, 256 bytes. */
kascade_status kascade_qk_norm_rope(const kascade_rope* rope, int32_t batch, int32_t n_tokens,
                                    int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                    int32_t dtype, const void* q, const void* k,
                                    const void* q_weight, const void* k_weight, float eps,
                                    const int32_t* positions, void* q_out, void* k_out,
                                    const int64_t* strides, void* ws, size_t ws_bytes,
                                    void* stream);

/* ------------------------------------------- paged 4-bit key/value cache -- */
/* Decode for a server's cache: sequences of different lengths, each a list of
 * fixed-size blocks, keys and values held in 4 bits (the pages describe
 * neither; the layers over the cache are theirs, Methodology 2-3).
 *
 * pages [num_blocks][Hkv][block_size/16][18 d] bytes, one such buffer per
 * layer (kascade_qcache_bytes), 16-byte aligned. The last axis is a group of
 * 16 tokens: 16 rows of K codes (d/2 bytes each, element 2i in the low half
 * of byte i), 16 rows of K scales (d/16 bytes), 16 rows of V codes, 16 rows of
 * V scales. 16 consecutive elements of a row share one scale; with
 * x' = x / {k,v}_scale and amax the block's largest |x'|,
 *   s    = amax/6 rounded to e4m3 (ties to even, at most 448),
 *   code = x'/s rounded to e2m1 {0, .5, 1, 1.5, 2, 3, 4, 6} (same, at most 6),
 * and the stored element is code * s * {k,v}_scale, exact in bf16. Blocks with
 * amax/6 <= 2^-10 are stored as zeros, magnitudes above 2688 (infinities
 * among them) saturate, and a block that holds a NaN reads back as NaN.
 *
 * block_table [B][max_blocks] int32: entry j of row b is the block that holds
 * tokens j*block_size .. of sequence b (all layers share it). A slot is
 * block * block_size + offset. kv_lens [B] int32: cached tokens of each
 * sequence, 0 <= kv_lens[b] <= desc->kv_len, read on the device; a sequence
 * of length 0 outputs zeros. What the pages hold behind a sequence's last
 * token is never used. desc->kv_len <= max_blocks*block_size is the longest
 * length, the row stride of scores, and what workspaces and limits go by, so it
 * is best kept near the lengths in use where the table is wide. desc->dtype is
 * that of q, out and of appended rows: bf16, or fp32, for which a query's
 * elements keep 22 bits; sums are in fp32. A length out of
 * range, or a block id outside [0, num_blocks), sets KASCADE_ERR_BAD_INPUT on the device;
 * those keys are not read and count as masked.
 * In the product with V softmax weights are rounded to 11 bits (bf16) or 22
 * (fp32), and to multiples of at most 2^-38 of the row's largest one; their sum
 * is taken unrounded.
 * A sequence's keys are split over CTAs by rules that look at the whole batch,
 * so the last bits of its output may differ between batches; one call repeated
 * gives the same bits.
 * Limits beyond the descriptor's: num_blocks*block_size < 2^31, B*max_blocks
 * < 2^31, fewer than 2^28 new tokens in a call and, for attention,
 * num_blocks*Hkv*block_size/16 < 2^28 - 1 (KASCADE_ERR_UNSUPPORTED). */
typedef struct {
  int32_t block_size;   /* 16, 32, 64, 128 or 256 tokens */
  int32_t num_blocks;   /* blocks of the cache */
  int32_t max_blocks;   /* columns of a block table */
  float k_scale;        /* powers of two in [2^-32, 2^32]; 0 selects 1 */
  float v_scale;
} kascade_qcache;

/* Bytes of one layer's pages (0 for an invalid geometry). */
size_t kascade_qcache_bytes(const kascade_qcache* cache, int32_t n_kv_heads, int32_t head_dim);

/* Workspace of the attention calls below: topk = 0 for
 * kascade_qcache_dense_decode, the sets' size for the others. 0 if invalid.
 * Plan, append and read need only the workspace header, 256 bytes. */
size_t kascade_qcache_workspace_size(const kascade_desc* desc, const kascade_qcache* cache,
                                     int32_t topk);

/* What kascade_qcache_reuse_decode alone needs of that: it keeps no logits,
 * which are B*Hq*kv_len*4 bytes of an anchor layer's. */
size_t kascade_qcache_reuse_workspace_size(const kascade_desc* desc, const kascade_qcache* cache,
                                           int32_t topk);

/* Block tables and slots of one step, on the device. Sequence b goes from
 * L = kv_lens[b] to L' = max(0, L + new_lens[b]) tokens: it grows (new tokens
 * to append), shrinks (tokens taken back) or, with -L or less, ends. It then
 * holds ceil(L'/block_size) blocks: those it gives back are pushed on the
 * stack free_blocks [num_blocks] (free_count of them valid) in (sequence,
 * column) order, then those it takes are popped from it in that order. A block
 * is in one place, one sequence's part of the table or the stack: blocks that
 * sequences share are read correctly, but each of them would give it back.
 * Writes
 *   block_table     the entries of taken blocks (others are left as they are);
 *   kv_lens_out [B], free_count_out [1]   (may be kv_lens and free_count);
 *   cu_new [B+1]    running number of new tokens: sequence b's rows of this
 *                   step are cu_new[b] .. cu_new[b+1]-1;
 *   slot_map [max_new]   the slot of every new token, -1 behind the last.
 * A step that cannot be served (too few free blocks, more tokens than
 * max_blocks*block_size or than max_new, a length out of range, an id out of
 * range among the blocks given back, taken or written to by new tokens)
 * changes no table, stack, length or count, leaves every slot -1 and cu_new
 * 0, and sets KASCADE_ERR_BAD_INPUT on the device. n_seqs <= 16384. */
kascade_status kascade_qcache_plan(const kascade_qcache* cache, int32_t n_seqs,
                                   const int32_t* kv_lens, const int32_t* new_lens,
                                   int32_t* block_table, int32_t* free_blocks,
                                   const int32_t* free_count, int32_t* kv_lens_out,
                                   int32_t* free_count_out, int32_t* cu_new, int32_t* slot_map,
                                   int32_t max_new, void* ws, size_t ws_bytes, void* stream);

/* Quantise rows of new keys and values into their slots. k, v: row (t, g) of
 * head_dim contiguous elements at k + t*strides[0] + g*strides[1] and
 * v + t*strides[2] + g*strides[3] (host array of four element strides, each a
 * multiple of 16 bytes), so the decode layout [T,Hkv,d] and the prefill
 * layout [Hkv,N,d] are both taken as they are. slot_map [n_tokens]: distinct
 * slots; a negative one is padding (skipped), one beyond the cache sets
 * KASCADE_ERR_BAD_INPUT and is skipped. */
kascade_status kascade_qcache_append(const kascade_qcache* cache, int32_t n_kv_heads,
                                     int32_t head_dim, int32_t dtype, const void* k,
                                     const void* v, const int64_t* strides,
                                     const int32_t* slot_map, int32_t n_tokens, void* pages,
                                     void* ws, size_t ws_bytes, void* stream);

/* kascade_qcache_append of rows that are normalised (k_weight not NULL) and
 * turned on their way (kascade_qk_norm_rope; the turned key is quantised from
 * its fp32 elements; values are stored as they are), and the same for the queries
 * of the step (q not NULL; n_q_heads heads). Positions come in one of two ways:
 *   positions [n_axes][n_tokens]: row t of k, v and q is token t; cu_new and
 *     kv_lens are NULL and n_seqs 0;
 *   cu_new [n_seqs+1] and kv_lens [n_seqs] as kascade_qcache_plan wrote them
 *     (positions NULL): row t of k and v is its new token t, and row b of q
 *     the query of sequence b's last token. All axes have that one position.
 * With rope NULL (a norm alone) the first way needs no positions either.
 * strides: k (tokens, heads), v, q, q_out: eight. q_out may be q with the same
 * strides. Queries are written whatever their token's slot. A position outside
 * the table does what it does in kascade_qk_norm_rope; those of keys without a
 * slot are not looked at. */
kascade_status kascade_qcache_append_rope(const kascade_qcache* cache, const kascade_rope* rope,
                                          int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim, int32_t dtype, const void* k,
                                          const void* v, const void* q, const int64_t* strides,
                                          const void* k_weight, const void* q_weight, float eps,
                                          const int32_t* slot_map, int32_t n_tokens,
                                          const int32_t* positions, const int32_t* cu_new,
                                          const int32_t* kv_lens, int32_t n_seqs, void* pages,
                                          void* q_out, void* ws, size_t ws_bytes, void* stream);

/* The stored values of rows, in the same layouts, for the calls that take
 * contiguous keys and values (a prompt's prefill, which needs a query row for
 * every key, or a calibration); zeros for a negative slot. Slots may repeat.
 * The rows that are written must not overlap. */
kascade_status kascade_qcache_read(const kascade_qcache* cache, int32_t n_kv_heads,
                                   int32_t head_dim, int32_t dtype, const void* pages,
                                   const int32_t* slot_map, int32_t n_tokens, void* k, void* v,
                                   const int64_t* strides, void* ws, size_t ws_bytes,
                                   void* stream);

/* Exact attention of one query per sequence over its cached tokens (as
 * kascade_dense_decode). When scores_out is not NULL the fp32 logits
 * sigma*q.k are written there, [B,Hq,kv_len], -inf behind the last token. */
kascade_status kascade_qcache_dense_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                           const void* q, const void* pages,
                                           const int32_t* block_table, const int32_t* kv_lens,
                                           void* out, float* scores_out, void* ws,
                                           size_t ws_bytes, void* stream);

/* kascade_qcache_dense_decode for a batch whose sequences begin alike: the first
 * prefix_len tokens (a multiple of block_size, 0 <= prefix_len <= kv_len) of
 * every sequence with kv_lens[b] >= prefix_len lie in the same blocks, so that
 * these sequences' rows of block_table have the same first
 * prefix_len/block_size entries. The prefix is read, and its products are
 * taken, once for all of them; a shorter sequence (a padding row of length 0
 * too) is attended to on its own, whatever its blocks. Entries that differ set
 * KASCADE_ERR_BAD_INPUT on the device; the sequence's own ones are used then, or
 * those of the lowest sequence that holds the prefix.
 * Over kascade_qcache_plan a sequence of such a batch starts with kv_lens[b] =
 * prefix_len and its row's first entries set, and ends with new_lens[b] =
 * prefix_len - kv_lens[b], which gives back its own blocks alone.
 * Weights of the prefix are multiples of 2^-28 (bf16) or 2^-32 (fp32) of the
 * row's largest one at most. How the SMs are shared out goes by prefix_len and
 * desc->kv_len - prefix_len, not by the lengths (they are not known to the
 * host), so kv_len is best given as the longest length in use. So does whether
 * it is done at all: with `always` 0 a batch that sharing is not reckoned to
 * help (few sequences, a short prefix) is attended to one by one, with the same
 * check of the tables; with 1 the prefix is shared whatever it costs.
 * Workspace: kascade_qcache_prefix_workspace_size. */
size_t kascade_qcache_prefix_workspace_size(const kascade_desc* desc, const kascade_qcache* cache,
                                            int32_t prefix_len);
kascade_status kascade_qcache_prefix_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                            const void* q, const void* pages,
                                            const int32_t* block_table, const int32_t* kv_lens,
                                            int32_t prefix_len, int32_t always, void* out,
                                            void* ws, size_t ws_bytes, void* stream);

/* Anchor layer (as kascade_anchor_decode, both index modes): the exact output
 * and the exact Top-k of every row, min(topk, kv_lens[b]) ascending positions
 * and -1 behind them; 1 <= topk <= desc->kv_len. scores_out as there, -inf
 * behind the last token. */
kascade_status kascade_qcache_anchor_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                            const void* q, const void* pages,
                                            const int32_t* block_table, const int32_t* kv_lens,
                                            int32_t topk, void* out, int32_t* idx_out,
                                            float* scores_out, void* ws, size_t ws_bytes,
                                            void* stream);

/* Reuse layer (as kascade_reuse_decode, both index modes): idx rows hold
 * ascending distinct positions in [0, kv_lens[b]), then -1 entries; an empty
 * set outputs zeros. Entries that break this set KASCADE_ERR_BAD_INPUT and
 * are not read. Per query head sets need kv_len <= 262144. */
kascade_status kascade_qcache_reuse_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                           const void* q, const void* pages,
                                           const int32_t* block_table, const int32_t* kv_lens,
                                           int32_t topk, const int32_t* idx, void* out, void* ws,
                                           size_t ws_bytes, void* stream);

/* The device state one decode step works on. */
typedef struct {
  int32_t* block_table;       /* [B, max_blocks] */
  int32_t* kv_lens;           /* [B]; updated by the step's plan */
  const int32_t* new_lens;    /* [B], or NULL: no plan, kv_lens and slot_map are as given */
  int32_t* free_blocks;       /* [num_blocks], with new_lens only, as the next two */
  int32_t* free_count;        /* [1] */
  int32_t* cu_new;            /* [B + 1] */
  int32_t* slot_map;          /* [max_new] */
  int32_t max_new;            /* rows of every k_new[l], v_new[l] */
} kascade_qcache_step;

/* One decode step over a layer stack: the plan (when step->new_lens is not
 * NULL), then per layer l the append of k_new[l], v_new[l] [max_new,Hkv,d]
 * (skipped when k_new and v_new are NULL) and the anchor, reuse or dense
 * layer over pages[l], dispatched as kascade_run_stack does. q, k_new,
 * v_new, pages, out: host arrays of device pointers. A sequence's query
 * attends to its new tokens too. */
kascade_status kascade_qcache_run_stack(
    const kascade_desc* desc, const kascade_qcache* cache, const kascade_qcache_step* step,
    int32_t n_layers, const void* const* q, const void* const* k_new, const void* const* v_new,
    void* const* pages, int32_t topk, const int32_t* anchors, int32_t n_anchors, void* const* out,
    int32_t* idx_buf, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------ scheduling -- */

/* Cross-layer Top-k overlap for the anchor DP (Methodology 4). sets: device
 * int32 [n_layers, units, topk], each row distinct positions in [0, n_bits).
 * counts_out: device int64 [n_layers, n_layers], counts_out[i][l] =
 * sum over units of |S_i ∩ S_l| (symmetric). Needs ws of
 * kascade_overlap_workspace_size bytes. */
size_t kascade_overlap_workspace_size(int32_t n_layers, int32_t units, int32_t n_bits);
kascade_status kascade_layer_overlap(const int32_t* sets, int32_t n_layers, int32_t units,
                                     int32_t topk, int32_t n_bits, int64_t* counts_out,
                                     void* ws, size_t ws_bytes, void* stream);

/* Calibration for the anchor DP (Methodology 4) on decode inputs: runs
 * every layer l as an anchor (kascade_anchor_decode) writing its exact
 * Top-k sets to sets_buf + l*B*H*topk (device int32 [n_layers, B*H,
 * topk], H = Hq, or Hkv in pooled index mode; also the layer outputs to
 * out[l]), counts the cross-layer overlaps on the device and returns
 * sim_out[i*n_layers + l] = sum over (sequence, head) of |S_i ∩ S_l| /
 * (B*H*topk) (host float64 [n_layers^2]).
 * Synchronises `stream` before returning. ws must hold
 * kascade_calibrate_workspace_size bytes. */
size_t kascade_calibrate_workspace_size(const kascade_desc* desc, int32_t topk, int32_t n_layers);
kascade_status kascade_calibrate(const kascade_desc* desc, int32_t n_layers,
                                 const void* const* q, const void* const* k,
                                 const void* const* v, int32_t topk, void* const* out,
                                 int32_t* sets_buf, double* sim_out, void* ws, size_t ws_bytes,
                                 void* stream);

/* Calibration with the attention-mass-recall similarity, an alternative to
 * the set overlap of kascade_calibrate (the pages give the DP's similarity no
 * formula; euno.news summary, Methodology 4). Every layer runs as an anchor
 * exactly as there (sets_buf and out as there) and
 *   sim_out[i*n_layers + l] = mean over (sequence, query head) of
 *                             sum_{j in S_i} softmax_j(layer l's logits),
 * for i <= l: the share of layer l's exact attention mass that the set layer
 * i holds for that head (its own set, or its KV head's in pooled index mode)
 * would keep. Entries with i > l are 0; the anchor DP reads only i <= l.
 * sim_out: host float64 [n_layers^2]. Synchronises `stream` before
 * returning. ws must hold kascade_calibrate_recall_workspace_size bytes. */
size_t kascade_calibrate_recall_workspace_size(const kascade_desc* desc, int32_t topk,
                                               int32_t n_layers);
kascade_status kascade_calibrate_recall(const kascade_desc* desc, int32_t n_layers,
                                        const void* const* q, const void* const* k,
                                        const void* const* v, int32_t topk, void* const* out,
                                        int32_t* sets_buf, double* sim_out, void* ws,
                                        size_t ws_bytes, void* stream);

/* Host DP: choose n_anchors layers (always including 0) maximising
 * F(A) = sum_l sim[a(l) * n_layers + l], a(l) = most recent anchor <= l.
 * sim: host [n_layers * n_layers], row i = anchor layer. Ties go to the
 * lexicographically smallest list. anchors_out: host [n_anchors],
 * ascending. objective_out may be NULL. */
kascade_status kascade_schedule_anchors(const double* sim, int32_t n_layers, int32_t n_anchors,
                                        int32_t* anchors_out, double* objective_out);

#ifdef __cplusplus
}
#endif
#endif /* KASCADE_H */
