// qcache_api.cu — the C ABI of the paged 4-bit key/value cache (the
// kascade_qcache_* part of include/kascade.h): argument validation, workspace
// layout, and the decode step over a layer stack. The pages describe neither
// a paged nor a compressed cache; the anchor and reuse layers over it are
// theirs (euno.news summary, Methodology 2-3).
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "common.cuh"
#include "kascade.h"
#include "qcache.h"

namespace kascade {
namespace {

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void* p, uintptr_t n) {
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}
inline kascade_status status_of(cudaError_t e) {
  if (e == cudaErrorNotSupported) return KASCADE_ERR_UNSUPPORTED;
  return e == cudaSuccess ? KASCADE_OK : KASCADE_ERR_CUDA;
}
template <typename T>
inline T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

// 0 selects 1; otherwise a power of two between 2^-32 and 2^32.
bool check_scale(float x, float& out) {
  if (x == 0.f) x = 1.f;
  out = x;
  int e = 0;
  if (!(x > 0.f) || !isfinite(x)) return false;
  return frexpf(x, &e) == 0.5f && e >= -31 && e <= 33;
}

kascade_status check_qcache(const kascade_qcache* c, QCacheShape& s) {
  if (c == nullptr) return KASCADE_ERR_INVALID_ARG;
  s.block_size = c->block_size;
  s.num_blocks = c->num_blocks;
  s.max_blocks = c->max_blocks;
  if (s.num_blocks < 1 || s.max_blocks < 1) return KASCADE_ERR_INVALID_ARG;
  s.bs_shift = 0;
  for (int sh = 4; sh <= 8; ++sh)
    if (s.block_size == (1 << sh)) s.bs_shift = sh;
  if (s.bs_shift == 0) return KASCADE_ERR_UNSUPPORTED;
  if (static_cast<long long>(s.num_blocks) * s.block_size >= (1ll << 31))
    return KASCADE_ERR_UNSUPPORTED;   // slots are 32-bit
  if (!check_scale(c->k_scale, s.k_scale) || !check_scale(c->v_scale, s.v_scale))
    return KASCADE_ERR_INVALID_ARG;
  return KASCADE_OK;
}

struct QLayout {
  size_t counters, part;                                  // every attention call
  size_t plan, plan_count;                                // topk >= 1, sets per query head
  size_t spill, row_stat, pool;                           // topk >= 1, anchor layers
  size_t reuse, total;                                    // bytes: without an anchor layer, in all
};

QLayout qlayout(const Shape& s, int topk) {
  QLayout L{};
  L.counters = sizeof(WsHeader);
  size_t off = kWsStateBytes;
  L.part = off;
  off = align256(off + static_cast<size_t>(kQPieces) * qpart_floats(s.G, s.d) * 4);
  if (topk >= 1 && !s.pooled) {
    const size_t chunks = decode_union_chunks(s.B * s.Hkv, s.N);
    L.plan = off;
    off = align256(off + static_cast<size_t>(s.B) * s.Hkv * chunks * kPlanCapEntries * 4);
    L.plan_count = off;
    off = align256(off + static_cast<size_t>(s.B) * s.Hkv * chunks * 4);
  }
  L.reuse = off;
  if (topk >= 1) {
    L.spill = off;
    off = align256(off + static_cast<size_t>(s.B) * s.Hq * s.N * 4);
    if (s.pooled) {
      L.row_stat = off;
      off = align256(off + static_cast<size_t>(s.B) * s.Hq * 8);
      L.pool = off;
      off = align256(off + static_cast<size_t>(s.B) * s.Hkv * s.N * 4);
    }
  }
  L.total = off;
  return L;
}

// One call's validated geometry.
struct QCall {
  Shape s;
  QCacheShape c;
  QLayout L;
};

kascade_status check_call(const kascade_desc* desc, const kascade_qcache* cache, QCall& k) {
  kascade_status r = check_desc(desc, k.s);
  if (r != KASCADE_OK) return r;
  if ((r = check_qcache(cache, k.c)) != KASCADE_OK) return r;
  if (static_cast<long long>(k.c.max_blocks) * k.c.block_size < k.s.N)
    return KASCADE_ERR_INVALID_ARG;
  if (static_cast<long long>(k.s.B) * k.c.max_blocks >= (1ll << 31)) return KASCADE_ERR_UNSUPPORTED;
  // a group's number fits 28 bits (2^28 groups are more than any GPU's memory)
  if (static_cast<long long>(k.c.num_blocks) * k.s.Hkv * (k.c.block_size / kQGroup) >=
      (1ll << 28) - 1)
    return KASCADE_ERR_UNSUPPORTED;
  return KASCADE_OK;
}

kascade_status check_qws(QCall& k, int topk, void* ws, size_t ws_bytes, bool reuse = false) {
  k.L = qlayout(k.s, topk);
  if (!aligned(ws, 256) || ws_bytes < (reuse ? k.L.reuse : k.L.total))
    return KASCADE_ERR_WORKSPACE;
  return KASCADE_OK;
}

bool check_small_ws(const void* ws, size_t ws_bytes) {
  return aligned(ws, 256) && ws_bytes >= sizeof(WsHeader);
}

kascade_status check_attn_ptrs(const void* q, const void* cache, const int32_t* table,
                               const int32_t* lens, const void* out) {
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(out, 16))
    return KASCADE_ERR_INVALID_ARG;
  return KASCADE_OK;
}

void fill_qargs(QDecodeArgs& a, const QCall& k, const void* q, const void* cache,
                const int32_t* table, const int32_t* lens, void* out, void* ws) {
  memset(&a, 0, sizeof(a));
  a.q = q;
  a.cache = static_cast<const uint8_t*>(cache);
  a.table = table;
  a.lens = lens;
  a.out = out;
  a.part = at<float>(ws, k.L.part);
  a.counters = at<unsigned int>(ws, k.L.counters);
  a.err = at<unsigned int>(ws, 0);
  a.B = k.s.B;
  a.Hq = k.s.Hq;
  a.Hkv = k.s.Hkv;
  a.G = k.s.G;
  a.N = k.s.N;
  a.bs_shift = k.c.bs_shift;
  a.num_blocks = k.c.num_blocks;
  a.max_blocks = k.c.max_blocks;
  a.scale = k.s.scale * k.c.k_scale;
  a.v_scale = k.c.v_scale;
  for (int i = 0; i < k.s.Hq; ++i) a.heads[i] = k.s.heads[i];
}

kascade_status run_qdense(const QCall& k, const void* q, const void* cache, const int32_t* table,
                          const int32_t* lens, void* out, float* scores, bool fill_tail,
                          float2* row_stat, void* ws, cudaStream_t st) {
  QDecodeArgs a;
  fill_qargs(a, k, q, cache, table, lens, out, ws);
  a.scores = scores;
  a.fill_tail = fill_tail ? 1 : 0;
  a.row_stat = row_stat;
  return status_of(launch_qdecode_dense(a, k.s.d, k.s.dtype, st));
}

kascade_status run_qanchor(const QCall& k, const void* q, const void* cache, const int32_t* table,
                           const int32_t* lens, int topk, void* out, int32_t* idx_out,
                           float* scores_out, void* ws, cudaStream_t st) {
  const Shape& s = k.s;
  // per query head the caller's scores are the logits themselves; pooled
  // scores are the group sums of the softmax weights, from logits kept here
  float* spill = scores_out != nullptr && !s.pooled ? scores_out : at<float>(ws, k.L.spill);
  float2* stat = s.pooled ? at<float2>(ws, k.L.row_stat) : nullptr;
  kascade_status r = run_qdense(k, q, cache, table, lens, out, spill,
                                scores_out != nullptr && !s.pooled, stat, ws, st);
  if (r != KASCADE_OK) return r;
  const float* rows = spill;
  if (s.pooled) {
    float* pool = scores_out != nullptr ? scores_out : at<float>(ws, k.L.pool);
    r = status_of(launch_pool_decode(spill, stat, pool, true, s.heads, s.B, s.Hq, s.Hkv, s.G, s.N,
                                     st));
    if (r != KASCADE_OK) return r;
    if (scores_out != nullptr &&
        (r = status_of(launch_qfill_tail(pool, lens, s.B, s.Hkv, s.N, st))) != KASCADE_OK)
      return r;
    rows = pool;
  }
  TopkArgs t{};
  t.scores = rows;
  t.idx_out = idx_out;
  t.err = at<unsigned int>(ws, 0);
  t.rows = s.B * s.H_idx;
  t.n = s.N;
  t.k = topk;
  t.k_stride = topk;
  t.tile = 128;
  t.row_lens = lens;
  t.rows_per_len = s.H_idx;
  return status_of(launch_topk(t, st));
}

// The union plan of per query head sets (bf16 and fp32 alike).
kascade_status run_qplan_sets(const QCall& k, const int32_t* lens, const int32_t* idx, int topk,
                              void* ws, cudaStream_t st) {
  DecodeArgs a;
  memset(&a, 0, sizeof(a));
  a.idx = idx;
  a.lens = lens;
  a.topk = topk;
  a.B = k.s.B;
  a.Hq = k.s.Hq;
  a.Hkv = k.s.Hkv;
  a.N = k.s.N;
  a.G = k.s.G;
  a.err = at<unsigned int>(ws, 0);
  for (int i = 0; i < k.s.Hq; ++i) a.heads[i] = k.s.heads[i];
  return status_of(launch_build_union_plan(a, at<uint32_t>(ws, k.L.plan),
                                           at<int32_t>(ws, k.L.plan_count), st));
}

kascade_status run_qreuse(const QCall& k, const void* q, const void* cache, const int32_t* table,
                          const int32_t* lens, int topk, const int32_t* idx, void* out, void* ws,
                          bool plan_ready, cudaStream_t st) {
  QDecodeArgs a;
  fill_qargs(a, k, q, cache, table, lens, out, ws);
  a.topk = topk;
  if (k.s.pooled) {
    a.idx = idx;
  } else {
    a.plan_chunks = decode_union_chunks(k.s.B * k.s.Hkv, k.s.N);
    if (a.plan_chunks > kMaxSplits) return KASCADE_ERR_UNSUPPORTED;
    if (!plan_ready) {
      const kascade_status r = run_qplan_sets(k, lens, idx, topk, ws, st);
      if (r != KASCADE_OK) return r;
    }
    a.plan = at<uint32_t>(ws, k.L.plan);
    a.plan_count = at<int32_t>(ws, k.L.plan_count);
  }
  return status_of(launch_qdecode_reuse(a, k.s.d, k.s.dtype, st));
}

// New tokens of one call: grids and slots are numbered in 32 bits.
constexpr int kMaxNewTokens = (1 << 28) - 1;

// Rows of new keys and values.
kascade_status check_rows(const kascade_qcache* cache, int n_kv_heads, int head_dim, int dtype,
                          const void* k, const void* v, const int64_t* strides,
                          const int32_t* slot_map, int n_tokens, const void* pages,
                          QCacheShape& c) {
  kascade_status r = check_qcache(cache, c);
  if (r != KASCADE_OK) return r;
  if (dtype != KASCADE_F32 && dtype != KASCADE_BF16) return KASCADE_ERR_INVALID_ARG;
  if (n_kv_heads < 1 || n_kv_heads > kMaxQHeads || n_tokens < 0 || strides == nullptr)
    return KASCADE_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return KASCADE_ERR_UNSUPPORTED;
  if (n_tokens > kMaxNewTokens) return KASCADE_ERR_UNSUPPORTED;
  if (n_tokens == 0) return KASCADE_OK;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slot_map, 4) || !aligned(pages, 16))
    return KASCADE_ERR_INVALID_ARG;
  const int64_t unit = dtype == KASCADE_F32 ? 4 : 8;   // rows start on 16-byte boundaries
  for (int i = 0; i < 4; ++i)
    if (strides[i] < 0 || strides[i] % unit != 0) return KASCADE_ERR_INVALID_ARG;
  return KASCADE_OK;
}

QRowArgs row_args(const QCacheShape& c, int n_kv_heads, int head_dim, const int64_t* strides,
                  const int32_t* slot_map, int n_tokens, void* ws) {
  QRowArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.tok_stride[i] = strides[2 * i];
    a.head_stride[i] = strides[2 * i + 1];
  }
  a.slot_map = slot_map;
  a.err = static_cast<unsigned int*>(ws);
  a.T = n_tokens;
  a.Hkv = n_kv_heads;
  a.d = head_dim;
  a.bs_shift = c.bs_shift;
  a.num_blocks = c.num_blocks;
  return a;
}

kascade_status run_qplan(const QCacheShape& c, int n_seqs, const int32_t* kv_lens,
                         const int32_t* new_lens, int32_t* block_table, int32_t* free_blocks,
                         const int32_t* free_count, int32_t* kv_lens_out, int32_t* free_count_out,
                         int32_t* cu_new, int32_t* slot_map, int max_new, void* ws,
                         cudaStream_t st) {
  QPlanArgs a;
  a.kv_lens = kv_lens;
  a.new_lens = new_lens;
  a.table = block_table;
  a.free_blocks = free_blocks;
  a.free_count = free_count;
  a.kv_lens_out = kv_lens_out;
  a.free_count_out = free_count_out;
  a.cu_new = cu_new;
  a.slot_map = slot_map;
  a.err = static_cast<unsigned int*>(ws);
  a.flag = static_cast<WsHeader*>(ws)->pad;
  a.B = n_seqs;
  a.bs_shift = c.bs_shift;
  a.num_blocks = c.num_blocks;
  a.max_blocks = c.max_blocks;
  a.max_new = max_new;
  return status_of(launch_qplan(a, st));
}

kascade_status check_plan(const kascade_qcache* cache, int n_seqs, const int32_t* kv_lens,
                          const int32_t* new_lens, const int32_t* block_table,
                          const int32_t* free_blocks, const int32_t* free_count,
                          const int32_t* kv_lens_out, const int32_t* free_count_out,
                          const int32_t* cu_new, const int32_t* slot_map, int max_new,
                          QCacheShape& c) {
  kascade_status r = check_qcache(cache, c);
  if (r != KASCADE_OK) return r;
  if (n_seqs < 1 || max_new < 0) return KASCADE_ERR_INVALID_ARG;
  if (n_seqs > kMaxCounterUnits || max_new > kMaxNewTokens ||
      static_cast<long long>(n_seqs) * c.max_blocks >= (1ll << 31) ||
      static_cast<long long>(c.max_blocks) * c.block_size >= (1ll << 31))
    return KASCADE_ERR_UNSUPPORTED;
  const void* need[] = {kv_lens, new_lens, block_table, free_blocks, free_count,
                        kv_lens_out, free_count_out, cu_new};
  for (const void* p : need)
    if (!aligned(p, 4)) return KASCADE_ERR_INVALID_ARG;
  if (max_new > 0 && !aligned(slot_map, 4)) return KASCADE_ERR_INVALID_ARG;
  return KASCADE_OK;
}

}  // namespace
}  // namespace kascade

using namespace kascade;

extern "C" {

size_t kascade_qcache_bytes(const kascade_qcache* cache, int32_t n_kv_heads, int32_t head_dim) {
  QCacheShape c;
  if (check_qcache(cache, c) != KASCADE_OK || n_kv_heads < 1 || n_kv_heads > kMaxQHeads ||
      (head_dim != 64 && head_dim != 128))
    return 0;
  return static_cast<size_t>(c.num_blocks) * n_kv_heads * (c.block_size / kQGroup) *
         qgroup_bytes(head_dim);
}

size_t kascade_qcache_workspace_size(const kascade_desc* desc, const kascade_qcache* cache,
                                     int32_t topk) {
  QCall k;
  if (check_call(desc, cache, k) != KASCADE_OK || topk < 0) return 0;
  return qlayout(k.s, topk).total;
}

size_t kascade_qcache_reuse_workspace_size(const kascade_desc* desc, const kascade_qcache* cache,
                                           int32_t topk) {
  QCall k;
  if (check_call(desc, cache, k) != KASCADE_OK || topk < 1) return 0;
  return qlayout(k.s, topk).reuse;
}

kascade_status kascade_qcache_plan(const kascade_qcache* cache, int32_t n_seqs,
                                   const int32_t* kv_lens, const int32_t* new_lens,
                                   int32_t* block_table, int32_t* free_blocks,
                                   const int32_t* free_count, int32_t* kv_lens_out,
                                   int32_t* free_count_out, int32_t* cu_new, int32_t* slot_map,
                                   int32_t max_new, void* ws, size_t ws_bytes, void* stream) {
  QCacheShape c;
  const kascade_status r =
      check_plan(cache, n_seqs, kv_lens, new_lens, block_table, free_blocks, free_count,
                 kv_lens_out, free_count_out, cu_new, slot_map, max_new, c);
  if (r != KASCADE_OK) return r;
  if (!check_small_ws(ws, ws_bytes)) return KASCADE_ERR_WORKSPACE;
  return run_qplan(c, n_seqs, kv_lens, new_lens, block_table, free_blocks, free_count,
                   kv_lens_out, free_count_out, cu_new, slot_map, max_new, ws,
                   static_cast<cudaStream_t>(stream));
}

kascade_status kascade_qcache_append(const kascade_qcache* cache, int32_t n_kv_heads,
                                     int32_t head_dim, int32_t dtype, const void* k,
                                     const void* v, const int64_t* strides,
                                     const int32_t* slot_map, int32_t n_tokens, void* pages,
                                     void* ws, size_t ws_bytes, void* stream) {
  QCacheShape c;
  const kascade_status r = check_rows(cache, n_kv_heads, head_dim, dtype, k, v, strides, slot_map,
                                      n_tokens, pages, c);
  if (r != KASCADE_OK) return r;
  if (!check_small_ws(ws, ws_bytes)) return KASCADE_ERR_WORKSPACE;
  QRowArgs a = row_args(c, n_kv_heads, head_dim, strides, slot_map, n_tokens, ws);
  a.src[0] = k;
  a.src[1] = v;
  a.cache = static_cast<uint8_t*>(pages);
  a.scale[0] = 1.f / c.k_scale;
  a.scale[1] = 1.f / c.v_scale;
  return status_of(launch_qappend(a, dtype, static_cast<cudaStream_t>(stream)));
}

kascade_status kascade_qcache_read(const kascade_qcache* cache, int32_t n_kv_heads,
                                   int32_t head_dim, int32_t dtype, const void* pages,
                                   const int32_t* slot_map, int32_t n_tokens, void* k, void* v,
                                   const int64_t* strides, void* ws, size_t ws_bytes,
                                   void* stream) {
  QCacheShape c;
  const kascade_status r = check_rows(cache, n_kv_heads, head_dim, dtype, k, v, strides, slot_map,
                                      n_tokens, pages, c);
  if (r != KASCADE_OK) return r;
  if (!check_small_ws(ws, ws_bytes)) return KASCADE_ERR_WORKSPACE;
  QRowArgs a = row_args(c, n_kv_heads, head_dim, strides, slot_map, n_tokens, ws);
  a.dst[0] = k;
  a.dst[1] = v;
  a.cache = const_cast<uint8_t*>(static_cast<const uint8_t*>(pages));
  a.scale[0] = c.k_scale;
  a.scale[1] = c.v_scale;
  return status_of(launch_qread(a, dtype, static_cast<cudaStream_t>(stream)));
}

kascade_status kascade_qcache_dense_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                           const void* q, const void* pages,
                                           const int32_t* block_table, const int32_t* kv_lens,
                                           void* out, float* scores_out, void* ws,
                                           size_t ws_bytes, void* stream) {
  QCall k;
  kascade_status r = check_call(desc, cache, k);
  if (r != KASCADE_OK) return r;
  if ((r = check_attn_ptrs(q, pages, block_table, kv_lens, out)) != KASCADE_OK) return r;
  if (scores_out != nullptr && !aligned(scores_out, 16)) return KASCADE_ERR_INVALID_ARG;
  if ((r = check_qws(k, 0, ws, ws_bytes)) != KASCADE_OK) return r;
  return run_qdense(k, q, pages, block_table, kv_lens, out, scores_out, true, nullptr, ws,
                    static_cast<cudaStream_t>(stream));
}

kascade_status kascade_qcache_anchor_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                            const void* q, const void* pages,
                                            const int32_t* block_table, const int32_t* kv_lens,
                                            int32_t topk, void* out, int32_t* idx_out,
                                            float* scores_out, void* ws, size_t ws_bytes,
                                            void* stream) {
  QCall k;
  kascade_status r = check_call(desc, cache, k);
  if (r != KASCADE_OK) return r;
  if ((r = check_attn_ptrs(q, pages, block_table, kv_lens, out)) != KASCADE_OK) return r;
  if (topk < 1 || topk > k.s.N || !aligned(idx_out, 16)) return KASCADE_ERR_INVALID_ARG;
  if (scores_out != nullptr && !aligned(scores_out, 16)) return KASCADE_ERR_INVALID_ARG;
  if ((r = check_qws(k, topk, ws, ws_bytes)) != KASCADE_OK) return r;
  return run_qanchor(k, q, pages, block_table, kv_lens, topk, out, idx_out, scores_out, ws,
                     static_cast<cudaStream_t>(stream));
}

kascade_status kascade_qcache_reuse_decode(const kascade_desc* desc, const kascade_qcache* cache,
                                           const void* q, const void* pages,
                                           const int32_t* block_table, const int32_t* kv_lens,
                                           int32_t topk, const int32_t* idx, void* out, void* ws,
                                           size_t ws_bytes, void* stream) {
  QCall k;
  kascade_status r = check_call(desc, cache, k);
  if (r != KASCADE_OK) return r;
  if ((r = check_attn_ptrs(q, pages, block_table, kv_lens, out)) != KASCADE_OK) return r;
  if (topk < 1 || topk > k.s.N || !aligned(idx, 4)) return KASCADE_ERR_INVALID_ARG;
  if ((r = check_qws(k, topk, ws, ws_bytes, true)) != KASCADE_OK) return r;
  return run_qreuse(k, q, pages, block_table, kv_lens, topk, idx, out, ws, false,
                    static_cast<cudaStream_t>(stream));
}

kascade_status kascade_qcache_run_stack(
    const kascade_desc* desc, const kascade_qcache* cache, const kascade_qcache_step* step,
    int32_t n_layers, const void* const* q, const void* const* k_new, const void* const* v_new,
    void* const* pages, int32_t topk, const int32_t* anchors, int32_t n_anchors, void* const* out,
    int32_t* idx_buf, void* ws, size_t ws_bytes, void* stream) {
  QCall k;
  kascade_status r = check_call(desc, cache, k);
  if (r != KASCADE_OK) return r;
  if (step == nullptr || n_layers < 1 || q == nullptr || pages == nullptr || out == nullptr ||
      (k_new == nullptr) != (v_new == nullptr))
    return KASCADE_ERR_INVALID_ARG;
  if (n_anchors < 0 || (n_anchors > 0 && anchors == nullptr)) return KASCADE_ERR_INVALID_ARG;
  for (int i = 0; i < n_anchors; ++i) {
    if (anchors[i] < 0 || anchors[i] >= n_layers) return KASCADE_ERR_INVALID_ARG;
    if (i > 0 && anchors[i] <= anchors[i - 1]) return KASCADE_ERR_INVALID_ARG;
  }
  if (n_anchors > 0 && (topk < 1 || topk > k.s.N || !aligned(idx_buf, 16)))
    return KASCADE_ERR_INVALID_ARG;
  for (int l = 0; l < n_layers; ++l)
    if ((r = check_attn_ptrs(q[l], pages[l], step->block_table, step->kv_lens, out[l])) !=
        KASCADE_OK)
      return r;
  QCacheShape c = k.c;
  if (step->new_lens != nullptr &&
      (r = check_plan(cache, k.s.B, step->kv_lens, step->new_lens, step->block_table,
                      step->free_blocks, step->free_count, step->kv_lens, step->free_count,
                      step->cu_new, step->slot_map, step->max_new, c)) != KASCADE_OK)
    return r;
  const int64_t strides[4] = {static_cast<int64_t>(k.s.Hkv) * k.s.d, k.s.d,
                              static_cast<int64_t>(k.s.Hkv) * k.s.d, k.s.d};
  if (k_new != nullptr)
    for (int l = 0; l < n_layers; ++l)
      if ((r = check_rows(cache, k.s.Hkv, k.s.d, k.s.dtype, k_new[l], v_new[l], strides,
                          step->slot_map, step->max_new, pages[l], c)) != KASCADE_OK)
        return r;
  const int tk = n_anchors > 0 ? topk : 0;
  if (tk > 0 && !k.s.pooled && decode_union_chunks(k.s.B * k.s.Hkv, k.s.N) > kMaxSplits)
    return KASCADE_ERR_UNSUPPORTED;
  if ((r = check_qws(k, tk, ws, ws_bytes)) != KASCADE_OK) return r;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (step->new_lens != nullptr) {
    r = run_qplan(c, k.s.B, step->kv_lens, step->new_lens, step->block_table, step->free_blocks,
                  step->free_count, step->kv_lens, step->free_count, step->cu_new, step->slot_map,
                  step->max_new, ws, st);
    if (r != KASCADE_OK) return r;
  }
  bool held = false;
  int next = 0;
  for (int l = 0; l < n_layers; ++l) {
    if (k_new != nullptr) {
      QRowArgs a = row_args(c, k.s.Hkv, k.s.d, strides, step->slot_map, step->max_new, ws);
      a.src[0] = k_new[l];
      a.src[1] = v_new[l];
      a.cache = static_cast<uint8_t*>(pages[l]);
      a.scale[0] = 1.f / c.k_scale;
      a.scale[1] = 1.f / c.v_scale;
      if ((r = status_of(launch_qappend(a, k.s.dtype, st))) != KASCADE_OK) return r;
    }
    const bool is_anchor = next < n_anchors && anchors[next] == l;
    if (is_anchor) {
      ++next;
      r = run_qanchor(k, q[l], pages[l], step->block_table, step->kv_lens, tk, out[l], idx_buf,
                      nullptr, ws, st);
      // one union plan for every reuse layer of this anchor
      if (r == KASCADE_OK && !k.s.pooled)
        r = run_qplan_sets(k, step->kv_lens, idx_buf, tk, ws, st);
      held = true;
    } else if (held) {
      r = run_qreuse(k, q[l], pages[l], step->block_table, step->kv_lens, tk, idx_buf, out[l], ws,
                     true, st);
    } else {
      r = run_qdense(k, q[l], pages[l], step->block_table, step->kv_lens, out[l], nullptr, false,
                     nullptr, ws, st);
    }
    if (r != KASCADE_OK) return r;
  }
  return KASCADE_OK;
}

}  // extern "C"
