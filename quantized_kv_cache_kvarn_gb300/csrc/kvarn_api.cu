// extern "C" boundary of libkvarn: argument validation on the host, then the
// launches. Declarations and the contract of every call are in kvarn.h.
#include <cuda_runtime.h>

#include <algorithm>

#include "../../include/kvarn.h"
#include "kvarn_common.cuh"
#include "kvarn_launch.h"

using namespace kvarn;

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int32_t from_cuda(cudaError_t e) { return e == cudaSuccess ? KVARN_OK : KVARN_ECUDA; }

// Dense layout with a compiled codec variant.
int32_t check_dense(const kvarn_layout* L) {
  if (!L) return KVARN_EINVAL;
  if (L->page_tokens != kPageTokens) return KVARN_EUNSUPPORTED;
  if (L->head_dim != 128 && L->head_dim != 256) return KVARN_EUNSUPPORTED;
  if (L->tile_tokens != 128 && L->tile_tokens != 64) return KVARN_EUNSUPPORTED;
  if (L->scale_dtype != 0 && L->scale_dtype != 1) return KVARN_EUNSUPPORTED;
  if (!widths_supported(L->head_dim, L->k_bits, L->v_bits, L->scale_dtype == 1 ? 2 : 4))
    return KVARN_EUNSUPPORTED;
  if (L->norm_iters < 1 || L->norm_iters > 8) return KVARN_EUNSUPPORTED;
  if (L->rope_dim != 0) return KVARN_EINVAL;
  if (L->kv_dtype != 0 && L->kv_dtype != 1) return KVARN_EUNSUPPORTED;
  if (L->num_kv_heads < 1 || L->num_pages < 0) return KVARN_EINVAL;
  return KVARN_OK;
}

int32_t check_latent(const kvarn_layout* L) {
  if (!L) return KVARN_EINVAL;
  if (L->page_tokens != kPageTokens || L->head_dim != 512 || L->tile_tokens != 128 ||
      L->k_bits != 4 || L->v_bits != 0 || L->rope_dim != 64 || L->num_kv_heads != 1)
    return KVARN_EUNSUPPORTED;
  if (L->norm_iters < 1 || L->norm_iters > 8) return KVARN_EUNSUPPORTED;
  if (L->kv_dtype != 0 && L->kv_dtype != 1) return KVARN_EUNSUPPORTED;
  if (L->num_pages < 0) return KVARN_EINVAL;
  return KVARN_OK;
}

bool is_latent(const kvarn_layout* L) { return L && L->head_dim == 512 && L->rope_dim > 0; }

// Layout of the affine comparison codec: head_dim 128, 128-token tiles of
// 16-token pages, equal key and value widths from {2, 3, 4, 6, 8}.
int32_t check_affine(const kvarn_layout* L) {
  if (!L) return KVARN_EINVAL;
  if (L->page_tokens != kPageTokens || L->head_dim != 128 || L->tile_tokens != 128 || L->rope_dim != 0)
    return KVARN_EUNSUPPORTED;
  if (L->k_bits != L->v_bits || !affine_width_compiled(L->k_bits)) return KVARN_EUNSUPPORTED;
  if (L->kv_dtype != 0 && L->kv_dtype != 1) return KVARN_EUNSUPPORTED;
  if (L->num_kv_heads < 1 || L->num_pages < 0) return KVARN_EINVAL;
  return KVARN_OK;
}

// Layout of the 8-bit block cache: blocks of one page.
int32_t check_q8(const kvarn_layout* L) {
  if (!L) return KVARN_EINVAL;
  if (L->page_tokens != kPageTokens || L->tile_tokens != kPageTokens || L->k_bits != 8 || L->v_bits != 8 ||
      (L->head_dim != 128 && L->head_dim != 256) || L->rope_dim != 0)
    return KVARN_EUNSUPPORTED;
  if (L->kv_dtype != 0 && L->kv_dtype != 1) return KVARN_EUNSUPPORTED;
  if (L->num_kv_heads < 1 || L->num_pages < 0) return KVARN_EINVAL;
  return KVARN_OK;
}

int32_t check_q8(const kvarn_layout* L, int32_t code) {
  const int32_t s = check_q8(L);
  if (s != KVARN_OK) return s;
  return code == KVARN_Q8_E4M3 || code == KVARN_Q8_INT8 ? KVARN_OK : KVARN_EUNSUPPORTED;
}

}  // namespace

extern "C" {

int32_t kvarn_version(void) { return 100; }

const char* kvarn_status_string(int32_t s) {
  switch (s) {
    case KVARN_OK: return "ok";
    case KVARN_EINVAL: return "invalid argument";
    case KVARN_EUNSUPPORTED: return "unsupported shape or width";
    case KVARN_EALIGN: return "misaligned pointer or stride";
    case KVARN_ECUDA: return "CUDA runtime error";
    case KVARN_EWORKSPACE: return "workspace too small";
    default: return "unknown status";
  }
}

int32_t kvarn_layout_check(const kvarn_layout* L) {
  return is_latent(L) ? check_latent(L) : check_dense(L);
}

int64_t kvarn_page_bytes(const kvarn_layout* L) {
  if (kvarn_layout_check(L) != KVARN_OK) return -1;
  if (is_latent(L)) return LatentPage(L->head_dim, L->rope_dim, L->tile_tokens).bytes();
  return DensePage(L->head_dim, L->tile_tokens, L->k_bits, L->v_bits, L->scale_dtype == 1 ? 2 : 4).bytes();
}

// The k4v2 preset with fp32 scales: the page format of the append, fp16
// bypass and no-allocation paths.
static bool is_preset(const kvarn_layout* L) {
  return L->k_bits == 4 && L->v_bits == 2 && L->scale_dtype == 0;
}

static int32_t encode_tiles(const void* k, const void* v, int64_t seq_stride, int64_t head_stride,
                            int32_t num_seqs, int32_t chunk_tokens, const int32_t* tile_start,
                            const int32_t* block_table, int32_t bt_stride, const kvarn_layout* L,
                            void* cache, float* stages, uint32_t* error_flags, kvarn_stream_t stream,
                            bool affine = false) {
  int32_t s = affine ? check_affine(L) : check_dense(L);
  if (s != KVARN_OK) return s;
  if (num_seqs < 0 || chunk_tokens < 0 || chunk_tokens % L->tile_tokens) return KVARN_EINVAL;
  if (num_seqs == 0 || chunk_tokens == 0) return KVARN_OK;
  if (!k || !v || !tile_start || !block_table || !cache || !error_flags) return KVARN_EINVAL;
  if (seq_stride < 0 || head_stride < 0 || bt_stride < 1) return KVARN_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || seq_stride % 8 || head_stride % 8) return KVARN_EALIGN;
  if (!aligned(cache, 128) || !aligned(error_flags, 4)) return KVARN_EALIGN;
  EncodeParams p{};
  p.k = k;
  p.v = v;
  p.seq_stride = seq_stride;
  p.head_stride = head_stride;
  p.num_seqs = num_seqs;
  p.chunk_tokens = chunk_tokens;
  p.tile_start = tile_start;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.cache = cache;
  p.num_pages = L->num_pages;
  p.num_kv_heads = L->num_kv_heads;
  p.D = L->head_dim;
  p.N = L->tile_tokens;
  p.norm_iters = L->norm_iters;
  p.bf16 = L->kv_dtype == 1;
  p.err = error_flags;
  p.k_bits = L->k_bits;
  p.v_bits = L->v_bits;
  p.scale_bytes = L->scale_dtype == 1 ? 2 : 4;
  p.stages = stages;
  if (affine) return from_cuda(launch_encode_affine(p, reinterpret_cast<cudaStream_t>(stream)));
  return from_cuda(launch_encode_dense(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_encode_tiles(const void* k, const void* v, int64_t seq_stride, int64_t head_stride,
                           int32_t num_seqs, int32_t chunk_tokens, const int32_t* tile_start,
                           const int32_t* block_table, int32_t bt_stride,
                           const kvarn_layout* L, void* cache, uint32_t* error_flags,
                           kvarn_stream_t stream) {
  return encode_tiles(k, v, seq_stride, head_stride, num_seqs, chunk_tokens, tile_start, block_table,
                      bt_stride, L, cache, nullptr, error_flags, stream);
}

int64_t kvarn_encode_stage_floats(const kvarn_layout* L, int32_t num_seqs, int32_t chunk_tokens) {
  if (check_dense(L) != KVARN_OK || num_seqs < 0 || chunk_tokens < 0 || chunk_tokens % L->tile_tokens)
    return -1;
  return static_cast<int64_t>(num_seqs) * L->num_kv_heads * (chunk_tokens / L->tile_tokens) * 2 *
         stage_floats(L->head_dim, L->tile_tokens);
}

int32_t kvarn_encode_tiles_staged(const void* k, const void* v, int64_t seq_stride, int64_t head_stride,
                                  int32_t num_seqs, int32_t chunk_tokens, const int32_t* tile_start,
                                  const int32_t* block_table, int32_t bt_stride,
                                  const kvarn_layout* L, void* cache, float* stages,
                                  uint32_t* error_flags, kvarn_stream_t stream) {
  if (!stages) return KVARN_EINVAL;
  if (!aligned(stages, 16)) return KVARN_EALIGN;
  return encode_tiles(k, v, seq_stride, head_stride, num_seqs, chunk_tokens, tile_start, block_table,
                      bt_stride, L, cache, stages, error_flags, stream);
}

// max_seq_len here: the accepted length bound (sizes the tile splits); raw_max:
// raw (sink + tail) tokens a row may see (sizes the raw splits).
static DensePlan dense_plan(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                            int32_t num_queries, int32_t max_seq_len, int32_t raw_max, bool affine = false) {
  const int32_t G = num_q_heads / L->num_kv_heads;
  if (affine)
    return plan_dense_stream(num_seqs, L->num_kv_heads * row_groups(G, num_queries), max_seq_len / L->tile_tokens,
                             L->head_dim, L->tile_tokens, raw_max, L->k_bits, L->v_bits, 2,
                             affine_decode_ctas_per_sm(L->k_bits));
  return plan_dense_stream(num_seqs, L->num_kv_heads * row_groups(G, num_queries), max_seq_len / L->tile_tokens,
                           L->head_dim, L->tile_tokens, raw_max, L->k_bits ? L->k_bits : 4, L->v_bits ? L->v_bits : 2,
                           L->scale_dtype == 1 ? 2 : 4);
}

// Plan of the decode over uncompressed fp16 pages: 32-token tiles, the last
// one partial, no raw records.
static DensePlan fp16_plan(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads, int32_t max_seq_len) {
  const int32_t G = num_q_heads / L->num_kv_heads;
  return plan_dense_stream(num_seqs, L->num_kv_heads * row_groups(G, 1), (max_seq_len + 31) / 32, L->head_dim, 32, 0,
                           4, 2, 4, raw_decode_ctas_per_sm(L->head_dim));
}

static int64_t dense_ws(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads, int32_t num_queries,
                        const DensePlan& plan) {
  return dense_stream_workspace_bytes(static_cast<int64_t>(num_seqs) * num_q_heads * num_queries, L->head_dim, plan);
}

// Raw tokens a row can see: at most the sequence, and at most the sink, the
// newest records, a partial tile and the tokens under verification.
static int32_t raw_bound(const kvarn_layout* L, int32_t max_seq_len, int32_t num_queries, int32_t sink,
                         int32_t recent) {
  const int64_t r = static_cast<int64_t>(sink) + recent + L->tile_tokens + num_queries - 2;
  return static_cast<int32_t>(std::min<int64_t>(std::max(0, max_seq_len), std::max<int64_t>(0, r)));
}

int32_t kvarn_append(const void* k, const void* v, const int32_t* seq_lens, int32_t max_seq_len,
                     void* tail_k, void* tail_v, int32_t num_seqs, const int32_t* block_table,
                     int32_t bt_stride, const kvarn_layout* L, void* cache, uint32_t* error_flags,
                     kvarn_stream_t stream) {
  int32_t s = check_dense(L);
  if (s != KVARN_OK) return s;
  if (!is_preset(L)) return KVARN_EUNSUPPORTED;
  if (num_seqs < 0 || max_seq_len < 0) return KVARN_EINVAL;
  if (num_seqs == 0) return KVARN_OK;
  if (!k || !v || !seq_lens || !tail_k || !tail_v || !block_table || !cache || !error_flags || bt_stride < 1)
    return KVARN_EINVAL;
  if (bt_stride < (max_seq_len / L->tile_tokens) * (L->tile_tokens / kPageTokens)) return KVARN_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(tail_k, 16) || !aligned(tail_v, 16)) return KVARN_EALIGN;
  if (!aligned(cache, 128) || !aligned(error_flags, 4)) return KVARN_EALIGN;
  AppendParams p{};
  p.k = k;
  p.v = v;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.tail_k = tail_k;
  p.tail_v = tail_v;
  p.num_seqs = num_seqs;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.cache = cache;
  p.num_pages = L->num_pages;
  p.num_kv_heads = L->num_kv_heads;
  p.D = L->head_dim;
  p.N = L->tile_tokens;
  p.norm_iters = L->norm_iters;
  p.bf16 = L->kv_dtype == 1;
  p.err = error_flags;
  return from_cuda(launch_append_commit(p, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t kvarn_decode_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                     int32_t max_seq_len) {
  if (kvarn_layout_check(L) != KVARN_OK || num_seqs < 0 || num_q_heads < 1 || max_seq_len < 0)
    return -1;
  if (is_latent(L)) return mla_workspace_bytes(num_seqs, num_q_heads, plan_mla(num_seqs, max_seq_len));
  if (num_q_heads % L->num_kv_heads) return -1;
  const DensePlan plan = dense_plan(L, num_seqs, num_q_heads, 1, max_seq_len, raw_bound(L, max_seq_len, 1, 0, 0));
  int64_t ws16 = 0;
  if (L->head_dim == 128 || L->head_dim == 256)
    ws16 = dense_stream_workspace_bytes(static_cast<int64_t>(num_seqs) * num_q_heads, L->head_dim,
                                        fp16_plan(L, num_seqs, num_q_heads, max_seq_len));
  return std::max(dense_ws(L, num_seqs, num_q_heads, 1, plan), ws16);
}

int64_t kvarn_decode_window_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                            int32_t num_queries, int32_t max_seq_len, int32_t sink_tokens,
                                            int32_t recent_tokens) {
  if (kvarn_layout_check(L) != KVARN_OK || is_latent(L) || num_seqs < 0 || num_q_heads < 1 ||
      max_seq_len < 0 || num_queries < 1 || num_queries > KVARN_MAX_VERIFY_QUERIES ||
      num_q_heads % L->num_kv_heads || sink_tokens < 0 || recent_tokens < 0)
    return -1;
  const DensePlan plan =
      dense_plan(L, num_seqs, num_q_heads, num_queries, std::max(0, max_seq_len - num_queries + 1),
                 raw_bound(L, max_seq_len, num_queries, sink_tokens, recent_tokens));
  return dense_ws(L, num_seqs, num_q_heads, num_queries, plan);
}

int64_t kvarn_decode_verify_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                            int32_t num_queries, int32_t max_seq_len) {
  return kvarn_decode_window_workspace_bytes(L, num_seqs, num_q_heads, num_queries, max_seq_len, 0, 0);
}

static int32_t check_decode_common(const kvarn_layout* L, int32_t num_q_heads,
                                   const int32_t* block_table, int32_t bt_stride,
                                   const int32_t* seq_lens, int32_t max_seq_len, int32_t num_seqs,
                                   float* out, void* workspace, uint32_t* error_flags) {
  if (num_seqs < 0 || max_seq_len < 0 || num_q_heads < 1) return KVARN_EINVAL;
  if (num_seqs == 0) return KVARN_OK;
  if (!block_table || !seq_lens || !out || !workspace || !error_flags) return KVARN_EINVAL;
  if (num_q_heads % L->num_kv_heads) return KVARN_EINVAL;
  if (!aligned(out, 16) || !aligned(workspace, 16)) return KVARN_EALIGN;
  (void)bt_stride;
  return KVARN_OK;
}

// The tile masses of kvarn_decode_mass.
struct MassArgs {
  const float* in;
  float* out;
  int32_t stride;
  float decay;
};

static int32_t decode_dense_common(const void* q, int32_t num_q_heads, int32_t num_queries, float sm_scale,
                                   const void* cache, const kvarn_layout* L, const int32_t* block_table,
                                   int32_t bt_stride, const int32_t* seq_lens, int32_t max_seq_len,
                                   const void* tail_k, const void* tail_v, int32_t tail_cap,
                                   int32_t sink_tokens, const void* sink_k, const void* sink_v,
                                   int32_t recent_tokens, int32_t num_seqs, float* out, float* lse,
                                   void* workspace, int64_t workspace_bytes, uint32_t* error_flags,
                                   kvarn_stream_t stream, bool affine = false, const MassArgs* mass = nullptr) {
  int32_t s = affine ? check_affine(L) : check_dense(L);
  if (s != KVARN_OK) return s;
  s = check_decode_common(L, num_q_heads, block_table, bt_stride, seq_lens, max_seq_len, num_seqs,
                          out, workspace, error_flags);
  if (s != KVARN_OK || num_seqs == 0) return s;
  if (!q || !cache) return KVARN_EINVAL;
  if (num_q_heads / L->num_kv_heads > 8) return KVARN_EUNSUPPORTED;
  // committed tiles: those filled by the accepted tokens [0, len - Q + 1),
  // less the newest recent_tokens, never before the sink
  const int32_t accepted = std::max(0, max_seq_len - num_queries + 1);
  const int32_t end = std::max(sink_tokens, (std::max(0, accepted - recent_tokens) / L->tile_tokens) *
                                                L->tile_tokens);
  const int32_t committed_pages = end > sink_tokens ? end / kPageTokens : 0;
  if (bt_stride < committed_pages) return KVARN_EINVAL;
  if (!aligned(q, 16) || !aligned(cache, 128)) return KVARN_EALIGN;
  if ((tail_k && !aligned(tail_k, 16)) || (tail_v && !aligned(tail_v, 16))) return KVARN_EALIGN;
  if ((sink_k && !aligned(sink_k, 16)) || (sink_v && !aligned(sink_v, 16))) return KVARN_EALIGN;
  const DensePlan plan = dense_plan(L, num_seqs, num_q_heads, num_queries, accepted,
                                    raw_bound(L, max_seq_len, num_queries, sink_tokens, recent_tokens), affine);
  int64_t need = dense_ws(L, num_seqs, num_q_heads, num_queries, plan);
  if (mass) need += mass_workspace_bytes(static_cast<int64_t>(num_seqs) * num_q_heads, max_seq_len / L->tile_tokens);
  if (workspace_bytes < need) return KVARN_EWORKSPACE;
  DecodeParams p{};
  p.q = q;
  p.num_q_heads = num_q_heads;
  p.sm_scale = sm_scale;
  p.cache = static_cast<const uint8_t*>(cache);
  p.D = L->head_dim;
  p.N = L->tile_tokens;
  p.num_kv_heads = L->num_kv_heads;
  p.num_pages = L->num_pages;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.tail_k = tail_k;
  p.tail_v = tail_v;
  p.num_seqs = num_seqs;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  p.err = error_flags;
  p.bf16 = L->kv_dtype == 1;
  p.num_queries = num_queries;
  p.tail_cap = tail_cap;
  p.sink_tokens = sink_tokens;
  p.sink_k = sink_k;
  p.sink_v = sink_v;
  p.recent_tokens = recent_tokens;
  p.k_bits = L->k_bits;
  p.v_bits = L->v_bits;
  p.scale_bytes = affine ? 2 : (L->scale_dtype == 1 ? 2 : 4);
  p.codec = affine ? 1 : 0;
  if (mass) {
    p.mass_in = mass->in;
    p.mass_out = mass->out;
    p.mass_stride = mass->stride;
    p.mass_decay = mass->decay;
  }
  return from_cuda(launch_decode_dense(p, plan, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_decode(const void* q, int32_t num_q_heads, float sm_scale, const void* cache,
                     const kvarn_layout* L, const int32_t* block_table, int32_t bt_stride,
                     const int32_t* seq_lens, int32_t max_seq_len, const void* tail_k,
                     const void* tail_v, int32_t num_seqs, float* out, float* lse,
                     void* workspace, int64_t workspace_bytes, uint32_t* error_flags,
                     kvarn_stream_t stream) {
  if (!L) return KVARN_EINVAL;
  return decode_dense_common(q, num_q_heads, 1, sm_scale, cache, L, block_table, bt_stride, seq_lens,
                             max_seq_len, tail_k, tail_v, L->tile_tokens, 0, nullptr, nullptr, 0, num_seqs,
                             out, lse, workspace, workspace_bytes, error_flags, stream);
}

int32_t kvarn_decode_verify(const void* q, int32_t num_q_heads, int32_t num_queries, float sm_scale,
                            const void* cache, const kvarn_layout* L, const int32_t* block_table,
                            int32_t bt_stride, const int32_t* seq_lens, int32_t max_seq_len,
                            const void* tail_k, const void* tail_v, int32_t tail_capacity,
                            int32_t num_seqs, float* out, float* lse, void* workspace,
                            int64_t workspace_bytes, uint32_t* error_flags, kvarn_stream_t stream) {
  if (!L) return KVARN_EINVAL;
  if (num_queries < 1 || num_queries > KVARN_MAX_VERIFY_QUERIES) return KVARN_EUNSUPPORTED;
  if (tail_capacity < L->tile_tokens + num_queries - 2 || tail_capacity < 1) return KVARN_EINVAL;
  return decode_dense_common(q, num_q_heads, num_queries, sm_scale, cache, L, block_table, bt_stride,
                             seq_lens, max_seq_len, tail_k, tail_v, tail_capacity, 0, nullptr, nullptr, 0,
                             num_seqs, out, lse, workspace, workspace_bytes, error_flags, stream);
}

int32_t kvarn_decode_window(const void* q, int32_t num_q_heads, int32_t num_queries, float sm_scale,
                            const void* cache, const kvarn_layout* L, const int32_t* block_table,
                            int32_t bt_stride, const int32_t* seq_lens, int32_t max_seq_len,
                            int32_t sink_tokens, const void* sink_k, const void* sink_v,
                            int32_t recent_tokens, const void* tail_k, const void* tail_v,
                            int32_t tail_capacity, int32_t num_seqs, float* out, float* lse,
                            void* workspace, int64_t workspace_bytes, uint32_t* error_flags,
                            kvarn_stream_t stream) {
  if (!L) return KVARN_EINVAL;
  if (num_queries < 1 || num_queries > KVARN_MAX_VERIFY_QUERIES) return KVARN_EUNSUPPORTED;
  if (L->tile_tokens < 1 || sink_tokens < 0 || sink_tokens % L->tile_tokens || recent_tokens < 0)
    return KVARN_EINVAL;
  if (tail_capacity < 1 || static_cast<int64_t>(tail_capacity) <
                               static_cast<int64_t>(recent_tokens) + L->tile_tokens + num_queries - 2)
    return KVARN_EINVAL;
  return decode_dense_common(q, num_q_heads, num_queries, sm_scale, cache, L, block_table, bt_stride,
                             seq_lens, max_seq_len, tail_k, tail_v, tail_capacity, sink_tokens, sink_k,
                             sink_v, recent_tokens, num_seqs, out, lse, workspace, workspace_bytes,
                             error_flags, stream);
}

int64_t kvarn_fp16_page_bytes(const kvarn_layout* L) {
  if (!L || (L->head_dim != 128 && L->head_dim != 256) || L->page_tokens != kPageTokens) return -1;
  return 4LL * kPageTokens * L->head_dim;
}

int32_t kvarn_store_fp16(const void* k, const void* v, int64_t seq_stride, int64_t head_stride,
                         int32_t num_seqs, int32_t token0, int32_t count,
                         const int32_t* block_table, int32_t bt_stride, const kvarn_layout* L,
                         void* cache, uint32_t* error_flags, kvarn_stream_t stream) {
  if (kvarn_fp16_page_bytes(L) < 0) return KVARN_EUNSUPPORTED;
  if (L->kv_dtype != 0) return KVARN_EUNSUPPORTED;
  if (num_seqs < 0 || token0 < 0 || count < 0 || token0 % kPageTokens || count % kPageTokens)
    return KVARN_EINVAL;
  if (num_seqs == 0 || count == 0) return KVARN_OK;
  if (!k || !v || !block_table || !cache || !error_flags || bt_stride < 1 || L->num_kv_heads < 1)
    return KVARN_EINVAL;
  if (!aligned(cache, 128) || !aligned(k, 4) || !aligned(v, 4)) return KVARN_EALIGN;
  StoreFp16Params p{};
  p.k = k;
  p.v = v;
  p.seq_stride = seq_stride;
  p.head_stride = head_stride;
  p.num_seqs = num_seqs;
  p.token0 = token0;
  p.count = count;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.cache = cache;
  p.num_pages = L->num_pages;
  p.num_kv_heads = L->num_kv_heads;
  p.D = L->head_dim;
  p.err = error_flags;
  return from_cuda(launch_store_fp16(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_decode_fp16(const void* q, int32_t num_q_heads, float sm_scale, const void* cache,
                          const kvarn_layout* L, const int32_t* block_table, int32_t bt_stride,
                          const int32_t* seq_lens, int32_t max_seq_len, int32_t num_seqs,
                          float* out, float* lse, void* workspace, int64_t workspace_bytes,
                          uint32_t* error_flags, kvarn_stream_t stream) {
  if (kvarn_fp16_page_bytes(L) < 0 || L->kv_dtype != 0) return KVARN_EUNSUPPORTED;
  if (L->num_kv_heads < 1 || L->num_pages < 0) return KVARN_EINVAL;
  int32_t s = check_decode_common(L, num_q_heads, block_table, bt_stride, seq_lens, max_seq_len,
                                  num_seqs, out, workspace, error_flags);
  if (s != KVARN_OK || num_seqs == 0) return s;
  if (!q || !cache) return KVARN_EINVAL;
  if (num_q_heads / L->num_kv_heads > 8) return KVARN_EUNSUPPORTED;
  if (bt_stride < (max_seq_len + kPageTokens - 1) / kPageTokens) return KVARN_EINVAL;
  if (!aligned(q, 16) || !aligned(cache, 128)) return KVARN_EALIGN;
  const DensePlan plan = fp16_plan(L, num_seqs, num_q_heads, max_seq_len);
  if (workspace_bytes < dense_stream_workspace_bytes(static_cast<int64_t>(num_seqs) * num_q_heads, L->head_dim, plan))
    return KVARN_EWORKSPACE;
  DecodeParams p{};
  p.q = q;
  p.num_q_heads = num_q_heads;
  p.sm_scale = sm_scale;
  p.cache = static_cast<const uint8_t*>(cache);
  p.D = L->head_dim;
  p.N = 32;
  p.num_kv_heads = L->num_kv_heads;
  p.num_pages = L->num_pages;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.num_seqs = num_seqs;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  p.err = error_flags;
  p.num_queries = 1;
  p.tail_cap = 32;
  p.codec = 2;
  return from_cuda(launch_decode_dense(p, plan, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_encode_latent(const void* latent, int64_t seq_stride, const void* rope,
                            int64_t rope_seq_stride, int32_t num_seqs, int32_t chunk_tokens,
                            const int32_t* tile_start, const int32_t* block_table,
                            int32_t bt_stride, const kvarn_layout* L, void* cache,
                            uint32_t* error_flags, kvarn_stream_t stream) {
  int32_t s = check_latent(L);
  if (s != KVARN_OK) return s;
  if (num_seqs < 0 || chunk_tokens < 0 || chunk_tokens % L->tile_tokens) return KVARN_EINVAL;
  if (num_seqs == 0 || chunk_tokens == 0) return KVARN_OK;
  if (!latent || !rope || !tile_start || !block_table || !cache || !error_flags || bt_stride < 1)
    return KVARN_EINVAL;
  if (seq_stride < 0 || rope_seq_stride < 0) return KVARN_EINVAL;
  if (!aligned(latent, 16) || !aligned(rope, 16) || seq_stride % 8 || rope_seq_stride % 8)
    return KVARN_EALIGN;
  if (!aligned(cache, 128)) return KVARN_EALIGN;
  EncodeLatentParams p{};
  p.latent = latent;
  p.seq_stride = seq_stride;
  p.rope = rope;
  p.rope_seq_stride = rope_seq_stride;
  p.num_seqs = num_seqs;
  p.chunk_tokens = chunk_tokens;
  p.tile_start = tile_start;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.cache = cache;
  p.num_pages = L->num_pages;
  p.norm_iters = L->norm_iters;
  p.bf16 = L->kv_dtype == 1;
  p.err = error_flags;
  return from_cuda(launch_encode_latent(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_decode_mla(const void* q_latent, const void* q_rope, int32_t num_heads,
                         float sm_scale, const void* cache, const kvarn_layout* L,
                         const int32_t* block_table, int32_t bt_stride, const int32_t* seq_lens,
                         int32_t max_seq_len, const void* tail_latent, const void* tail_rope,
                         int32_t num_seqs, float* out, float* lse, void* workspace,
                         int64_t workspace_bytes, uint32_t* error_flags, kvarn_stream_t stream) {
  int32_t s = check_latent(L);
  if (s != KVARN_OK) return s;
  s = check_decode_common(L, num_heads, block_table, bt_stride, seq_lens, max_seq_len, num_seqs, out,
                          workspace, error_flags);
  if (s != KVARN_OK || num_seqs == 0) return s;
  if (!q_latent || !q_rope || !cache) return KVARN_EINVAL;
  if (num_heads % 16 || num_heads > 128) return KVARN_EUNSUPPORTED;
  if (bt_stride < (max_seq_len / L->tile_tokens) * (L->tile_tokens / kPageTokens)) return KVARN_EINVAL;
  if (!aligned(q_latent, 16) || !aligned(q_rope, 16) || !aligned(cache, 128)) return KVARN_EALIGN;
  if ((tail_latent && !aligned(tail_latent, 16)) || (tail_rope && !aligned(tail_rope, 16)))
    return KVARN_EALIGN;
  const SplitPlan plan = plan_mla(num_seqs, max_seq_len);
  if (workspace_bytes < mla_workspace_bytes(num_seqs, num_heads, plan)) return KVARN_EWORKSPACE;
  DecodeParams p{};
  p.q = q_latent;
  p.q_rope = q_rope;
  p.num_q_heads = num_heads;
  p.sm_scale = sm_scale;
  p.cache = static_cast<const uint8_t*>(cache);
  p.D = 512;
  p.N = L->tile_tokens;
  p.num_kv_heads = 1;
  p.num_pages = L->num_pages;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.tail_k = tail_latent;
  p.tail_v = tail_rope;
  p.num_seqs = num_seqs;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  p.err = error_flags;
  p.bf16 = L->kv_dtype == 1;
  return from_cuda(launch_decode_mla(p, plan, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t kvarn_affine_page_bytes(const kvarn_layout* L) {
  if (check_affine(L) != KVARN_OK) return -1;
  return AffinePage(L->head_dim, L->k_bits, L->v_bits).bytes();
}

int32_t kvarn_affine_encode_tiles(const void* k, const void* v, int64_t seq_stride, int64_t head_stride,
                                  int32_t num_seqs, int32_t chunk_tokens, const int32_t* tile_start,
                                  const int32_t* block_table, int32_t bt_stride, const kvarn_layout* L,
                                  void* cache, uint32_t* error_flags, kvarn_stream_t stream) {
  return encode_tiles(k, v, seq_stride, head_stride, num_seqs, chunk_tokens, tile_start, block_table, bt_stride, L,
                      cache, nullptr, error_flags, stream, true);
}

int64_t kvarn_affine_decode_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                            int32_t max_seq_len) {
  if (check_affine(L) != KVARN_OK || num_seqs < 0 || num_q_heads < 1 || max_seq_len < 0 ||
      num_q_heads % L->num_kv_heads)
    return -1;
  const DensePlan plan =
      dense_plan(L, num_seqs, num_q_heads, 1, max_seq_len, raw_bound(L, max_seq_len, 1, 0, 0), true);
  return dense_ws(L, num_seqs, num_q_heads, 1, plan);
}

int32_t kvarn_affine_decode(const void* q, int32_t num_q_heads, float sm_scale, const void* cache,
                            const kvarn_layout* L, const int32_t* block_table, int32_t bt_stride,
                            const int32_t* seq_lens, int32_t max_seq_len, const void* tail_k,
                            const void* tail_v, int32_t num_seqs, float* out, float* lse, void* workspace,
                            int64_t workspace_bytes, uint32_t* error_flags, kvarn_stream_t stream) {
  if (!L) return KVARN_EINVAL;
  return decode_dense_common(q, num_q_heads, 1, sm_scale, cache, L, block_table, bt_stride, seq_lens,
                             max_seq_len, tail_k, tail_v, L->tile_tokens, 0, nullptr, nullptr, 0, num_seqs,
                             out, lse, workspace, workspace_bytes, error_flags, stream, true);
}

static int32_t check_mass(const kvarn_layout* L) {
  const int32_t s = check_dense(L);
  if (s != KVARN_OK) return s;
  return mass_widths_supported(L->k_bits, L->v_bits, L->scale_dtype == 1 ? 2 : 4) ? KVARN_OK : KVARN_EUNSUPPORTED;
}

int64_t kvarn_decode_mass_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                          int32_t max_seq_len) {
  if (check_mass(L) != KVARN_OK || num_seqs < 0 || num_q_heads < 1 || max_seq_len < 0 ||
      num_q_heads % L->num_kv_heads)
    return -1;
  const DensePlan plan = dense_plan(L, num_seqs, num_q_heads, 1, max_seq_len, raw_bound(L, max_seq_len, 1, 0, 0));
  return dense_ws(L, num_seqs, num_q_heads, 1, plan) +
         mass_workspace_bytes(static_cast<int64_t>(num_seqs) * num_q_heads, max_seq_len / L->tile_tokens);
}

int32_t kvarn_decode_mass(const void* q, int32_t num_q_heads, float sm_scale, const void* cache,
                          const kvarn_layout* L, const int32_t* block_table, int32_t bt_stride,
                          const int32_t* seq_lens, int32_t max_seq_len, const void* tail_k, const void* tail_v,
                          int32_t num_seqs, float* out, float* lse, const float* mass_in, float* mass_out,
                          int32_t mass_stride, float decay, void* workspace, int64_t workspace_bytes,
                          uint32_t* error_flags, kvarn_stream_t stream) {
  if (!L) return KVARN_EINVAL;
  const int32_t s = check_mass(L);
  if (s != KVARN_OK) return s;
  if (num_seqs > 0) {
    const int32_t tiles = std::max(0, max_seq_len) / L->tile_tokens;
    if (tiles > 0 && (!mass_in || !mass_out || mass_stride < tiles)) return KVARN_EINVAL;
    if (!(decay >= 0.f && decay <= 1.f)) return KVARN_EINVAL;
    if (!aligned(mass_in, 4) || !aligned(mass_out, 4)) return KVARN_EALIGN;
    if (num_seqs > 65535) return KVARN_EUNSUPPORTED;
  }
  // without a committed tile there is no mass to write
  const MassArgs m{mass_in, mass_out, mass_stride, decay};
  return decode_dense_common(q, num_q_heads, 1, sm_scale, cache, L, block_table, bt_stride, seq_lens, max_seq_len,
                             tail_k, tail_v, L->tile_tokens, 0, nullptr, nullptr, 0, num_seqs, out, lse, workspace,
                             workspace_bytes, error_flags, stream, false, &m);
}

// Plan of a decode over a shared prefix (whole tiles) and the tokens past it.
static SharedPlan shared_plan(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads, int32_t num_queries,
                              int32_t max_seq_len, int32_t prefix_tokens) {
  const int32_t own = std::max(0, max_seq_len - num_queries + 1 - prefix_tokens);
  return plan_shared(num_seqs, L->num_kv_heads, num_q_heads / L->num_kv_heads, num_queries,
                     prefix_tokens / L->tile_tokens, own / L->tile_tokens, L->head_dim, L->tile_tokens,
                     raw_bound(L, std::max(0, max_seq_len - prefix_tokens), num_queries, 0, 0), L->k_bits, L->v_bits,
                     L->scale_dtype == 1 ? 2 : 4);
}

static bool shared_sizes_ok(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads, int32_t num_queries,
                            int32_t max_seq_len, int32_t prefix_tokens) {
  return num_seqs >= 0 && num_q_heads >= 1 && max_seq_len >= 0 && num_queries >= 1 &&
         num_queries <= KVARN_MAX_VERIFY_QUERIES && num_q_heads % L->num_kv_heads == 0 && prefix_tokens > 0 &&
         prefix_tokens % L->tile_tokens == 0 &&
         static_cast<int64_t>(num_seqs) * num_queries * num_q_heads <= (1 << 30);
}

int64_t kvarn_decode_shared_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                            int32_t num_queries, int32_t max_seq_len, int32_t prefix_tokens) {
  if (check_dense(L) != KVARN_OK ||
      !shared_sizes_ok(L, num_seqs, num_q_heads, num_queries, max_seq_len, prefix_tokens))
    return -1;
  return shared_workspace_bytes(static_cast<int64_t>(num_seqs) * num_queries * num_q_heads, L->head_dim,
                                shared_plan(L, num_seqs, num_q_heads, num_queries, max_seq_len, prefix_tokens));
}

int32_t kvarn_decode_shared(const void* q, int32_t num_q_heads, int32_t num_queries, float sm_scale,
                            const void* cache, const kvarn_layout* L, const int32_t* prefix_table,
                            int32_t prefix_tokens, const int32_t* block_table, int32_t bt_stride,
                            const int32_t* seq_lens, int32_t max_seq_len, const void* tail_k, const void* tail_v,
                            int32_t tail_capacity, int32_t num_seqs, float* out, float* lse, void* workspace,
                            int64_t workspace_bytes, uint32_t* error_flags, kvarn_stream_t stream) {
  int32_t s = check_dense(L);
  if (s != KVARN_OK) return s;
  if (num_queries < 1 || num_queries > KVARN_MAX_VERIFY_QUERIES) return KVARN_EUNSUPPORTED;
  s = check_decode_common(L, num_q_heads, block_table, bt_stride, seq_lens, max_seq_len, num_seqs, out, workspace,
                          error_flags);
  if (s != KVARN_OK || num_seqs == 0) return s;
  if (!shared_sizes_ok(L, num_seqs, num_q_heads, num_queries, max_seq_len, prefix_tokens)) return KVARN_EINVAL;
  if (tail_capacity < L->tile_tokens + num_queries - 2 || tail_capacity < 1) return KVARN_EINVAL;
  if (!q || !cache || !prefix_table || L->num_pages < 1) return KVARN_EINVAL;
  if (num_q_heads / L->num_kv_heads > 8) return KVARN_EUNSUPPORTED;
  const int32_t committed = std::max(0, max_seq_len - num_queries + 1) / L->tile_tokens * L->tile_tokens;
  if (committed > prefix_tokens && bt_stride < committed / kPageTokens) return KVARN_EINVAL;
  if (!aligned(q, 16) || !aligned(cache, 128)) return KVARN_EALIGN;
  if ((tail_k && !aligned(tail_k, 16)) || (tail_v && !aligned(tail_v, 16))) return KVARN_EALIGN;
  const SharedPlan plan = shared_plan(L, num_seqs, num_q_heads, num_queries, max_seq_len, prefix_tokens);
  if (workspace_bytes <
      shared_workspace_bytes(static_cast<int64_t>(num_seqs) * num_queries * num_q_heads, L->head_dim, plan))
    return KVARN_EWORKSPACE;
  DecodeParams p{};
  p.q = q;
  p.num_q_heads = num_q_heads;
  p.sm_scale = sm_scale;
  p.cache = static_cast<const uint8_t*>(cache);
  p.D = L->head_dim;
  p.N = L->tile_tokens;
  p.num_kv_heads = L->num_kv_heads;
  p.num_pages = L->num_pages;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.tail_k = tail_k;
  p.tail_v = tail_v;
  p.num_seqs = num_seqs;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  p.err = error_flags;
  p.bf16 = L->kv_dtype == 1;
  p.num_queries = num_queries;
  p.tail_cap = tail_capacity;
  p.k_bits = L->k_bits;
  p.v_bits = L->v_bits;
  p.scale_bytes = L->scale_dtype == 1 ? 2 : 4;
  p.skip_tokens = prefix_tokens;
  return from_cuda(launch_decode_shared(p, plan, prefix_table, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_evict_tiles(const float* mass_in, float* mass_out, int32_t mass_stride, const int32_t* block_table,
                          int32_t* block_table_out, int32_t* freed, int32_t bt_stride, const int32_t* seq_lens,
                          int32_t* seq_lens_out, int32_t* freed_count, int32_t max_seq_len, int32_t num_seqs,
                          const kvarn_layout* L, int32_t keep_tiles, int32_t sink_tiles, int32_t recent_tiles,
                          uint32_t* error_flags, kvarn_stream_t stream) {
  const int32_t s = check_dense(L);
  if (s != KVARN_OK) return s;
  if (num_seqs < 0 || max_seq_len < 0 || sink_tiles < 0 || recent_tiles < 0 || keep_tiles < sink_tiles ||
      keep_tiles - sink_tiles < recent_tiles)
    return KVARN_EINVAL;
  if (num_seqs == 0) return KVARN_OK;
  if (num_seqs > 65535) return KVARN_EUNSUPPORTED;
  const int32_t tiles = max_seq_len / L->tile_tokens;
  if (!seq_lens || !seq_lens_out || !freed_count || !error_flags) return KVARN_EINVAL;
  if (tiles > 0 && (!mass_in || !mass_out || !block_table || !block_table_out || !freed || mass_stride < tiles ||
                    bt_stride < tiles * (L->tile_tokens / kPageTokens) || freed == block_table ||
                    freed == block_table_out))
    return KVARN_EINVAL;
  if (!aligned(mass_in, 4) || !aligned(mass_out, 4) || !aligned(block_table, 4) || !aligned(block_table_out, 4) ||
      !aligned(freed, 4) || !aligned(seq_lens, 4) || !aligned(seq_lens_out, 4) || !aligned(freed_count, 4) ||
      !aligned(error_flags, 4))
    return KVARN_EALIGN;
  if (freed_count == seq_lens_out || freed_count == seq_lens) return KVARN_EINVAL;
  EvictParams p{};
  p.mass = mass_in;
  p.mass_out = mass_out;
  p.mass_stride = mass_stride;
  p.table = block_table;
  p.table_out = block_table_out;
  p.freed = freed;
  p.freed_count = freed_count;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.lens_out = seq_lens_out;
  p.max_seq_len = max_seq_len;
  p.num_seqs = num_seqs;
  p.N = L->tile_tokens;
  p.keep = keep_tiles;
  p.sink = sink_tiles;
  p.recent = recent_tiles;
  p.err = error_flags;
  return from_cuda(launch_evict(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_rope(const kvarn_rope_tensor* tensors, int32_t num_tensors, int32_t dtype, int32_t num_seqs,
                   int32_t num_tokens, const int32_t* positions, int64_t pos_stride, const double* inv_freq,
                   int32_t rope_dim, int32_t rope_offset, int32_t interleaved, float scale, int32_t inverse,
                   kvarn_stream_t stream) {
  if (!tensors || num_tensors < 1 || num_tensors > KVARN_ROPE_MAX_TENSORS) return KVARN_EINVAL;
  if (dtype < 0 || dtype > 2) return KVARN_EUNSUPPORTED;
  if (num_seqs < 0 || num_tokens < 0 || rope_dim < 2 || rope_dim % 2 || rope_offset < 0 || pos_stride < 0 ||
      (interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return KVARN_EINVAL;
  const uintptr_t size = dtype == 2 ? 4 : 2;
  RopeParams p{};
  int64_t heads = 0;
  for (int32_t k = 0; k < num_tensors; ++k) {
    const kvarn_rope_tensor& t = tensors[k];
    if (t.num_heads < 0 || t.head_dim < 1) return KVARN_EINVAL;
    if (static_cast<int64_t>(rope_offset) + rope_dim > t.head_dim) return KVARN_EINVAL;
    if (t.head_dim > KVARN_ROPE_MAX_DIM) return KVARN_EUNSUPPORTED;
    heads += t.num_heads;
  }
  if (heads > (1 << 20) || static_cast<int64_t>(num_seqs) * num_tokens > (1 << 30)) return KVARN_EUNSUPPORTED;
  if (num_seqs == 0 || num_tokens == 0 || heads == 0) return KVARN_OK;
  if (!positions || !inv_freq) return KVARN_EINVAL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return KVARN_EALIGN;
  for (int32_t k = 0; k < num_tensors; ++k) {
    kvarn_rope_tensor t = tensors[k];
    if (t.num_heads == 0) continue;
    // the stride of an axis of length one says nothing
    if (num_seqs == 1) t.in_seq_stride = t.out_seq_stride = 0;
    if (num_tokens == 1) t.in_token_stride = t.out_token_stride = 0;
    if (t.num_heads == 1) t.in_head_stride = t.out_head_stride = 0;
    if (!t.in || !t.out) return KVARN_EINVAL;
    if (!aligned(t.in, size) || !aligned(t.out, size)) return KVARN_EALIGN;
    // in place: every element is written where it was read
    if (t.in == t.out && (t.in_seq_stride != t.out_seq_stride || t.in_token_stride != t.out_token_stride ||
                          t.in_head_stride != t.out_head_stride))
      return KVARN_EINVAL;
    // a tensor is written while the others are read and written
    for (int32_t j = 0; j < p.num_tensors; ++j)
      if (t.out == p.t[j].out || t.out == p.t[j].in || t.in == p.t[j].out) return KVARN_EINVAL;
    p.t[p.num_tensors++] = {t.in,            t.out,            t.in_seq_stride,   t.in_token_stride, t.in_head_stride,
                            t.out_seq_stride, t.out_token_stride, t.out_head_stride, t.num_heads,      t.head_dim};
  }
  p.total_heads = static_cast<int32_t>(heads);
  p.dtype = dtype;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.inv_freq = inv_freq;
  p.rope_dim = rope_dim;
  p.offset = rope_offset;
  p.interleaved = interleaved;
  p.scale = scale;
  p.inverse = inverse;
  return from_cuda(launch_rope(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_fork_sequences(const int32_t* parents, int32_t num_in, int32_t num_out, const int32_t* seq_lens,
                             int32_t* seq_lens_out, int32_t max_seq_len, const int32_t* block_table,
                             int32_t* block_table_out, int32_t bt_stride, const int32_t* page_refs,
                             int32_t* page_refs_out, int32_t* freed, int32_t* freed_count,
                             const kvarn_fork_tail* tails, int32_t num_tails, const kvarn_layout* L,
                             int32_t recent_tokens, int32_t window, int32_t sink_tokens, uint32_t* error_flags,
                             kvarn_stream_t stream) {
  if (!L) return KVARN_EINVAL;
  if (L->page_tokens != kPageTokens || L->tile_tokens < kPageTokens || L->tile_tokens % kPageTokens ||
      L->tile_tokens > 1024)
    return KVARN_EUNSUPPORTED;
  if (num_in < 0 || num_out < 0 || max_seq_len < 0 || num_tails < 0 || recent_tokens < 0 || window < 0 ||
      sink_tokens < 0 || L->num_pages < 0)
    return KVARN_EINVAL;
  if (num_in > kForkMaxRows || num_out > kForkMaxRows || num_tails > kForkMaxTails || L->num_pages > kForkMaxPages)
    return KVARN_EUNSUPPORTED;
  const int32_t entries = max_seq_len / L->tile_tokens * (L->tile_tokens / kPageTokens);
  if ((num_out > 0 && (!parents || !seq_lens_out)) || (num_in > 0 && !seq_lens) || !freed_count || !error_flags)
    return KVARN_EINVAL;
  if (entries > 0 && ((num_in > 0 && !block_table) || (num_out > 0 && !block_table_out) || bt_stride < entries))
    return KVARN_EINVAL;
  if (L->num_pages > 0 && (!page_refs || !page_refs_out || !freed)) return KVARN_EINVAL;
  const void* ints[] = {parents,   seq_lens, seq_lens_out, block_table, block_table_out, page_refs, page_refs_out,
                        freed,     freed_count, error_flags};
  for (const void* p : ints)
    if (!aligned(p, 4)) return KVARN_EALIGN;
  // outputs are buffers of their own
  const void* outs[] = {seq_lens_out, block_table_out, freed, freed_count, error_flags};
  for (const void* o : outs) {
    int n = 0;
    for (const void* p : ints) n += o && p == o;
    if (n > 1) return KVARN_EINVAL;
  }
  if (page_refs_out && (page_refs_out == parents || page_refs_out == seq_lens || page_refs_out == block_table))
    return KVARN_EINVAL;
  ForkParams p{};
  for (int32_t k = 0; k < num_tails; ++k) {
    if (!tails) return KVARN_EINVAL;
    const kvarn_fork_tail& t = tails[k];
    if (t.num_heads < 0 || t.capacity < 0 || t.row_bytes < 0 || (t.whole != 0 && t.whole != 1)) return KVARN_EINVAL;
    if (t.num_heads > (1 << 20) || t.row_bytes > (1 << 20)) return KVARN_EUNSUPPORTED;
    if (t.num_heads == 0 || t.capacity == 0 || t.row_bytes == 0) continue;
    if ((!t.in && num_in > 0) || (!t.out && num_out > 0) || (t.in && t.in == t.out)) return KVARN_EINVAL;
    if (t.row_bytes % 16 || !aligned(t.in, 16) || !aligned(t.out, 16)) return KVARN_EALIGN;
    for (int32_t j = 0; j < p.num_rows; ++j)
      if ((t.out && (t.out == p.rows[j].out || t.out == p.rows[j].in)) || (t.in && t.in == p.rows[j].out)) return KVARN_EINVAL;
    p.rows[p.num_rows++] = {t.in, t.out, t.num_heads, t.capacity, t.row_bytes, t.whole, 0};
  }
  p.parents = parents;
  p.num_in = num_in;
  p.num_out = num_out;
  p.seq_lens = seq_lens;
  p.lens_out = seq_lens_out;
  p.max_seq_len = max_seq_len;
  p.table = block_table;
  p.table_out = block_table_out;
  p.bt_stride = bt_stride;
  p.entries = entries;
  p.refs = page_refs;
  p.refs_out = page_refs_out;
  p.num_pages = static_cast<int32_t>(L->num_pages);
  p.freed = freed;
  p.freed_count = freed_count;
  p.N = L->tile_tokens;
  p.pages_per_tile = L->tile_tokens / kPageTokens;
  p.recent = recent_tokens;
  p.window = window;
  p.sinks = sink_tokens;
  p.err = error_flags;
  return from_cuda(launch_fork(p, reinterpret_cast<cudaStream_t>(stream)));
}

int64_t kvarn_compact_workspace_bytes(int64_t num_pages) {
  return num_pages < 0 || num_pages > (1 << 30) ? -1 : compact_workspace_bytes(num_pages);
}

int32_t kvarn_compact_pages(void* cache, int64_t page_stride, int64_t num_pages, const int32_t* page_refs,
                            int32_t* page_refs_out, const int32_t* block_table, int32_t* block_table_out,
                            int32_t num_rows, int32_t entries, int32_t bt_stride, int32_t* remap,
                            int32_t* live_count, void* workspace, int64_t workspace_bytes, uint32_t* error_flags,
                            kvarn_stream_t stream) {
  if (num_pages < 0 || page_stride < 1 || num_rows < 0 || entries < 0) return KVARN_EINVAL;
  if (num_pages > (1 << 30) || page_stride > (1LL << 30)) return KVARN_EUNSUPPORTED;
  if (!live_count || !workspace || !error_flags) return KVARN_EINVAL;
  if (num_pages > 0 && (!cache || !page_refs || !page_refs_out || !remap)) return KVARN_EINVAL;
  const bool tables = num_rows > 0 && entries > 0;
  if (tables && (!block_table || !block_table_out || (num_rows > 1 && bt_stride < entries))) return KVARN_EINVAL;
  if (!aligned(cache, 16) || page_stride % 16 || !aligned(workspace, 16)) return KVARN_EALIGN;
  const void* ints[] = {page_refs, page_refs_out, block_table, block_table_out, remap, live_count, error_flags};
  for (const void* p : ints)
    if (!aligned(p, 4)) return KVARN_EALIGN;
  for (const void* o : {static_cast<const void*>(remap), static_cast<const void*>(live_count)}) {
    int n = 0;
    for (const void* p : ints) n += o && p == o;
    if (n > 1) return KVARN_EINVAL;
  }
  if (tables && (block_table_out == page_refs || block_table_out == page_refs_out || page_refs_out == block_table))
    return KVARN_EINVAL;
  if (workspace_bytes < compact_workspace_bytes(num_pages)) return KVARN_EWORKSPACE;
  CompactParams p{};
  p.cache = static_cast<uint8_t*>(cache);
  p.page_bytes = page_stride;
  p.num_pages = static_cast<int32_t>(num_pages);
  p.refs = page_refs;
  p.refs_out = page_refs_out;
  p.table = block_table;
  p.table_out = block_table_out;
  p.rows = tables ? num_rows : 0;
  p.entries = tables ? entries : 1;
  p.bt_stride = bt_stride;
  p.remap = remap;
  p.live = live_count;
  p.err = error_flags;
  return from_cuda(launch_compact(p, workspace, reinterpret_cast<cudaStream_t>(stream)));
}

static bool norm_sizes_ok(int32_t num_tensors, int32_t head_dim, int32_t num_seqs, int32_t num_tokens) {
  return num_tensors >= 1 && num_tensors <= KVARN_ROPE_MAX_TENSORS && head_dim >= 1 && num_seqs >= 0 && num_tokens >= 0;
}

int64_t kvarn_norm_rope_backward_workspace_bytes(const int32_t* num_heads, int32_t num_tensors, int32_t head_dim,
                                                 int32_t num_seqs, int32_t num_tokens) {
  if (!num_heads || !norm_sizes_ok(num_tensors, head_dim, num_seqs, num_tokens) || head_dim > KVARN_ROPE_MAX_DIM ||
      static_cast<int64_t>(num_seqs) * num_tokens > (1 << 30))
    return -1;
  int64_t heads = 0;
  for (int32_t k = 0; k < num_tensors; ++k) {
    if (num_heads[k] < 0) return -1;
    heads += num_heads[k];
  }
  if (heads > (1 << 20)) return -1;
  return norm_rope_workspace_bytes(num_tensors, num_heads, head_dim, static_cast<int64_t>(num_seqs) * num_tokens);
}

static int32_t norm_rope(const kvarn_norm_rope_tensor* tensors, int32_t num_tensors, int32_t head_dim, int32_t dtype,
                         int32_t weight_dtype, int32_t num_seqs, int32_t num_tokens, const int32_t* positions,
                         int64_t pos_stride, const double* inv_freq, int32_t rope_dim, int32_t rope_offset,
                         int32_t interleaved, float scale, float eps, float weight_offset, bool backward,
                         void* workspace, int64_t workspace_bytes, kvarn_stream_t stream) {
  if (!tensors || !norm_sizes_ok(num_tensors, head_dim, num_seqs, num_tokens)) return KVARN_EINVAL;
  if (dtype < 0 || dtype > 2 || weight_dtype < 0 || weight_dtype > 2) return KVARN_EUNSUPPORTED;
  if (rope_dim < 0 || rope_dim % 2 || rope_offset < 0 || pos_stride < 0 || (interleaved != 0 && interleaved != 1) ||
      !(eps >= 0.f) || static_cast<int64_t>(rope_offset) + rope_dim > head_dim)
    return KVARN_EINVAL;
  if (head_dim > KVARN_ROPE_MAX_DIM) return KVARN_EUNSUPPORTED;
  const uintptr_t size = dtype == 2 ? 4 : 2, wsize = weight_dtype == 2 ? 4 : 2;
  NormParams p{};
  int64_t heads = 0;
  int32_t every[KVARN_ROPE_MAX_TENSORS];
  bool sums = false;
  for (int32_t k = 0; k < num_tensors; ++k) {
    if (tensors[k].num_heads < 0) return KVARN_EINVAL;
    every[k] = tensors[k].num_heads;
    heads += tensors[k].num_heads;
    sums = sums || (backward && tensors[k].dweight);
  }
  const int64_t tokens = static_cast<int64_t>(num_seqs) * num_tokens;
  if (heads > (1 << 20) || tokens > (1 << 30)) return KVARN_EUNSUPPORTED;
  const int64_t space = backward ? norm_rope_workspace_bytes(num_tensors, every, head_dim, tokens) : 0;
  if (space < 0) return KVARN_EUNSUPPORTED;
  // the gradient of the weights over no tokens or heads is still written
  if ((tokens == 0 || heads == 0) && !sums) return KVARN_OK;
  if (rope_dim > 0 && tokens > 0 && (!positions || !inv_freq)) return KVARN_EINVAL;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return KVARN_EALIGN;
  for (int32_t k = 0; k < num_tensors; ++k) {
    kvarn_norm_rope_tensor t = tensors[k];
    if (!backward) t.dweight = nullptr, t.dy = nullptr;
    if (!aligned(t.weight, wsize) || !aligned(t.dweight, 4)) return KVARN_EALIGN;
    if (t.num_heads == 0 || tokens == 0) {
      t.num_heads = 0;
    } else {
      // the stride of an axis of length one says nothing
      if (num_seqs == 1) t.x_seq_stride = t.dy_seq_stride = t.out_seq_stride = 0;
      if (num_tokens == 1) t.x_token_stride = t.dy_token_stride = t.out_token_stride = 0;
      if (t.num_heads == 1) t.x_head_stride = t.dy_head_stride = t.out_head_stride = 0;
      if (!backward) t.dy_seq_stride = t.dy_token_stride = t.dy_head_stride = 0;
      if (!t.x || !t.out || (backward && !t.dy)) return KVARN_EINVAL;
      if (!aligned(t.x, size) || !aligned(t.dy, size) || !aligned(t.out, size)) return KVARN_EALIGN;
      // in place: every element is written where it was read
      if (t.x == t.out && (t.x_seq_stride != t.out_seq_stride || t.x_token_stride != t.out_token_stride ||
                           t.x_head_stride != t.out_head_stride))
        return KVARN_EINVAL;
      if (backward && t.dy == t.out && (t.dy_seq_stride != t.out_seq_stride || t.dy_token_stride != t.out_token_stride ||
                                        t.dy_head_stride != t.out_head_stride))
        return KVARN_EINVAL;
    }
    const void* dw = t.dweight;
    if ((dw && (dw == t.weight || dw == t.out || dw == t.x || dw == t.dy)) || (t.weight && t.weight == t.out))
      return KVARN_EINVAL;
    // a tensor is written while the others are read and written
    for (int32_t j = 0; j < p.num_tensors; ++j) {
      const NormTensor& o = p.t[j];
      if (t.num_heads && o.heads && (t.out == o.out || t.out == o.x || t.x == o.out)) return KVARN_EINVAL;
      if (t.num_heads && o.heads && backward && (t.out == o.dy || t.dy == o.out)) return KVARN_EINVAL;
      if (dw && (dw == o.dw || dw == o.w || dw == o.x || dw == o.dy || dw == o.out)) return KVARN_EINVAL;
      if (o.dw && (o.dw == t.weight || o.dw == t.x || o.dw == t.dy || o.dw == t.out)) return KVARN_EINVAL;
      if ((t.weight && t.weight == o.out) || (o.w && o.w == t.out)) return KVARN_EINVAL;
    }
    p.t[p.num_tensors++] = {t.x,           t.dy,            t.out,          t.weight,        t.dweight,
                            t.x_seq_stride, t.x_token_stride, t.x_head_stride, t.dy_seq_stride, t.dy_token_stride,
                            t.dy_head_stride, t.out_seq_stride, t.out_token_stride, t.out_head_stride, t.num_heads};
  }
  if (sums) {
    if (!workspace && tokens > 0 && heads > 0) return KVARN_EINVAL;
    if (!aligned(workspace, 16)) return KVARN_EALIGN;
    if (workspace_bytes < space) return KVARN_EWORKSPACE;
  }
  p.dim = head_dim;
  p.dtype = dtype;
  p.wdtype = weight_dtype;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.inv_freq = inv_freq;
  p.rope_dim = rope_dim;
  p.offset = rope_offset;
  p.interleaved = interleaved;
  p.scale = scale;
  p.eps = eps;
  p.weight_offset = weight_offset;
  p.backward = backward;
  p.parts = static_cast<float*>(workspace);
  return from_cuda(launch_norm_rope(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_norm_rope(const kvarn_norm_rope_tensor* tensors, int32_t num_tensors, int32_t head_dim, int32_t dtype,
                        int32_t weight_dtype, int32_t num_seqs, int32_t num_tokens, const int32_t* positions,
                        int64_t pos_stride, const double* inv_freq, int32_t rope_dim, int32_t rope_offset,
                        int32_t interleaved, float scale, float eps, float weight_offset, kvarn_stream_t stream) {
  return norm_rope(tensors, num_tensors, head_dim, dtype, weight_dtype, num_seqs, num_tokens, positions, pos_stride,
                   inv_freq, rope_dim, rope_offset, interleaved, scale, eps, weight_offset, false, nullptr, 0, stream);
}

int32_t kvarn_norm_rope_backward(const kvarn_norm_rope_tensor* tensors, int32_t num_tensors, int32_t head_dim,
                                 int32_t dtype, int32_t weight_dtype, int32_t num_seqs, int32_t num_tokens,
                                 const int32_t* positions, int64_t pos_stride, const double* inv_freq,
                                 int32_t rope_dim, int32_t rope_offset, int32_t interleaved, float scale, float eps,
                                 float weight_offset, void* workspace, int64_t workspace_bytes,
                                 kvarn_stream_t stream) {
  return norm_rope(tensors, num_tensors, head_dim, dtype, weight_dtype, num_seqs, num_tokens, positions, pos_stride,
                   inv_freq, rope_dim, rope_offset, interleaved, scale, eps, weight_offset, true, workspace,
                   workspace_bytes, stream);
}

int64_t kvarn_q8_page_bytes(const kvarn_layout* L) { return check_q8(L) == KVARN_OK ? 32 * L->head_dim + 32 : -1; }

static Q8BlockParams q8_params(const kvarn_layout* L, int32_t code, const void* cache, uint32_t* error_flags) {
  Q8BlockParams p{};
  p.cache = const_cast<void*>(cache);
  p.num_pages = L->num_pages;
  p.num_kv_heads = L->num_kv_heads;
  p.D = L->head_dim;
  p.bf16 = L->kv_dtype == 1;
  p.code = code;
  p.err = error_flags;
  return p;
}

static int32_t q8_blocks(const void* k, const void* v, int64_t seq_stride, int64_t head_stride, int64_t token_stride,
                         int32_t num_seqs, int32_t chunk_tokens, const int32_t* block_start,
                         const int32_t* block_table, int32_t bt_stride, const kvarn_layout* L, int32_t code,
                         const void* cache, uint32_t* error_flags, kvarn_stream_t stream, bool read) {
  const int32_t s = check_q8(L, code);
  if (s != KVARN_OK) return s;
  if (num_seqs < 0 || chunk_tokens < 0 || chunk_tokens % kPageTokens) return KVARN_EINVAL;
  if (num_seqs == 0 || chunk_tokens == 0) return KVARN_OK;
  if (!k || !v || !block_start || !block_table || !cache || !error_flags) return KVARN_EINVAL;
  if (seq_stride < 0 || head_stride < 0 || token_stride < 0 || bt_stride < 1) return KVARN_EINVAL;
  if (read && k == v) return KVARN_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || seq_stride % 8 || head_stride % 8 || token_stride % 8) return KVARN_EALIGN;
  if (!aligned(cache, 128) || !aligned(error_flags, 4) || !aligned(block_start, 4) || !aligned(block_table, 4))
    return KVARN_EALIGN;
  // two items a block and head, four to a CTA
  if (static_cast<int64_t>(num_seqs) * L->num_kv_heads > (1LL << 31) / (chunk_tokens / kPageTokens))
    return KVARN_EUNSUPPORTED;
  Q8BlockParams p = q8_params(L, code, cache, error_flags);
  p.k = k;
  p.v = v;
  p.seq_stride = seq_stride;
  p.head_stride = head_stride;
  p.token_stride = token_stride;
  p.num_seqs = num_seqs;
  p.blocks = chunk_tokens / kPageTokens;
  p.block_start = block_start;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  return from_cuda(launch_q8_blocks(p, read, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_q8_encode_blocks(const void* k, const void* v, int64_t seq_stride, int64_t head_stride,
                               int64_t token_stride, int32_t num_seqs, int32_t chunk_tokens,
                               const int32_t* block_start, const int32_t* block_table, int32_t bt_stride,
                               const kvarn_layout* L, int32_t code, void* cache, uint32_t* error_flags,
                               kvarn_stream_t stream) {
  return q8_blocks(k, v, seq_stride, head_stride, token_stride, num_seqs, chunk_tokens, block_start, block_table,
                   bt_stride, L, code, cache, error_flags, stream, false);
}

int32_t kvarn_q8_read_blocks(void* k, void* v, int64_t seq_stride, int64_t head_stride, int64_t token_stride,
                             int32_t num_seqs, int32_t chunk_tokens, const int32_t* block_start,
                             const int32_t* block_table, int32_t bt_stride, const kvarn_layout* L, int32_t code,
                             const void* cache, uint32_t* error_flags, kvarn_stream_t stream) {
  return q8_blocks(k, v, seq_stride, head_stride, token_stride, num_seqs, chunk_tokens, block_start, block_table,
                   bt_stride, L, code, cache, error_flags, stream, true);
}

int32_t kvarn_q8_append(const void* k, const void* v, const int32_t* seq_lens, int32_t max_seq_len, void* tail_k,
                        void* tail_v, int32_t tail_capacity, int32_t num_seqs, const int32_t* block_table,
                        int32_t bt_stride, const kvarn_layout* L, int32_t code, void* cache, uint32_t* error_flags,
                        kvarn_stream_t stream) {
  const int32_t s = check_q8(L, code);
  if (s != KVARN_OK) return s;
  if (num_seqs < 0 || max_seq_len < 0) return KVARN_EINVAL;
  if (num_seqs == 0) return KVARN_OK;
  if (!k || !v || !seq_lens || !tail_k || !tail_v || !block_table || !cache || !error_flags || bt_stride < 1)
    return KVARN_EINVAL;
  if (tail_k == tail_v || tail_capacity < kPageTokens - 1 || bt_stride < max_seq_len / kPageTokens) return KVARN_EINVAL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(tail_k, 16) || !aligned(tail_v, 16)) return KVARN_EALIGN;
  if (!aligned(cache, 128) || !aligned(error_flags, 4) || !aligned(seq_lens, 4) || !aligned(block_table, 4))
    return KVARN_EALIGN;
  if (static_cast<int64_t>(num_seqs) * L->num_kv_heads > (1LL << 31)) return KVARN_EUNSUPPORTED;
  Q8BlockParams p = q8_params(L, code, cache, error_flags);
  p.k = k;
  p.v = v;
  p.num_seqs = num_seqs;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.tail_k = tail_k;
  p.tail_v = tail_v;
  p.tail_cap = tail_capacity;
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  return from_cuda(launch_q8_append(p, reinterpret_cast<cudaStream_t>(stream)));
}

static bool q8_decode_sizes_ok(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads, int32_t num_queries,
                               int32_t max_seq_len, int32_t window, int32_t sink_tokens) {
  return num_seqs >= 0 && num_q_heads >= 1 && num_q_heads % L->num_kv_heads == 0 && num_queries >= 1 &&
         num_queries <= KVARN_MAX_VERIFY_QUERIES && max_seq_len >= 0 && window >= 0 && sink_tokens >= 0;
}

int64_t kvarn_q8_decode_workspace_bytes(const kvarn_layout* L, int32_t num_seqs, int32_t num_q_heads,
                                        int32_t num_queries, int32_t max_seq_len, int32_t window,
                                        int32_t sink_tokens) {
  if (check_q8(L) != KVARN_OK ||
      !q8_decode_sizes_ok(L, num_seqs, num_q_heads, num_queries, max_seq_len, window, sink_tokens))
    return -1;
  return q8_decode_workspace_bytes(num_seqs, num_q_heads / L->num_kv_heads * num_queries, L->head_dim);
}

int32_t kvarn_q8_decode(const void* q, int32_t num_q_heads, int32_t num_queries, float sm_scale, const void* cache,
                        const kvarn_layout* L, int32_t code, const int32_t* block_table, int32_t bt_stride,
                        const int32_t* seq_lens, int32_t max_seq_len, const void* tail_k, const void* tail_v,
                        int32_t tail_capacity, int32_t window, int32_t sink_tokens, int32_t num_seqs, float* out,
                        float* lse, void* workspace, int64_t workspace_bytes, uint32_t* error_flags,
                        kvarn_stream_t stream) {
  int32_t s = check_q8(L, code);
  if (s != KVARN_OK) return s;
  if (!q8_decode_sizes_ok(L, num_seqs, num_q_heads, num_queries, max_seq_len, window, sink_tokens))
    return KVARN_EINVAL;
  s = check_decode_common(L, num_q_heads, block_table, bt_stride, seq_lens, max_seq_len, num_seqs, out, workspace,
                          error_flags);
  if (s != KVARN_OK || num_seqs == 0) return s;
  if (num_q_heads / L->num_kv_heads > 8 || static_cast<int64_t>(num_seqs) * num_queries * num_q_heads > (1 << 30))
    return KVARN_EUNSUPPORTED;
  if (!q || !cache || tail_capacity < num_queries + kPageTokens - 2) return KVARN_EINVAL;
  const int32_t blocks = std::max(0, max_seq_len - num_queries + 1) / kPageTokens;
  if (bt_stride < blocks || (blocks > 0 && L->num_pages < 1)) return KVARN_EINVAL;
  if (!aligned(q, 16) || !aligned(cache, 128) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(lse, 4) || !aligned(error_flags, 4))
    return KVARN_EALIGN;
  if ((tail_k && !aligned(tail_k, 16)) || (tail_v && !aligned(tail_v, 16))) return KVARN_EALIGN;
  if (workspace_bytes <
      q8_decode_workspace_bytes(num_seqs, num_q_heads / L->num_kv_heads * num_queries, L->head_dim))
    return KVARN_EWORKSPACE;
  Q8DecodeParams p{};
  p.q = q;
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.seq_lens = seq_lens;
  p.max_seq_len = max_seq_len;
  p.num_seqs = num_seqs;
  p.num_queries = num_queries;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = L->num_kv_heads;
  p.D = L->head_dim;
  p.num_pages = L->num_pages;
  p.tail_k = tail_k;
  p.tail_v = tail_v;
  p.tail_cap = tail_capacity;
  p.window = window;
  p.sinks = sink_tokens;
  p.sm_scale = sm_scale;
  p.bf16 = L->kv_dtype == 1;
  p.code = code;
  p.out = out;
  p.lse = lse;
  p.workspace = workspace;
  p.err = error_flags;
  return from_cuda(launch_q8_decode(p, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t kvarn_set_copy_wait_test(int64_t cycles, int32_t withhold) {
  if (cycles < 0 || (withhold != 0 && withhold != 1)) return KVARN_EINVAL;
  set_copy_wait_test(cycles, withhold ? 16 : 0);
  return KVARN_OK;
}

int32_t kvarn_read_error_flags(const uint32_t* error_flags, uint32_t* host_out,
                               kvarn_stream_t stream) {
  if (!error_flags || !host_out) return KVARN_EINVAL;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(host_out, error_flags, 4, cudaMemcpyDeviceToHost, st) != cudaSuccess)
    return KVARN_ECUDA;
  return from_cuda(cudaStreamSynchronize(st));
}

}  // extern "C"
