// Internal launch parameters shared by the C-ABI layer and the kernels.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

namespace kvarn {

struct EncodeParams {
  const void* k;
  const void* v;
  int64_t seq_stride, head_stride;
  int32_t num_seqs, chunk_tokens;
  const int32_t* tile_start;
  const int32_t* block_table;
  int32_t bt_stride;
  void* cache;
  int64_t num_pages;
  int32_t num_kv_heads, D, N, norm_iters;
  bool bf16;
  uint32_t* err;
  int32_t k_bits, v_bits, scale_bytes;  // 4, 2, 4 for the k4v2 preset with fp32 scales
  float* stages;  // optional fp32 stage records of the encoded tiles (null: none)
};

// Code widths and scale sizes with compiled kernels: every pair of a key
// width and a value width from {2, 3, 4, 5, 6, 8} (the gmlx page sets the
// two widths separately), with fp16 or fp32 scales at head_dim 128 and with
// fp16 scales at head_dim 256, where (4, 2) also takes fp32 scales.
inline bool width_compiled(int32_t b) { return b == 2 || b == 3 || b == 4 || b == 5 || b == 6 || b == 8; }
inline bool widths_supported(int32_t D, int32_t kb, int32_t vb, int32_t sb) {
  if (kb == 4 && vb == 2 && sb == 4) return true;
  if (!width_compiled(kb) || !width_compiled(vb)) return false;
  if (D == 256) return sb == 2;
  return D == 128 && (sb == 2 || sb == 4);
}

// X(KB, VB) for every compiled (key width, value width) pair with fp16
// scales; the key used by the dispatch switches is 16 KB + VB.
#define KVARN_WIDTH_ROW(X, K) X(K, 2) X(K, 3) X(K, 4) X(K, 5) X(K, 6) X(K, 8)
#define KVARN_WIDTH_PAIRS(X)                                                         \
  KVARN_WIDTH_ROW(X, 2) KVARN_WIDTH_ROW(X, 3) KVARN_WIDTH_ROW(X, 4) KVARN_WIDTH_ROW(X, 5) \
  KVARN_WIDTH_ROW(X, 6) KVARN_WIDTH_ROW(X, 8)
// X(KB, VB) for the pairs compiled at head_dim 256 (fp16 scales): all.
#define KVARN_WIDTH_PAIRS_256(X) KVARN_WIDTH_PAIRS(X)
// X(KB, VB) for the pairs compiled with fp32 scales at head_dim 128 besides
// the preset (4, 2), which has its own instantiation.
#define KVARN_WIDTH_ROW_NO42(X, K) X(K, 3) X(K, 4) X(K, 5) X(K, 6) X(K, 8)
#define KVARN_WIDTH_PAIRS_S32(X)                                                              \
  KVARN_WIDTH_ROW(X, 2) KVARN_WIDTH_ROW(X, 3) KVARN_WIDTH_ROW_NO42(X, 4) KVARN_WIDTH_ROW(X, 5) \
  KVARN_WIDTH_ROW(X, 6) KVARN_WIDTH_ROW(X, 8)

struct AppendParams {
  const void* k;  // newest token per (sequence, KV head): [B][Hkv][D]
  const void* v;
  const int32_t* seq_lens;  // lengths including the newest token
  int32_t max_seq_len;
  void* tail_k;  // [B][Hkv][N][D]
  void* tail_v;
  int32_t num_seqs;
  const int32_t* block_table;
  int32_t bt_stride;
  void* cache;
  int64_t num_pages;
  int32_t num_kv_heads, D, N, norm_iters;
  bool bf16;
  uint32_t* err;
};
cudaError_t launch_append_commit(const AppendParams& p, cudaStream_t st);

struct EncodeLatentParams {
  const void* latent;
  int64_t seq_stride;
  const void* rope;
  int64_t rope_seq_stride;
  int32_t num_seqs, chunk_tokens;
  const int32_t* tile_start;
  const int32_t* block_table;
  int32_t bt_stride;
  void* cache;
  int64_t num_pages;
  int32_t norm_iters;
  bool bf16;
  uint32_t* err;
};

struct DecodeParams {
  const void* q;            // [B][Hq][D] (dense) or q_latent [B][H][Dl] (MLA)
  const void* q_rope;       // MLA only
  int32_t num_q_heads;
  float sm_scale;
  const uint8_t* cache;
  int32_t D, N, num_kv_heads;
  int64_t num_pages;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* seq_lens;
  int32_t max_seq_len;
  const void* tail_k;       // tail_latent for MLA
  const void* tail_v;       // tail_rope for MLA
  int32_t num_seqs;
  float* out;
  float* lse;
  void* workspace;
  uint32_t* err;
  bool bf16;
  int32_t num_queries;  // dense: query tokens per sequence (0 or 1: plain decode)
  int32_t tail_cap;     // dense: tail rows per (sequence, KV head) (0: N)
  int32_t sink_tokens;  // dense: raw sink records (a multiple of N; 0: none)
  int32_t recent_tokens;  // dense: newest accepted tokens kept raw (0: none)
  const void* sink_k;   // dense: [B][Hkv][sink_tokens][D]
  const void* sink_v;
  int32_t k_bits, v_bits, scale_bytes;  // dense code widths and scale size (0: the k4v2 preset, fp32)
  int32_t codec;        // dense: 0 the KVarN pages, 1 the affine comparison pages
  int32_t skip_tokens;  // dense: tokens before the first tile taken from block_table (a shared prefix; 0: none)
  const float* mass_in;  // dense: tile masses to add to (null: none are gathered)
  float* mass_out;
  int32_t mass_stride;
  float mass_decay;
};

// (query head, query token) row groups of eight per KV head.
inline int32_t row_groups(int32_t G, int32_t Q) { return (G * Q + 7) / 8; }

// Split-K plan: tiles per split and the number of splits (+1 slot for the
// tail partial). Depends only on the arguments and the device's SM count.
struct SplitPlan {
  int32_t tiles_per_split;
  int32_t nsplit;  // splits over committed tiles
  int32_t slots;   // nsplit + 1 (the tail)
};

// Smallest split of the raw (sink and tail) records of the dense decode's stream-K plan, largest of its pieces' (down to 32).
constexpr int32_t kRawChunk = 128;

// Plan of the compressed decode: `ctas` persistent CTAs share the flattened
// list of compressed tiles (stream-K), each taking at least `min_tiles` of
// them, so a unit of n tiles writes at most 1 + ceil((n - 1) / min_tiles)
// tile partials; raw partials (raw_chunk raw tokens each) follow them.
struct DensePlan {
  int32_t ctas;
  int32_t min_tiles;
  int32_t tile_slots;  // partial slots per row reserved for tiles
  int32_t raw_splits;
  int32_t raw_chunk;   // raw tokens per raw split (kRawChunk times a power of two, over one in the pieces' plan)
  int32_t slots;       // tile_slots + raw_splits
  int32_t piece;       // > 0: pieces of so many tiles within each unit instead of stream-K ranges
  int32_t raw_last;    // raw items from the last CTA down (the grid has CTAs to spare for them)
};

// units_per_seq: KV heads x row groups; max_tiles: compressed tiles a unit
// can hold; raw_max: raw tokens a row can see.
DensePlan plan_dense_stream(int32_t num_seqs, int32_t units_per_seq, int32_t max_tiles, int32_t D, int32_t N,
                            int32_t raw_max, int32_t kb = 4, int32_t vb = 2, int32_t sb = 4,
                            int32_t ctas_per_sm = 0);
// The same work in pieces: for many short units with a raw tail each, whose
// longest (max_tiles, raw_max) sizes the grid.
DensePlan plan_dense_pieces(int32_t num_seqs, int32_t units_per_seq, int32_t max_tiles, int32_t D, int32_t N,
                            int32_t raw_max, int32_t kb, int32_t vb, int32_t sb);
// Partials of `rows` output rows, then one int32 tile-partial count per row.
int64_t dense_stream_workspace_bytes(int64_t rows, int32_t D, const DensePlan& plan);
int dense_decode_warps(int32_t D);
int dense_decode_ctas_per_sm(int32_t D, int32_t N, int32_t kb = 4, int32_t vb = 2, int32_t sb = 4);
cudaError_t launch_encode_dense(const EncodeParams& p, cudaStream_t st);

// The affine comparison codec (per-token groups of 64 channels, an fp16
// scale and offset per group; head_dim 128, 128-token tiles, equal key and
// value widths): whether a width is compiled, the encoder, and the decode
// kernel's residency (the decode runs through launch_decode_dense with
// DecodeParams::codec = 1).
inline bool affine_width_compiled(int32_t b) { return b == 2 || b == 3 || b == 4 || b == 6 || b == 8; }
cudaError_t launch_encode_affine(const EncodeParams& p, cudaStream_t st);
int affine_decode_ctas_per_sm(int32_t bits);
cudaError_t launch_encode_latent(const EncodeLatentParams& p, cudaStream_t st);
cudaError_t launch_decode_dense(const DecodeParams& p, const DensePlan& plan, cudaStream_t st);

struct StoreFp16Params {
  const void* k;
  const void* v;
  int64_t seq_stride, head_stride;
  int32_t num_seqs, token0, count;
  const int32_t* block_table;
  int32_t bt_stride;
  void* cache;
  int64_t num_pages;
  int32_t num_kv_heads, D;
  uint32_t* err;
};
cudaError_t launch_store_fp16(const StoreFp16Params& p, cudaStream_t st);
// Resident CTAs per SM of the decode over uncompressed fp16 pages (the dense
// decode kernel with no codec: DecodeParams::codec = 2, N = 32).
int raw_decode_ctas_per_sm(int32_t D);

// Widths whose decode gathers tile masses: the preset, and with fp16 scales
// K4V2 and equal widths of 4, 6 and 8 bits.
inline bool mass_widths_supported(int32_t kb, int32_t vb, int32_t sb) {
  if (kb == 4 && vb == 2) return true;
  return sb == 2 && kb == vb && (kb == 4 || kb == 6 || kb == 8);
}
// Tile masses of the dense decode: one (base-2 maximum, sum) pair per output
// row and committed tile in the workspace.
int64_t mass_workspace_bytes(int64_t rows, int32_t max_tiles);

// Rotary positions (kvarn_rope.cu).
constexpr int kRopeMaxTensors = 4;
struct RopeTensor {
  const void* in;
  void* out;
  int64_t in_seq, in_tok, in_head, out_seq, out_tok, out_head;  // elements
  int32_t heads, dim;
};
struct RopeParams {
  RopeTensor t[kRopeMaxTensors];
  int32_t num_tensors, total_heads;
  int32_t dtype;  // 0 fp16, 1 bf16, 2 fp32
  int32_t num_seqs, num_tokens;
  const int32_t* positions;
  int64_t pos_stride;
  const double* inv_freq;
  int32_t rope_dim, offset;
  int32_t interleaved;
  float scale;
  int32_t inverse;
};
cudaError_t launch_rope(const RopeParams& p, cudaStream_t st);

// Norms of queries and keys with their rotation (kvarn_norm_rope.cu).
struct NormTensor {
  const void* x;
  const void* dy;   // gradient of the output (backward)
  void* out;        // the output, or the gradient of x
  const void* w;    // [dim] or null: ones
  float* dw;        // gradient of w (backward; null: not wanted)
  int64_t x_seq, x_tok, x_head, g_seq, g_tok, g_head, o_seq, o_tok, o_head;  // elements
  int32_t heads;
};
struct NormParams {
  NormTensor t[kRopeMaxTensors];
  int32_t num_tensors;
  int32_t dim, dtype, wdtype;  // 0 fp16, 1 bf16, 2 fp32
  int32_t num_seqs, num_tokens;
  const int32_t* positions;
  int64_t pos_stride;
  const double* inv_freq;
  int32_t rope_dim, offset, interleaved;
  float scale, eps, weight_offset;
  int32_t backward;
  float* parts;  // backward: sums of the CTAs
};
int64_t norm_rope_workspace_bytes(int32_t num_tensors, const int32_t* heads, int32_t dim, int64_t tokens);
cudaError_t launch_norm_rope(const NormParams& p, cudaStream_t st);

// Eviction of tiles (kvarn_evict.cu).
struct EvictParams {
  const float* mass;
  float* mass_out;
  int32_t mass_stride;
  const int32_t* table;
  int32_t* table_out;
  int32_t* freed;
  int32_t* freed_count;
  int32_t bt_stride;
  const int32_t* seq_lens;
  int32_t* lens_out;
  int32_t max_seq_len, num_seqs, N;
  int32_t keep, sink, recent;
  int32_t range;  // tiles of a CTA (set by the launch)
  int32_t held;   // whether they fit its shared memory
  uint32_t* err;
};
cudaError_t launch_evict(const EvictParams& p, cudaStream_t st);

// Decode over a prefix that the whole batch shares (kvarn_shared.cu): the
// prefix's partials, the own tokens' decode, one merge.
struct SharedPlan {
  DensePlan own;     // each sequence's tokens past the prefix
  DensePlan prefix;  // the prefix as one sequence whose query rows are the batch's
  int32_t tc_units;  // > 0: the tensor-core kernel takes the prefix in so many (KV head, 128 rows) units,
  int32_t tc_tps;    // tiles per split
};                   // (and prefix.slots splits)
SharedPlan plan_shared(int32_t num_seqs, int32_t num_kv_heads, int32_t G, int32_t num_queries, int32_t prefix_tiles,
                       int32_t own_tiles, int32_t D, int32_t N, int32_t raw_max, int32_t kb, int32_t vb, int32_t sb);
int64_t shared_workspace_bytes(int64_t rows, int32_t D, const SharedPlan& plan);
cudaError_t launch_decode_shared(const DecodeParams& p, const SharedPlan& plan, const int32_t* prefix_table,
                                 cudaStream_t st);

SplitPlan plan_mla(int32_t num_seqs, int32_t max_seq_len);
int64_t mla_workspace_bytes(int32_t num_seqs, int32_t num_heads, const SplitPlan& plan);
cudaError_t launch_decode_mla(const DecodeParams& p, const SplitPlan& plan, cudaStream_t st);

// Pages of a cache (kvarn_pages.cu): sequences that fork, end and leave their
// windows; compaction.
constexpr int kForkMaxTails = 4, kForkMaxRows = 32768, kForkMaxPages = 1 << 23;
struct ForkRows {
  const void* in;  // [num_in][heads][capacity][row_bytes]
  void* out;       // [num_out]...
  int32_t heads, capacity;
  int64_t row_bytes;
  int32_t whole;   // all rows, not the live ones alone
  int64_t pieces;  // set by the launch
};
struct ForkParams {
  const int32_t* parents;
  int32_t num_in, num_out;
  const int32_t* seq_lens;
  int32_t* lens_out;
  int32_t max_seq_len;
  const int32_t* table;
  int32_t* table_out;
  int32_t bt_stride, entries;  // entries: of max_seq_len's whole tiles
  const int32_t* refs;
  int32_t* refs_out;
  int32_t num_pages;
  int32_t* freed;
  int32_t* freed_count;
  int32_t N, pages_per_tile, recent, window, sinks;
  ForkRows rows[kForkMaxTails];
  int32_t num_rows;
  int64_t tail_pieces;  // set by the launch
  int32_t vectors;      // the counts' addresses are multiples of 16 (set by the launch)
  uint32_t* err;
};
cudaError_t launch_fork(const ForkParams& p, cudaStream_t st);

struct CompactParams {
  uint8_t* cache;
  int64_t page_bytes;
  int32_t num_pages;
  const int32_t* refs;
  int32_t* refs_out;
  const int32_t* table;
  int32_t* table_out;
  int32_t rows, entries, bt_stride;
  int32_t* remap;
  int32_t* live;
  uint32_t* err;
  int32_t* block_live;  // in the workspace, set by the launch, as the rest
  int32_t* moves;
  int2* movers;         // page, count
  int32_t* holes;
};
int64_t compact_workspace_bytes(int64_t num_pages);
cudaError_t launch_compact(const CompactParams& p, void* workspace, cudaStream_t st);

// The 8-bit block cache (kvarn_q8.cu): blocks of 16 tokens written, read back
// or completed by an appended token.
struct Q8BlockParams {
  const void* k;  // tokens (written by the read)
  const void* v;
  int64_t seq_stride, head_stride, token_stride;  // elements
  int32_t num_seqs, blocks;
  const int32_t* block_start;
  const int32_t* seq_lens;  // append
  int32_t max_seq_len;
  void* tail_k;  // [B][Hkv][tail_cap][D]
  void* tail_v;
  int32_t tail_cap;
  const int32_t* block_table;
  int32_t bt_stride;
  void* cache;
  int64_t num_pages;
  int32_t num_kv_heads, D;
  bool bf16;
  int32_t code;  // 0 e4m3, 1 int8
  uint32_t* err;
};
cudaError_t launch_q8_blocks(const Q8BlockParams& p, bool read, cudaStream_t st);
cudaError_t launch_q8_append(const Q8BlockParams& p, cudaStream_t st);

// Decode over the 8-bit block cache, with a sliding window (kvarn_q8_decode.cu).
struct Q8DecodeParams {
  const void* q;  // [B][Q][Hq][D]
  const uint8_t* cache;
  const int32_t* block_table;
  int32_t bt_stride;
  const int32_t* seq_lens;
  int32_t max_seq_len, num_seqs, num_queries, num_q_heads, num_kv_heads, D;
  int64_t num_pages;
  const void* tail_k;
  const void* tail_v;
  int32_t tail_cap;
  int32_t window, sinks;  // window 0: none
  float sm_scale;
  bool bf16;
  int32_t code;
  float* out;
  float* lse;
  void* workspace;
  uint32_t* err;
};
int64_t q8_decode_workspace_bytes(int32_t num_seqs, int32_t rows, int32_t D);
cudaError_t launch_q8_decode(const Q8DecodeParams& p, cudaStream_t st);

int device_sm_count();

// A launch as a programmatic dependent of the kernel before it on the stream:
// the kernel waits (pdl_wait_primary) before it touches memory.
template <typename... P, typename... Args>
cudaError_t chained(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// A kernel's limit of dynamic shared memory, raised once per device to one
// value whatever the call (a static object per kernel).
class SmemLimit {
 public:
  template <typename K>
  cudaError_t set(K* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }

 private:
  std::atomic<uint64_t> done_{0};
};
// Diagnostic: clock cycles the dense decode kernels wait for a page copy (0:
// default) and whether each copy is announced larger than it is (so that its
// phase never completes and every wait runs out).
void set_copy_wait_test(long long cycles, int withhold);
long long copy_wait_limit();  // cycles, the default where none is set
int copy_withhold();

}  // namespace kvarn
