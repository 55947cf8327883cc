// KVarN decode attention: split planning and launch (kernels in
// kvarn_decode_kernel.cuh; the k4v2 preset with fp32 scales is instantiated
// here, the other code widths in kvarn_decode_k*{lo,hi}.cu and
// kvarn_decode_d256{a,b}.cu).
#include <cudaTypedefs.h>

#include <atomic>

#include "kvarn_decode_kernel.cuh"

namespace kvarn {

// Clock cycles the dense decode kernels wait for a page copy before they
// give up (flag KVARN_DEVERR_TIMEOUT and return); 0: the default, about a
// second. Read when a call launches.
static std::atomic<long long> g_copy_wait_limit{0};
static std::atomic<int> g_copy_withhold{0};
constexpr long long kDefaultCopyWait = 2000000000LL;

void set_copy_wait_test(long long cycles, int withhold) {
  g_copy_wait_limit.store(cycles, std::memory_order_relaxed);
  g_copy_withhold.store(withhold, std::memory_order_relaxed);
}

long long copy_wait_limit() {
  const long long w = g_copy_wait_limit.load(std::memory_order_relaxed);
  return w > 0 ? w : kDefaultCopyWait;
}
int copy_withhold() { return g_copy_withhold.load(std::memory_order_relaxed); }

// ------------------------------------------------------------- planning
int device_sm_count() {
  static std::atomic<int> known[64];  // by device; a device's count does not change
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

int dense_decode_warps(int32_t D) { return D == 256 ? 2 : 4; }

DensePlan plan_dense_stream(int32_t num_seqs, int32_t units_per_seq, int32_t max_tiles, int32_t D, int32_t N,
                            int32_t raw_max, int32_t kb, int32_t vb, int32_t sb, int32_t ctas_per_sm) {
  DensePlan p{};
  // tiles a CTA has in flight: one per warp, one per warp pair at head_dim 256
  const int in_flight = D == 256 ? dense_decode_warps(D) / 2 : dense_decode_warps(D);
  const int64_t resident = static_cast<int64_t>(device_sm_count()) *
                           (ctas_per_sm > 0 ? ctas_per_sm : dense_decode_ctas_per_sm(D, N, kb, vb, sb));
  const int64_t units = static_cast<int64_t>(num_seqs) * units_per_seq;
  const int64_t most = units * std::max(0, max_tiles);
  // four tiles in flight per CTA slot at least, fewer (down to one round)
  // when the whole batch is too small to fill the GPU; a multiple of the
  // tiles in flight, the granularity of the CTA ranges
  const int64_t want = std::max<int64_t>(in_flight, std::min<int64_t>(4 * in_flight, most / resident));
  p.min_tiles = static_cast<int32_t>((want + in_flight - 1) / in_flight * in_flight);
  p.tile_slots = max_tiles > 0 ? 1 + (max_tiles - 1 + p.min_tiles - 1) / p.min_tiles : 0;
  // raw tokens per split: the size with the shortest estimated raw phase,
  // (splits per CTA slot, rounded up) x (tokens of a split + about 96 tokens'
  // worth of fixed cost per split: its query rows, barriers and merge).
  // Larger splits cost less each but can leave a few CTAs with two of them.
  p.raw_chunk = kRawChunk;
  {
    int64_t best = -1;
    for (int32_t ch = kRawChunk; ch <= 16 * kRawChunk; ch *= 2) {
      const int64_t splits = raw_max > ch ? (raw_max + ch - 1) / ch : 1;
      const int64_t rounds = (units * splits + resident - 1) / resident;
      const int64_t cost = rounds * (std::min<int64_t>(ch, std::max(0, raw_max)) + 96);
      if (best < 0 || cost < best) {
        best = cost;
        p.raw_chunk = ch;
      }
      if (splits == 1) break;
    }
  }
  p.raw_splits = raw_max > p.raw_chunk ? (raw_max + p.raw_chunk - 1) / p.raw_chunk : 1;
  p.slots = p.tile_slots + p.raw_splits;
  const int64_t tile_ctas = (most + p.min_tiles - 1) / p.min_tiles;
  const int64_t raw_items = units * p.raw_splits;
  p.ctas = static_cast<int32_t>(std::max<int64_t>(1, std::min(resident, tile_ctas + raw_items)));
  p.raw_last = tile_ctas + raw_items <= resident;
  return p;
}

DensePlan plan_dense_pieces(int32_t num_seqs, int32_t units_per_seq, int32_t max_tiles, int32_t D, int32_t N,
                            int32_t raw_max, int32_t kb, int32_t vb, int32_t sb) {
  DensePlan p{};
  const int in_flight = D == 256 ? dense_decode_warps(D) / 2 : dense_decode_warps(D);
  const int64_t resident = static_cast<int64_t>(device_sm_count()) * dense_decode_ctas_per_sm(D, N, kb, vb, sb);
  const int64_t units = static_cast<int64_t>(num_seqs) * units_per_seq;
  // a piece: as many rounds of the CTA's tiles in flight as the CTA slots
  // need when the units are half of the longest on average
  const int64_t rounds = std::max<int64_t>(1, units * max_tiles / (2 * in_flight * resident));
  p.piece = p.min_tiles = static_cast<int32_t>(std::min<int64_t>(rounds * in_flight, std::max(1, max_tiles)));
  p.tile_slots = (max_tiles + p.piece - 1) / p.piece;
  // raw records: splits of 128 down to 32 while the CTA slots hold them all
  // (a split of 32 takes about half the time of one of 128, most of it fixed)
  p.raw_chunk = kRawChunk;
  while (p.raw_chunk > 32 && units * ((raw_max + p.raw_chunk / 2 - 1) / (p.raw_chunk / 2)) <= resident) p.raw_chunk /= 2;
  p.raw_splits = raw_max > p.raw_chunk ? (raw_max + p.raw_chunk - 1) / p.raw_chunk : 1;
  p.slots = p.tile_slots + p.raw_splits;
  p.ctas = static_cast<int32_t>(std::max<int64_t>(1, std::min(resident, units * (p.tile_slots + p.raw_splits))));
  p.raw_last = 1;
  return p;
}

int64_t dense_stream_workspace_bytes(int64_t rows, int32_t D, const DensePlan& plan) {
  return rows * plan.slots * kPStride(D) * 4 + (rows * 4 + 15) / 16 * 16;
}

// CTAs of the compressed decode kernel of these widths that fit on one SM at
// once (same for fp16 and bf16 queries, which share the register and smem
// footprint); computed once per combination.
int dense_decode_ctas_per_sm(int32_t D, int32_t N, int32_t kb, int32_t vb, int32_t sb) {
  // one entry per combination, filled by whichever host thread asks first
  // (threads racing on an empty entry compute the same value)
  static std::atomic<int> cache[2][2][9][9][2] = {};
  const int di = D == 256, ni = N == 64, si = sb == 2;
  if (kb < 0 || kb > 8 || vb < 0 || vb > 8) return 1;
  const int known = cache[di][ni][kb][vb][si].load(std::memory_order_relaxed);
  if (known) return known;
  int c = 0;
  {
    if (kb == 4 && vb == 2 && sb == 4) {
      if (D == 128 && N == 128) c = resident_dense<128, 128, 4, 4, 2, 4>();
      else if (D == 128) c = resident_dense<128, 64, 4, 4, 2, 4>();
      else if (N == 128) c = resident_dense<256, 128, 2, 4, 2, 4>();
      else c = resident_dense<256, 64, 2, 4, 2, 4>();
    } else if (D == 128 && sb == 2) {
      switch (16 * kb + vb) {
#define KVARN_RES_CASE(K, V) \
  case 16 * K + V: c = resident_widths<K, V, 2>(D, N); break;
        KVARN_WIDTH_PAIRS(KVARN_RES_CASE)
#undef KVARN_RES_CASE
        default: c = 1; break;
      }
    } else if (D == 128 && sb == 4) {
      switch (16 * kb + vb) {
#define KVARN_RES_CASE(K, V) \
  case 16 * K + V: c = resident_widths<K, V, 4>(D, N); break;
        KVARN_WIDTH_PAIRS_S32(KVARN_RES_CASE)
#undef KVARN_RES_CASE
        default: c = 1; break;
      }
    } else if (D == 256 && sb == 2) {
      switch (16 * kb + vb) {
#define KVARN_RES_CASE(K, V) \
  case 16 * K + V: c = resident_widths256<K, V, 2>(N); break;
        KVARN_WIDTH_PAIRS_256(KVARN_RES_CASE)
#undef KVARN_RES_CASE
        default: c = 1; break;
      }
    } else {
      c = 1;
    }
  }
  cache[di][ni][kb][vb][si].store(c, std::memory_order_relaxed);
  return c;
}

// cuTensorMapEncodeTiled of the driver, found once through the runtime.
static PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  // a function-local static: initialised once, thread-safe
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// The cache as rows of 8-byte elements, one row per (page, KV head); the box
// is one row high and `box_bytes` wide (a page's K or V part, or one of its
// two pieces).
static cudaError_t cache_tensor_map(CUtensorMap* map, const void* cache, int64_t rows, int page_bytes,
                                    int box_bytes) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(page_bytes / 8), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(page_bytes)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / 8), 1u};
  const cuuint32_t estr[2] = {1u, 1u};
  auto encode = [&] {
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<void*>(cache), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  };
  CUresult r = encode();
  if (r == CUDA_ERROR_INVALID_CONTEXT) {
    // the driver call asks for a current context, which the runtime makes only
    // with a host thread's first call that needs one; this may be it
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);
    if (e != cudaSuccess) return e;
    r = encode();
  }
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t dense_args(const DecodeParams& p, const DensePlan& plan, DecArgs& A) {
  A = DecArgs{};
  {
    const int kb = p.k_bits ? p.k_bits : 4, vb = p.v_bits ? p.v_bits : 2, sb = p.scale_bytes ? p.scale_bytes : 4;
    const bool aff = p.codec == 1;
    const int kpart = aff ? AffinePage(p.D, kb, vb).k_part() : DensePage(p.D, p.N, kb, vb, sb).k_part();
    const int vpart = aff ? AffinePage(p.D, kb, vb).v_part() : DensePage(p.D, p.N, kb, vb, sb).v_part();
    if (p.codec != 2 && parts_gather(p.D, p.N, kpart, vpart, kb, vb)) {
      const int page = kpart + vpart;
      const int64_t rows = static_cast<int64_t>(p.num_pages) * p.num_kv_heads;
      // a part wider than one box is gathered as two (split where its
      // codes' first half ends); the second map is unused otherwise
      const int ks = gather_split(kpart, 2 * p.D * kb), vs = gather_split(vpart, 2 * p.D * vb);
      cudaError_t e = cache_tensor_map(&A.tmk, p.cache, rows, page, ks);
      if (e == cudaSuccess) e = cache_tensor_map(&A.tmv, p.cache, rows, page, vs);
      if (e == cudaSuccess && ks < kpart) e = cache_tensor_map(&A.tmk2, p.cache, rows, page, kpart - ks);
      if (e == cudaSuccess && vs < vpart) e = cache_tensor_map(&A.tmv2, p.cache, rows, page, vpart - vs);
      if (e != cudaSuccess) return e;
    }
  }
  A.q = p.q;
  A.kappa = p.sm_scale * kLog2e;
  A.cache = p.cache;
  A.Hq = p.num_q_heads;
  A.Hkv = p.num_kv_heads;
  A.G = p.num_q_heads / p.num_kv_heads;
  A.Q = p.num_queries > 0 ? p.num_queries : 1;
  A.tail_cap = p.tail_cap > 0 ? p.tail_cap : p.N;
  A.sink_tiles = (p.skip_tokens + p.sink_tokens) / p.N;
  A.sink_raw = p.sink_tokens;
  A.recent = p.recent_tokens;
  A.sink_k = p.sink_k;
  A.sink_v = p.sink_v;
  A.num_pages = p.num_pages;
  A.bt = p.block_table;
  A.bt_stride = p.bt_stride;
  A.seq_lens = p.seq_lens;
  A.max_seq_len = p.max_seq_len;
  A.tail_k = p.tail_k;
  A.tail_v = p.tail_v;
  A.ws = static_cast<float*>(p.workspace);
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * A.Q * p.num_q_heads;
  A.counts = reinterpret_cast<int32_t*>(A.ws + rows * plan.slots * kPStride(p.D));
  A.num_seqs = p.num_seqs;
  A.X = p.num_kv_heads * row_groups(A.G, A.Q);
  A.min_tiles = plan.min_tiles;
  A.tile_slots = plan.tile_slots;
  A.raw_splits = plan.raw_splits;
  A.raw_chunk = plan.raw_chunk;
  A.slots = plan.slots;
  A.piece = plan.piece;
  A.raw_last = plan.raw_last;
  A.err = p.err;
  A.bf16 = p.bf16 ? 1 : 0;
  A.partial_tiles = p.codec == 2;
  A.wait_limit = copy_wait_limit();
  A.withhold = copy_withhold();
  return cudaSuccess;
}

cudaError_t run_decode_kernel(const DecodeParams& p, const DecArgs& A, int ctas, cudaStream_t st) {
  cudaError_t e = cudaErrorInvalidValue;
  const int kb = p.k_bits ? p.k_bits : 4, vb = p.v_bits ? p.v_bits : 2, sb = p.scale_bytes ? p.scale_bytes : 4;
  if (p.codec == 2) {  // the uncompressed fp16 pages (tiles of 32 tokens)
    return p.D == 128   ? run_raw<128>(A, ctas, st)
           : p.D == 256 ? run_raw<256>(A, ctas, st)
                        : cudaErrorInvalidValue;
  }
  if (p.codec == 1) {
    if (p.D != 128 || p.N != 128 || kb != vb) return cudaErrorInvalidValue;
    switch (kb) {
#define KVARN_AFF_CASE(K) \
  case K: e = run_affine_widths<K>(A, p.bf16, ctas, st); break;
      KVARN_AFFINE_WIDTHS(KVARN_AFF_CASE)
#undef KVARN_AFF_CASE
      default: break;
    }
    return e;
  }
  if (A.stats) {
#define KVARN_MASS_CASE(K, V, S) \
  if (kb == K && vb == V && sb == S) return run_mass_widths<K, V, S>(A, p.D, p.N, ctas, st);
    KVARN_MASS_WIDTHS(KVARN_MASS_CASE)
#undef KVARN_MASS_CASE
    return cudaErrorInvalidValue;
  }
  if (kb == 4 && vb == 2 && sb == 4) {
#define KV_DISPATCH(DD, NN, WW)                                                              \
  if (p.D == DD && p.N == NN)                                                                \
    e = run_dense<DD, NN, WW, 4, 2, 4>(A, ctas, st);
    KV_DISPATCH(128, 128, 4)
    KV_DISPATCH(128, 64, 4)
    KV_DISPATCH(256, 128, 2)
    KV_DISPATCH(256, 64, 2)
#undef KV_DISPATCH
  } else if (sb == 2 && p.D == 256) {
    switch (16 * kb + vb) {
#define KVARN_RUN_CASE(K, V) \
  case 16 * K + V: e = run_dense_widths256<K, V, 2>(A, p.N, p.bf16, ctas, st); break;
      KVARN_WIDTH_PAIRS_256(KVARN_RUN_CASE)
#undef KVARN_RUN_CASE
      default: break;
    }
  } else if (sb == 2) {
    switch (16 * kb + vb) {
#define KVARN_RUN_CASE(K, V) \
  case 16 * K + V: e = run_dense_widths<K, V, 2>(A, p.D, p.N, p.bf16, ctas, st); break;
      KVARN_WIDTH_PAIRS(KVARN_RUN_CASE)
#undef KVARN_RUN_CASE
      default: break;
    }
  } else if (sb == 4 && p.D == 128) {
    switch (16 * kb + vb) {
#define KVARN_RUN_CASE(K, V) \
  case 16 * K + V: e = run_dense_widths<K, V, 4>(A, p.D, p.N, p.bf16, ctas, st); break;
      KVARN_WIDTH_PAIRS_S32(KVARN_RUN_CASE)
#undef KVARN_RUN_CASE
      default: break;
    }
  }
  return e;
}

// The merge, and beside it in the same launch (CTAs from merge_ctas on) the
// attention mass of the tiles: weights summed over the query heads, from each
// head's (maximum, sum) of the tile and of its whole row, l 2^(m - M) / L. A
// mass CTA takes 32 tiles of a sequence: its threads form M and 1 / L of up
// to 128 heads from the decode's partials (so that it does not wait for the
// merge), then a warp takes every fourth head and the lanes the tiles, whose
// pairs are contiguous; the warps' sums are added in a fixed order. Reads 8
// bytes per head and tile; two dependent trips to memory bound it: 16
// sequences of 128 tiles and 64 heads 6.9 us with the merge under a profiler,
// 7 ragged ones of 32 heads 5.2.
template <int D>
__global__ void __launch_bounds__(128) merge_mass_kernel(const __grid_constant__ DecArgs A, int N, int rows,
                                                         int merge_ctas, int mass_x, float* out, float* lse,
                                                         const float* mass_in, float* mass_out, int mass_stride,
                                                         float decay) {
  constexpr int S = kPStride(D);
  __shared__ float2 whole[128];  // M, 1 / L of a head
  __shared__ float part[4][32];
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (static_cast<int>(blockIdx.x) < merge_ctas) {
    const int row = blockIdx.x * 4 + warp;
    if (row < rows) merge_row<D, true>(A.ws, A.slots, row, A.counts, 0, A.tile_slots, out, lse);
    return;
  }
  const int item = blockIdx.x - merge_ctas, b = item / mass_x;
  const int t = item % mass_x * 32 + lane, C = seq_tiles(A, N, b);
  float sum = 0.f;
  for (int h0 = 0; h0 < A.Hq; h0 += 128) {
    const int h = h0 + threadIdx.x;
    if (h < A.Hq) {
      const int row = b * A.Hq + h, nt = min(A.counts[row], A.tile_slots);
      const float* P = A.ws + static_cast<int64_t>(row) * A.slots * S;
      float M = -INFINITY, L = 0.f;
      for (int s0 = 0; s0 < A.slots; s0 += 8) {  // eight slots in flight
        float2 v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int s = s0 + i;
          const bool used = s < A.slots && (s < nt || s >= A.tile_slots);
          v[i] = used ? *reinterpret_cast<const float2*>(P + s * S) : make_float2(-INFINITY, 0.f);
        }
        float Mn = M;
#pragma unroll
        for (int i = 0; i < 8; ++i) Mn = fmaxf(Mn, v[i].x);
        if (Mn == -INFINITY) continue;
        L *= exp2f(M - Mn);
#pragma unroll
        for (int i = 0; i < 8; ++i) L = fmaf(v[i].y, exp2f(v[i].x - Mn), L);
        M = Mn;
      }
      whole[threadIdx.x] = make_float2(M, L > 0.f ? 1.f / L : 0.f);
    }
    __syncthreads();
    if (t < C) {
      const float2* st = A.stats + (static_cast<int64_t>(b) * A.Hq + h0) * A.stat_tiles + t;
      const int n = min(128, A.Hq - h0);
#pragma unroll 8
      for (int i = warp; i < n; i += 4) {
        const float2 v = st[static_cast<int64_t>(i) * A.stat_tiles], w = whole[i];
        sum = fmaf(v.y, exp2f(v.x - w.x) * w.y, sum);
      }
    }
    __syncthreads();
  }
  part[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && t < A.stat_tiles) {
    const int64_t at = static_cast<int64_t>(b) * mass_stride + t;
    sum = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    // decay 0 does not look at what was there (it may be anything)
    mass_out[at] = t >= C ? 0.f : decay == 0.f ? sum : fmaf(decay, mass_in[at], sum);
  }
}

int64_t mass_workspace_bytes(int64_t rows, int32_t max_tiles) { return (rows * max_tiles * 8 + 15) / 16 * 16; }

template <int D>
static cudaError_t launch_merge_mass(const DecArgs& A, int rows, const DecodeParams& p, cudaStream_t st) {
  const int merge_ctas = (rows + 3) / 4, mass_x = (A.stat_tiles + 31) / 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(merge_ctas + mass_x * p.num_seqs);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, merge_mass_kernel<D>, A, p.N, rows, merge_ctas, mass_x, p.out, p.lse, p.mass_in,
                            p.mass_out, p.mass_stride, p.mass_decay);
}

cudaError_t launch_decode_dense(const DecodeParams& p, const DensePlan& plan, cudaStream_t st) {
  if (p.num_seqs == 0) return cudaSuccess;
  DecArgs A;
  cudaError_t e = dense_args(p, plan, A);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * A.Q * p.num_q_heads;
  if (p.mass_out) {
    A.stat_tiles = p.max_seq_len / p.N;
    A.stats = reinterpret_cast<float2*>(static_cast<char*>(p.workspace) + dense_stream_workspace_bytes(rows, p.D, plan));
  }
  e = run_decode_kernel(p, A, plan.ctas, st);
  if (e != cudaSuccess) return e;
  if (p.codec != 0)  // the affine and fp16 pages are in the original basis
    return p.D == 128 ? launch_merge<128, false>(A.ws, A.slots, rows, A.counts, 0, A.tile_slots, p.out, p.lse, st)
                      : launch_merge<256, false>(A.ws, A.slots, rows, A.counts, 0, A.tile_slots, p.out, p.lse, st);
  if (p.mass_out && A.stat_tiles > 0)
    return p.D == 128 ? launch_merge_mass<128>(A, static_cast<int>(rows), p, st)
                      : launch_merge_mass<256>(A, static_cast<int>(rows), p, st);
  return p.D == 128 ? launch_merge<128>(A.ws, A.slots, rows, A.counts, 0, A.tile_slots, p.out, p.lse, st)
                    : launch_merge<256>(A.ws, A.slots, rows, A.counts, 0, A.tile_slots, p.out, p.lse, st);
}

}  // namespace kvarn
