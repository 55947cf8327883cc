// Eviction of whole tiles by accumulated attention mass, sm_103a.
//
// A sequence of C committed tiles over its budget keeps its first `sink` and
// newest `recent` tiles and, of the others, those of the largest mass, equal
// ones by the lowest index. The order of the kept tiles does not change (the
// decode takes a sequence's tiles in any order; the raw tail follows them).
//
// A cluster of CTAs per sequence, each with a consecutive range of its tiles
// (one CTA where the whole row has at most kOneCta tiles). The masses become
// 32-bit keys of the same order; the smallest kept key is found by radix
// selection, eight bits a pass from the top: every CTA counts its tiles'
// digits in shared memory (each warp adds its equal digits at once), the
// cluster meets, and every CTA adds up all histograms through distributed
// shared memory and finds the same digit. The last pass also says how many
// tiles of that key stay. Each CTA then counts its kept tiles, the cluster
// meets again, and the counts of the ranges before it give a CTA's first
// output rank. Page ids and masses were read into shared memory before that
// meeting, so that the outputs may be the inputs. Rows whose ranges do not
// fit shared memory take one CTA, which reads its keys again in every pass
// and compacts chunk by chunk.
// Latency bounds it: six cluster meetings (four passes, the counts, the one
// before the fill) and two trips to memory. 8 sequences of up to 16384 tiles
// take 20 us (one CTA per sequence 50), 32 of up to 128 tiles 11, of which the
// launch and the host are the most.
#include <cooperative_groups.h>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace cg = cooperative_groups;

namespace kvarn {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kCluster = 8;
constexpr int kOneCta = 512;             // tiles that one CTA takes alone
constexpr int kEvictSmem = 200 * 1024;   // dynamic shared memory of a range

// Total order of the masses: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// Exclusive block scan of two 16-bit counts packed in a word; returns the
// thread's exclusive value, and the block's sum in *total. `sums` alternates
// between two buffers so that one barrier a scan is enough after the sums.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  uint32_t s = sums[lane];  // every warp scans the warps' sums
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += y;
  }
  *total = __shfl_sync(0xffffffffu, s, 31);
  const uint32_t upto = __shfl_sync(0xffffffffu, s, warp ? warp - 1 : 0);
  return (warp ? upto : 0u) + x - v;
}

template <int PPT>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams A) {
  extern __shared__ __align__(16) unsigned char dyn[];
  __shared__ __align__(16) uint32_t hist[4][256];
  __shared__ uint32_t sums[2][32], found[4][2];
  __shared__ uint32_t counts[2];  // this CTA's tiles that surely stay, and its ties
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.y, tid = threadIdx.x, nc = gridDim.x, rank_in = blockIdx.x;  // the cluster is grid row b
  const int N = PPT * kPageTokens;
  int len = A.seq_lens[b];
  if (len < 0 || len > A.max_seq_len) {
    if (tid == 0) set_error(A.err, KVARN_DEVERR_SEQ_LEN);
    len = len < 0 ? 0 : A.max_seq_len;
  }
  const int C = len / N, most = A.max_seq_len / N;
  const float* mass = A.mass + static_cast<int64_t>(b) * A.mass_stride;
  const int32_t* table = A.table + static_cast<int64_t>(b) * A.bt_stride;
  float* mass_out = A.mass_out + static_cast<int64_t>(b) * A.mass_stride;
  int32_t* table_out = A.table_out + static_cast<int64_t>(b) * A.bt_stride;
  int32_t* freed = A.freed + static_cast<int64_t>(b) * A.bt_stride;
  const bool cut = C > A.keep;
  const int lo = A.sink, hi = C - A.recent;  // tiles that may go: [lo, hi)
  // this CTA's tiles [r0, r1), held in shared memory if the ranges fit
  const int per = (C + nc - 1) / nc, r0 = min(C, rank_in * per), r1 = min(C, r0 + per), n = r1 - r0;
  const bool held = A.held;
  float* mass_s = reinterpret_cast<float*>(dyn);
  int32_t* page_s = reinterpret_cast<int32_t*>(dyn) + A.range;
  if (held) {
    for (int i = tid; i < n; i += kEvictThreads) mass_s[i] = mass[r0 + i];
    const int32_t* src = table + static_cast<int64_t>(r0) * PPT;
    if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
      for (int i = tid; i < n * PPT / 4; i += kEvictThreads)
        reinterpret_cast<int4*>(page_s)[i] = reinterpret_cast<const int4*>(src)[i];
    } else {
      for (int i = tid; i < n * PPT; i += kEvictThreads) page_s[i] = src[i];
    }
  }
  for (int i = tid; i < 4 * 256; i += kEvictThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto mass_at = [&](int t) { return held ? mass_s[t - r0] : mass[t]; };

  uint32_t thr = 0;  // smallest kept key
  int ties = 0;      // tiles of that key that stay
  if (cut) {         // the same in every CTA of the cluster
    int want = A.keep - A.sink - A.recent;  // tiles of [lo, hi) that stay
    if (want == 0) {
      thr = 0xffffffffu;
    } else {
      const int l0 = max(lo, r0), l1 = min(hi, r1);
      for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        const uint32_t mask = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
        for (int t0 = l0; t0 < l1; t0 += kEvictThreads) {
          const int t = t0 + tid;
          uint32_t k = 0;
          bool on = t < l1;
          if (on) {
            k = mass_key(mass_at(t));
            on = (k & mask) == thr;
          }
          const uint32_t digit = on ? (k >> shift) & 255u : 256u;
          const unsigned same = __match_any_sync(0xffffffffu, digit);
          if (on && (same & ((1u << (tid & 31)) - 1)) == 0) atomicAdd(&hist[pass][digit], __popc(same));
        }
        if (nc > 1) cluster.sync();
        else __syncthreads();
        if (tid < 32) {
          // digits from the top: lane l holds digits 255 - 8 l down to 248 - 8 l
          uint32_t c[8] = {0, 0, 0, 0, 0, 0, 0, 0}, sum = 0;
          for (int r = 0; r < nc; ++r) {
            const uint32_t* h = nc > 1 ? cluster.map_shared_rank(&hist[pass][0], r) : &hist[pass][0];
            const uint4 x = *reinterpret_cast<const uint4*>(h + 252 - 8 * tid);
            const uint4 y = *reinterpret_cast<const uint4*>(h + 248 - 8 * tid);
            c[0] += x.w;
            c[1] += x.z;
            c[2] += x.y;
            c[3] += x.x;
            c[4] += y.w;
            c[5] += y.z;
            c[6] += y.y;
            c[7] += y.x;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += c[j];
          uint32_t incl = sum;
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
            if (tid >= o) incl += y;
          }
          uint32_t above = incl - sum;
          if (above < static_cast<uint32_t>(want) && incl >= static_cast<uint32_t>(want)) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (above < static_cast<uint32_t>(want) && above + c[j] >= static_cast<uint32_t>(want)) {
                found[pass][0] = 255 - 8 * tid - j;
                found[pass][1] = above;
              }
              above += c[j];
            }
          }
        }
        __syncthreads();
        thr |= found[pass][0] << shift;
        want -= static_cast<int>(found[pass][1]);
      }
      ties = want;
    }
  }

  // ---- tiles of this range that stay, by kind, and those of the ranges before
  auto kind = [&](int t, float m) -> uint32_t {  // 1: surely, 1 << 16: a tie, 0: neither
    if (!cut || t < lo || t >= hi) return 1u;
    const uint32_t k = mass_key(m);
    return k > thr ? 1u : k == thr ? 1u << 16 : 0u;
  };
  int kept_before = 0, ties_before = 0;
  if (nc > 1) {
    uint32_t s = 0, e = 0;
    for (int t = r0 + tid; t < r1; t += kEvictThreads) {
      const uint32_t k = kind(t, mass_at(t));
      s += k & 1u;
      e += k >> 16;
    }
    s = __reduce_add_sync(0xffffffffu, s);
    e = __reduce_add_sync(0xffffffffu, e);
    if ((tid & 31) == 0) {
      sums[0][tid >> 5] = s;
      sums[1][tid >> 5] = e;
    }
    __syncthreads();
    if (tid < 32) {
      s = __reduce_add_sync(0xffffffffu, sums[0][tid]);
      e = __reduce_add_sync(0xffffffffu, sums[1][tid]);
      if (tid == 0) {
        counts[0] = s;
        counts[1] = e;
      }
    }
    cluster.sync();  // every range is read and counted
    for (int r = 0; r < rank_in; ++r) {
      const uint32_t* c = cluster.map_shared_rank(&counts[0], r);
      kept_before += static_cast<int>(c[0]);
      ties_before += static_cast<int>(c[1]);
    }
  }

  // ---- compaction of the range in chunks, in order
  for (int t0 = r0, buf = 0; t0 < r1; t0 += kEvictThreads, buf ^= 1) {
    const int t = t0 + tid;
    uint32_t k = 0;
    float m = 0.f;
    int32_t page[PPT];
    if (t < r1) {
      m = mass_at(t);
#pragma unroll
      for (int j = 0; j < PPT; ++j) page[j] = held ? page_s[(t - r0) * PPT + j] : table[static_cast<int64_t>(t) * PPT + j];
      k = kind(t, m);
    }
    uint32_t total;
    const uint32_t ex = block_scan(k, sums[buf], &total);
    const int tie_rank = ties_before + static_cast<int>(ex >> 16);
    const int rank = kept_before + static_cast<int>(ex & 0xffffu) + min(tie_rank, ties);
    if (t < r1) {
      int32_t* dst;
      if (k == 1u || (k != 0u && tie_rank < ties)) {
        mass_out[rank] = m;
        dst = table_out + static_cast<int64_t>(rank) * PPT;
      } else {
        dst = freed + static_cast<int64_t>(t - rank) * PPT;
      }
      if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
#pragma unroll
        for (int j = 0; j < PPT; j += 4)
          *reinterpret_cast<int4*>(dst + j) = make_int4(page[j], page[j + 1], page[j + 2], page[j + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < PPT; ++j) dst[j] = page[j];
      }
    }
    kept_before += static_cast<int>(total & 0xffffu);
    ties_before += static_cast<int>(total >> 16);
  }

  // ---- behind the kept tiles and the freed pages: every CTA fills its share
  const int kept = cut ? A.keep : C, gone = C - kept;
  const int step = kEvictThreads * nc, at = rank_in * kEvictThreads + tid;
  // a chunk's late threads may still read their inputs; and with several
  // CTAs no one leaves while another reads its counts
  if (nc > 1) cluster.sync();
  else __syncthreads();
  for (int t = kept + at; t < most; t += step) mass_out[t] = 0.f;
  for (int64_t i = static_cast<int64_t>(kept) * PPT + at; i < static_cast<int64_t>(most) * PPT; i += step) table_out[i] = -1;
  for (int64_t i = static_cast<int64_t>(gone) * PPT + at; i < static_cast<int64_t>(most) * PPT; i += step) freed[i] = -1;
  if (tid == 0 && rank_in == 0) {
    A.lens_out[b] = len - gone * N;
    A.freed_count[b] = gone * PPT;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t st) {
  EvictParams A = p;
  const int tiles = A.max_seq_len / A.N, ppt = A.N / kPageTokens;
  // a cluster where one CTA would walk several chunks and the ranges fit
  int nc = tiles > kOneCta ? kCluster : 1;
  A.range = (tiles + nc - 1) / nc;
  A.range = (A.range + 3) / 4 * 4;  // keeps the page ids 16-byte aligned
  A.held = static_cast<int64_t>(A.range) * 4 * (1 + ppt) <= kEvictSmem;
  if (!A.held) nc = 1;
  const int smem = A.held ? A.range * 4 * (1 + ppt) : 0;
  auto kern = A.N == 128 ? evict_kernel<8> : evict_kernel<4>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvictSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, A.num_seqs);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, A);
}

}  // namespace kvarn
