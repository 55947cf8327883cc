// Eviction of whole tiles by accumulated attention mass, sm_103a.
//
// A sequence of C committed tiles over its budget keeps its first `sink` and
// newest `recent` tiles and, of the others, those of the largest mass, equal
// ones by the lowest index. The order of the kept tiles does not change (the
// decode takes a sequence's tiles in any order; the raw tail follows them).
//
// One CTA per sequence. The masses become 32-bit keys of the same order; the
// smallest kept key is found by radix selection, eight bits a pass from the
// top (a histogram in shared memory, each warp adding its equal digits at
// once), which also says how many of the tiles with that key stay. Then
// chunks of 1024 tiles are compacted in order: a block scan ranks the kept
// tiles, whose page ids and masses are read before any thread writes, so that
// the outputs may be the inputs. Latency bounds it: a dozen block barriers
// and one chain of loads per pass.
#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace kvarn {

namespace {

constexpr int kEvictThreads = 1024;
constexpr int kKeyCap = 24576;  // keys kept in shared memory (96 KB); longer rows are read again each pass

// Total order of the masses: NaN below everything, -0 equal to +0.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t u = __float_as_uint(m + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

// Exclusive block scan of two 16-bit counts packed in a word; returns the
// thread's exclusive value, and the block's sum in *total.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sums, uint32_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint32_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  *total = warp_sums[31];
  const uint32_t before = warp ? warp_sums[warp - 1] : 0u;
  __syncthreads();  // warp_sums is written again by the next scan
  return before + x - v;
}

template <int PPT>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams A) {
  extern __shared__ uint32_t keys[];
  __shared__ uint32_t hist[256], warp_sums[32], found[2];
  const int b = blockIdx.x, tid = threadIdx.x;
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
  uint32_t thr = 0;  // smallest kept key
  int ties = 0;      // tiles of that key that stay
  const bool in_smem = cut && C <= A.key_cap;
  if (cut) {
    if (in_smem)
      for (int t = tid; t < C; t += kEvictThreads) keys[t] = mass_key(mass[t]);
    int want = A.keep - A.sink - A.recent;  // tiles of [lo, hi) that stay
    if (want == 0) {
      thr = 0xffffffffu;
    } else {
      uint32_t prefix = 0;
      for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
        const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int t0 = lo; t0 < hi; t0 += kEvictThreads) {
          const int t = t0 + tid;
          uint32_t k = 0;
          bool on = t < hi;
          if (on) {
            k = in_smem ? keys[t] : mass_key(mass[t]);
            on = (k & mask) == prefix;
          }
          const uint32_t digit = on ? (k >> shift) & 255u : 256u;
          const unsigned same = __match_any_sync(0xffffffffu, digit);
          if (on && (same & ((1u << (tid & 31)) - 1)) == 0) atomicAdd(hist + digit, __popc(same));
        }
        __syncthreads();
        if (tid < 32) {
          // digits from the top: lane l holds digits 255 - 8 l down to 248 - 8 l
          uint32_t c[8], sum = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) sum += c[j] = hist[255 - 8 * tid - j];
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
                found[0] = 255 - 8 * tid - j;
                found[1] = above;
              }
              above += c[j];
            }
          }
        }
        __syncthreads();
        prefix |= found[0] << shift;
        want -= static_cast<int>(found[1]);
        // hist and found are rewritten after the next pass's barrier; `found`
        // is read by every thread before that
      }
      thr = prefix;
      ties = want;
    }
  }
  __syncthreads();

  int kept_before = 0, ties_before = 0;  // over the chunks so far: tiles above the threshold or safe, ties
  int out_at = 0;
  for (int t0 = 0; t0 < C; t0 += kEvictThreads) {
    const int t = t0 + tid;
    bool sure = false, tie = false;
    float m = 0.f;
    int32_t page[PPT];
    if (t < C) {
      m = mass[t];
#pragma unroll
      for (int j = 0; j < PPT; ++j) page[j] = table[static_cast<int64_t>(t) * PPT + j];
      const uint32_t k = mass_key(m);
      sure = !cut || t < lo || t >= hi || k > thr;
      tie = !sure && k == thr;
    }
    uint32_t total;
    const uint32_t ex = block_scan((sure ? 1u : 0u) | (tie ? 1u << 16 : 0u), warp_sums, &total);
    const int tie_rank = ties_before + static_cast<int>(ex >> 16);
    const int rank = kept_before + static_cast<int>(ex & 0xffffu) + min(tie_rank, ties);
    const bool stays = sure || (tie && tie_rank < ties);
    if (t < C) {
      if (stays) {
        mass_out[rank] = m;
#pragma unroll
        for (int j = 0; j < PPT; ++j) table_out[static_cast<int64_t>(rank) * PPT + j] = page[j];
      } else {
#pragma unroll
        for (int j = 0; j < PPT; ++j) freed[static_cast<int64_t>(t - rank) * PPT + j] = page[j];
      }
    }
    kept_before += static_cast<int>(total & 0xffffu);
    ties_before += static_cast<int>(total >> 16);
    out_at = kept_before + min(ties_before, ties);
  }
  const int gone = C - out_at;
  for (int t = out_at + tid; t < most; t += kEvictThreads) mass_out[t] = 0.f;
  for (int64_t i = static_cast<int64_t>(out_at) * PPT + tid; i < static_cast<int64_t>(most) * PPT; i += kEvictThreads)
    table_out[i] = -1;
  for (int64_t i = static_cast<int64_t>(gone) * PPT + tid; i < static_cast<int64_t>(most) * PPT; i += kEvictThreads)
    freed[i] = -1;
  if (tid == 0) {
    A.lens_out[b] = len - gone * N;
    A.freed_count[b] = gone * PPT;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t st) {
  EvictParams A = p;
  A.key_cap = kKeyCap;
  const int tiles = A.max_seq_len / A.N;
  const int smem = 4 * (tiles < kKeyCap ? tiles : kKeyCap);
  auto kern = A.N == 128 ? evict_kernel<8> : evict_kernel<4>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kKeyCap);
  if (e != cudaSuccess) return e;
  kern<<<A.num_seqs, kEvictThreads, smem, st>>>(A);
  return cudaGetLastError();
}

}  // namespace kvarn
