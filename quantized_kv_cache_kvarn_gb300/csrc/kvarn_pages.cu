// Pages of a cache: sequences that fork, end and leave their windows, and the
// compaction of what is left, sm_103a.
//
// Fork. Whole tiles are never written again, so a sequence that forks shares
// its pages: its table row is copied and the pages' reference counts rise;
// only the raw tail rows are copied. Three kernels, chained as programmatic
// dependents:
//   copy   tails (live rows), lengths, tables; the counts to their new place
//   count  an old row's pages by (children that keep them) - 1, nothing where
//          that is 0; a page whose count passes between above 0 and not above
//          turns its bit in a bitmap kept where the list of freed pages will be
//   list   one cluster turns the bitmap into the list, in order
// The counts are whole numbers and a bit says how often a count has passed, odd
// or even, so the order of the atomics does not matter, whatever the counts.
//
// Compact. n live pages move to the lowest ids: the k-th free page below n
// (a hole) receives the k-th live page at or above n. Up to three kernels: live
// pages per block of pages; their prefix sums and with them the list of
// moves; the moves, beside the tables. A page's move is read and written once
// (HBM bounds it), a hole is never a source, so moves need no order.
//
// Measured: 32 sequences of 2000 to 16384 tokens that fork among four beams 12
// us on the GPU, 512 of an 8-bit cache of 1.3 million pages behind a window 21 us
// (41 MB), both bound by the three launches' latencies; 126 MB of pages moved
// (252 MB of traffic) 52 us, of which the moves 36 to 43, 0.9 of the measured
// copy bandwidth and more.
#include <cooperative_groups.h>

#include <algorithm>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace cg = cooperative_groups;

namespace kvarn {

namespace {

constexpr int kThreads = 256, kWarpsPerCta = kThreads / 32;
constexpr int kPiece = 4096;      // bytes a warp copies at a time, all in flight
constexpr int kCopyCtas = 4;      // resident CTAs of the kernels that copy: 126 MB of pages in 53 us, 68 with six
constexpr int kEntries = 256;     // table entries a warp takes at a time
constexpr int kCounts = 1024;       // reference counts a warp takes at a time
constexpr int kPagesPerCta = 2048;  // compaction: pages of a block

// Compaction: up to so many pages every CTA of the plan counts for itself what
// is in use, without a kernel for the blocks' sums: 6.2 us against 8.2 for 1531
// pages, 8.8 against 9.7 for 16384, 12.3 against 10.9 for 32768.
constexpr int kDirectPages = 16384;

// `bytes` (a multiple of 16) by one warp, at most kPiece.
__device__ __forceinline__ void copy_piece(void* dst, const void* src, int bytes) {
  const int lane = threadIdx.x & 31;
  const uint4* s = static_cast<const uint4*>(src);
  uint4* d = static_cast<uint4*>(dst);
  const int n = bytes >> 4;
  uint4 v[kPiece / 512];
#pragma unroll
  for (int i = 0; i < kPiece / 512; ++i)
    if (lane + 32 * i < n) v[i] = s[lane + 32 * i];
#pragma unroll
  for (int i = 0; i < kPiece / 512; ++i)
    if (lane + 32 * i < n) d[lane + 32 * i] = v[i];
}

// ---------------------------------------------------------------- fork
__device__ __forceinline__ int length_of(const ForkParams& A, int a) {
  const int L = A.seq_lens[a];
  if (L < 0 || L > A.max_seq_len) {
    set_error(A.err, KVARN_DEVERR_SEQ_LEN);
    return min(max(L, 0), A.max_seq_len);
  }
  return L;
}

// The old row of new row b, or -1.
__device__ __forceinline__ int parent_of(const ForkParams& A, int b) {
  const int p = A.parents[b];
  if (p >= A.num_in) {
    set_error(A.err, KVARN_DEVERR_INDEX);
    return -1;
  }
  return p < 0 ? -1 : p;
}

__device__ __forceinline__ int whole_tiles(const ForkParams& A, int L) { return max(0, L - A.recent) / A.N; }

// Entries that the next token of a sequence of L tokens, or its sinks, sees:
// those below `sinks` and those from `first` on.
struct Seen {
  int sinks, first;
  __device__ __forceinline__ Seen(const ForkParams& A, int L) : sinks(0), first(0) {
    if (A.window == 0) return;
    const int s = min(A.sinks, A.max_seq_len);
    sinks = (s / A.N + (s % A.N != 0)) * A.pages_per_tile;
    // tile t holds a token after position L - window where t >= (L + 1 - window) / N
    first = max(0, L - (A.window - 1)) / A.N * A.pages_per_tile;
  }
  __device__ __forceinline__ bool operator()(int e) const { return e < sinks || e >= first; }
};

// Entry e of old row a, which holds `held`: the page, -1 where there is none.
__device__ __forceinline__ int entry_of(const ForkParams& A, int a, int held, int e) {
  if (e >= held) return -1;
  const int id = A.table[static_cast<int64_t>(a) * A.bt_stride + e];
  if (id >= A.num_pages) {
    set_error(A.err, KVARN_DEVERR_PAGE_RANGE);
    return -1;
  }
  return id < 0 ? -1 : id;
}

// Items of a warp: pieces of the tails, pieces of the table rows (with the
// lengths), pieces of the counts, each item one chain of loads. Four CTAs an SM
// leave it 64 registers, of which 56 bytes spill.
__global__ void __launch_bounds__(kThreads, kCopyCtas) fork_copy_kernel(const __grid_constant__ ForkParams A) {
  pdl_wait_primary();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarpsPerCta;
  const int pieces = max(1, (A.entries + kEntries - 1) / kEntries);
  const int64_t table_items = static_cast<int64_t>(A.num_out) * pieces, count_items = (A.num_pages + kCounts - 1) / kCounts;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
       i < A.tail_pieces + table_items + count_items; i += warps) {
    if (i < A.tail_pieces) {
      int k = 0;
      int64_t j = i;
      while (j >= A.rows[k].pieces) j -= A.rows[k++].pieces;
      const ForkRows& R = A.rows[k];
      const int64_t size = static_cast<int64_t>(R.capacity) * R.row_bytes, per = (size + kPiece - 1) / kPiece;
      const int64_t unit = j / per;
      const int b = static_cast<int>(unit / R.heads), h = static_cast<int>(unit % R.heads);
      const int p = parent_of(A, b);
      if (p < 0) continue;
      const int L = length_of(A, p);
      const int live = R.whole ? R.capacity : min(R.capacity, L - whole_tiles(A, L) * A.N);
      const int64_t at = (j - unit * per) * kPiece, end = live * R.row_bytes;
      if (at >= end) continue;
      copy_piece(static_cast<char*>(R.out) + unit * size + at,
                 static_cast<const char*>(R.in) + (static_cast<int64_t>(p) * R.heads + h) * size + at,
                 static_cast<int>(min(static_cast<int64_t>(kPiece), end - at)));
    } else if (i < A.tail_pieces + table_items) {
      const int64_t j = i - A.tail_pieces;
      const int b = static_cast<int>(j / pieces), e0 = static_cast<int>(j % pieces) * kEntries;
      const int p = parent_of(A, b);
      const int L = p < 0 ? 0 : length_of(A, p), held = p < 0 ? 0 : whole_tiles(A, L) * A.pages_per_tile;
      const Seen seen(A, L);
      if (e0 == 0 && lane == 0) A.lens_out[b] = L;
      int v[kEntries / 32];
#pragma unroll
      for (int k = 0; k < kEntries / 32; ++k) {
        const int e = e0 + 32 * k + lane;
        v[k] = seen(e) ? entry_of(A, p, held, e) : -1;
      }
#pragma unroll
      for (int k = 0; k < kEntries / 32; ++k) {
        const int e = e0 + 32 * k + lane;
        if (e < A.entries) A.table_out[static_cast<int64_t>(b) * A.bt_stride + e] = v[k];
      }
    } else {
      // the counts, an empty bitmap, -1 behind it
      const int words = (A.num_pages + 31) / 32, p0 = static_cast<int>(i - A.tail_pieces - table_items) * kCounts;
      const bool copy = A.refs_out != A.refs;
      if (A.vectors && p0 + kCounts <= A.num_pages) {
        int4 v[kCounts / 128];
        if (copy) {
#pragma unroll
          for (int k = 0; k < kCounts / 128; ++k) v[k] = reinterpret_cast<const int4*>(A.refs + p0)[32 * k + lane];
#pragma unroll
          for (int k = 0; k < kCounts / 128; ++k) reinterpret_cast<int4*>(A.refs_out + p0)[32 * k + lane] = v[k];
        }
#pragma unroll
        for (int k = 0; k < kCounts / 128; ++k) {
          const int at = p0 + 4 * (32 * k + lane);
          reinterpret_cast<int4*>(A.freed + p0)[32 * k + lane] =
              make_int4(at < words ? 0 : -1, at + 1 < words ? 0 : -1, at + 2 < words ? 0 : -1, at + 3 < words ? 0 : -1);
        }
      } else {
        for (int at = p0 + lane; at < min(A.num_pages, p0 + kCounts); at += 32) {
          if (copy) A.refs_out[at] = A.refs[at];
          A.freed[at] = at < words ? 0 : -1;
        }
      }
    }
  }
}

// Children of every old row, counted by each CTA for itself, then the rows'
// entries a warp at a time. What is read before pdl_wait_primary no kernel of
// this call writes, and what came before the call had finished when the copy
// kernel let this one start.
__global__ void __launch_bounds__(kThreads) fork_count_kernel(const __grid_constant__ ForkParams A) {
  extern __shared__ int children[];
  for (int a = threadIdx.x; a < A.num_in; a += kThreads) children[a] = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < A.num_out; b += kThreads) {
    const int p = A.parents[b];
    if (p >= 0 && p < A.num_in) atomicAdd(&children[p], 1);
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, pieces = (A.entries + kEntries - 1) / kEntries;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarpsPerCta;
  bool waited = false;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5);
       i < static_cast<int64_t>(A.num_in) * pieces; i += warps) {
    const int a = static_cast<int>(i / pieces), e0 = static_cast<int>(i % pieces) * kEntries;
    const int c = children[a];
    if (c == 1 && A.window == 0) continue;
    const int L = length_of(A, a), held = whole_tiles(A, L) * A.pages_per_tile;
    if (e0 >= held) continue;
    const Seen seen(A, L);
    int id[kEntries / 32], d[kEntries / 32];
#pragma unroll
    for (int k = 0; k < kEntries / 32; ++k) {
      const int e = e0 + 32 * k + lane;
      d[k] = (seen(e) ? c : 0) - 1;
      id[k] = d[k] && e < A.entries ? entry_of(A, a, held, e) : -1;
    }
    if (!waited) pdl_wait_primary();
    waited = true;
    // all atomics of the piece in flight together
    int old[kEntries / 32];
#pragma unroll
    for (int k = 0; k < kEntries / 32; ++k) old[k] = id[k] >= 0 ? atomicAdd(A.refs_out + id[k], d[k]) : 0;
#pragma unroll
    for (int k = 0; k < kEntries / 32; ++k)
      if (id[k] >= 0 && (old[k] > 0) != (old[k] + d[k] > 0))
        atomicXor(A.freed + (id[k] >> 5), static_cast<int>(1u << (id[k] & 31)));
  }
  // the list kernel may start once every CTA is here, and waits for the end
  if (!waited) pdl_wait_primary();
  pdl_launch_dependents();
}

constexpr int kListCtas = 8, kListThreads = 1024;

// One cluster: thread t takes an equal run of the bitmap's words. Nothing is
// written before every word has been read (the list takes their place).
__global__ void __cluster_dims__(kListCtas, 1, 1) __launch_bounds__(kListThreads) fork_list_kernel(const __grid_constant__ ForkParams A) {
  extern __shared__ uint32_t bits[];  // this CTA's words
  __shared__ int warp_sum[32];
  __shared__ int cta_sum;
  cg::cluster_group cluster = cg::this_cluster();
  pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31, rank = static_cast<int>(cluster.block_rank());
  const int words = (A.num_pages + 31) / 32, share = (words + kListCtas - 1) / kListCtas;
  const int w0 = min(words, rank * share), n = min(words, w0 + share) - w0;
  constexpr int kWords = 8;  // of a thread, in flight together
  for (int i0 = tid; i0 < n; i0 += kWords * kListThreads) {
    uint32_t word[kWords];
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int i = i0 + j * kListThreads;
      word[j] = i < n ? static_cast<uint32_t>(A.freed[w0 + i]) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kWords; ++j) {
      const int i = i0 + j * kListThreads;
      if (i >= n) break;
      // of the counts that ended on the other side than they began, those that
      // are not above 0 now
      uint32_t b = word[j], keep = 0;
      while (b) {
        int bit[4], refs[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // four counts in flight
          bit[k] = __ffs(b) - 1;
          b &= b - 1;
          refs[k] = bit[k] >= 0 ? A.refs_out[(w0 + i) * 32 + bit[k]] : 1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) keep |= refs[k] <= 0 ? 1u << bit[k] : 0u;
      }
      bits[i] = keep;
    }
  }
  __syncthreads();
  const int per = (n + kListThreads - 1) / kListThreads, i0 = min(n, tid * per), i1 = min(n, i0 + per);
  int mine = 0;
  for (int i = i0; i < i1; ++i) mine += __popc(bits[i]);
  int before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) warp_sum[tid >> 5] = before;
  before -= mine;
  __syncthreads();
  for (int w = 0; w < tid >> 5; ++w) before += warp_sum[w];
  if (tid == kListThreads - 1) cta_sum = before + mine;
  cluster.sync();
  int total = 0;
  for (int r = 0; r < kListCtas; ++r) {
    const int s = *cluster.map_shared_rank(&cta_sum, r);
    if (r < rank) before += s;
    total += s;
  }
  for (int i = i0; i < i1; ++i) {
    uint32_t b = bits[i];
    while (b) {
      const int bit = __ffs(b) - 1;
      b &= b - 1;
      A.freed[before++] = (w0 + i) * 32 + bit;
    }
  }
  // what is left of the bitmap's place
  for (int i = total + rank * kListThreads + tid; i < words; i += kListCtas * kListThreads) A.freed[i] = -1;
  if (rank == 0 && tid == 0) *A.freed_count = total;
  cluster.sync();  // no CTA leaves while its sum is read
}

// ------------------------------------------------------------- compaction
// Exclusive prefix of a value per thread over the CTA; the sum to *total.
__device__ __forceinline__ int block_prefix(int v, int* total) {
  __shared__ int sums[kWarpsPerCta];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kWarpsPerCta; ++w) {
    if (w < warp) before += sums[w];
    all += sums[w];
  }
  *total = all;
  return before + x - v;
}

// Live pages of every block of kPagesPerCta.
__global__ void __launch_bounds__(kThreads) compact_count_kernel(const __grid_constant__ CompactParams A) {
  pdl_wait_primary();
  pdl_launch_dependents();
  int mine = 0, total;
  for (int i = threadIdx.x; i < kPagesPerCta; i += kThreads) {
    const int page = blockIdx.x * kPagesPerCta + i;
    mine += page < A.num_pages && A.refs[page] > 0;
  }
  block_prefix(mine, &total);
  if (threadIdx.x == 0) A.block_live[blockIdx.x] = total;
}

// Moves, new counts and new ids (a mover's: -2 - its rank, until it moves).
// DIRECT: every CTA counts the live pages for itself, from all counts, instead
// of from the blocks' sums.
template <bool DIRECT>
__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const __grid_constant__ CompactParams A, int blocks) {
  pdl_wait_primary();
  pdl_launch_dependents();
  // live pages before this block, in all, and below the `live`-th page
  int b = 0, a = 0, c = 0, live, before, below;
  if constexpr (DIRECT) {
#pragma unroll 8
    for (int page = threadIdx.x; page < A.num_pages; page += kThreads) {
      const int used = A.refs[page] > 0;
      a += used;
      if (page < static_cast<int>(blockIdx.x) * kPagesPerCta) b += used;
    }
  } else {
    for (int i = threadIdx.x; i < blocks; i += kThreads) {
      const int s = A.block_live[i];
      a += s;
      if (i < static_cast<int>(blockIdx.x)) b += s;
    }
  }
  block_prefix(b, &before);
  block_prefix(a, &live);
  const int edge = DIRECT ? 0 : live / kPagesPerCta;
  for (int i = threadIdx.x; i < edge; i += kThreads) c += A.block_live[i];
#pragma unroll 8
  for (int page = edge * kPagesPerCta + threadIdx.x; page < live; page += kThreads) c += A.refs[page] > 0;
  block_prefix(c, &below);
  constexpr int kPer = kPagesPerCta / kThreads;
  int refs[kPer], mine = 0, all;
  const int p0 = blockIdx.x * kPagesPerCta + threadIdx.x * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    refs[i] = p0 + i < A.num_pages ? A.refs[p0 + i] : 0;
    mine += refs[i] > 0;
  }
  int rank = before + block_prefix(mine, &all);  // live pages before p0
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int page = p0 + i;
    if (page >= A.num_pages) break;
    const bool used = refs[i] > 0;
    if (page < live) {
      A.remap[page] = used ? page : -1;
      if (used)
        A.refs_out[page] = refs[i];
      else
        A.holes[page - rank] = page;  // its count comes with the page that moves in
    } else {
      A.remap[page] = used ? -2 - (rank - below) : -1;
      if (used) A.movers[rank - below] = make_int2(page, refs[i]);
      A.refs_out[page] = 0;
    }
    rank += used;
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *A.live = live;
    *A.moves = live - below;
  }
}

// Items of a warp: 32 table entries (a chain of three loads, so they come
// first), then pieces of kPiece bytes of the pages that move.
__global__ void __launch_bounds__(kThreads, kCopyCtas) compact_move_kernel(const __grid_constant__ CompactParams A) {
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, moves = *A.moves;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kWarpsPerCta;
  const int64_t per = (A.page_bytes + kPiece - 1) / kPiece;
  const int64_t cells = static_cast<int64_t>(A.rows) * A.entries, table_items = (cells + 31) / 32;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarpsPerCta + (threadIdx.x >> 5); i < table_items + moves * per;
       i += warps) {
    if (i < table_items) {
      const int64_t cell = i * 32 + lane;
      if (cell >= cells) continue;
      const int64_t at = cell / A.entries * A.bt_stride + cell % A.entries;
      int id = A.table[at];
      if (id >= A.num_pages) {
        set_error(A.err, KVARN_DEVERR_PAGE_RANGE);
        id = -1;
      } else if (id >= 0) {
        // a mover's new id is written while this runs: either form names it
        id = *static_cast<volatile const int32_t*>(A.remap + id);
        if (id == -1) set_error(A.err, KVARN_DEVERR_PAGE_RANGE);  // a free page
        if (id <= -2) id = A.holes[-2 - id];
      } else {
        id = -1;
      }
      A.table_out[at] = id;
    } else {
      const int64_t j = i - table_items, k = j / per, at = (j - k * per) * kPiece;
      const int2 from = A.movers[k];
      const int to = A.holes[k];
      copy_piece(A.cache + to * A.page_bytes + at, A.cache + from.x * A.page_bytes + at,
                 static_cast<int>(min(static_cast<int64_t>(kPiece), A.page_bytes - at)));
      if (at == 0 && lane == 0) {
        A.refs_out[to] = from.y;
        A.remap[from.x] = to;
      }
    }
  }
}

// CTAs of kThreads for so many warp items, at most `per_sm` an SM.
int ctas_for(int64_t items, int per_sm) {
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((items + kWarpsPerCta - 1) / kWarpsPerCta,
                                                                 static_cast<int64_t>(per_sm) * device_sm_count())));
}

}  // namespace

cudaError_t launch_fork(const ForkParams& p, cudaStream_t st) {
  ForkParams A = p;
  A.tail_pieces = 0;
  for (int k = 0; k < A.num_rows; ++k) {
    ForkRows& R = A.rows[k];
    R.pieces = static_cast<int64_t>(A.num_out) * R.heads *
               ((static_cast<int64_t>(R.capacity) * R.row_bytes + kPiece - 1) / kPiece);
    A.tail_pieces += R.pieces;
  }
  A.vectors = ((reinterpret_cast<uintptr_t>(A.refs) | reinterpret_cast<uintptr_t>(A.refs_out) |
                reinterpret_cast<uintptr_t>(A.freed)) % 16) == 0;
  const int pieces = (A.entries + kEntries - 1) / kEntries;
  const int64_t copies = A.tail_pieces + static_cast<int64_t>(A.num_out) * std::max(1, pieces) + (A.num_pages + kCounts - 1) / kCounts;
  // as many CTAs as are resident
  cudaError_t e = chained(fork_copy_kernel, ctas_for(copies, kCopyCtas), kThreads, 0, st, A);
  if (e != cudaSuccess) return e;
  const int smem = 4 * A.num_in;
  static SmemLimit count_limit, list_limit;
  e = count_limit.set(fork_count_kernel, 4 * kForkMaxRows);
  if (e != cudaSuccess) return e;
  e = chained(fork_count_kernel, ctas_for(static_cast<int64_t>(A.num_in) * pieces, 4), kThreads, smem, st, A);
  if (e != cudaSuccess) return e;
  const int words = (A.num_pages + 31) / 32;
  e = list_limit.set(fork_list_kernel, 4 * ((kForkMaxPages / 32 + kListCtas - 1) / kListCtas));
  if (e != cudaSuccess) return e;
  return chained(fork_list_kernel, kListCtas, kListThreads, 4 * std::max(1, (words + kListCtas - 1) / kListCtas), st, A);
}

int64_t compact_workspace_bytes(int64_t num_pages) {
  const int64_t blocks = (num_pages + kPagesPerCta - 1) / kPagesPerCta;
  // at most half of the pages move
  return (4 * (blocks + 1) + 15) / 16 * 16 + 8 * (num_pages / 2 + 1) + 4 * (num_pages / 2 + 1);
}

cudaError_t launch_compact(const CompactParams& p, void* workspace, cudaStream_t st) {
  CompactParams A = p;
  const int blocks = std::max(1, (A.num_pages + kPagesPerCta - 1) / kPagesPerCta);
  A.block_live = static_cast<int32_t*>(workspace);
  A.moves = A.block_live + blocks;
  A.movers = reinterpret_cast<int2*>(static_cast<char*>(workspace) + (4LL * (blocks + 1) + 15) / 16 * 16);
  A.holes = reinterpret_cast<int32_t*>(A.movers + A.num_pages / 2 + 1);
  cudaError_t e;
  // (in place a CTA would count pages whose counts another one has written)
  if (A.refs_out != A.refs && A.num_pages <= kDirectPages) {
    e = chained(compact_plan_kernel<true>, blocks, kThreads, 0, st, A, blocks);
  } else {
    e = chained(compact_count_kernel, blocks, kThreads, 0, st, A);
    if (e != cudaSuccess) return e;
    e = chained(compact_plan_kernel<false>, blocks, kThreads, 0, st, A, blocks);
  }
  if (e != cudaSuccess) return e;
  const int64_t per = (A.page_bytes + kPiece - 1) / kPiece;
  const int64_t items = A.num_pages / 2 * per + (static_cast<int64_t>(A.rows) * A.entries + 31) / 32;
  return chained(compact_move_kernel, ctas_for(items, kCopyCtas), kThreads, 0, st, A);  // as many as are resident
}

}  // namespace kvarn
