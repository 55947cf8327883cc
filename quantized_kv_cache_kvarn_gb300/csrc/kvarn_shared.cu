// Decode attention of a batch whose sequences share their first tokens,
// sm_103a.
//
// The shared prefix is one sequence whose query rows are the rows of the
// whole batch: its pages are read and converted once per eight rows of a KV
// head by the dense decode kernel, not once per sequence. Each sequence's own
// tokens (tiles past the prefix, raw tail) go through the dense decode as
// ever, starting at the prefix's end. Both leave (maximum, sum, output)
// partials per row, which one merge joins by log-sum-exp.
#include <math.h>

#include <algorithm>

#include "kvarn_decode_kernel.cuh"

namespace kvarn {

namespace {

// One warp per output row: partials of the prefix (slots [0, pcounts[row])
// of `pre`), of the row's own tiles ([0, counts[row]) of `own`) and of its
// raw tail ([raw_begin, slots)), the first two through the inverse Hadamard
// transform. A sequence of length 0 has no prefix either: out = 0, lse =
// -inf; one shorter than the prefix and its queries is flagged.
template <int D>
__global__ void __launch_bounds__(128) shared_merge_kernel(const float* __restrict__ pre, int pslots,
                                                           const int32_t* __restrict__ pcounts,
                                                           const float* __restrict__ own, int slots,
                                                           const int32_t* __restrict__ counts, int raw_begin, int rows,
                                                           int rows_per_seq, const int32_t* __restrict__ seq_lens,
                                                           int shortest, float* out, float* lse, uint32_t* err) {
  constexpr int E = D / 32, S = kPStride(D);
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const int row = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= rows) return;
  const int len = seq_lens[row / rows_per_seq];
  float* o = out + static_cast<int64_t>(row) * D + lane * E;
  if (len < shortest) {
    if (len != 0 && lane == 0) set_error(err, KVARN_DEVERR_SEQ_LEN);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (lse && lane == 0) lse[row] = -INFINITY;
    return;
  }
  const int np = min(pcounts[row], pslots), nt = min(counts[row], raw_begin);
  const float* P = pre + static_cast<int64_t>(row) * pslots * S;
  const float* O = own + static_cast<int64_t>(row) * slots * S;
  auto used = [&](int s) { return s < nt || s >= raw_begin; };
  float M = -INFINITY;
  for (int s = lane; s < np; s += 32) M = fmaxf(M, P[s * S]);
  for (int s = lane; s < slots; s += 32)
    if (used(s)) M = fmaxf(M, O[s * S]);
  M = warp_max_xor(M, 1, 32);
  if (M == -INFINITY) {  // nothing to see, as in the plain decode's merge
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    if (lse && lane == 0) lse[row] = -INFINITY;
    return;
  }
  float L = 0.f;
  for (int s = lane; s < np; s += 32) L = fmaf(P[s * S + 1], exp2f(P[s * S] - M), L);
  for (int s = lane; s < slots; s += 32)
    if (used(s)) L = fmaf(O[s * S + 1], exp2f(O[s * S] - M), L);
  L = warp_sum_xor(L, 1, 32);
  float rot[E], more[E], raw[E];
  accumulate_slots<E>(P, S, 0, np, M, rot);
  accumulate_slots<E>(O, S, 0, nt, M, more);
  accumulate_slots<E>(O, S, raw_begin, slots, M, raw);
#pragma unroll
  for (int e = 0; e < E; ++e) rot[e] += more[e];
  warp_fwht<E>(rot);
  const float invL = 1.f / L, sc = invL / sqrtf(static_cast<float>(D));
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = fmaf(rot[e], sc, raw[e] * invL);
  if (lse && lane == 0) lse[row] = (M + log2f(L)) * kLn2;
}

template <int D>
cudaError_t launch_shared_merge(const DecArgs& P, const DecArgs& A, int rows, int shortest, float* out, float* lse,
                                cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((rows + 3) / 4);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D>, static_cast<const float*>(P.ws), P.slots,
                            static_cast<const int32_t*>(P.counts), static_cast<const float*>(A.ws), A.slots,
                            static_cast<const int32_t*>(A.counts), A.tile_slots, rows, rows / A.num_seqs, A.seq_lens,
                            shortest, out, lse, A.err);
}

}  // namespace

SharedPlan plan_shared(int32_t num_seqs, int32_t num_kv_heads, int32_t G, int32_t num_queries, int32_t prefix_tiles,
                       int32_t own_tiles, int32_t D, int32_t N, int32_t raw_max, int32_t kb, int32_t vb, int32_t sb) {
  SharedPlan s{};
  s.own = plan_dense_stream(num_seqs, num_kv_heads * row_groups(G, num_queries), own_tiles, D, N, raw_max, kb, vb, sb);
  s.prefix = plan_dense_stream(1, num_kv_heads * row_groups(G, num_seqs * num_queries), prefix_tiles, D, N, 0, kb, vb, sb);
  s.prefix.raw_splits = 0;  // whole tiles only
  s.prefix.slots = s.prefix.tile_slots;
  return s;
}

int64_t shared_workspace_bytes(int64_t rows, int32_t D, const SharedPlan& plan) {
  return dense_stream_workspace_bytes(rows, D, plan.own) + dense_stream_workspace_bytes(rows, D, plan.prefix);
}

cudaError_t launch_decode_shared(const DecodeParams& p, const SharedPlan& plan, const int32_t* prefix_table,
                                 cudaStream_t st) {
  if (p.num_seqs == 0) return cudaSuccess;
  const int Q = p.num_queries > 0 ? p.num_queries : 1;
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * Q * p.num_q_heads;
  DecArgs A, P;
  cudaError_t e = dense_args(p, plan.own, A);
  if (e != cudaSuccess) return e;
  DecodeParams pp = p;
  pp.num_seqs = 1;
  pp.num_queries = p.num_seqs * Q;
  pp.block_table = prefix_table;
  pp.skip_tokens = 0;
  pp.workspace = static_cast<char*>(p.workspace) + dense_stream_workspace_bytes(rows, p.D, plan.own);
  e = dense_args(pp, plan.prefix, P);
  if (e != cudaSuccess) return e;
  P.fixed_tiles = p.skip_tokens / p.N;
  e = run_decode_kernel(pp, P, plan.prefix.ctas, st);
  if (e == cudaSuccess) e = run_decode_kernel(p, A, plan.own.ctas, st);
  if (e != cudaSuccess) return e;
  const int shortest = p.skip_tokens + Q - 1 > 0 ? p.skip_tokens + Q - 1 : 1;
  return p.D == 128 ? launch_shared_merge<128>(P, A, static_cast<int>(rows), shortest, p.out, p.lse, st)
                    : launch_shared_merge<256>(P, A, static_cast<int>(rows), shortest, p.out, p.lse, st);
}

}  // namespace kvarn
