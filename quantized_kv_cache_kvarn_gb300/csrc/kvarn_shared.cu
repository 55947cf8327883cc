// Decode attention of a batch whose sequences share their first tokens,
// sm_103a.
//
// The shared prefix is one sequence whose query rows are the rows of the
// whole batch. Its pages are read once per 128 rows of a KV head by the
// tensor-core kernel (kvarn_shared_tc.cu), or, where there are few rows and
// at head_dim 256, once per eight rows by the dense decode kernel. Each
// sequence's own tokens (tiles past the prefix, raw tail) go through the
// dense decode as ever, starting at the prefix's end. Both leave (maximum,
// sum, output) partials per row, which one merge joins by log-sum-exp.
#include <math.h>

#include <algorithm>

#include "kvarn_decode_kernel.cuh"
#include "kvarn_shared.cuh"

namespace kvarn {

namespace {

// Four warps per output row: partials of the prefix (slots [0, pcounts[row])
// of `pre`), of the row's own tiles ([0, counts[row]) of `own`) and of its
// raw tail ([raw_begin, slots)), the first two through the inverse Hadamard
// transform. Each warp takes every fourth slot of each kind (a slot is one
// dependent load, and a wide head's row may have thirty), the sums meet in
// shared memory. A sequence of length 0 has no prefix either: out = 0, lse =
// -inf; one shorter than the prefix and its queries is flagged.
template <int D>
__global__ void __launch_bounds__(128) shared_merge_kernel(const float* __restrict__ pre, int pslots,
                                                           const int32_t* __restrict__ pcounts,
                                                           const float* __restrict__ own, int slots,
                                                           const int32_t* __restrict__ counts, int raw_begin,
                                                           int rows_per_seq, const int32_t* __restrict__ seq_lens,
                                                           int shortest, float* out, float* lse, uint32_t* err) {
  constexpr int E = D / 32, S = kPStride(D);
  __shared__ float part[4][2 * D + 4];  // per warp: rotated part, raw part, sum
  pdl_wait_primary();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x;
  const int len = seq_lens[row / rows_per_seq];
  float* o = out + static_cast<int64_t>(row) * D;
  const int np = pcounts ? min(pcounts[row], pslots) : pslots, nt = min(counts[row], raw_begin);
  const float* P = pre + static_cast<int64_t>(row) * pslots * S;
  const float* O = own + static_cast<int64_t>(row) * slots * S;
  auto used = [&](int s) { return s < nt || s >= raw_begin; };
  float M = -INFINITY;  // every warp takes the maximum over all slots
  for (int s = lane; s < np; s += 32) M = fmaxf(M, P[s * S]);
  for (int s = lane; s < slots; s += 32)
    if (used(s)) M = fmaxf(M, O[s * S]);
  M = warp_max_xor(M, 1, 32);
  if (len < shortest || M == -INFINITY) {
    // a padding row; or a row that sees the prefix without one finite score
    // (a query of nan or infinities), whose softmax is undefined
    const bool undefined = len >= shortest;
    if (len != 0 && !undefined && threadIdx.x == 0) set_error(err, KVARN_DEVERR_SEQ_LEN);
    for (int j = threadIdx.x; j < D; j += 128) o[j] = undefined ? NAN : 0.f;
    if (lse && threadIdx.x == 0) lse[row] = undefined ? NAN : -INFINITY;
    return;
  }
  float rot[E], raw[E], L = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) rot[e] = raw[e] = 0.f;
  auto take = [&](const float* p, float (&dst)[E]) {
    const float w = exp2f(p[0] - M);
    L = fmaf(p[1], w, L);
    p += 4 + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + e);
      dst[e] = fmaf(v.x, w, dst[e]);
      dst[e + 1] = fmaf(v.y, w, dst[e + 1]);
      dst[e + 2] = fmaf(v.z, w, dst[e + 2]);
      dst[e + 3] = fmaf(v.w, w, dst[e + 3]);
    }
  };
#pragma unroll 4
  for (int s = warp; s < np; s += 4) take(P + static_cast<int64_t>(s) * S, rot);
#pragma unroll 2
  for (int s = warp; s < nt; s += 4) take(O + static_cast<int64_t>(s) * S, rot);
  for (int s = raw_begin + warp; s < slots; s += 4) take(O + static_cast<int64_t>(s) * S, raw);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    part[warp][lane * E + e] = rot[e];
    part[warp][D + lane * E + e] = raw[e];
  }
  if (lane == 0) part[warp][2 * D] = L;
  __syncthreads();
  if (warp != 0) return;
  L = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) L += part[w][2 * D];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    rot[e] = (part[0][lane * E + e] + part[1][lane * E + e]) + (part[2][lane * E + e] + part[3][lane * E + e]);
    raw[e] = (part[0][D + lane * E + e] + part[1][D + lane * E + e]) + (part[2][D + lane * E + e] + part[3][D + lane * E + e]);
  }
  warp_fwht<E>(rot);
  const float invL = 1.f / L, sc = invL / sqrtf(static_cast<float>(D));
#pragma unroll
  for (int e = 0; e < E; ++e) o[lane * E + e] = fmaf(rot[e], sc, raw[e] * invL);
  if (lse && lane == 0) lse[row] = (M + log2f(L)) * kLn2;
}

template <int D>
cudaError_t launch_shared_merge(const float* pre, int pslots, const int32_t* pcounts, const DecArgs& A, int rows,
                                int shortest, float* out, float* lse, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows);
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<D>, pre, pslots, pcounts, static_cast<const float*>(A.ws), A.slots,
                            static_cast<const int32_t*>(A.counts), A.tile_slots, rows / A.num_seqs, A.seq_lens,
                            shortest, out, lse, A.err);
}

// Whether the tensor-core kernel takes the prefix (head_dim 128). It spends
// the time of 128 rows on any number of them and starts later (its CTAs need
// an SM each), so the dense decode kernel keeps short prefixes and few rows.
// Estimated beyond what both share, in ns of the whole GPU, from calls
// with 16 to 256 rows of 1 and 8 KV heads over 1024 to 16384 tokens (K4V2,
// us, dense / tensor cores: 8 x 32 rows over 16384 tokens 34 / 44, 8 x 64 rows
// 46 / 44, 8 x 256 rows 127 / 68; over 4096 tokens 8 x 96 rows 28 / 32, 8 x 128
// rows 36 / 33; over 1024 tokens 8 x 128 rows 18 / 28):
//   dense: 4.5 per (eight rows, 128 tokens), 2.5 more for a width of two code
//          planes (K or V each), 4 more for 8-bit K and V (two-warp CTAs)
//   tensor cores: 10000, and 11.5 per (128 rows, 64 tokens)
bool prefix_on_tensor_cores(int64_t rows_per_head, int64_t heads, int64_t tokens, int kb, int vb) {
  const double per = 4.5 + (plane_w1(kb) ? 2.5 : 0.0) + (plane_w1(vb) ? 2.5 : 0.0) + (kb + vb == 16 ? 4.0 : 0.0);
  const double dense = per * static_cast<double>((rows_per_head + 7) / 8 * heads) * static_cast<double>(tokens) / 128.0;
  const double tc = 10000.0 + 11.5 * static_cast<double>((rows_per_head + 127) / 128 * heads) * static_cast<double>(tokens) / 64.0;
  return dense > tc;
}

}  // namespace

SharedPlan plan_shared(int32_t num_seqs, int32_t num_kv_heads, int32_t G, int32_t num_queries, int32_t prefix_tiles,
                       int32_t own_tiles, int32_t D, int32_t N, int32_t raw_max, int32_t kb, int32_t vb, int32_t sb) {
  SharedPlan s{};
  // Own tokens: pieces of units while they are short, equal ranges of the
  // flattened tile list where every CTA has about six rounds of tiles or
  // more (32 sequences of 8 KV heads over a 4096-token prefix, us, ranges /
  // pieces: 300 own tokens 52 / 50, up to 2000 of ragged length 74 / 59, 8000
  // 105 / 114, up to 8000 78 / 88; 4 sequences of one head, 8000: 20 / 14).
  constexpr int64_t kOwnRounds = 6;
  const int32_t per_seq = num_kv_heads * row_groups(G, num_queries);
  const int64_t slots = static_cast<int64_t>(device_sm_count()) * dense_decode_ctas_per_sm(D, N, kb, vb, sb) *
                        (D == 256 ? dense_decode_warps(D) / 2 : dense_decode_warps(D));
  s.own = static_cast<int64_t>(num_seqs) * per_seq * own_tiles >= kOwnRounds * slots
              ? plan_dense_stream(num_seqs, per_seq, own_tiles, D, N, raw_max, kb, vb, sb)
              : plan_dense_pieces(num_seqs, per_seq, own_tiles, D, N, raw_max, kb, vb, sb);
  const int64_t rows = static_cast<int64_t>(num_seqs) * num_queries * G;
  const int64_t units = (rows + 127) / 128 * num_kv_heads;
  if (D == 128 && units <= 65535 && prefix_on_tensor_cores(rows, num_kv_heads, static_cast<int64_t>(prefix_tiles) * N, kb, vb)) {
    s.tc_units = static_cast<int32_t>(units);
    s.prefix.slots = s.prefix.tile_slots = shared_tc_splits(s.tc_units, prefix_tiles, N / 64, &s.tc_tps);
    return s;
  }
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
  DecArgs A;
  cudaError_t e = dense_args(p, plan.own, A);
  if (e != cudaSuccess) return e;
  // The own tokens go first: their CTAs end at different times, and the
  // prefix's, which need an SM each, start as they leave.
  A.late_trigger = 1;
  e = run_decode_kernel(p, A, plan.own.ctas, st);
  if (e != cudaSuccess) return e;
  float* pre = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + dense_stream_workspace_bytes(rows, p.D, plan.own));
  const int32_t* pcounts = nullptr;
  const int kb = p.k_bits ? p.k_bits : 4, vb = p.v_bits ? p.v_bits : 2, sb = p.scale_bytes ? p.scale_bytes : 4;
  if (plan.tc_units > 0) {
    SharedTcArgs T{};
    const DensePage pg(p.D, p.N, kb, vb, sb);
    T.q = p.q;
    T.qscale = p.sm_scale * kLog2e / sqrtf(static_cast<float>(p.D));
    T.bf16 = p.bf16 ? 1 : 0;
    T.cache = p.cache;
    T.num_pages = p.num_pages;
    T.table = prefix_table;
    T.Hq = p.num_q_heads;
    T.Hkv = p.num_kv_heads;
    T.G = A.G;
    T.rows_per_head = p.num_seqs * Q * A.G;
    T.N = p.N;
    T.tiles = p.skip_tokens / p.N;
    T.tps = plan.tc_tps;
    T.k_bits = kb;
    T.v_bits = vb;
    T.scale_bytes = sb;
    T.page_bytes = pg.bytes();
    T.k_part = pg.k_part();
    T.tile_bytes = p.N / kPageTokens * pg.bytes();
    T.ws = pre;
    T.slots = plan.prefix.slots;
    T.wait_limit = A.wait_limit;
    T.withhold = A.withhold;
    T.err = p.err;
    e = launch_shared_tc(T, plan.tc_units, st);
  } else {
    DecArgs P;
    DecodeParams pp = p;
    pp.num_seqs = 1;
    pp.num_queries = p.num_seqs * Q;
    pp.block_table = prefix_table;
    pp.skip_tokens = 0;
    pp.workspace = pre;
    e = dense_args(pp, plan.prefix, P);
    if (e != cudaSuccess) return e;
    P.fixed_tiles = p.skip_tokens / p.N;
    pcounts = P.counts;
    P.late_wait = 1;
    e = run_decode_kernel(pp, P, plan.prefix.ctas, st);
  }
  if (e != cudaSuccess) return e;
  const int shortest = p.skip_tokens + Q - 1 > 0 ? p.skip_tokens + Q - 1 : 1;
  return p.D == 128 ? launch_shared_merge<128>(pre, plan.prefix.slots, pcounts, A, static_cast<int>(rows), shortest, p.out, p.lse, st)
                    : launch_shared_merge<256>(pre, plan.prefix.slots, pcounts, A, static_cast<int>(rows), shortest, p.out, p.lse, st);
}

}  // namespace kvarn
