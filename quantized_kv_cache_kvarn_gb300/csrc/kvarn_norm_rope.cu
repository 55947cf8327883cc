// Norms of queries and keys for each head with their rotary positions in the
// same pass, and the gradient, sm_103a.
//
// A head x of D channels becomes y = R(p) z, z_d = x_d r (w_d + o), with r =
// (sum x^2 / D + eps)^-1/2 and R(p) the rotation of kvarn_rope.cu (scaled).
// Backward, with h = x r, g = R(p)^T dy (scaled likewise) and u = g (w + o):
//   dx = r (u - h (u . h) / D),   dw = sum over tokens and heads of g h.
//
// Vector path: a group of 4 to 32 lanes takes a head, each lane two 16-byte
// vectors that hold both channels of its pairs (or two vectors of channels
// that are not turned), so that the rotation needs no exchange and the norm
// one butterfly over the group. A CTA takes `tok` tokens of one tensor: their
// cosines and sines are formed once in shared memory, and a lane keeps those
// of its token and the weights of its channels in registers while it walks
// the heads. The gradient of the weights stays in registers too, is joined
// over the CTA's groups in a fixed order and leaves as one row per CTA, which
// a second kernel sums in fp64: no atomics, the same bits every time. The pass
// forward is bound by HBM (0.85 of the measured copy bandwidth), the one
// backward by the latency of its two sums at 16 warps an SM (0.56).
#include <algorithm>

#include "kvarn_launch.h"
#include "kvarn_rope.cuh"

namespace kvarn {

namespace {

constexpr int kThreads = 256;

// Work of a launch: tiles of `tok` tokens of each tensor, `per` consecutive
// tiles to a CTA, CTAs [cta0[k], cta0[k + 1]) for tensor k. Backward, heads are
// shared out too: CTA i of a tensor takes span i % spans of `span` heads.
struct NormPlan {
  int32_t cta0[kRopeMaxTensors + 1];
  int32_t tok[kRopeMaxTensors];
  int32_t per[kRopeMaxTensors];
  int32_t span[kRopeMaxTensors];
  int32_t spans[kRopeMaxTensors];
  int32_t lanes;  // of a head's group (vector path)
};
constexpr int kMaxRounds = 128;  // terms of the weights' gradient that are added up in a row

__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
  if (!w) return 1.f;
  if (dtype == 2) return static_cast<const float*>(w)[i];
  if (dtype == 1) return __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i]);
  return __half2float(static_cast<const __half*>(w)[i]);
}

__device__ __forceinline__ int tensor_of(const NormPlan& P, int n) {
  int k = 0;
  while (k + 1 < n && static_cast<int>(blockIdx.x) >= P.cta0[k + 1]) ++k;
  return k;
}

// Rounds whose vectors are under way to shared memory (32 bytes a lane and
// round forward, 64 backward), and CTAs per SM that registers leave room for:
// 4 x 4096 tokens of 72 bf16 heads of 128 take 106 us with three CTAs (80
// registers) as with two, 118 with four (spills); backward two CTAs of at most
// 128 registers, two to four rounds under way make no difference (2 x 4093
// tokens of 28 heads of 256: 94 to 97 us). (Compared with each other before the
// launches were chained, which took the two kept ones to 104 and 93.)
constexpr int kFwdCtas = 3, kFwdDepth = 4, kBackCtas = 2, kBackDepth = 2;

// 16 bytes to shared memory, zeros where there is nothing to read.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}

// The vector pair of a lane as its pairs' channels, a[e] and b[e].
template <int N, bool INTERLEAVED>
__device__ __forceinline__ void to_pairs(const float (&f)[2 * N], float2 (&a)[N / 2], float2 (&b)[N / 2]) {
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    a[e] = INTERLEAVED ? make_float2(f[4 * e], f[4 * e + 2]) : make_float2(f[2 * e], f[2 * e + 1]);
    b[e] = INTERLEAVED ? make_float2(f[4 * e + 1], f[4 * e + 3]) : make_float2(f[N + 2 * e], f[N + 2 * e + 1]);
  }
}
template <int N, bool INTERLEAVED>
__device__ __forceinline__ void from_pairs(const float2 (&a)[N / 2], const float2 (&b)[N / 2], float (&f)[2 * N]) {
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    f[INTERLEAVED ? 4 * e : 2 * e] = a[e].x;
    f[INTERLEAVED ? 4 * e + 2 : 2 * e + 1] = a[e].y;
    f[INTERLEAVED ? 4 * e + 1 : N + 2 * e] = b[e].x;
    f[INTERLEAVED ? 4 * e + 3 : N + 2 * e + 1] = b[e].y;
  }
}

template <typename T, int LANES, bool INTERLEAVED, bool BACK>
__global__ void __launch_bounds__(kThreads, BACK ? kBackCtas : kFwdCtas)
    norm_rope_kernel(const __grid_constant__ NormParams A, const __grid_constant__ NormPlan P) {
  using V = RopeVec<T>;
  constexpr int N = V::N, M = N / 2;
  constexpr int VECS = BACK ? 4 : 2, DEPTH = BACK ? kBackDepth : kFwdDepth;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = tensor_of(P, A.num_tensors), tok = P.tok[k];
  const NormTensor& t = A.t[k];
  const int pairs = A.rope_dim / 2, chunks = pairs / N, columns = A.dim / (2 * N);
  uint4* ring = reinterpret_cast<uint4*>(smem);  // [depth][vector][thread]
  unsigned char* rest = smem + DEPTH * VECS * kThreads * 16;
  uint64_t* frac = reinterpret_cast<uint64_t*>(rest);                     // [pairs]
  float2* cs = reinterpret_cast<float2*>(rest + 8 * ((pairs + 1) & ~1));  // [tok][pairs]
  const int tokens = A.num_seqs * A.num_tokens;  // fits 32 bits
  const int tid = threadIdx.x;
  pdl_wait_primary();
  pdl_launch_dependents();

  const int c = tid % LANES, tt = tid / LANES % tok, hs = tid / (LANES * tok), slots = kThreads / (LANES * tok);
  const bool on = c < columns, turn = c < chunks;
  int first = 0, second = 0;
  if (turn) {
    first = A.offset + (INTERLEAVED ? 2 * N * c : N * c);
    second = first + (INTERLEAVED ? N : pairs);
  } else if (on) {
    const int j = 2 * N * (c - chunks);  // of the channels that are not turned
    first = j < A.offset ? j : j + A.rope_dim;
    second = j + N < A.offset ? j + N : j + N + A.rope_dim;
  }
  // A round is one head of every group's token; the rounds of all the CTA's
  // tiles are asked for in one sequence, DEPTH ahead, each lane its own
  // vectors into its own slots: no barrier, and nothing held in registers.
  const int per = BACK ? P.per[k] : 1;  // forward: one tile, all heads
  const int cta = static_cast<int>(blockIdx.x) - P.cta0[k], spans = BACK ? P.spans[k] : 1;
  const int tile0 = (BACK ? cta / spans : cta) * per;
  const int h0 = BACK ? cta % spans * P.span[k] : 0, heads = BACK ? min(P.span[k], t.heads - h0) : t.heads;
  const int rounds = (heads + slots - 1) / slots;  // of a tile
  int ahead_tile = tile0, ahead_left = rounds, ahead_mine = 0, slot = 0;
  const T* ahead_x = nullptr;
  const T* ahead_g = nullptr;
  auto at_tile = [&](int tile) {
    const int n = tile * tok + tt;
    ahead_mine = 0;  // rounds in which this lane has a head
    ahead_x = static_cast<const T*>(t.x);
    ahead_g = static_cast<const T*>(t.dy);
    if (tile < tile0 + per && n < tokens && on) {
      const int seq = n / A.num_tokens, pos_in = n % A.num_tokens;
      ahead_x += seq * t.x_seq + pos_in * t.x_tok + (h0 + hs) * t.x_head + first;
      if (BACK) ahead_g += seq * t.g_seq + pos_in * t.g_tok + (h0 + hs) * t.g_head + first;
      ahead_mine = (heads - hs + slots - 1) / slots;
    }
  };
  at_tile(tile0);
  const int64_t x_step = slots * t.x_head, g_step = slots * t.g_head;
  const int apart = second - first;
  auto ask = [&]() {
    const bool there = ahead_mine > 0;
    const uint32_t dst = smem_addr(ring + slot * VECS * kThreads + tid);
    cp_async16_or_zero(dst, ahead_x, there);
    cp_async16_or_zero(dst + kThreads * 16, there ? ahead_x + apart : ahead_x, there);
    if constexpr (BACK) {
      cp_async16_or_zero(dst + 2 * kThreads * 16, ahead_g, there);
      cp_async16_or_zero(dst + 3 * kThreads * 16, there ? ahead_g + apart : ahead_g, there);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (--ahead_mine > 0) {
      ahead_x += x_step;
      if (BACK) ahead_g += g_step;
    }
    if (BACK && --ahead_left == 0) {
      ahead_left = rounds;
      at_tile(++ahead_tile);
    }
  };
#pragma unroll
  for (int i = 0; i < DEPTH; ++i) {
    slot = i;
    ask();
  }
  slot = 0;
  auto take = [&](uint4 (&v)[VECS]) {
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
#pragma unroll
    for (int i = 0; i < VECS; ++i) v[i] = ring[(slot * VECS + i) * kThreads + tid];
  };
  // The slot's next round, once its values have gone into a sum.
  auto refill = [&]() {
    ask();
    if (++slot == DEPTH) slot = 0;
  };

  for (int i = tid; i < pairs; i += kThreads) frac[i] = turn_fraction(A.inv_freq[i]);
  float2 wa[M], wb[M], da[BACK ? M : 1], db[BACK ? M : 1];  // weights and their gradients by pair
  {
    float w[2 * N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      w[e] = on ? weight_at(t.w, A.wdtype, first + e) + A.weight_offset : 0.f;
      w[N + e] = on ? weight_at(t.w, A.wdtype, second + e) + A.weight_offset : 0.f;
    }
    to_pairs<N, INTERLEAVED>(w, wa, wb);
  }
#pragma unroll
  for (int e = 0; e < (BACK ? M : 1); ++e) da[e] = db[e] = f2(0.f);
  const float inv_dim = 1.f / static_cast<float>(A.dim);
  __syncthreads();
  auto group_sum = [](float s) {
#pragma unroll
    for (int d = 1; d < LANES; d <<= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    return s;
  };

  for (int tile = tile0; tile < tile0 + per; ++tile) {
    const int n0 = tile * tok;
    if (n0 >= tokens) break;
    for (int i = tid; i < tok * pairs; i += kThreads) {
      const int n = n0 + i / pairs;
      if (n < tokens) {
        const int p = A.positions[static_cast<int64_t>(n / A.num_tokens) * A.pos_stride + n % A.num_tokens];
        cs[i] = turn_cos_sin(frac[i % pairs] * static_cast<uint64_t>(static_cast<int64_t>(p)), A.scale, BACK);
      }
    }
    __syncthreads();
    const int n = min(n0 + tt, tokens - 1);
    const bool live = on && n0 + tt < tokens;
    const int seq = n / A.num_tokens, pos_in = n % A.num_tokens;
    float2 cv[M], sv[M];
#pragma unroll
    for (int e = 0; e < M; ++e) {
      const float4 v = turn && live ? *reinterpret_cast<const float4*>(cs + tt * pairs + c * N + 2 * e) : make_float4(1.f, 0.f, 1.f, 0.f);
      cv[e] = make_float2(v.x, v.z);
      sv[e] = make_float2(v.y, v.w);
    }
    T* dst = static_cast<T*>(t.out) + seq * t.o_seq + pos_in * t.o_tok + (h0 + hs) * t.o_head + first;
    const int64_t o_step = slots * t.o_head;
    // Every lane of the CTA makes every round, so that the sums' exchanges are
    // those of whole warps.
    if constexpr (!BACK) {
      // y_a = r (w_a c x_a - w_b s x_b), y_b = r (w_a s x_a + w_b c x_b): the
      // weights go into the turn's coefficients once per token
      float2 aa[M], ab[M], ba[M], bb[M];
#pragma unroll
      for (int e = 0; e < M; ++e) {
        aa[e] = f2mul(wa[e], cv[e]);
        ab[e] = f2mul(wb[e], make_float2(-sv[e].x, -sv[e].y));
        ba[e] = f2mul(wa[e], sv[e]);
        bb[e] = f2mul(wb[e], cv[e]);
      }
      for (int h = hs; h - hs < heads; h += slots) {
        uint4 v[VECS];
        take(v);
        float f[2 * N];
        V::unpack(v[0], f);
        V::unpack(v[1], f + N);
        float2 fa[M], fb[M], s2 = f2(0.f);
        to_pairs<N, INTERLEAVED>(f, fa, fb);
#pragma unroll
        for (int e = 0; e < M; ++e) s2 = f2fma(fa[e], fa[e], f2fma(fb[e], fb[e], s2));
        const float2 rs = f2(rsqrtf(fmaf(group_sum(s2.x + s2.y), inv_dim, A.eps)));
        refill();
        if (live && h < heads) {
          float2 ya[M], yb[M];
#pragma unroll
          for (int e = 0; e < M; ++e) {
            ya[e] = f2mul(rs, f2fma(fa[e], aa[e], f2mul(fb[e], ab[e])));
            yb[e] = f2mul(rs, f2fma(fa[e], ba[e], f2mul(fb[e], bb[e])));
          }
          from_pairs<N, INTERLEAVED>(ya, yb, f);
          *reinterpret_cast<uint4*>(dst) = V::pack(f);
          *reinterpret_cast<uint4*>(dst + apart) = V::pack(f + N);
        }
        dst += o_step;
      }
    } else {
      for (int h = hs; h - hs < heads; h += slots) {
        uint4 v[VECS];
        const bool here = live && h < heads;
        take(v);
        float f[2 * N];
        float2 xa[M], xb[M], ga[M], gb[M], s2 = f2(0.f), q2 = f2(0.f);
        V::unpack(v[2], f);
        V::unpack(v[3], f + N);
        to_pairs<N, INTERLEAVED>(f, xa, xb);
#pragma unroll
        for (int e = 0; e < M; ++e) {  // the turn back: sv has its sign
          ga[e] = f2fma(xa[e], cv[e], f2mul(xb[e], make_float2(-sv[e].x, -sv[e].y)));
          gb[e] = f2fma(xa[e], sv[e], f2mul(xb[e], cv[e]));
        }
        V::unpack(v[0], f);
        V::unpack(v[1], f + N);
        to_pairs<N, INTERLEAVED>(f, xa, xb);
#pragma unroll
        for (int e = 0; e < M; ++e) {
          s2 = f2fma(xa[e], xa[e], f2fma(xb[e], xb[e], s2));
          q2 = f2fma(f2mul(ga[e], wa[e]), xa[e], f2fma(f2mul(gb[e], wb[e]), xb[e], q2));
        }
        float ss = s2.x + s2.y, qs = q2.x + q2.y;
#pragma unroll
        for (int d = 1; d < LANES; d <<= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, d);
          qs += __shfl_xor_sync(0xffffffffu, qs, d);
        }
        refill();
        const float root = rsqrtf(fmaf(ss, inv_dim, A.eps));
        const float rs1 = n0 + tt < tokens && h < heads ? root : 0.f;  // no row: nothing, even with eps 0
        const float m = qs * rs1 * inv_dim;  // (u . h) / D
        const float2 rs = f2(rs1), mm = f2(-m);
#pragma unroll
        for (int e = 0; e < M; ++e) {
          xa[e] = f2mul(xa[e], rs);
          xb[e] = f2mul(xb[e], rs);
          da[e] = f2fma(ga[e], xa[e], da[e]);
          db[e] = f2fma(gb[e], xb[e], db[e]);
          xa[e] = f2mul(rs, f2fma(ga[e], wa[e], f2mul(xa[e], mm)));
          xb[e] = f2mul(rs, f2fma(gb[e], wb[e], f2mul(xb[e], mm)));
        }
        if (here) {
          from_pairs<N, INTERLEAVED>(xa, xb, f);
          *reinterpret_cast<uint4*>(dst) = V::pack(f);
          *reinterpret_cast<uint4*>(dst + apart) = V::pack(f + N);
        }
        dst += o_step;
      }
    }
    __syncthreads();
  }
  if constexpr (BACK) {
    if (!t.dw) return;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* rows = reinterpret_cast<float*>(smem);  // [groups][dim]
    constexpr int groups = kThreads / LANES;
    const int g = tid / LANES;
    if (on) {
      float f[2 * N];
      from_pairs<N, INTERLEAVED>(da, db, f);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        rows[g * A.dim + first + e] = f[e];
        rows[g * A.dim + second + e] = f[N + e];
      }
    }
    __syncthreads();
    for (int d = tid; d < A.dim; d += kThreads) {
      float s = 0.f;
      for (int i = 0; i < groups; ++i) s += rows[i * A.dim + d];
      A.parts[static_cast<int64_t>(blockIdx.x) * A.dim + d] = s;
    }
  }
}

// Any alignment: one warp per (token, head), two or three passes over the
// head; a lane owns every 32nd pair and every 32nd channel that is not turned,
// and forms their cosines anew for every head (backward twice), which bounds it:
// 4 x 4096 tokens of 72 bf16 heads of 128 that begin at odd channels take 667 us
// where the vector path takes 106, their gradient 1465 where it takes 181.
template <typename T, bool BACK>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const __grid_constant__ NormParams A,
                                                                 const __grid_constant__ NormPlan P) {
  using V = RopeVec<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = tensor_of(P, A.num_tensors), tok = P.tok[k];
  const NormTensor& t = A.t[k];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pairs = A.rope_dim / 2, rest = A.dim - A.rope_dim;
  float* mine = reinterpret_cast<float*>(smem) + warp * A.dim;  // this warp's gradient of the weights
  pdl_wait_primary();
  pdl_launch_dependents();
  if constexpr (BACK)
    for (int d = lane; d < A.dim; d += 32) mine[d] = 0.f;
  __syncwarp();
  const int tokens = A.num_seqs * A.num_tokens;
  const int cta = static_cast<int>(blockIdx.x) - P.cta0[k];
  const int64_t n0 = static_cast<int64_t>(cta / P.spans[k]) * P.per[k] * tok;
  const int64_t n1 = min(static_cast<int64_t>(tokens), n0 + static_cast<int64_t>(P.per[k]) * tok);
  const int h0 = cta % P.spans[k] * P.span[k], heads = min(P.span[k], t.heads - h0);
  for (int64_t i = n0 * heads + warp; i < n1 * heads; i += kThreads / 32) {
    const int64_t n = i / heads, h = h0 + i % heads, seq = n / A.num_tokens, pos_in = n % A.num_tokens;
    const T* x = static_cast<const T*>(t.x) + seq * t.x_seq + pos_in * t.x_tok + h * t.x_head;
    const T* dy = static_cast<const T*>(t.dy) + (BACK ? seq * t.g_seq + pos_in * t.g_tok + h * t.g_head : 0);
    T* out = static_cast<T*>(t.out) + seq * t.o_seq + pos_in * t.o_tok + h * t.o_head;
    // f(a, b, cos, sin) of this lane's pairs, f(a, -1, 1, 0) of its other channels
    auto each = [&](auto f) {
      const int p = pairs ? A.positions[seq * A.pos_stride + pos_in] : 0;
      for (int j = lane; j < pairs; j += 32) {
        const float2 v = turn_cos_sin(turn_fraction(A.inv_freq[j]) * static_cast<uint64_t>(static_cast<int64_t>(p)),
                                      A.scale, BACK);
        const int a = A.offset + (A.interleaved ? 2 * j : j);
        f(a, A.interleaved ? a + 1 : a + pairs, v.x, v.y);
      }
      for (int j = lane; j < rest; j += 32) f(j < A.offset ? j : j + A.rope_dim, -1, 1.f, 0.f);
    };
    float s = 0.f, q = 0.f;
    for (int d = lane; d < A.dim; d += 32) {
      const float f = V::load(x + d);
      s = fmaf(f, f, s);
    }
    const float inv_dim = 1.f / static_cast<float>(A.dim);
    const float rs = rsqrtf(fmaf(warp_sum_xor(s, 1, 32), inv_dim, A.eps));
    if constexpr (!BACK) {
      each([&](int a, int b, float cv, float sv) {
        const float za = V::load(x + a) * rs * (weight_at(t.w, A.wdtype, a) + A.weight_offset);
        if (b < 0) {
          V::store(out + a, za);
        } else {
          const float zb = V::load(x + b) * rs * (weight_at(t.w, A.wdtype, b) + A.weight_offset);
          V::store(out + a, fmaf(za, cv, -zb * sv));
          V::store(out + b, fmaf(za, sv, zb * cv));
        }
      });
    } else {
      each([&](int a, int b, float cv, float sv) {
        const float da = V::load(dy + a), db = b < 0 ? 0.f : V::load(dy + b);
        q = fmaf(fmaf(da, cv, -db * sv) * (weight_at(t.w, A.wdtype, a) + A.weight_offset), V::load(x + a), q);
        if (b >= 0) q = fmaf(fmaf(da, sv, db * cv) * (weight_at(t.w, A.wdtype, b) + A.weight_offset), V::load(x + b), q);
      });
      const float m = warp_sum_xor(q, 1, 32) * rs * inv_dim;
      each([&](int a, int b, float cv, float sv) {
        const float da = V::load(dy + a), db = b < 0 ? 0.f : V::load(dy + b);
        const float ga = fmaf(da, cv, -db * sv), gb = fmaf(da, sv, db * cv);
        const float ha = V::load(x + a) * rs, hb = b < 0 ? 0.f : V::load(x + b) * rs;
        mine[a] = fmaf(ga, ha, mine[a]);
        V::store(out + a, rs * fmaf(ga, weight_at(t.w, A.wdtype, a) + A.weight_offset, -ha * m));
        if (b >= 0) {
          mine[b] = fmaf(gb, hb, mine[b]);
          V::store(out + b, rs * fmaf(gb, weight_at(t.w, A.wdtype, b) + A.weight_offset, -hb * m));
        }
      });
    }
  }
  if constexpr (BACK) {
    if (!t.dw) return;
    __syncthreads();
    const float* rows = reinterpret_cast<const float*>(smem);
    for (int d = threadIdx.x; d < A.dim; d += kThreads) {
      float sum = 0.f;
      for (int i = 0; i < kThreads / 32; ++i) sum += rows[i * A.dim + d];
      A.parts[static_cast<int64_t>(blockIdx.x) * A.dim + d] = sum;
    }
  }
}

// Sums of the CTAs' rows: a CTA takes 32 channels of a tensor, its warps every
// 32nd row, in fp64.
__global__ void __launch_bounds__(1024) norm_weight_sum_kernel(const __grid_constant__ NormParams A,
                                                               const __grid_constant__ NormPlan P) {
  __shared__ double part[32][32];
  const int k = blockIdx.y, lane = threadIdx.x & 31, d = blockIdx.x * 32 + lane, w = threadIdx.x >> 5;
  pdl_wait_primary();
  if (!A.t[k].dw) return;
  double s = 0.;
  if (d < A.dim) {
#pragma unroll 8
    for (int i = P.cta0[k] + w; i < P.cta0[k + 1]; i += 32) s += A.parts[static_cast<int64_t>(i) * A.dim + d];
  }
  part[w][lane] = s;
  __syncthreads();
  if (w == 0 && d < A.dim) {
    for (int i = 1; i < 32; ++i) s += part[i][lane];
    A.t[k].dw[d] = static_cast<float>(s);
  }
}

// Tiles and CTAs of every tensor; the number of CTAs, or -1 where a grid does not
// hold them. Forward a CTA takes one tile (several, with their vectors asked for
// in one sequence, took 122 to 156 us where one takes 106). Backward the CTAs
// fill the SMs once, shared out by the tensors' work (a tile's rounds and about
// one more for its cosines and barriers), but none adds up more than kMaxRounds
// rounds: a tile of more heads than that is cut into spans of them.
int64_t plan_norm(NormPlan& P, int num_tensors, const int32_t* heads, int dim, int64_t tokens, int lanes, bool backward) {
  P = NormPlan{};
  P.lanes = lanes;
  const int groups = kThreads / lanes;
  const int64_t sms = device_sm_count();
  int64_t tiles[kRopeMaxTensors], rounds[kRopeMaxTensors], all = 0, ctas = 0;
  for (int k = 0; k < num_tensors; ++k) {
    // tokens of a tile: as many as leave each group a head, halved while
    // fewer than four CTAs per SM remain
    int tok = 1;
    while (tok < 8 && tok * 2 <= groups && (tok * heads[k] < groups || (tokens + 2 * tok - 1) / (2 * tok) >= 4 * sms)) tok *= 2;
    P.tok[k] = tok;
    const int slots = groups / tok;  // heads of a round
    P.span[k] = backward ? std::min(heads[k], kMaxRounds * slots) : heads[k];
    P.spans[k] = heads[k] ? (heads[k] + P.span[k] - 1) / P.span[k] : 1;
    tiles[k] = heads[k] ? (tokens + tok - 1) / tok : 0;
    rounds[k] = (P.span[k] + slots - 1) / slots;
    all += tiles[k] * P.spans[k] * (rounds[k] + 1);
  }
  for (int k = 0; k < num_tensors; ++k) {
    int64_t per = 1;
    if (backward && tiles[k]) {
      const int64_t work = tiles[k] * P.spans[k];
      const int64_t want = std::max<int64_t>(1, 2 * sms * work * (rounds[k] + 1) / all);
      per = std::max<int64_t>(1, std::min<int64_t>((work + want - 1) / want, kMaxRounds / std::max<int64_t>(1, rounds[k])));
    }
    P.per[k] = static_cast<int32_t>(per);
    ctas += (tiles[k] + per - 1) / per * P.spans[k];
    if (ctas > 0x7fffffff) return -1;
    P.cta0[k + 1] = static_cast<int32_t>(ctas);
  }
  return ctas;
}

int vector_lanes(int dim, int n) {
  int lanes = 4;
  while (lanes * 2 * n < dim) lanes *= 2;
  return lanes;
}

template <typename T, int LANES, bool INTERLEAVED, bool BACK>
cudaError_t run_vector(const NormParams& A, const NormPlan& P, int rest, cudaStream_t st) {
  constexpr int kRing = (BACK ? kBackDepth * 4 : kFwdDepth * 2) * kThreads * 16;
  static SmemLimit limit;
  auto* kernel = norm_rope_kernel<T, LANES, INTERLEAVED, BACK>;
  // beside the ring at most 512 fractions, 8 x 512 cosines and sines
  const cudaError_t e = limit.set(kernel, kRing + 8 * 512 + 8 * 8 * 512);
  if (e != cudaSuccess) return e;
  return chained(kernel, dim3(static_cast<unsigned>(P.cta0[A.num_tensors])), kThreads,
                 std::max(kRing + rest, BACK ? kThreads / LANES * A.dim * 4 : 0), st, A, P);
}
template <typename T, int LANES>
cudaError_t run_lanes(const NormParams& A, const NormPlan& P, int rest, cudaStream_t st) {
  if (A.interleaved)
    return A.backward ? run_vector<T, LANES, true, true>(A, P, rest, st) : run_vector<T, LANES, true, false>(A, P, rest, st);
  return A.backward ? run_vector<T, LANES, false, true>(A, P, rest, st) : run_vector<T, LANES, false, false>(A, P, rest, st);
}

template <typename T>
cudaError_t launch(const NormParams& A, cudaStream_t st) {
  constexpr int N = RopeVec<T>::N;
  const int64_t tokens = static_cast<int64_t>(A.num_seqs) * A.num_tokens;
  const int pairs = A.rope_dim / 2;
  bool vec = A.dim % (2 * N) == 0 && A.dim <= 64 * N && pairs % N == 0 && A.offset % N == 0;
  int32_t heads[kRopeMaxTensors];
  bool sums = false;
  for (int k = 0; k < A.num_tensors; ++k) {
    const NormTensor& t = A.t[k];
    heads[k] = t.heads;
    sums = sums || (A.backward && t.dw);
    uintptr_t at = reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.out);
    int64_t strides = t.x_seq | t.x_tok | t.x_head | t.o_seq | t.o_tok | t.o_head;
    if (A.backward) {
      at |= reinterpret_cast<uintptr_t>(t.dy);
      strides |= t.g_seq | t.g_tok | t.g_head;
    }
    vec = vec && at % 16 == 0 && strides % N == 0;
  }
  // one warp per head: the plan of a group of 32
  NormPlan P;
  const int64_t ctas = plan_norm(P, A.num_tensors, heads, A.dim, tokens, vec ? vector_lanes(A.dim, N) : 32, A.backward);
  if (ctas < 0) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaSuccess;
  if (ctas == 0) {
    // no heads or tokens: the sums over nothing
  } else if (vec) {
    int tok = 1;
    for (int k = 0; k < A.num_tensors; ++k) tok = std::max(tok, P.tok[k]);
    const int rest = 8 * ((pairs + 1) & ~1) + 8 * tok * pairs;
    e = P.lanes == 4    ? run_lanes<T, 4>(A, P, rest, st)
        : P.lanes == 8  ? run_lanes<T, 8>(A, P, rest, st)
        : P.lanes == 16 ? run_lanes<T, 16>(A, P, rest, st)
                        : run_lanes<T, 32>(A, P, rest, st);
  } else {
    const int smem = A.backward ? kThreads / 32 * A.dim * 4 : 0;
    e = chained(A.backward ? norm_rope_any_kernel<T, true> : norm_rope_any_kernel<T, false>, dim3(static_cast<unsigned>(ctas)), kThreads, smem, st, A, P);
  }
  if (e != cudaSuccess || !sums) return e;
  return chained(norm_weight_sum_kernel, dim3((A.dim + 31) / 32, A.num_tensors), 1024, 0, st, A, P);
}

}  // namespace

// One row of `dim` per CTA, of the plan with the most CTAs; -1 where a plan has
// more than a grid.
int64_t norm_rope_workspace_bytes(int32_t num_tensors, const int32_t* heads, int32_t dim, int64_t tokens) {
  int64_t most = 0;
  for (int lanes = 4; lanes <= 32; lanes *= 2) {
    NormPlan P;
    const int64_t ctas = plan_norm(P, num_tensors, heads, dim, tokens, lanes, true);
    if (ctas < 0) return -1;
    most = std::max(most, ctas);
  }
  return most * dim * 4;
}

cudaError_t launch_norm_rope(const NormParams& A, cudaStream_t st) {
  switch (A.dtype) {
    case 0: return launch<__half>(A, st);
    case 1: return launch<__nv_bfloat16>(A, st);
    case 2: return launch<float>(A, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvarn
