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
// a second kernel sums in fp64: no atomics, the same bits every time.
#include <algorithm>

#include "kvarn_launch.h"
#include "kvarn_rope.cuh"

namespace kvarn {

namespace {

constexpr int kThreads = 256;

// Work of a launch: tiles of `tok` tokens of each tensor, `per` consecutive
// tiles to a CTA, CTAs [cta0[k], cta0[k + 1]) for tensor k.
struct NormPlan {
  int32_t cta0[kRopeMaxTensors + 1];
  int32_t tok[kRopeMaxTensors];
  int32_t per[kRopeMaxTensors];
  int32_t lanes;  // of a head's group (vector path)
};

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

template <typename T, bool INTERLEAVED, bool BACK>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ NormParams A,
                                                             const __grid_constant__ NormPlan P) {
  using V = RopeVec<T>;
  constexpr int N = V::N;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = tensor_of(P, A.num_tensors), tok = P.tok[k], lanes = P.lanes;
  const NormTensor& t = A.t[k];
  const int pairs = A.rope_dim / 2, chunks = pairs / N, columns = A.dim / (2 * N);
  uint64_t* frac = reinterpret_cast<uint64_t*>(smem);                     // [pairs]
  float2* cs = reinterpret_cast<float2*>(smem + 8 * ((pairs + 1) & ~1));  // [tok][pairs]
  const int tokens = A.num_seqs * A.num_tokens;  // fits 32 bits
  const int tid = threadIdx.x, lane = tid & 31;
  for (int i = tid; i < pairs; i += kThreads) frac[i] = turn_fraction(A.inv_freq[i]);

  const int c = tid % lanes, tt = tid / lanes % tok, hs = tid / (lanes * tok), slots = kThreads / (lanes * tok);
  const uint32_t group = lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u) << (lane & ~(lanes - 1));
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
  float w[2 * N], dw[BACK ? 2 * N : 1];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    w[e] = on ? weight_at(t.w, A.wdtype, first + e) + A.weight_offset : 0.f;
    w[N + e] = on ? weight_at(t.w, A.wdtype, second + e) + A.weight_offset : 0.f;
  }
#pragma unroll
  for (int e = 0; e < (BACK ? 2 * N : 1); ++e) dw[e] = 0.f;
  const float inv_dim = 1.f / static_cast<float>(A.dim);
  __syncthreads();

  const int tile0 = (static_cast<int>(blockIdx.x) - P.cta0[k]) * P.per[k];
  for (int tile = tile0; tile < tile0 + P.per[k]; ++tile) {
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
    const int n = n0 + tt;
    if (n < tokens && hs < slots) {
      const int seq = n / A.num_tokens, pos_in = n % A.num_tokens;
      float cv[N], sv[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float2 v = turn ? cs[tt * pairs + c * N + e] : make_float2(1.f, 0.f);
        cv[e] = v.x;
        sv[e] = v.y;
      }
      const T* x0 = static_cast<const T*>(t.x) + seq * t.x_seq + pos_in * t.x_tok;
      const T* g0 = static_cast<const T*>(t.dy) + (BACK ? seq * t.g_seq + pos_in * t.g_tok : 0);
      T* o0 = static_cast<T*>(t.out) + seq * t.o_seq + pos_in * t.o_tok;
      auto rotate = [&](const float* f, float* r) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int a = INTERLEAVED ? 2 * e : e, b = INTERLEAVED ? 2 * e + 1 : N + e;
          r[a] = fmaf(f[a], cv[e], -f[b] * sv[e]);
          r[b] = fmaf(f[a], sv[e], f[b] * cv[e]);
        }
      };
      auto group_sum = [&](float s) {
        for (int d = 1; d < lanes; d <<= 1) s += __shfl_xor_sync(group, s, d);
        return s;
      };
      if constexpr (!BACK) {
        constexpr int kBatch = 2;
        for (int h = hs; h < t.heads; h += kBatch * slots) {
          uint4 x[kBatch], y[kBatch];
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            x[u] = y[u] = make_uint4(0, 0, 0, 0);
            const int hh = h + u * slots;
            if (on && hh < t.heads) {
              x[u] = *reinterpret_cast<const uint4*>(x0 + hh * t.x_head + first);
              y[u] = *reinterpret_cast<const uint4*>(x0 + hh * t.x_head + second);
            }
          }
#pragma unroll
          for (int u = 0; u < kBatch; ++u) {
            const int hh = h + u * slots;
            if (hh >= t.heads) break;
            float f[2 * N], r[2 * N];
            V::unpack(x[u], f);
            V::unpack(y[u], f + N);
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) s = fmaf(f[e], f[e], s);
            const float rs = rsqrtf(fmaf(group_sum(s), inv_dim, A.eps));
#pragma unroll
            for (int e = 0; e < 2 * N; ++e) f[e] = f[e] * rs * w[e];
            if (on) {
              T* dst = o0 + hh * t.o_head;
              if (turn) rotate(f, r);
              *reinterpret_cast<uint4*>(dst + first) = V::pack(turn ? r : f);
              *reinterpret_cast<uint4*>(dst + second) = V::pack(turn ? r + N : f + N);
            }
          }
        }
      } else {
        for (int h = hs; h < t.heads; h += slots) {
          uint4 v[4] = {};
          if (on) {
            v[0] = *reinterpret_cast<const uint4*>(x0 + h * t.x_head + first);
            v[1] = *reinterpret_cast<const uint4*>(x0 + h * t.x_head + second);
            v[2] = *reinterpret_cast<const uint4*>(g0 + h * t.g_head + first);
            v[3] = *reinterpret_cast<const uint4*>(g0 + h * t.g_head + second);
          }
          float f[2 * N], d[2 * N], g[2 * N];
          V::unpack(v[0], f);
          V::unpack(v[1], f + N);
          V::unpack(v[2], d);
          V::unpack(v[3], d + N);
          float s = 0.f, q = 0.f;
          rotate(d, g);
#pragma unroll
          for (int e = 0; e < 2 * N; ++e) {
            if (!turn) g[e] = d[e];
            s = fmaf(f[e], f[e], s);
            q = fmaf(g[e] * w[e], f[e], q);
          }
          s = group_sum(s);
          q = group_sum(q);
          const float rs = rsqrtf(fmaf(s, inv_dim, A.eps));
          const float m = q * rs * inv_dim;  // (u . h) / D
#pragma unroll
          for (int e = 0; e < 2 * N; ++e) {
            const float hd = f[e] * rs;
            dw[e] = fmaf(g[e], hd, dw[e]);
            f[e] = rs * fmaf(g[e], w[e], -hd * m);
          }
          if (on) {
            T* dst = o0 + h * t.o_head;
            *reinterpret_cast<uint4*>(dst + first) = V::pack(f);
            *reinterpret_cast<uint4*>(dst + second) = V::pack(f + N);
          }
        }
      }
    }
    __syncthreads();
  }
  if constexpr (BACK) {
    if (!t.dw) return;
    float* rows = reinterpret_cast<float*>(smem);  // [groups][dim]
    const int groups = kThreads / lanes, g = tid / lanes;
    if (on) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        rows[g * A.dim + first + e] = dw[e];
        rows[g * A.dim + second + e] = dw[N + e];
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
// head; a lane owns every 32nd pair and every 32nd channel that is not turned.
template <typename T, bool BACK>
__global__ void __launch_bounds__(kThreads) norm_rope_any_kernel(const __grid_constant__ NormParams A,
                                                                 const __grid_constant__ NormPlan P) {
  using V = RopeVec<T>;
  extern __shared__ __align__(16) unsigned char smem[];
  const int k = tensor_of(P, A.num_tensors), tok = P.tok[k];
  const NormTensor& t = A.t[k];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pairs = A.rope_dim / 2, rest = A.dim - A.rope_dim;
  float* mine = reinterpret_cast<float*>(smem) + warp * A.dim;  // this warp's gradient of the weights
  if constexpr (BACK)
    for (int d = lane; d < A.dim; d += 32) mine[d] = 0.f;
  __syncwarp();
  const int tokens = A.num_seqs * A.num_tokens;
  const int64_t n0 = static_cast<int64_t>(static_cast<int>(blockIdx.x) - P.cta0[k]) * P.per[k] * tok;
  const int64_t n1 = min(static_cast<int64_t>(tokens), n0 + static_cast<int64_t>(P.per[k]) * tok);
  for (int64_t i = n0 * t.heads + warp; i < n1 * t.heads; i += kThreads / 32) {
    const int64_t n = i / t.heads, h = i % t.heads, seq = n / A.num_tokens, pos_in = n % A.num_tokens;
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
// eighth row, in fp64.
__global__ void __launch_bounds__(256) norm_weight_sum_kernel(const __grid_constant__ NormParams A,
                                                              const __grid_constant__ NormPlan P) {
  __shared__ double part[8][32];
  const int k = blockIdx.y, d = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  pdl_wait_primary();
  if (!A.t[k].dw) return;
  double s = 0.;
  if (d < A.dim) {
#pragma unroll 8
    for (int i = P.cta0[k] + w; i < P.cta0[k + 1]; i += 8) s += A.parts[static_cast<int64_t>(i) * A.dim + d];
  }
  part[w][threadIdx.x & 31] = s;
  __syncthreads();
  if (w == 0 && d < A.dim) {
    for (int i = 1; i < 8; ++i) s += part[i][threadIdx.x];
    A.t[k].dw[d] = static_cast<float>(s);
  }
}

// CTAs of tensor k. Backward: rows of the weights' gradient, so a CTA takes
// up to about 64 tokens' worth of heads, fewer where that leaves SMs idle.
NormPlan plan_norm(int num_tensors, const int32_t* heads, int dim, int64_t tokens, int lanes, bool backward) {
  NormPlan P{};
  P.lanes = lanes;
  const int groups = kThreads / lanes;
  const int64_t sms = device_sm_count();
  int64_t all = 0;
  for (int k = 0; k < num_tensors; ++k) all += heads[k];
  for (int k = 0; k < num_tensors; ++k) {
    // tokens of a tile: as many as leave each group a head, halved while
    // fewer than four CTAs per SM remain
    int tok = 1;
    while (tok < 8 && tok * 2 <= groups && (tok * heads[k] < groups || (tokens + 2 * tok - 1) / (2 * tok) >= 4 * sms)) tok *= 2;
    const int64_t tiles = (tokens + tok - 1) / tok;
    int64_t per = 1;
    if (backward) {
      // CTAs in proportion to the heads, about eight per SM over all tensors
      const int64_t want = std::max<int64_t>(1, 8 * sms * heads[k] / std::max<int64_t>(1, all));
      per = std::max<int64_t>(1, std::min<int64_t>((tiles + want - 1) / want, std::max(1, 64 / tok)));
    }
    P.tok[k] = tok;
    P.per[k] = static_cast<int32_t>(per);
    P.cta0[k + 1] = P.cta0[k] + (heads[k] ? static_cast<int32_t>((tiles + per - 1) / per) : 0);
  }
  return P;
}

int vector_lanes(int dim, int n) {
  int lanes = 4;
  while (lanes * 2 * n < dim) lanes *= 2;
  return lanes;
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
  const NormPlan P = plan_norm(A.num_tensors, heads, A.dim, tokens, vec ? vector_lanes(A.dim, N) : 32, A.backward);
  const unsigned ctas = P.cta0[A.num_tensors];
  if (ctas == 0) {
    // no heads or tokens: the sums over nothing
  } else if (vec) {
    int tok = 1;
    for (int k = 0; k < A.num_tensors; ++k) tok = std::max(tok, P.tok[k]);
    int smem = 8 * ((pairs + 1) & ~1) + 8 * tok * pairs;
    if (A.backward) smem = std::max(smem, kThreads / P.lanes * A.dim * 4);
    auto* kernel = A.interleaved ? (A.backward ? norm_rope_kernel<T, true, true> : norm_rope_kernel<T, true, false>)
                                 : (A.backward ? norm_rope_kernel<T, false, true> : norm_rope_kernel<T, false, false>);
    kernel<<<ctas, kThreads, smem, st>>>(A, P);
  } else {
    const int smem = A.backward ? kThreads / 32 * A.dim * 4 : 0;
    if (A.backward)
      norm_rope_any_kernel<T, true><<<ctas, kThreads, smem, st>>>(A, P);
    else
      norm_rope_any_kernel<T, false><<<ctas, kThreads, smem, st>>>(A, P);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !sums) return e;
  norm_weight_sum_kernel<<<dim3((A.dim + 31) / 32, A.num_tensors), 256, 0, st>>>(A, P);
  return cudaGetLastError();
}

}  // namespace

// One row of `dim` per CTA, of the plan with the most CTAs.
int64_t norm_rope_workspace_bytes(int32_t num_tensors, const int32_t* heads, int32_t dim, int64_t tokens) {
  int64_t ctas = 0;
  for (int lanes = 4; lanes <= 32; lanes *= 2)
    ctas = std::max<int64_t>(ctas, plan_norm(num_tensors, heads, dim, tokens, lanes, true).cta0[num_tensors]);
  return ctas * dim * 4;
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
