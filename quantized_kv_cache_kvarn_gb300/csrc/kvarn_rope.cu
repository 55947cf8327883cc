// Rotary positions of queries and keys, sm_103a.
//
// Channels a and b of pair i of a token at position p become
//   y_a = s (x_a cos t - x_b sin t),  y_b = s (x_a sin t + x_b cos t),
//   t = p f_i,
// with a = i, b = i + R/2 (half layout) or a = 2i, b = 2i + 1 (interleaved)
// of the R rotated channels. The gradient is the same map with -t.
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: F_i =
// f_i / 2 pi as a 64-bit fraction (formed with integer products from the
// fp64 frequency, off by less than 2^-64 turns plus the frequency's own
// rounding), and p F_i modulo 2^64 drops the whole turns exactly, so a
// position of 2^31 costs no accuracy and no fp64 arithmetic (a GB300 SM has
// about two fp64 lanes). Cosine and sine are taken of the signed fraction
// rounded to fp32, which turns by at most 2^-24 of the angle, itself at most
// half a turn, more or less: as much as the fp32 arithmetic behind it.
//
// A CTA takes `tok` tokens: its threads form the tok x R/2 cosines and sines
// once in shared memory, each thread keeps those of its token and pair chunk
// in registers and walks the heads of every tensor of the call with them, two
// 16-byte vectors a head, kBatch heads in flight (in place, a load can not
// move above a store by itself). What bounds it is HBM for prompts and the
// launch for single tokens: 4 x 4096 tokens of 72 fp16 heads of 128 take 97
// us, 0.92 of the measured copy bandwidth; 8 x 1021 tokens of 28 bf16 heads of
// 256 with 64 turned channels 43 us, 0.80 (87 with the copied channels in a
// loop of their own); 32 single tokens of 72 heads 3.4 us under a profiler.
#include <algorithm>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"

namespace kvarn {

namespace {

constexpr int kRopeThreads = 256;
// Heads a thread has in flight. Two keep 64 registers, and so more CTAs than
// four (80) do: us with 1 / 2 / 3 / 4 / 8 heads, 8 x 1021 tokens of 256-wide
// heads partly turned 48 / 44 / 48 / 48 / 50, 4 x 4096 tokens of 72 heads
// 106 / 98 / 99 / 99 / 102, fp32 25 / 23 / 23 / 24 / 28.
constexpr int kBatch = 2;

// f / 2 pi modulo 1 as a 64-bit fraction, rounded to nearest. f = m 2^e with
// a 53-bit m; 1 / 2 pi as a 128-bit fraction times m, shifted.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(f));
  const int ex = static_cast<int>((bits >> 52) & 0x7ff);
  const uint64_t m = (bits & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0ull);
  const int e = (ex ? ex : 1) - 1075;
  constexpr uint64_t kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;  // 1 / 2 pi
  uint64_t lo = m * kHi, hi = __umul64hi(m, kHi);
  const uint64_t add = __umul64hi(m, kLo);
  lo += add;
  hi += lo < add;
  uint64_t F;
  if (e >= 64) {
    F = 0;
  } else if (e >= 0) {
    F = lo << e;
  } else if (e > -64) {
    const uint64_t half = (lo >> (-e - 1)) & 1;
    F = (hi << (64 + e)) | (lo >> -e);
    F += half;
  } else if (e > -128) {
    const int s = -e - 64;
    const uint64_t half = s ? (hi >> (s - 1)) & 1 : lo >> 63;
    F = (hi >> s) + half;
  } else {
    F = 0;
  }
  return (bits >> 63) ? 0 - F : F;
}

// (cos, sin) of 2 pi times a signed 64-bit fraction of a turn, times `scale`.
__device__ __forceinline__ float2 turn_cos_sin(uint64_t phase, float scale, bool inverse) {
  const float x = __ll2float_rn(static_cast<long long>(phase)) * 0x1p-63f;  // half turns in [-1, 1]
  float s, c;
  sincospif(x, &s, &c);
  return make_float2(c * scale, (inverse ? -s : s) * scale);
}

template <typename T> struct RopeVec;
template <> struct RopeVec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = __half22float2(u32_as_h2(w[k]));
      f[2 * k] = v.x;
      f[2 * k + 1] = v.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = h2_as_u32(__floats2half2_rn(f[2 * k], f[2 * k + 1]));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float load(const __half* p) { return __half2float(*p); }
  static __device__ __forceinline__ void store(__half* p, float v) { *p = __float2half_rn(v); }
};
template <> struct RopeVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(uint4 u, float* f) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(w[k] << 16);
      f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};
template <> struct RopeVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(uint4 u, float* f) {
    f[0] = __uint_as_float(u.x);
    f[1] = __uint_as_float(u.y);
    f[2] = __uint_as_float(u.z);
    f[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};

// Element offsets of head g (over the heads of all tensors) of token
// (seq, tok), and its tensor.
struct HeadAt {
  int k;
  int64_t in, out;
  __device__ __forceinline__ HeadAt(const RopeParams& A, int g, int64_t seq, int64_t tok) : k(0) {
    while (g >= A.t[k].heads) g -= A.t[k++].heads;
    const RopeTensor& t = A.t[k];
    in = seq * t.in_seq + tok * t.in_tok + g * t.in_head;
    out = seq * t.out_seq + tok * t.out_tok + g * t.out_head;
  }
};

// Every address a multiple of 16 bytes. A thread owns one column of the head,
// two vectors of V = 16 / sizeof(T) elements: a pair chunk (V pairs; `chunks` =
// R / (2 V) of them) or, where outputs are not in place, two vectors of the
// channels outside the rotated ones.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams A, int columns, int tok,
                                                            int head_slots, int heads_per_y) {
  using V = RopeVec<T>;
  constexpr int N = V::N;
  extern __shared__ __align__(16) unsigned char smem[];
  const int pairs = A.rope_dim / 2, chunks = pairs / N;
  uint64_t* frac = reinterpret_cast<uint64_t*>(smem);                   // [pairs]
  float2* cs = reinterpret_cast<float2*>(smem + 8 * ((pairs + 1) & ~1));  // [tok][pairs]
  const int tokens = A.num_seqs * A.num_tokens;  // fits 32 bits
  const int tok0 = blockIdx.x * tok;
  for (int i = threadIdx.x; i < pairs; i += kRopeThreads) frac[i] = turn_fraction(A.inv_freq[i]);
  __syncthreads();
  for (int i = threadIdx.x; i < tok * pairs; i += kRopeThreads) {
    const int n = tok0 + i / pairs;
    if (n < tokens) {
      const int p = A.positions[static_cast<int64_t>(n / A.num_tokens) * A.pos_stride + n % A.num_tokens];
      cs[i] = turn_cos_sin(frac[i % pairs] * static_cast<uint64_t>(static_cast<int64_t>(p)), A.scale, A.inverse);
    }
  }
  __syncthreads();

  const int h0 = blockIdx.y * heads_per_y, h1 = min(A.total_heads, h0 + heads_per_y);
  const int c = threadIdx.x % columns, tt = (threadIdx.x / columns) % tok, hs = threadIdx.x / (columns * tok);
  const int n = tok0 + tt;
  if (hs >= head_slots || n >= tokens) return;
  const int seq = n / A.num_tokens, pos_in = n % A.num_tokens;
  const bool turn = c < chunks;
  float cv[N], sv[N];
  int first, second;
  if (turn) {
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float4 v = *reinterpret_cast<const float4*>(cs + tt * pairs + c * N + e);
      cv[e] = v.x;
      sv[e] = v.y;
      cv[e + 1] = v.z;
      sv[e + 1] = v.w;
    }
    first = A.offset + (INTERLEAVED ? 2 * N * c : N * c);
    second = first + (INTERLEAVED ? N : pairs);
  } else {
    const int j = 2 * N * (c - chunks);  // of the channels left over
    first = j < A.offset ? j : j + A.rope_dim;
    second = j + N < A.offset ? j + N : j + N + A.rope_dim;
  }
  for (int h = h0 + hs; h < h1; h += kBatch * head_slots) {
    uint4 x[kBatch], y[kBatch];
    T* dst[kBatch];
    int width[kBatch];  // channels to write; 0: none
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int hh = h + u * head_slots;
      width[u] = 0;
      if (hh < h1) {
        const HeadAt at(A, hh, seq, pos_in);
        const RopeTensor& t = A.t[at.k];
        const T* src = static_cast<const T*>(t.in) + at.in;
        dst[u] = static_cast<T*>(t.out) + at.out;
        width[u] = turn || t.in != t.out ? t.dim : 0;
        if (first < width[u]) x[u] = *reinterpret_cast<const uint4*>(src + first);
        if (second < width[u]) y[u] = *reinterpret_cast<const uint4*>(src + second);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (turn && width[u]) {
        float f[2 * N], r[2 * N];
        V::unpack(x[u], f);
        V::unpack(y[u], f + N);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int a = INTERLEAVED ? 2 * e : e, b = INTERLEAVED ? 2 * e + 1 : N + e;
          r[a] = fmaf(f[a], cv[e], -f[b] * sv[e]);
          r[b] = fmaf(f[a], sv[e], f[b] * cv[e]);
        }
        x[u] = V::pack(r);
        y[u] = V::pack(r + N);
      }
      if (first < width[u]) *reinterpret_cast<uint4*>(dst[u] + first) = x[u];
      if (second < width[u]) *reinterpret_cast<uint4*>(dst[u] + second) = y[u];
    }
  }
}

// Any alignment: one thread per pair or copied channel of a (token, head),
// which forms its own cosine and sine. That bounds it: 4 x 4096 tokens of 72
// fp16 heads of 128 take 808 us with 64 channels turned from channel 4 on and
// 1021 us with 20 turned, 0.6 to 0.75 TB/s; 32 single tokens 9.6 us a call.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_any_kernel(const __grid_constant__ RopeParams A) {
  using V = RopeVec<T>;
  const int pairs = A.rope_dim / 2;
  int dim_max = 0;
  for (int k = 0; k < A.num_tensors; ++k) dim_max = max(dim_max, A.t[k].dim);
  const int per = pairs + (dim_max - A.rope_dim);
  const int64_t total = static_cast<int64_t>(A.num_seqs) * A.num_tokens * A.total_heads * per;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRopeThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kRopeThreads) {
    const int w = static_cast<int>(i % per);
    const int64_t q = i / per;
    const int64_t n = q / A.total_heads;
    const int64_t seq = n / A.num_tokens, tok = n % A.num_tokens;
    const HeadAt at(A, static_cast<int>(q % A.total_heads), seq, tok);
    const RopeTensor& t = A.t[at.k];
    const T* src = static_cast<const T*>(t.in) + at.in;
    T* dst = static_cast<T*>(t.out) + at.out;
    if (w < pairs) {
      const int p = A.positions[seq * A.pos_stride + tok];
      const float2 v = turn_cos_sin(turn_fraction(A.inv_freq[w]) * static_cast<uint64_t>(static_cast<int64_t>(p)),
                                    A.scale, A.inverse);
      const int a = A.offset + (A.interleaved ? 2 * w : w), b = A.interleaved ? a + 1 : a + pairs;
      const float xa = V::load(src + a), xb = V::load(src + b);
      V::store(dst + a, fmaf(xa, v.x, -xb * v.y));
      V::store(dst + b, fmaf(xa, v.y, xb * v.x));
    } else {
      const int r = w - pairs, ch = r < A.offset ? r : r + A.rope_dim;
      if (ch < t.dim && t.in != t.out) dst[ch] = src[ch];
    }
  }
}

template <typename T>
cudaError_t launch(const RopeParams& A, cudaStream_t st) {
  constexpr int N = RopeVec<T>::N;
  const int64_t tokens = static_cast<int64_t>(A.num_seqs) * A.num_tokens;
  const int pairs = A.rope_dim / 2, chunks = pairs / N;
  bool vec = pairs % N == 0 && A.offset % N == 0 && chunks >= 1;  // at most 128 + 128 columns
  for (int k = 0; k < A.num_tensors; ++k) {
    const RopeTensor& t = A.t[k];
    vec = vec && t.dim % N == 0 && (reinterpret_cast<uintptr_t>(t.in) | reinterpret_cast<uintptr_t>(t.out)) % 16 == 0 &&
          (t.in_seq | t.in_tok | t.in_head | t.out_seq | t.out_tok | t.out_head) % N == 0;
  }
  const int sms = device_sm_count();
  if (!vec) {
    const int64_t items = tokens * A.total_heads * A.t[0].dim;
    const int64_t ctas = (items + kRopeThreads - 1) / kRopeThreads;
    rope_any_kernel<T><<<static_cast<unsigned>(ctas < 16LL * sms ? ctas : 16LL * sms), kRopeThreads, 0, st>>>(A);
    return cudaGetLastError();
  }
  // columns: the pair chunks, then the vectors left over two by two
  int rest = 0;
  for (int k = 0; k < A.num_tensors; ++k)
    if (A.t[k].in != A.t[k].out) rest = std::max(rest, (A.t[k].dim - A.rope_dim) / N);
  const int columns = chunks + (rest + 1) / 2;
  // Tokens per CTA: as many as the CTA's threads hold (at most eight), halved
  // while fewer than four CTAs per SM remain. More tokens share the fractions
  // of a CTA; the cosines and sines cost the same per token.
  const int slots = kRopeThreads / columns;
  int tok = 1;
  while (tok * 2 <= slots && tok < 8 && tok * 2 * pairs <= 2048 && (tokens + 2 * tok - 1) / (2 * tok) >= 4LL * sms) tok *= 2;
  const int head_slots = slots / tok;
  const int64_t gx = (tokens + tok - 1) / tok;
  // heads split over grid.y where the tokens alone leave SMs idle
  const int rounds = (A.total_heads + head_slots - 1) / head_slots;
  int64_t gy = gx >= 2LL * sms ? 1 : (2LL * sms + gx - 1) / gx;
  if (gy > rounds) gy = rounds;
  const int heads_per_y = (rounds + static_cast<int>(gy) - 1) / static_cast<int>(gy) * head_slots;
  gy = (A.total_heads + heads_per_y - 1) / heads_per_y;
  const int smem = 8 * ((pairs + 1) & ~1) + 8 * tok * pairs;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (A.interleaved)
    rope_kernel<T, true><<<grid, kRopeThreads, smem, st>>>(A, columns, tok, head_slots, heads_per_y);
  else
    rope_kernel<T, false><<<grid, kRopeThreads, smem, st>>>(A, columns, tok, head_slots, heads_per_y);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& A, cudaStream_t st) {
  switch (A.dtype) {
    case 0: return launch<__half>(A, st);
    case 1: return launch<__nv_bfloat16>(A, st);
    case 2: return launch<float>(A, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvarn
