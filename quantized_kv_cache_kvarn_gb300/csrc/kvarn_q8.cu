// Writing, reading and appending to the 8-bit block cache, sm_103a.
//
// One warp takes one block (16 tokens x D of a KV head) of K or of V: 16-byte
// loads (a lane holds eight channels of 16 D / 256 tokens), the largest
// magnitude by integer maxima over the bit patterns (which order NaN above
// infinity above every number), the scale, the codes. Key codes leave in
// token order, eight bytes a lane; value codes are put in the decode's operand
// order through 2 KB (4 KB at head_dim 256) of shared memory per warp, whose
// 16-byte units are exchanged so that neither side meets a bank conflict.
// Bounded by HBM: 4 bytes read and 2 written per channel and token (K and V);
// 4 x 4096 tokens of 8 bf16 heads of 128 written and read back take 32.5 us,
// 0.92 of the measured copy bandwidth, 7 x 2032 tokens of 4 heads of 256 29 us,
// 0.89. An append is one launch, a warp per sequence, head and side: replayed
// from a graph 1.6 us for 32 sequences of 8 heads, 2.3 where all complete a
// block, 2.6 and 6.1 for 512.
#include "kvarn_launch.h"
#include "kvarn_q8.cuh"

namespace kvarn {

namespace {

constexpr int kWarps = 4;

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t w);
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t w) { return __half22float2(u32_as_h2(w)); }
template <> __device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  return h2_as_u32(__floats2half2_rn(a, b));
}
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What a lane holds of a block: eight channels from 8 nc on, of the tokens
// token(i), i < I. At D = 128 the half-warps share the tokens so that each
// has the four of a V word: the first takes t = 0, 1 (tokens 2t, 2t + 1,
// 2t + 8, 2t + 9), the second t = 2, 3.
template <int D> struct Lanes {
  static constexpr int I = D / 16;
  static __device__ __forceinline__ int chunk(int lane) { return D == 128 ? lane & 15 : lane; }
  // index i = 4 u + 2 h + j of t = t0 + u: token 8 h + 2 t + j
  static __device__ __forceinline__ int t0(int lane) { return D == 128 ? lane >> 4 << 1 : 0; }
  static __device__ __forceinline__ int token(int lane, int i) {
    return 8 * (i >> 1 & 1) + 2 * (t0(lane) + (i >> 2)) + (i & 1);
  }
};

// Byte offset of 16-byte unit u of token `token` in the K codes.
template <int D>
__device__ __forceinline__ int k_unit(int token, int u) {
  return token * D + 16 * (u ^ (4 * (token & 1)));
}
// Shared slot of the 16-byte unit 32 w + L of the V codes.
__device__ __forceinline__ int v_slot(int w, int L) { return 32 * w + (L ^ ((w & 1) | (w & 2) << 1)); }

// raw[i]: eight channels of token(i).
template <int D, typename T, int CODE, bool VALUES>
__device__ __forceinline__ void encode_block(const uint4 (&raw)[D / 16], uint8_t* page, unsigned char* sm) {
  using LN = Lanes<D>;
  const int lane = threadIdx.x & 31;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < LN::I; ++i)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu),
                                 __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu)));
  const uint32_t bits = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  const bool finite = bits < (sizeof(T) == 2 && std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u);
  const float A = finite ? fmaxf(unpack2<T>(bits).x, kQ8Tiny) : 1.f;
  const float scale = finite ? __fmul_rn(A, 1.f / q8_top<CODE>()) : __int_as_float(0x7fc00000);
  const float inv = __fmul_rn(__frcp_rn(A), q8_top<CODE>());
  uint32_t lo[LN::I], hi[LN::I];  // codes of channels 0-3 and 4-7
  constexpr uint32_t kZero = CODE == kQ8Int8 ? 0x80808080u : 0u;
#pragma unroll
  for (int i = 0; i < LN::I; ++i) {
    const float2 a = unpack2<T>(raw[i].x), b = unpack2<T>(raw[i].y), c = unpack2<T>(raw[i].z), d = unpack2<T>(raw[i].w);
    lo[i] = finite ? q8_code4<CODE>(a.x, a.y, b.x, b.y, inv) : kZero;
    hi[i] = finite ? q8_code4<CODE>(c.x, c.y, d.x, d.y, inv) : kZero;
  }
  const int nc = LN::chunk(lane);
  if constexpr (!VALUES) {
#pragma unroll
    for (int i = 0; i < LN::I; ++i) {
      const int tok = LN::token(lane, i);
      *reinterpret_cast<uint2*>(page + k_unit<D>(tok, nc >> 1) + 8 * (nc & 1)) = make_uint2(lo[i], hi[i]);
    }
    if (lane == 0) *reinterpret_cast<float*>(page + q8_scales(D)) = scale;
  } else {
    // word (nc, L = 4 g + t): byte j + 2 h is channel g of token 8 h + 2 t + j
#pragma unroll
    for (int u = 0; u < LN::I / 4; ++u) {
      uint32_t x[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t* c = half ? hi : lo;
        const uint32_t a0 = c[4 * u], a1 = c[4 * u + 1], a2 = c[4 * u + 2], a3 = c[4 * u + 3];
        const uint32_t p01 = __byte_perm(a0, a1, 0x5140), p23 = __byte_perm(a2, a3, 0x5140);  // channels 0, 1
        const uint32_t q01 = __byte_perm(a0, a1, 0x7362), q23 = __byte_perm(a2, a3, 0x7362);  // channels 2, 3
        x[4 * half] = __byte_perm(p01, p23, 0x5410);
        x[4 * half + 1] = __byte_perm(p01, p23, 0x7632);
        x[4 * half + 2] = __byte_perm(q01, q23, 0x5410);
        x[4 * half + 3] = __byte_perm(q01, q23, 0x7632);
      }
#pragma unroll
      for (int g = 0; g < 8; ++g)
        *reinterpret_cast<uint32_t*>(sm + 16 * v_slot(nc >> 2, 4 * g + LN::t0(lane) + u) + 4 * (nc & 3)) = x[g];
    }
    __syncwarp();
#pragma unroll
    for (int w = 0; w < D / 32; ++w)
      *reinterpret_cast<uint4*>(page + 16 * D + 16 * (32 * w + lane)) =
          *reinterpret_cast<const uint4*>(sm + 16 * v_slot(w, lane));
    if (lane == 0) *reinterpret_cast<float*>(page + q8_scales(D) + 4) = scale;
    __syncwarp();
  }
}

// Page of logical block `block` of sequence b, or null (flagged).
__device__ __forceinline__ uint8_t* page_of(const Q8BlockParams& A, int b, int h, int64_t block, int page_bytes) {
  const int32_t id = block >= 0 && block < A.bt_stride ? A.block_table[static_cast<int64_t>(b) * A.bt_stride + block] : -1;
  if (id < 0 || id >= A.num_pages) {
    if ((threadIdx.x & 31) == 0) set_error(A.err, KVARN_DEVERR_PAGE_RANGE);
    return nullptr;
  }
  return static_cast<uint8_t*>(A.cache) + (static_cast<int64_t>(id) * A.num_kv_heads + h) * page_bytes;
}

template <int D, typename T, int CODE, bool VALUES>
__device__ __forceinline__ void encode_at(const Q8BlockParams& A, const T* src, int64_t token_stride, uint8_t* page,
                                          unsigned char* sm) {
  using LN = Lanes<D>;
  const int lane = threadIdx.x & 31;
  uint4 raw[LN::I];
#pragma unroll
  for (int i = 0; i < LN::I; ++i)
    raw[i] = __ldg(reinterpret_cast<const uint4*>(src + LN::token(lane, i) * token_stride + 8 * LN::chunk(lane)));
  encode_block<D, T, CODE, VALUES>(raw, page, sm);
}

template <int D, typename T, int CODE, bool VALUES>
__device__ __forceinline__ void read_at(uint8_t* page, T* dst, int64_t token_stride, unsigned char* sm) {
  using LN = Lanes<D>;
  const int lane = threadIdx.x & 31, nc = LN::chunk(lane);
  const float scale = *reinterpret_cast<const float*>(page + q8_scales(D) + (VALUES ? 4 : 0));
  uint32_t lo[LN::I], hi[LN::I];
  if constexpr (!VALUES) {
#pragma unroll
    for (int i = 0; i < LN::I; ++i) {
      const uint2 v = *reinterpret_cast<const uint2*>(page + k_unit<D>(LN::token(lane, i), nc >> 1) + 8 * (nc & 1));
      lo[i] = v.x;
      hi[i] = v.y;
    }
  } else {
    uint4 v[D / 32];
#pragma unroll
    for (int w = 0; w < D / 32; ++w) v[w] = *reinterpret_cast<const uint4*>(page + 16 * D + 16 * (32 * w + lane));
#pragma unroll
    for (int w = 0; w < D / 32; ++w) *reinterpret_cast<uint4*>(sm + 16 * v_slot(w, lane)) = v[w];
    __syncwarp();
#pragma unroll
    for (int u = 0; u < LN::I / 4; ++u) {
      uint32_t x[8];
#pragma unroll
      for (int g = 0; g < 8; ++g)
        x[g] = *reinterpret_cast<const uint32_t*>(sm + 16 * v_slot(nc >> 2, 4 * g + LN::t0(lane) + u) + 4 * (nc & 3));
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint32_t p = __byte_perm(x[4 * half], x[4 * half + 1], 0x5140), q = __byte_perm(x[4 * half + 2], x[4 * half + 3], 0x5140);
        const uint32_t r = __byte_perm(x[4 * half], x[4 * half + 1], 0x7362), s = __byte_perm(x[4 * half + 2], x[4 * half + 3], 0x7362);
        uint32_t* c = half ? hi : lo;
        c[4 * u] = __byte_perm(p, q, 0x5410);
        c[4 * u + 1] = __byte_perm(p, q, 0x7632);
        c[4 * u + 2] = __byte_perm(r, s, 0x5410);
        c[4 * u + 3] = __byte_perm(r, s, 0x7632);
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < LN::I; ++i) {
    uint32_t p[4], w[4];
    q8_pairs<CODE>(lo[i], p[0], p[1]);
    q8_pairs<CODE>(hi[i], p[2], p[3]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(u32_as_h2(p[k]));
      w[k] = pack2<T>(__fmul_rn(f.x, scale), __fmul_rn(f.y, scale));
    }
    *reinterpret_cast<uint4*>(dst + LN::token(lane, i) * token_stride + 8 * nc) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Warp item ((b blocks + u) Hkv + h) 2 + (0: K, 1: V): the heads are innermost, so that token-major inputs are read in whole rows.
template <int D, typename T, int CODE, bool READ>
__global__ void __launch_bounds__(32 * kWarps) q8_block_kernel(const __grid_constant__ Q8BlockParams A) {
  __shared__ __align__(16) unsigned char sm[kWarps][16 * D];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t n = item >> 1;
  const int h = static_cast<int>(n % A.num_kv_heads);
  const int64_t m = n / A.num_kv_heads;
  const int u = static_cast<int>(m % A.blocks);
  const int64_t b = m / A.blocks;
  if (b >= A.num_seqs) return;
  const int start = A.block_start[b];
  if (start < 0) return;
  uint8_t* page = page_of(A, static_cast<int>(b), h, static_cast<int64_t>(start) + u, q8_page(D));
  if (!page) return;
  const int64_t at = b * A.seq_stride + h * A.head_stride + static_cast<int64_t>(u) * kPageTokens * A.token_stride;
  unsigned char* mine = sm[threadIdx.x >> 5];
  if constexpr (READ) {
    if (item & 1)
      read_at<D, T, CODE, true>(page, static_cast<T*>(const_cast<void*>(A.v)) + at, A.token_stride, mine);
    else
      read_at<D, T, CODE, false>(page, static_cast<T*>(const_cast<void*>(A.k)) + at, A.token_stride, mine);
  } else {
    if (item & 1)
      encode_at<D, T, CODE, true>(A, static_cast<const T*>(A.v) + at, A.token_stride, page, mine);
    else
      encode_at<D, T, CODE, false>(A, static_cast<const T*>(A.k) + at, A.token_stride, page, mine);
  }
}

// One warp per (sequence, KV head, K or V): the newest token goes to its row
// of the raw tail, or completes a block, which is coded into its page.
template <int D, typename T, int CODE, bool VALUES>
__device__ __forceinline__ void append_one(const Q8BlockParams& A, int b, int h, int L, unsigned char* sm) {
  using LN = Lanes<D>;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(b) * A.num_kv_heads + h;
  const T* x = static_cast<const T*>(VALUES ? A.v : A.k) + unit * D;
  T* tail = static_cast<T*>(VALUES ? A.tail_v : A.tail_k) + unit * A.tail_cap * D;
  const int row = (L - 1) % kPageTokens;
  if (row != kPageTokens - 1) {
    if (lane < D / 8) reinterpret_cast<uint4*>(tail + row * D)[lane] = __ldg(reinterpret_cast<const uint4*>(x) + lane);
    return;
  }
  uint8_t* page = page_of(A, b, h, L / kPageTokens - 1, q8_page(D));
  if (!page) return;
  uint4 raw[LN::I];
#pragma unroll
  for (int i = 0; i < LN::I; ++i) {
    const int tok = LN::token(lane, i);
    raw[i] = *reinterpret_cast<const uint4*>((tok == kPageTokens - 1 ? x : tail + tok * D) + 8 * LN::chunk(lane));
  }
  encode_block<D, T, CODE, VALUES>(raw, page, sm);
}

template <int D, typename T, int CODE>
__global__ void __launch_bounds__(32 * kWarps) q8_append_kernel(const __grid_constant__ Q8BlockParams A) {
  __shared__ __align__(16) unsigned char sm[kWarps][16 * D];
  pdl_wait_primary();
  pdl_launch_dependents();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t n = item >> 1;
  const int h = static_cast<int>(n % A.num_kv_heads);
  const int64_t b = n / A.num_kv_heads;
  if (b >= A.num_seqs) return;
  const int L = A.seq_lens[b];
  if (L < 0 || L > A.max_seq_len) {
    if ((threadIdx.x & 31) == 0) set_error(A.err, KVARN_DEVERR_SEQ_LEN);
    return;
  }
  if (L == 0) return;
  if (item & 1)
    append_one<D, T, CODE, true>(A, static_cast<int>(b), h, L, sm[threadIdx.x >> 5]);
  else
    append_one<D, T, CODE, false>(A, static_cast<int>(b), h, L, sm[threadIdx.x >> 5]);
}

// f(D, T, code) of the parameters.
template <typename F>
cudaError_t with_types(const Q8BlockParams& p, F&& f) {
  using std::integral_constant;
  auto typed = [&](auto d) {
    auto coded = [&](auto tag) {
      using T = decltype(tag);
      return p.code == kQ8Int8 ? f(d, T{}, integral_constant<int, kQ8Int8>{}) : f(d, T{}, integral_constant<int, kQ8E4M3>{});
    };
    return p.bf16 ? coded(__nv_bfloat16{}) : coded(__half{});
  };
  return p.D == 128 ? typed(integral_constant<int, 128>{}) : typed(integral_constant<int, 256>{});
}

}  // namespace

cudaError_t launch_q8_blocks(const Q8BlockParams& p, bool read, cudaStream_t st) {
  const int64_t items = 2LL * p.num_seqs * p.num_kv_heads * p.blocks;
  const int64_t ctas = (items + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return with_types(p, [&](auto d, auto t, auto c) {
    using T = decltype(t);
    return chained(read ? q8_block_kernel<decltype(d)::value, T, decltype(c)::value, true>
                        : q8_block_kernel<decltype(d)::value, T, decltype(c)::value, false>,
                   dim3(static_cast<unsigned>(ctas)), 32 * kWarps, 0, st, p);
  });
}

cudaError_t launch_q8_append(const Q8BlockParams& p, cudaStream_t st) {
  const int64_t items = 2LL * p.num_seqs * p.num_kv_heads;
  const int64_t ctas = (items + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return with_types(p, [&](auto d, auto t, auto c) {
    return chained(q8_append_kernel<decltype(d)::value, decltype(t), decltype(c)::value>, dim3(static_cast<unsigned>(ctas)),
                   32 * kWarps, 0, st, p);
  });
}

}  // namespace kvarn
