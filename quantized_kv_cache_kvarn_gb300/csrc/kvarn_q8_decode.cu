// Decode attention over the 8-bit block cache, with a sliding window and
// sinks, sm_103a.
//
// Query j of sequence b sits at position p = L - Q + j and sees the tokens
// i <= p with i < S or i > p - W (W = 0: all). Its output is
//   sum_i 2^(s_i) v_i / sum_i 2^(s_i),  s_i = sm_scale log2(e) q . k_i,
// k_i = K scale of i's block times codes, v_i likewise.
//
// Work. The visible blocks of a sequence (those of the sinks, those from the
// window's start on) form one list, taken two at a time as items; up to
// sixteen raw tail tokens are an item too. The items of all units (sequence,
// KV head, group of R query rows) are one list, and every warp of the grid
// takes an equal contiguous range of it, so that neither a long sequence nor
// a short window leaves SMs idle and no page outside a window is touched. A
// unit that lies in one range is written out by its warp; the parts of others
// go to the workspace (two slots per range: of its first and its last unit)
// and a second kernel joins them.
//
// A warp works alone: a ring of kStages items in shared memory, filled by one
// bulk copy per page (lane 0, bounded waits on the stage's mbarrier), and the
// tensor cores' m16n8k16 with fp16 operands. Codes of both kinds are exact in
// fp16, and so is a row of queries scaled by a power of two, so that Q K needs
// one product. The weights go in as fp16 hi + lo: with up to eight rows (R =
// 8) they fill the two halves of the m16 tile, with more (R = 16) they are two
// products into one accumulator.
//
// Two running maxima per row, both whole numbers (so that rescaling is exact):
// m of s for the sum of the weights, and mt of s + e, 2^e the power of two in
// the block's V scale, for the output, so that blocks of any scales add up
// without leaving fp16's range: the operand is 2^(s + e - mt + 12) times the
// scale's mantissa, and a weight counts down to 2^-36 of the largest share. Both
// are floats, so beyond scores of 2^24 (fp32 counts in twos there) mt is rounded
// up, by at most the step of the score: at 2^27 that leaves the weights 20 bits.
//
// At head_dim 256 two warps share an item, 128 channels each (one warp's output
// alone would take 128 registers a thread): they add each other's scores by way
// of shared memory, meeting once an item at a named barrier, and do the softmax
// twice. That barrier has no time limit, so a warp whose wait ran out says so
// beside its scores and both leave behind the same meeting.
//
// The raw tail (at most Q + 14 tokens a sequence) is done in fp32 without the
// tensor cores: hidden tokens' values are never multiplied, whatever they are.
//
// Measured: 32 x 16384 tokens of 64/8 heads of 128 (1.08 GB) 174 us, 0.92 of
// the measured copy bandwidth, of 24/4 heads of 256 186; 3 queries of 24/4 heads
// of 256 behind a window of 4096 tokens, 32 sequences of 2000 to 65536, 145 us:
// there two groups of rows read the pages and dependent instructions at two warps
// a scheduler bound it (issue slots 40%, tensor pipe 31%). What the compiler can
// not reorder is put in an order without waits: the products are volatile
// statements, taken in turn into four accumulators (one after another into the
// same one: 180 and 172 us, when the rest took 176 and 146).
#include <math.h>

#include <algorithm>

#include "kvarn_launch.h"
#include "kvarn_merge.cuh"
#include "kvarn_q8.cuh"

namespace kvarn {

namespace {

constexpr float kOff = 12.f;  // exponent of the weights' operands over mt
// Raw rows are any bf16 numbers, up to 2^128. Products of keys beyond 2^105 may
// add up past a float, which those with the queries at 2^-26 of their scaled size
// do not (at most 2^(15 - 26 + 128 + 8)). Values go in with weights of at most
// 2^-6, so that those of 22 tokens add up to a float.
constexpr float kRawQ = 0x1p-26f, kRawUp = kOff + 6.f;

struct Q8Args {
  const void* q;
  const uint8_t* cache;
  const int32_t* table;
  int32_t bt_stride;
  const int32_t* lens;
  int32_t max_len, B, Q, Hq, Hkv, G, groups;
  int64_t num_pages;
  const void* tail_k;
  const void* tail_v;
  int32_t tail_cap;
  int32_t window, sinks;
  float scale_log2;
  int32_t bf16;
  float* out;
  float* lse;
  int64_t* offs;  // [B + 1]: items before each sequence
  float* part;    // [teams][2][R][D + 4]
  uint32_t* err;
  long long wait_limit;
  int32_t withhold;
};

constexpr int kDW = 128;  // channels of a warp

// One CTA of eight warps per SM, each with a ring of three items. Twelve warps
// of 168 registers with two items each spill and take 192 us where eight take
// 180 (32 x 16384 tokens, 64/8 heads), ten 222.
constexpr int kWarps = 8, kStages = 3;

template <int D, int R> struct Shape {
  static constexpr int HV = D / kDW, TEAMS = kWarps / HV;
  static constexpr int PB = q8_page(D), STAGE = 2 * PB;
  static constexpr int XLANE = R;  // floats that a lane exchanges: 32 tokens' scores of its rows over four lanes
  static constexpr int XBUF = HV == 2 ? 2 * 2 * XLANE * 32 * 4 : 0;  // [parity][half][value][lane], per team
  static constexpr int XCHG = TEAMS * kStages * STAGE;
  static constexpr int FLAGS = XCHG + TEAMS * XBUF;  // [team][parity][half]
  static constexpr int BARS = FLAGS + (HV == 2 ? TEAMS * 16 : 0);
  static constexpr int SMEM = BARS + TEAMS * kStages * 8;
  static_assert(SMEM + 512 <= 227 * 1024, "shared memory of a CTA");
};
// Floats of a partial row: m, l, mt, pad, output.
__host__ __device__ constexpr int part_row(int D) { return D + 4; }

// a / b of non-negative numbers, by the short division where both fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// What a sequence's queries see: blocks [0, sp) and [wp, C) of C whole ones,
// then `tail` raw tokens.
struct Seq {
  int L, C, sp, wp, np, tail, page_items, items;
  __device__ __forceinline__ void load(const Q8Args& A, int b) {
    L = min(max(A.lens[b], 0), A.max_len);
    C = max(0, L - A.Q + 1) / kPageTokens;
    sp = C;
    wp = C;
    if (A.window > 0) {
      wp = min(C, max(0, L - A.Q + 1 - A.window) / kPageTokens);
      sp = min(C, A.sinks / kPageTokens + (A.sinks % kPageTokens != 0));
      if (sp >= wp) sp = wp = C;
    }
    np = sp + C - wp;
    tail = L - C * kPageTokens;
    page_items = (np + 1) >> 1;
    items = page_items + (tail + 15) / 16;
  }
  __device__ __forceinline__ int block(int i) const { return i < sp ? i : wp + i - sp; }
};

// A place in the item list: item i of row group grp of KV head h of sequence b.
struct Place {
  int b, h, grp, i;
  Seq s;
  __device__ __forceinline__ void next(const Q8Args& A) {
    if (++i < s.items) return;
    i = 0;
    if (++grp < A.groups) return;
    grp = 0;
    if (++h < A.Hkv) return;
    h = 0;
    do {
      if (++b >= A.B) return;
      s.load(A, b);
    } while (s.items == 0);
  }
};

// d = A B: the accumulators need not be cleared before.
__device__ __forceinline__ void mma_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// x as fp16 hi + lo (the weights stay below 2^(kOff + 1), so nothing saturates).
__device__ __forceinline__ void split_sat(float2 x, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(hi) : "f"(x.x), "f"(x.y));
  const float2 r = f2fma(__half22float2(u32_as_h2(hi)), f2(-1.f), x);
  asm("cvt.rn.satfinite.f16x2.f32 %0, %2, %1;" : "=r"(lo) : "f"(r.x), "f"(r.y));
}

__device__ __forceinline__ float ex2(float x) { return fast_exp2(x); }
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

// Four consecutive 16-bit elements as floats.
__device__ __forceinline__ void raw4(uint32_t a, uint32_t b, bool bf16, float* f) {
  if (bf16) {
    f[0] = __uint_as_float(a << 16);
    f[1] = __uint_as_float(a & 0xffff0000u);
    f[2] = __uint_as_float(b << 16);
    f[3] = __uint_as_float(b & 0xffff0000u);
  } else {
    const float2 x = __half22float2(u32_as_h2(a)), y = __half22float2(u32_as_h2(b));
    f[0] = x.x;
    f[1] = x.y;
    f[2] = y.x;
    f[3] = y.y;
  }
}

// Sixteen consecutive 16-bit elements (32 bytes, aligned to 16) as floats.
__device__ __forceinline__ void raw16(const uint16_t* p, bool bf16, float* f) {
  const uint4 x = *reinterpret_cast<const uint4*>(p), y = *reinterpret_cast<const uint4*>(p + 8);
  raw4(x.x, x.y, bf16, f);
  raw4(x.z, x.w, bf16, f + 4);
  raw4(y.x, y.y, bf16, f + 8);
  raw4(y.z, y.w, bf16, f + 12);
}

// The rows of a unit that a lane holds: row lane / 4, and row 8 + lane / 4
// where R is 16; of D channels those from c0 on.
template <int D, int R>
struct Rows {
  static constexpr int NR = R / 8;
  uint32_t q[kDW / 16][2 * NR];  // k-step: (a0, a2) of the first row, then (a1, a3) of the second
  float qi[NR];                  // what a row's products are times, per unit of K scale and scale_log2 (a power of two)
  int pos[NR];                   // position of the row's query
  float m[NR], mt[NR], l[NR];
  float o[kDW / 8][4];

  // q channels c0 + 16 (t + 4 c) + 4 s .. + 3 are k-step 4 c + s of lane column t.
  __device__ __forceinline__ void load(const Q8Args& A, int b, int h, int grp, const Seq& s, int c0) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int rr = grp * R + 8 * r + g;
      const bool real = rr < A.G * A.Q;
      const int j = real ? rr / A.G : 0, hg = real ? rr % A.G : 0;
      pos[r] = real ? s.L - A.Q + j : -1;
      const uint16_t* src = static_cast<const uint16_t*>(A.q) +
                            ((static_cast<int64_t>(b) * A.Q + j) * A.Hq + h * A.G + hg) * D + c0;
      float top = 0.f;
      bool finite = true;
#pragma unroll
      for (int c = 0; c < kDW / 64; ++c) {
        float f[16];
        raw16(src + 16 * (t + 4 * c), A.bf16, f);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          top = fmaxf(top, fabsf(f[k]));
          finite = finite && fabsf(f[k]) < INFINITY;
        }
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t votes = __ballot_sync(0xffffffffu, finite);
      finite = ((votes >> (lane & 28)) & 15u) == 15u;
      // the largest element to [2^14, 2^15); smaller ones stay normal fp16
      // numbers down to 2^-28 of it. At most 2^110 times: there every bf16
      // number, a multiple of 2^-133, is one of fp16's, and 2^-e is a float of
      // full precision, as it has to be where large keys make up for it.
      const int e = finite && top > 0.f ? min(141 - static_cast<int>(__float_as_uint(top) >> 23), 110) : 0;
      const float f1 = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      qi[r] = finite ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : nan_f();
#pragma unroll
      for (int c = 0; c < kDW / 64; ++c) {
        float f[16];
        raw16(src + 16 * (t + 4 * c), A.bf16, f);
#pragma unroll
        for (int k = 0; k < 16; ++k) f[k] = finite && real ? f[k] * f1 : 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          q[4 * c + k][2 * r] = h2_as_u32(__floats2half2_rn(f[4 * k], f[4 * k + 1]));
          q[4 * c + k][2 * r + 1] = h2_as_u32(__floats2half2_rn(f[4 * k + 2], f[4 * k + 3]));
        }
      }
      m[r] = mt[r] = -INFINITY;
      l[r] = 0.f;
    }
#pragma unroll
    for (int n = 0; n < kDW / 8; ++n)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[n][x] = 0.f;
  }

  __device__ __forceinline__ bool sees(const Q8Args& A, int r, int token) const {
    return token <= pos[r] && (A.window == 0 || token < A.sinks || token > pos[r] - A.window);
  }

  // New maxima over this lane's scores' maxima; rescales what was added up.
  __device__ __forceinline__ void raise(const float (&ms)[NR], const float (&mts)[NR]) {
    float a[NR];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float x = ms[r], y = mts[r];
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
      y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 1));
      x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
      y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, 2));
      x = fmaxf(m[r], ceilf(x));
      y = fmaxf(mt[r], ceilf(y));
      l[r] *= x == m[r] ? 1.f : ex2(m[r] - x);
      a[r] = y == mt[r] ? 1.f : ex2(mt[r] - y);
      moved = moved || y != mt[r];
      m[r] = x;
      mt[r] = y;
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int n = 0; n < kDW / 8; ++n) {
        o[n][0] *= a[0];
        o[n][1] *= a[0];
        o[n][2] *= a[NR - 1];
        o[n][3] *= a[NR - 1];
      }
    }
  }

  // Two scores of a row to their weights for the sum, 2^(s - m), and for the
  // output, 2^(s - mt + kOff) times the V scale, below 2^(kOff + 1); cm = -m. Next
  // to scores of more than 24 bits fp32 has no room for kOff and the scale's
  // exponent ev. With eight rows they come after s - m: ct = kOff + (m - mt) + ev,
  // the factor is the scale's mantissa. With sixteen that wait shows, and they are
  // in the factor but for what would leave 2^(s - mt) no room: ct = add - mt. (One
  // way for both: 32 x 16384 tokens 175.0 us and window_verify 147.3, or 177.6 and
  // 144.8; each its own 174.3 and 145.2.)
  static constexpr bool kExponents = NR == 1;
  static __device__ __forceinline__ float2 weigh(float2 s, float cm, float ct, float factor, float2& sum) {
    const float2 x = f2add(s, f2(cm)), y = f2add(kExponents ? x : s, f2(ct));
    sum = f2add(sum, make_float2(ex2(x.x), ex2(x.y)));
    return f2mul(make_float2(ex2(y.x), ex2(y.y)), f2(factor));
  }
  // m and mt with 0 for a row that has seen nothing.
  __device__ __forceinline__ float base(float x) const { return x == -INFINITY ? 0.f : x; }

  // This warp's part of the scores of an item's two pages, the second one the
  // first again where the list ends (n = 1): token 8 e + 2 t + j of page p for
  // row r at s[8 r + 4 p + 2 e + j].
  template <int CODE>
  __device__ __forceinline__ void page_scores(const Q8Args& A, const unsigned char* pg0, const unsigned char* pg1, int half,
                                              float (&s)[R]) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float acc[2][2][4];
    // products in turn into four accumulators, so that none waits for the one before
#pragma unroll
    for (int c = 0; c < kDW / 64; ++c) {
      uint32_t x[4][4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {  // half n & 1 of page n >> 1
        const uint4 v = *reinterpret_cast<const uint4*>((n >> 1 ? pg1 : pg0) + (8 * (n & 1) + g) * D + half * kDW +
                                                        16 * ((t + 4 * c) ^ (4 * (g & 1))));
        x[n][0] = v.x;
        x[n][1] = v.y;
        x[n][2] = v.z;
        x[n][3] = v.w;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t* a = q[4 * c + k];
        uint32_t b[4][2];
#pragma unroll
        for (int n = 0; n < 4; ++n) q8_pairs<CODE>(x[n][k], b[n][0], b[n][1]);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          float* to = acc[n >> 1][n & 1];
          if (c == 0 && k == 0)
            mma_first(to, a[0], NR == 2 ? a[2 * NR - 2] : 0u, a[1], NR == 2 ? a[2 * NR - 1] : 0u, b[n][0], b[n][1]);
          else
            mma_f16(to, a[0], NR == 2 ? a[2 * NR - 2] : 0u, a[1], NR == 2 ? a[2 * NR - 1] : 0u, b[n][0], b[n][1]);
        }
      }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float ks = *reinterpret_cast<const float*>((p ? pg1 : pg0) + q8_scales(D)) * A.scale_log2;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float k = ks * qi[r];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 v = f2mul(make_float2(acc[p][e][2 * r], acc[p][e][2 * r + 1]), f2(k));
          s[8 * r + 4 * p + 2 * e] = v.x;
          s[8 * r + 4 * p + 2 * e + 1] = v.y;
        }
      }
    }
  }

  template <int CODE>
  __device__ __forceinline__ void add_pages(const Q8Args& A, const unsigned char* pg0, const unsigned char* pg1, int half,
                                            const Seq& sq, int i0, int n, float (&s)[R]) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float ev[2], add[2], factor[2];  // exponent of the V scale; its shares of weigh's ct and factor
    int first[2];
    bool edge = n < 2, bad[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t bits = *reinterpret_cast<const uint32_t*>((p ? pg1 : pg0) + q8_scales(D) + 4);
      ev[p] = static_cast<float>(static_cast<int>(bits >> 23) - 127);
      bad[p] = bits >= 0x7f800000u;  // not a scale: the block reads as NaN
      if constexpr (kExponents) {
        add[p] = ev[p];
        factor[p] = bad[p] ? nan_f() : __uint_as_float((bits & 0x7fffffu) | 0x3f800000u);
      } else {
        // the largest share of a block has s - mt <= -ev: with the scales of 2^64 and more that is taken up again
        const bool large = ev[p] >= 64.f;
        add[p] = large ? 64.f : 0.f;
        factor[p] = bad[p] ? nan_f() : __uint_as_float(bits) * (large ? 0x1p-52f : 0x1p12f);
      }
      first[p] = p < n ? sq.block(i0 + p) * kPageTokens : 0;
      if (A.window > 0 && first[p] + kPageTokens > A.sinks && first[p] <= sq.L - 1 - A.window) edge = true;
    }
    if (edge) {
#pragma unroll
      for (int x = 0; x < R; ++x) {
        const int p = x >> 2 & 1;
        if (p >= n || !sees(A, x >> 3, first[p] + 8 * (x >> 1 & 1) + 2 * t + (x & 1))) s[x] = -INFINITY;
      }
    }
    float ms[NR], mts[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float top[2];
#pragma unroll
      for (int p = 0; p < 2; ++p)
        top[p] = fmaxf(fmaxf(s[8 * r + 4 * p], s[8 * r + 4 * p + 1]), fmaxf(s[8 * r + 4 * p + 2], s[8 * r + 4 * p + 3]));
      ms[r] = fmaxf(top[0], top[1]);
      mts[r] = fmaxf(__fadd_ru(top[0], ev[0]), __fadd_ru(top[1], ev[1]));  // a bound of every share
    }
    raise(ms, mts);
    float2 w[NR][2][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float2 sum = f2(0.f);
      const float cm = -base(m[r]), ct = kExponents ? kOff + (base(m[r]) - base(mt[r])) : -base(mt[r]);
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int x = 8 * r + 4 * p + 2 * e;
          w[r][p][e] = weigh(make_float2(s[x], s[x + 1]), cm, ct + add[p], factor[p], sum);
        }
      l[r] += sum.x + sum.y;
    }
    if (edge && (bad[0] || bad[1])) {  // 0 times NaN where a token is hidden
#pragma unroll
      for (int x = 0; x < R; x += 2) {
        float2& v = w[x >> 3][x >> 2 & 1][x >> 1 & 1];
        v = make_float2(s[x] == -INFINITY ? 0.f : v.x, s[x + 1] == -INFINITY ? 0.f : v.y);
      }
    }
    uint32_t hi[2][2][NR], lo[2][2][NR];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int e = 0; e < 2; ++e) split_sat(w[r][p][e], hi[p][e][r], lo[p][e][r]);
    // The products of the two pages start from zero and join the output by
    // rounded additions: the tensor cores truncate what they accumulate, which
    // over thousands of tokens adds up to 4e-6 where this leaves 6e-7.
#pragma unroll
    for (int w = 0; w < kDW / 32; ++w) {
      uint32_t x[2][4];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint4 v = *reinterpret_cast<const uint4*>((p ? pg1 : pg0) + 16 * D + 16 * (32 * (4 * half + w) + lane));
        x[p][0] = v.x;
        x[p][1] = v.y;
        x[p][2] = v.z;
        x[p][3] = v.w;
      }
      float d[4][4];
      uint32_t b[4][2][2];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q8_pairs<CODE>(x[0][k], b[k][0][0], b[k][0][1]);
        q8_pairs<CODE>(x[1][k], b[k][1][0], b[k][1][1]);
      }
      // four accumulators in turn
      if constexpr (NR == 1) {
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_first(d[k], hi[0][0][0], lo[0][0][0], hi[0][1][0], lo[0][1][0], b[k][0][0], b[k][0][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) mma_f16(d[k], hi[1][0][0], lo[1][0][0], hi[1][1][0], lo[1][1][0], b[k][1][0], b[k][1][1]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_first(d[k], lo[0][0][0], lo[0][0][NR - 1], lo[0][1][0], lo[0][1][NR - 1], b[k][0][0], b[k][0][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f16(d[k], lo[1][0][0], lo[1][0][NR - 1], lo[1][1][0], lo[1][1][NR - 1], b[k][1][0], b[k][1][1]);
#pragma unroll
        for (int p = 0; p < 2; ++p)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16(d[k], hi[p][0][0], hi[p][0][NR - 1], hi[p][1][0], hi[p][1][NR - 1], b[k][p][0], b[k][p][1]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          float* to = o[4 * w + k] + i;
          const float2 v = f2add(make_float2(to[0], to[1]), make_float2(d[k][i], d[k][i + 1]));
          to[0] = v.x;
          to[1] = v.y;
        }
    }
  }

  // Raw tokens of the tail in fp32, n <= 16 rows of the stage: token 8 e + 2 t +
  // j for row r at s[8 r + 2 e + j], without the row's and the softmax's scales;
  // queries times kRawQ where SMALL. Four tokens at a time (rows behind the n-th
  // are hidden afterwards).
  template <bool SMALL>
  __device__ __forceinline__ void raw_products(const Q8Args& A, const uint16_t* K, int n, float (&s)[R]) const {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int x = 0; x < R; ++x) s[x] = 0.f;
#pragma unroll(SMALL && NR == 2 ? 1 : 4)
    for (int i = 0; i < ((n + 3) & ~3); ++i) {
      float d[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) d[r] = 0.f;
#pragma unroll
      for (int c = 0; c < kDW / 64; ++c) {
        float f[16];
        raw16(K + i * D + 16 * (t + 4 * c), A.bf16, f);
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            float2 a = __half22float2(u32_as_h2(q[4 * c + k][2 * r]));
            float2 b = __half22float2(u32_as_h2(q[4 * c + k][2 * r + 1]));
            if constexpr (SMALL) {
              a = f2mul(a, f2(kRawQ));
              b = f2mul(b, f2(kRawQ));
            }
            d[r] = fmaf(a.x, f[4 * k], d[r]);
            d[r] = fmaf(a.y, f[4 * k + 1], d[r]);
            d[r] = fmaf(b.x, f[4 * k + 2], d[r]);
            d[r] = fmaf(b.y, f[4 * k + 3], d[r]);
          }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        d[r] += __shfl_xor_sync(0xffffffffu, d[r], 1);
        d[r] += __shfl_xor_sync(0xffffffffu, d[r], 2);
#pragma unroll
        for (int x = 0; x < 4; ++x)
          if (i == 8 * (x >> 1) + 2 * t + (x & 1)) s[8 * r + x] = d[r];
      }
    }
  }

  __device__ __forceinline__ void raw_scores(const Q8Args& A, const uint16_t* K, int n, float (&s)[R]) const {
    // a large scale comes before the row's power of two, a small one after it: what lies between is a float
    const bool large = fabsf(A.scale_log2) >= 1.f;
    float before = large ? A.scale_log2 : 1.f;
    const float after = (large ? 1.f : A.scale_log2) * (1.f / kRawQ);
    if constexpr (NR == 1) {
      raw_products<true>(A, K, n, s);
    } else {  // the factor on sixteen rows' queries costs more than a look at the products
      raw_products<false>(A, K, n, s);
      const int t = threadIdx.x & 3;
      bool fine = true;
#pragma unroll
      for (int x = 0; x < R; ++x)
        if ((x & 7) < 4) fine = fine && (8 * (x >> 1 & 1) + 2 * t + (x & 1) >= n || fabsf(s[x]) < INFINITY);
      if (__builtin_expect(__any_sync(0xffffffffu, !fine), 0))
        raw_products<true>(A, K, n, s);
      else
        before *= kRawQ;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int x = 0; x < 4; ++x) s[8 * r + x] = s[8 * r + x] * before * qi[r] * after;
  }

  __device__ __forceinline__ void add_raw(const Q8Args& A, const uint16_t* V, int token0, int n, const float (&s)[R]) {
    const int lane = threadIdx.x & 31, t = lane & 3;
    float w[NR][4], ms[NR], mts[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      ms[r] = -INFINITY;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 8 * (x >> 1) + 2 * t + (x & 1);
        w[r][x] = i < n && sees(A, r, token0 + i) ? s[8 * r + x] : -INFINITY;
        ms[r] = fmaxf(ms[r], w[r][x]);
      }
      mts[r] = __fadd_ru(ms[r], kRawUp);
    }
    raise(ms, mts);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float2 sum = f2(0.f);
      const float cm = -base(m[r]), ct = kExponents ? kOff + (base(m[r]) - base(mt[r])) : -base(mt[r]);
#pragma unroll
      for (int x = 0; x < 4; x += 2) {
        const float2 v = weigh(make_float2(w[r][x], w[r][x + 1]), cm, ct, kExponents ? 1.f : 0x1p12f, sum);
        w[r][x] = v.x;
        w[r][x + 1] = v.y;
      }
      l[r] += sum.x + sum.y;
    }
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const int x = 2 * (i >> 3) + (i & 1), from = (lane & 28) | (i & 7) >> 1;
      float wi[NR];
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const float v = x == 0 ? w[r][0] : x == 1 ? w[r][1] : x == 2 ? w[r][2] : w[r][3];
        wi[r] = __shfl_sync(0xffffffffu, v, from);
      }
      const uint32_t* src = reinterpret_cast<const uint32_t*>(V + i * D) + t;
#pragma unroll
      for (int c = 0; c < kDW / 8; ++c) {
        float f[4];
        raw4(src[4 * c], 0u, A.bf16, f);
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (wi[r] != 0.f) {  // a hidden token's value may be anything
            o[c][2 * r] = fmaf(wi[r], f[0], o[c][2 * r]);
            o[c][2 * r + 1] = fmaf(wi[r], f[1], o[c][2 * r + 1]);
          }
      }
    }
  }
};

// out and lse of a row from its sums: O 2^(mt - kOff) / (l 2^m).
__device__ __forceinline__ float out_factor(float m, float mt, float l) {
  return l == 0.f ? 0.f : exp2f(mt - m - kOff) / l;
}
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }

template <int D, int R, int CODE>
__global__ void __launch_bounds__(32 * kWarps, 1) q8_decode_kernel(const __grid_constant__ Q8Args A) {
  using S = Shape<D, R>;
  constexpr int W = kWarps, HV = S::HV, TEAMS = S::TEAMS, ROW = part_row(D);
  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BARS);
  __shared__ int64_t sum_of[W], range_at[TEAMS], start_at[TEAMS];
  __shared__ int start_b[TEAMS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < TEAMS * kStages) mbar_init(bars + tid, 1);
  fence_mbar_init();
  pdl_wait_primary();
  pdl_launch_dependents();

  // Items before each sequence: thread i counts those of an equal share of
  // the sequences.
  const int units = A.Hkv * A.groups;
  const int per = (A.B + 32 * W - 1) / (32 * W), b0 = min(A.B, tid * per), b1 = min(A.B, b0 + per);
  int64_t mine = 0;
  Place at;
  for (int b = b0; b < b1; ++b) {
    at.s.load(A, b);
    mine += static_cast<int64_t>(at.s.items) * units;
    if (blockIdx.x == 0) {
      if (A.lens[b] != at.s.L) set_error(A.err, KVARN_DEVERR_SEQ_LEN);
      if (at.s.tail > 0 && (!A.tail_k || !A.tail_v)) set_error(A.err, KVARN_DEVERR_NO_TAIL);
    }
  }
  int64_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += x;
  }
  if (lane == 31) sum_of[warp] = before;
  before -= mine;
  __syncthreads();
  int64_t total = 0;
  for (int w = 0; w < W; ++w) {
    if (w < warp) before += sum_of[w];
    total += sum_of[w];
  }
  // Range e of as many as there are teams (warps, or pairs of them), at most
  // one per item, is that of team e / grid of CTA e % grid: few items spread
  // over the SMs.
  const int64_t teams = min(total, static_cast<int64_t>(gridDim.x) * TEAMS);
  auto range_of = [&](int w) { return static_cast<int64_t>(w) * gridDim.x + blockIdx.x; };
  if (tid < TEAMS) range_at[tid] = range_of(tid) < teams ? quotient(range_of(tid) * total, teams) : -1;
  __syncthreads();
  for (int b = b0; b < b1; ++b) {
    if (blockIdx.x == 0) A.offs[b] = before;
    at.s.load(A, b);
    const int64_t n = static_cast<int64_t>(at.s.items) * units;
    for (int w = 0; w < TEAMS; ++w) {
      const int64_t x = range_at[w];
      if (x >= before && x < before + n) {
        start_b[w] = b;
        start_at[w] = x - before;
      }
    }
    before += n;
  }
  if (blockIdx.x == 0 && tid == 0) A.offs[A.B] = total;
  __syncthreads();
  const int team = warp / HV, half = warp % HV;
  const int64_t range = range_of(team);
  if (range >= teams) return;
  const int64_t x0 = range_at[team], x1 = quotient((range + 1) * total, teams);

  at.b = start_b[team];
  at.s.load(A, at.b);
  const int unit = static_cast<int>(quotient(start_at[team], at.s.items));
  at.i = static_cast<int>(start_at[team] - static_cast<int64_t>(unit) * at.s.items);
  at.h = unit / A.groups;
  at.grp = unit % A.groups;
  Place ahead = at;
  const int count = static_cast<int>(x1 - x0);  // items of this team
  unsigned char* ring = smem + team * kStages * S::STAGE;
  uint64_t* bar = bars + team * kStages;

  // Copies of the next item that none has been asked for into its stage. ids:
  // 32 entries of the block list of sequence ids_b from ids_at on.
  const bool has_tail = A.tail_k && A.tail_v;
  int ids = 0, ids_b = -1, ids_at = 0, issued = 0, issue_st = 0;
  auto issue = [&]() {
    if (ahead.i < ahead.s.page_items) {
      const int i = 2 * ahead.i, n = min(2, ahead.s.np - i);
      if (ids_b != ahead.b || ids_at != (i & ~31)) {
        ids_b = ahead.b;
        ids_at = i & ~31;
        const int k = ids_at + lane;
        ids = 0;
        if (k < ahead.s.np) {
          ids = A.table[static_cast<int64_t>(ahead.b) * A.bt_stride + ahead.s.block(k)];
          if (ids < 0 || ids >= A.num_pages) {
            set_error(A.err, KVARN_DEVERR_PAGE_RANGE);
            ids = 0;
          }
        }
      }
      const int p0 = __shfl_sync(0xffffffffu, ids, i & 31), p1 = __shfl_sync(0xffffffffu, ids, (i + 1) & 31);
      if (lane == 0) {
        unsigned char* dst = ring + issue_st * S::STAGE;
        mbar_arrive_expect_tx(bar + issue_st, n * S::PB + A.withhold);
        bulk_g2s(dst, A.cache + (static_cast<int64_t>(p0) * A.Hkv + ahead.h) * S::PB, S::PB, bar + issue_st);
        if (n == 2)
          bulk_g2s(dst + S::PB, A.cache + (static_cast<int64_t>(p1) * A.Hkv + ahead.h) * S::PB, S::PB, bar + issue_st);
      }
    } else if (lane == 0) {  // raw tokens: their key rows, then at 16 rows their value rows
      const int r0 = 16 * (ahead.i - ahead.s.page_items), bytes = has_tail ? min(16, ahead.s.tail - r0) * 2 * D : 0;
      mbar_arrive_expect_tx(bar + issue_st, 2 * bytes + (bytes ? A.withhold : 0));
      if (bytes) {
        unsigned char* dst = ring + issue_st * S::STAGE;
        const int64_t from = ((static_cast<int64_t>(ahead.b) * A.Hkv + ahead.h) * A.tail_cap + r0) * D;
        bulk_g2s(dst, static_cast<const uint16_t*>(A.tail_k) + from, bytes, bar + issue_st);
        bulk_g2s(dst + 32 * D, static_cast<const uint16_t*>(A.tail_v) + from, bytes, bar + issue_st);
      }
    }
    if (++issue_st == kStages) issue_st = 0;
    if (++issued < count) ahead.next(A);
  };
  if (half == 0)
    for (int k = 0; k < min(kStages, count); ++k) issue();

  Rows<D, R> rows;
  bool fresh = true, whole = false;  // whole: the unit's first item was this team's
  int seg_item = 0;                  // the range's item that the segment began with
  int st = 0;
  uint32_t parity = 0;
  for (int k = 0; k < count; ++k) {
    if (fresh) {
      rows.load(A, at.b, at.h, at.grp, at.s, half * kDW);
      fresh = false;
      whole = at.i == 0;
      seg_item = k;
    }
    bool came = mbar_test_phase(bar + st, parity);
    if (!__all_sync(0xffffffffu, came))
      came = __all_sync(0xffffffffu, mbar_wait_bounded(bar + st, parity, A.wait_limit));
    const bool paged = at.i < at.s.page_items;
    const int i0 = 2 * at.i, n = min(2, at.s.np - i0);
    const unsigned char* pg0 = ring + st * S::STAGE;
    const unsigned char* pg1 = n == 2 ? pg0 + S::PB : pg0;
    const bool raw = !paged && has_tail;
    int r0 = 0, nraw = 0;
    if (!paged) {
      r0 = 16 * (at.i - at.s.page_items);
      nraw = min(16, at.s.tail - r0);
    }
    float s[R];
    if (paged)
      rows.template page_scores<CODE>(A, pg0, pg1, half, s);
    else if (raw)
      rows.raw_scores(A, reinterpret_cast<const uint16_t*>(pg0) + half * kDW, nraw, s);
    bool dead = !came;
    if constexpr (HV == 2) {
      float* mine = reinterpret_cast<float*>(smem + S::XCHG + team * S::XBUF) + ((k & 1) * 2 + half) * S::XLANE * 32;
      const float* other = mine + (half ? -1 : 1) * S::XLANE * 32;
      volatile int* flag = reinterpret_cast<volatile int*>(smem + S::FLAGS) + (team * 2 + (k & 1)) * 2;
#pragma unroll
      for (int x = 0; x < R; ++x) mine[x * 32 + lane] = s[x];
      if (lane == 0) flag[half] = dead;
      asm volatile("bar.sync %0, 64;" ::"r"(1 + team) : "memory");
#pragma unroll
      for (int x = 0; x < R; ++x) s[x] += other[x * 32 + lane];
      dead = dead || flag[half ^ 1];
      // both warps have left the item before this one
      if (half == 0 && !dead && k > 0 && issued < count) issue();
    }
    if (dead) {
      // give up: the copies under way have to land before the CTA leaves, which
      // the warp that asked for them sees to (the other does not know how many
      // they are, and a stage that was not asked for would hold it to the limit)
      if (!came) set_error(A.err, KVARN_DEVERR_TIMEOUT);
      if (half == 0)
        for (int j = k; j < issued; ++j) mbar_wait_bounded(bar + j % kStages, (j / kStages) & 1, 100000000LL);
      return;
    }
    if (paged)
      rows.template add_pages<CODE>(A, pg0, pg1, half, at.s, i0, n, s);
    else if (raw)
      rows.add_raw(A, reinterpret_cast<const uint16_t*>(pg0 + 32 * D) + half * kDW, at.s.C * kPageTokens + r0, nraw, s);
    __syncwarp();
    if (HV == 1 && issued < count) issue();
    const bool last = at.i + 1 == at.s.items;
    if (last || k + 1 == count) {
      const int g = lane >> 2, t = lane & 3;
#pragma unroll
      for (int r = 0; r < rows.NR; ++r) {
        float l = rows.l[r];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        const int rr = at.grp * R + 8 * r + g;
        float f = 1.f;
        float* dst = nullptr;
        if (last && whole) {
          if (rr < A.G * A.Q) {
            const int64_t row = (static_cast<int64_t>(at.b) * A.Q + rr / A.G) * A.Hq + at.h * A.G + rr % A.G;
            f = out_factor(rows.m[r], rows.mt[r], l);
            dst = A.out + row * D;
            if (A.lse && t == 0 && half == 0) A.lse[row] = lse_of(rows.m[r], l);
          }
        } else {
          dst = A.part + ((2 * range + (seg_item == 0 ? 0 : 1)) * R + 8 * r + g) * ROW;
          if (t == 0 && half == 0) *reinterpret_cast<float4*>(dst) = make_float4(rows.m[r], l, rows.mt[r], 0.f);
          dst += 4;
        }
        if (dst) {
          dst += half * kDW + 2 * t;
#pragma unroll
          for (int c = 0; c < kDW / 8; ++c) {
            const float a = rows.NR == 2 ? rows.o[c][2 * r] : rows.o[c][0] + rows.o[c][2];
            const float b = rows.NR == 2 ? rows.o[c][2 * r + 1] : rows.o[c][1] + rows.o[c][3];
            *reinterpret_cast<float2*>(dst + 8 * c) = make_float2(a * f, b * f);
          }
        }
      }
      fresh = true;
    }
    if (++st == kStages) {
      st = 0;
      parity ^= 1;
    }
    if (k + 1 < count) at.next(A);
  }
}

// One warp per output row: joins the parts of units that several warps took,
// writes the rows of empty sequences. 3 to 6 us of two dependent trips to memory
// and the parts, four to eight under way.
template <int D, int R>
__global__ void __launch_bounds__(128) q8_merge_kernel(const __grid_constant__ Q8Args A, int64_t grid_teams) {
  constexpr int E = D / 32, ROW = part_row(D);
  pdl_wait_primary();
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= static_cast<int64_t>(A.B) * A.Q * A.Hq) return;
  const int at = static_cast<int>(row) / A.Hq, hq = static_cast<int>(row) % A.Hq;  // at most 2^30 rows
  const int b = at / A.Q, j = at % A.Q;
  const int h = hq / A.G, rr = j * A.G + hq % A.G, units = A.Hkv * A.groups;
  const int64_t o0 = A.offs[b], o1 = A.offs[b + 1], total = A.offs[A.B];
  const int64_t items = quotient(o1 - o0, units), teams = min(total, grid_teams);
  float* dst = A.out + row * D + lane * E;
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float M = -INFINITY, L = 0.f, f = 0.f;
  if (items > 0) {
    const int64_t p0 = o0 + (static_cast<int64_t>(h) * A.groups + rr / R) * items, p1 = p0 + items;
    // the range of item x is the last that begins at or before it
    const int64_t w0 = quotient((p0 + 1) * teams - 1, total), w1 = quotient(p1 * teams - 1, total);
    if (w0 == w1) return;
    const bool inside = quotient(w0 * total, teams) < p0;  // the first range begins before the unit
    const int n = static_cast<int>(w1 - w0 + 1);
    const float* part = A.part + (2 * w0 * R + rr % R) * ROW;
    auto slot = [&](int i) { return part + static_cast<int64_t>(2 * i + (i == 0 && inside ? 1 : 0)) * R * ROW; };
    // a lane keeps the head (m, l, mt) of every 32nd part: the maxima first
    float MT = -INFINITY;
    float4 head = make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
    for (int i = lane; i < n; i += 32) {
      const float4 v = *reinterpret_cast<const float4*>(slot(i));
      M = fmaxf(M, v.x);
      MT = fmaxf(MT, v.z);
      if (i < 32) head = v;
    }
    M = warp_max_xor(M, 1, 32);
    MT = warp_max_xor(MT, 1, 32);
    const float mu = M == -INFINITY ? 0.f : M, mtu = MT == -INFINITY ? 0.f : MT;
    for (int i0 = 0; i0 < n; i0 += 32) {
      if (i0 > 0 && i0 + lane < n) head = *reinterpret_cast<const float4*>(slot(i0 + lane));
      const bool mine = i0 + lane < n;
      const float w = mine ? exp2f(head.z - mtu) : 0.f;
      L += mine ? head.y * exp2f(head.x - mu) : 0.f;
      const int count = min(32, n - i0);
#pragma unroll 8
      for (int i = 0; i < count; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        const float* p = slot(i0 + i) + 4 + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 v = *reinterpret_cast<const float4*>(p + e);
          acc[e] = fmaf(v.x, wi, acc[e]);
          acc[e + 1] = fmaf(v.y, wi, acc[e + 1]);
          acc[e + 2] = fmaf(v.z, wi, acc[e + 2]);
          acc[e + 3] = fmaf(v.w, wi, acc[e + 3]);
        }
      }
    }
    L = warp_sum_xor(L, 1, 32);
    f = out_factor(mu, mtu, L);
    M = mu;
  }
#pragma unroll
  for (int e = 0; e < E; e += 4)
    *reinterpret_cast<float4*>(dst + e) = make_float4(acc[e] * f, acc[e + 1] * f, acc[e + 2] * f, acc[e + 3] * f);
  if (A.lse && lane == 0) A.lse[row] = lse_of(M, L);
}

// Sixteen rows to a group wherever there are more than eight. 32 sequences of
// 24/4 heads of 256 behind a window of 4096 tokens: 2 queries (12 rows) 94 us as
// one group of sixteen, 121 as two of eight; 3 queries (18 rows) 153 as two, 167
// as three. 2 queries of 64/8 heads of 128 (16 rows) over 32 x 8192 tokens 138
// and 185.
int rows_per_group(int rows) { return rows > 8 ? 16 : 8; }

template <int D, int R, int CODE>
cudaError_t run(const Q8Args& A, int ctas, cudaStream_t st) {
  using S = Shape<D, R>;
  auto* kernel = q8_decode_kernel<D, R, CODE>;
  static SmemLimit limit;
  cudaError_t e = limit.set(kernel, S::SMEM);
  if (e != cudaSuccess) return e;
  e = chained(kernel, dim3(ctas), 32 * kWarps, S::SMEM, st, A);
  if (e != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(A.B) * A.Q * A.Hq;
  return chained(q8_merge_kernel<D, R>, dim3(static_cast<unsigned>((rows + 3) / 4)), 128, 0, st, A,
                 static_cast<int64_t>(ctas) * S::TEAMS);
}

}  // namespace

// Offsets, then two partial slots per team.
int64_t q8_decode_workspace_bytes(int32_t num_seqs, int32_t rows, int32_t D) {
  const int64_t teams = static_cast<int64_t>(device_sm_count()) * (kWarps * kDW / D);
  return (8LL * (num_seqs + 1) + 127) / 128 * 128 + teams * 2 * rows_per_group(rows) * part_row(D) * 4;
}

cudaError_t launch_q8_decode(const Q8DecodeParams& p, cudaStream_t st) {
  Q8Args A{};
  A.q = p.q;
  A.cache = p.cache;
  A.table = p.block_table;
  A.bt_stride = p.bt_stride;
  A.lens = p.seq_lens;
  A.max_len = p.max_seq_len;
  A.B = p.num_seqs;
  A.Q = p.num_queries;
  A.Hq = p.num_q_heads;
  A.Hkv = p.num_kv_heads;
  A.G = p.num_q_heads / p.num_kv_heads;
  const int R = rows_per_group(A.G * A.Q);
  A.groups = (A.G * A.Q + R - 1) / R;
  A.num_pages = p.num_pages;
  A.tail_k = p.tail_k;
  A.tail_v = p.tail_v;
  A.tail_cap = p.tail_cap;
  // every query sees at most the whole sequence
  A.window = p.window >= p.max_seq_len ? 0 : p.window;
  A.sinks = std::min(p.sinks, p.max_seq_len);
  A.scale_log2 = p.sm_scale * 1.4426950408889634f;
  A.bf16 = p.bf16;
  A.out = p.out;
  A.lse = p.lse;
  A.offs = static_cast<int64_t*>(p.workspace);
  A.part = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + (8LL * (p.num_seqs + 1) + 127) / 128 * 128);
  A.err = p.err;
  A.wait_limit = copy_wait_limit();
  A.withhold = copy_withhold();
  const int ctas = device_sm_count();
  const bool i8 = p.code == kQ8Int8;
  if (p.D == 128) {
    if (R == 8) return i8 ? run<128, 8, kQ8Int8>(A, ctas, st) : run<128, 8, kQ8E4M3>(A, ctas, st);
    return i8 ? run<128, 16, kQ8Int8>(A, ctas, st) : run<128, 16, kQ8E4M3>(A, ctas, st);
  }
  if (R == 8) return i8 ? run<256, 8, kQ8Int8>(A, ctas, st) : run<256, 8, kQ8E4M3>(A, ctas, st);
  return i8 ? run<256, 16, kQ8Int8>(A, ctas, st) : run<256, 16, kQ8E4M3>(A, ctas, st);
}

}  // namespace kvarn
