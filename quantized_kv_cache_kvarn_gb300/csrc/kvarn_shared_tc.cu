// Scores and values of a shared prefix on the fifth-generation tensor cores,
// sm_103a, head_dim 128.
//
// The prefix's pages meet the query rows of the whole batch (R = sequences x
// queries x G rows per KV head), so the products are matrix products: a CTA
// takes 128 rows of one KV head and a run of the prefix's tiles, 64 tokens (a
// stage) at a time, flash-attention style:
//   S = q' K^T   (128 x 64, K = 128)     P = 2^(S - m)     O += P V
// with q' = kappa q H / sqrt(D) (rotated basis, base-2 scores), K and V the
// dequantised rotated rows c (a code + b).
//
// fp32 results need more than one fp16 product: every operand is x = hi + lo
// in fp16 (off by 2^-22 of its tile's or row's magnitude, which a power of two
// brings to about 1 first: 2^eK, 2^eV per tile, 2^eq per row), and each
// product is hi hi + lo hi + hi lo, three MMAs with fp32 accumulators in
// tensor memory. eK and eq return with the scores' scale. eV goes into the
// weights: P = 2^(S + eV - m), where m follows the largest S + eV of the row,
// the bound of a token's share of the output, instead of the largest S alone.
// So O = sum P V 2^-eV is in units of 2^m whichever tiles it adds up, tiles of
// values of any sizes fit fp16 as operands, and what P loses below 2^-25 is
// lost against the largest share. The sum of the weights takes 2^-eV back in
// fp32. Codes as exact operands with the scales folded around them (as in the
// dense decode) would need two, but their column scales change q' with every
// tile and their row scales the output: 576 + 320 more issue slots per SM and
// tile than this form spends.
//
// Roles (896 threads, one CTA per SM; registers moved to them with setmaxnreg):
//   warps 0-7    softmax: two threads per row (= tensor-memory lane), 32 of
//                the stage's 64 tokens each; a pair of warps exchanges its
//                maxima through shared memory. Keeps the running maximum
//                of S + eV (an integer, so that it adds to eV and to the
//                partial's exponent without rounding; raised only when passed
//                by 2^8, so that O is rescaled a few times at most) and sum,
//                writes P hi / lo over the scores as the A operand
//   warps 8-23   dequantisation, K on eight and V on eight, warp = (page of the
//                stage, 64-channel group): code planes -> exact fp16 (the
//                decode's conversions) -> fp32 c (a code + b) -> hi and lo,
//                stored in the B operands' 128-byte-swizzled rows: K as token
//                rows of channels, V as channel rows of tokens, which is how
//                the pages' fragments pair their codes, so every store is one
//                conflict-free word
//   warp 24      MMA issue: QK of stage s + 2 behind PV of stage s, so that the
//                tensor pipe has work while the softmax runs
//   warps 25, 26 page copies (bulk copies, up to four tiles in flight) and, per
//                tile, the scales of K and of V unpacked to fp32 and their
//                exponents
// Tensor memory: q' hi, lo 128 columns; S (then P) 2 x 64; O 128, and 128 for
// the sum of its small products (lo hi + hi lo): the tensor cores truncate the
// accumulator at every step, so the long sum takes four steps a stage instead
// of twelve (error against 64 bits at 16384 tokens with one accumulator:
// 5.4e-6, with two 2.7e-6, of the fp32 form 2.6e-6).
// A stage costs the tensor pipe 24 MMAs of N = 64 and 12 of N = 128: 1536
// cycles per 64 tokens and 128 rows. Measured, 256 rows of 8 KV heads over
// 16384 tokens: 56 us, about 2870 cycles a stage, tensor pipe 43% and issue
// slots 66% of active cycles: the conversions of the hi / lo splits and the
// softmax share the issue slots, DRAM (16.4 MB) does not matter.
#include <math.h>

#include <algorithm>

#include "kvarn_common.cuh"
#include "kvarn_launch.h"
#include "kvarn_merge.cuh"
#include "kvarn_shared.cuh"
#include "kvarn_tcgen05.cuh"

namespace kvarn {

namespace {

constexpr int kD = 128, kM = 128, kStage = 64;  // channels, rows of a CTA, tokens of a stage
constexpr int kSoftmax = 256, kDequant = 512, kThreads = kSoftmax + kDequant + 128;
constexpr int kMmaWarp = (kSoftmax + kDequant) / 32;  // then the page copies' and scales' two
// registers per thread: at launch, then per role (whole warpgroups)
constexpr int kRegs = 72, kRegsSoftmax = 96, kRegsDequant = 64, kRegsOther = 56;
static_assert(kSoftmax * kRegsSoftmax + kDequant * kRegsDequant + 128 * kRegsOther <= kThreads * kRegs, "register split");
constexpr int kPlane = kStage * kD * 2;   // hi or lo operand plane: 16 KB
constexpr int kRing = 2;                  // stages of K and of V in flight
constexpr int kPages = 4;                 // most tiles whose pages are in shared memory or on their way
constexpr int kMetaSlots = 8;             // tiles whose scales are kept: past kPages, the softmax may be three behind
constexpr int kMeta = 6 * 128 * 4 + 16;   // cK, cV, aK, bK, aV, bV, 2^eK, eV, 2^-eV
constexpr int kOffK = 0, kOffV = kRing * 2 * kPlane, kOffMeta = 2 * kOffV, kOffScale = kOffMeta + kMetaSlots * kMeta;
constexpr int kBarBytes = 320, kOffMax = kOffScale + kM * 4, kOffBar = kOffMax + 4 * kM * 4, kOffRaw = kOffBar + kBarBytes;
constexpr int kQRow = 2 * kD * 2 + 16;    // staged query row: hi, lo, padding
static_assert(kM * kQRow <= kOffMeta, "query rows are staged in the operand rings");
static_assert(kOffRaw % 16 == 0 && kOffMeta % 1024 == 0, "layout");
enum { B_KF = 0, B_KE = 2, B_VF = 4, B_VE = 6, B_SF = 8, B_PF = 10, B_OF = 12, B_FIN = 14, B_RF = 15, B_RE = B_RF + kPages,
       B_META = B_RE + kPages, kBars = B_META + kMetaSlots };
static_assert(kBars * 8 + 8 <= kBarBytes, "barriers");
constexpr uint32_t kColQ = 0, kColS = 128, kColO = 256, kColL = 384;  // tensor-memory columns
constexpr uint32_t kIdQK = tc_idesc_f16(kM, kStage, false, false), kIdPV = tc_idesc_f16(kM, kD, false, false);
constexpr int kSmemMax = 232448;
static_assert(kOffRaw + 2 * 8 * DensePage(kD, 128, 8, 8, 4).bytes() + 1024 <= kSmemMax, "two tiles of the widest pages");
constexpr long long kMmaWait = 2000000000LL, kDrainWait = 100000000LL;  // cycles: about a second, 50 ms
constexpr uint32_t kGone = 0x7f800badu;  // in place of a value between a pair's warps: one of them gives up
constexpr float kRaise = 8.f;  // log2 of how far a share may pass the running maximum
// Exponents of a tile's values: between them 2^-eV times a sum of weights (at
// most 2^8 a token) stays in fp32's range, and values to 2^125 in fp16's. A
// tile of zeros takes no share: an exponent kZeros below that of the tile
// before (the least where there is none) keeps it from raising the maximum
// unless its scores are as far above, and its weights, down to 2^-126 of the
// maximum, in the sum.
constexpr int kLeastExp = -90, kMostExp = 110, kZeros = 40, kLeastZeros = -100;

// Barriers by shared-memory address: one probe (the hardware may hold the
// thread a short time; with a time hint it would poll with sleeps between),
// and an arrival.
__device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// One thread of the warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

template <int R> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }

// D (tensor memory) = A (tensor memory) * B^T (+ D if `accumulate`).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u));
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }
// Exponent of a positive normal float, 0 for others (zero, inf, nan, subnormal).
__device__ __forceinline__ int exponent_of(float x) {
  const int e = (__float_as_int(x) >> 23) & 255;
  return e == 0 || e == 255 ? 0 : e - 127;
}

// hi and lo words of a pair at `off` of the two planes of an operand stage.
__device__ __forceinline__ void put_pair(unsigned char* plane, uint32_t off, float2 x) {
  uint32_t hi, lo;
  split_hi_lo2(x, hi, lo);
  *reinterpret_cast<uint32_t*>(plane + off) = hi;
  *reinterpret_cast<uint32_t*>(plane + kPlane + off) = lo;
}

// The code words of one lane for eight fragments, taken W0 times F0 = 8 / W0
// fragments: after a step the words move down, so that a step's fragments
// are always slots 0 .. F0 - 1 of the first word of each plane and the loop
// over the steps stays rolled (unrolled, the six widths of K and of V, the
// softmax and the MMA issue of one scheduler do not fit its instruction
// cache: no-instruction stalls were the largest).
template <int B>
struct CodeWords {
  static constexpr int W0 = plane_w0(B), W1 = plane_w1(B), F0 = 8 / W0;
  uint32_t x0[W0], x1[W1 ? W1 : 1];
  template <int SLOT>
  __device__ __forceinline__ void pair(uint32_t& b0, uint32_t& b1) const {
    code_pair<B, SLOT, SLOT>(x0[0], x1[0], b0, b1);
  }
  __device__ __forceinline__ void next() {
#pragma unroll
    for (int i = 0; i + 1 < W0; ++i) x0[i] = x0[i + 1];
    if constexpr (W1 == 4) {  // two fragments a word, as in the first plane
#pragma unroll
      for (int i = 0; i + 1 < W1; ++i) x1[i] = x1[i + 1];
    } else if constexpr (W1 == 2) {  // four a word, a byte each: two bytes on
      x1[0] = __funnelshift_r(x1[0], x1[1], 16);
      x1[1] >>= 16;
    } else if constexpr (W1 == 1) {  // eight a word, a bit of each byte each
      x1[0] >>= F0;
    }
  }
};

// K of one page and one group of 64 channels (ch): 16 pairs a lane. page: the
// raw K part; a, b: the page's 16 row scales (a / kappa, b + a centre); c: the
// tile's column scales; tok0: the page's first token in the stage.
template <int KB>
__device__ __forceinline__ void dequant_k(const unsigned char* page, const float* a, const float* b, const float* c,
                                          unsigned char* plane, int ch, int tok0, int lane) {
  using C = CodeWords<KB>;
  constexpr int W0 = C::W0, W1 = C::W1;
  constexpr int U0 = kD * W0 / 64 < 4 ? kD * W0 / 64 : 4, U1 = W1 ? (kD * W1 / 64 < 4 ? kD * W1 / 64 : 4) : 1;
  const int g = lane >> 2, t = lane & 3;
  C x;
  load_words<W0>(page + 4 * U0 * (32 * ((ch * W0) / U0) + lane) + 4 * ((ch * W0) % U0), x.x0);
  if constexpr (W1 != 0)
    load_words<W1>(page + 2 * kD * W0 + 4 * U1 * (32 * ((ch * W1) / U1) + lane) + 4 * ((ch * W1) % U1), x.x1);
  const float2 a2[2] = {f2(a[g]), f2(a[8 + g])}, b2[2] = {f2(b[g]), f2(b[8 + g])};
  unsigned char* dst = plane + ch * (kStage * 128) + (tok0 + g) * 128 + 4 * t;  // row g of the first token block
  c += 64 * ch + 2 * t;
#pragma unroll 1
  for (int step = 0; step < W0; ++step) {
    static_for<0, C::F0 / 2>([&](auto kq) {  // k-chunks of the step (16 channels), two token blocks each
      constexpr int q = decltype(kq)::value;
      const int kc = step * (C::F0 / 2) + q;
      const float2 c0 = *reinterpret_cast<const float2*>(c + 16 * kc);
      const float2 c1 = *reinterpret_cast<const float2*>(c + 16 * kc + 8);
      const uint32_t u0 = ((2 * kc) ^ g) << 4, u1 = ((2 * kc + 1) ^ g) << 4;  // 128-byte swizzle (rows are g modulo 8)
      static_for<0, 2>([&](auto ec) {
        constexpr int e = decltype(ec)::value;
        uint32_t w0, w1;
        x.template pair<2 * q + e>(w0, w1);
        put_pair(dst, 1024 * e + u0, f2mul(c0, f2fma(a2[e], __half22float2(u32_as_h2(w0)), b2[e])));
        put_pair(dst, 1024 * e + u1, f2mul(c1, f2fma(a2[e], __half22float2(u32_as_h2(w1)), b2[e])));
      });
    });
    x.next();
  }
}

// V of one page (p of the stage) and one group of 64 channels (hq).
template <int VB>
__device__ __forceinline__ void dequant_v(const unsigned char* page, const float* a, const float* b, const float* c,
                                          unsigned char* plane, int hq, int p, int lane) {
  using C = CodeWords<VB>;
  constexpr int W0 = C::W0, W1 = C::W1;
  const int g = lane >> 2, t = lane & 3;
  C x;
  load_words<W0>(page + 4 * W0 * (32 * hq + lane), x.x0);
  if constexpr (W1 != 0) load_words<W1>(page + 2 * kD * W0 + 4 * W1 * (32 * hq + lane), x.x1);
  const float2 a0 = *reinterpret_cast<const float2*>(a + 2 * t), a1 = *reinterpret_cast<const float2*>(a + 8 + 2 * t);
  const float2 b0 = *reinterpret_cast<const float2*>(b + 2 * t), b1 = *reinterpret_cast<const float2*>(b + 8 + 2 * t);
  unsigned char* dst0 = plane + (64 * hq + g) * 128 + (((2 * p) ^ g) << 4) + 4 * t;  // channel row g of the first block
  unsigned char* dst1 = plane + (64 * hq + g) * 128 + (((2 * p + 1) ^ g) << 4) + 4 * t;
  c += 64 * hq + g;
#pragma unroll 1
  for (int step = 0; step < W0; ++step) {
    static_for<0, C::F0>([&](auto kc) {  // channel blocks of the step
      constexpr int k = decltype(kc)::value;
      uint32_t w0, w1;
      x.template pair<k>(w0, w1);
      const float2 c2 = f2(c[8 * k]);
      put_pair(dst0, 1024 * k, f2mul(c2, f2fma(a0, __half22float2(u32_as_h2(w0)), b0)));
      put_pair(dst1, 1024 * k, f2mul(c2, f2fma(a1, __half22float2(u32_as_h2(w1)), b1)));
    });
    x.next();
    c += 8 * C::F0;
    dst0 += 1024 * C::F0;
    dst1 += 1024 * C::F0;
  }
}

// POLL: a call whose waits are limited to less than kPollWaitBelow, which a
// probe's own suspension may outlast, keeps the limit by tests that do not
// suspend. A diagnostic's setting, so a kernel of its own: asked at run time,
// it cost 32 x 64 heads over 16384 tokens 2.7 us of 87.
template <bool POLL>
__global__ void __launch_bounds__(kThreads, 1) shared_tc_kernel(const __grid_constant__ SharedTcArgs A) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int split = blockIdx.x, unit = blockIdx.y;
  const int kvh = unit % A.Hkv, blk = unit / A.Hkv;
  const int t0 = split * A.tps, n = min(A.tps, A.tiles - t0);  // this CTA's tiles (n >= 1)
  const int ppt = A.N / kPageTokens, spt = A.N / kStage, stages = n * spt;
  unsigned char* sm = smem + ((1024u - (smem_addr(smem) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kOffBar);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(sm + kOffBar + kBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + kOffBar + kBars * 8 + 4);
  float* rscale = reinterpret_cast<float*>(sm + kOffScale);
  const uint32_t bar0 = smem_addr(bars);
  // Bounded wait, uniform over the warp; gives up (and tells every role to)
  // after the call's limit or once another warp has given up. The clock and the
  // flag are looked at every 32 probes only: a waiting warp takes issue slots
  // from the working ones.
  auto wait = [&](int bar, uint32_t parity) -> bool {
    const uint32_t at = bar0 + 8 * bar;
    if (!POLL && __all_sync(0xffffffffu, probe(at, parity))) return true;
    bool ok = false;
    const long long start = clock64();
    do {
      if (POLL) ok = mbar_test_phase(bars + bar, parity);
#pragma unroll 1
      for (int i = 0; !POLL && i < 32 && !ok; ++i) ok = probe(at, parity);
    } while (!ok && !*abort_flag && clock64() - start <= A.wait_limit);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *abort_flag = 1;
    return ok;
  };

  if (warp == kMmaWarp) tc_alloc(tslot, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bars + B_KF + i, kDequant / 64);
      mbar_init(bars + B_KE + i, 1);
      mbar_init(bars + B_VF + i, kDequant / 64);
      mbar_init(bars + B_VE + i, 1);
      mbar_init(bars + B_SF + i, 1);
      mbar_init(bars + B_PF + i, kSoftmax / 32);
      mbar_init(bars + B_OF + i, 1);
    }
    for (int i = 0; i < kPages; ++i) {
      mbar_init(bars + B_RF + i, 1);
      mbar_init(bars + B_RE + i, kDequant / 32);
    }
    for (int i = 0; i < kMetaSlots; ++i) mbar_init(bars + B_META + i, 2);
    mbar_init(bars + B_FIN, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // Launched as the dependent of the own tokens' decode, which lets it go
  // once the call's inputs are complete (DecArgs::late_trigger): it starts as
  // that kernel's CTAs leave and waits for its end only before ending itself.
  pdl_launch_dependents();

  // ---- query rows: rotated, scaled, hi and lo, by way of shared memory into
  //      tensor memory. Row r of the block is row 128 blk + r of the KV head:
  //      token row (128 blk + r) / G, head kvh G + (128 blk + r) % G.
  const int rows = A.rows_per_head - kM * blk;  // rows used (the others are zero)
  {
    constexpr int kWarps = kThreads / 32, kIter = (kM + kWarps - 1) / kWarps;
    uint2 raw[kIter];
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = warp + i * kWarps;
      raw[i] = make_uint2(0u, 0u);
      if (r < kM && r < rows) {
        const int pr = kM * blk + r;
        const int64_t row = static_cast<int64_t>(pr / A.G) * A.Hq + kvh * A.G + pr % A.G;
        raw[i] = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(A.q) + row * kD + 4 * lane));
      }
    }
#pragma unroll
    for (int i = 0; i < kIter; ++i) {
      const int r = warp + i * kWarps;
      if (r >= kM) break;
      float v[4];
      if (A.bf16) {
        v[0] = __uint_as_float(raw[i].x << 16);
        v[1] = __uint_as_float(raw[i].x & 0xffff0000u);
        v[2] = __uint_as_float(raw[i].y << 16);
        v[3] = __uint_as_float(raw[i].y & 0xffff0000u);
      } else {
        const float2 f0 = __half22float2(u32_as_h2(raw[i].x)), f1 = __half22float2(u32_as_h2(raw[i].y));
        v[0] = f0.x;
        v[1] = f0.y;
        v[2] = f1.x;
        v[3] = f1.y;
      }
      warp_fwht<4>(v);
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] *= A.qscale;
        mx = fmaxf(mx, fabsf(v[e]));
      }
      mx = warp_max_xor(mx, 1, 32);
      const int e = exponent_of(mx);
      // two factors, each a normal power of two
      const float down0 = pow2i(-(e / 2)), down1 = pow2i(-(e - e / 2));
      uint32_t h0, l0, h1, l1;
      split_hi_lo2(make_float2(v[0] * down0 * down1, v[1] * down0 * down1), h0, l0);
      split_hi_lo2(make_float2(v[2] * down0 * down1, v[3] * down0 * down1), h1, l1);
      unsigned char* dst = sm + r * kQRow + 8 * lane;
      *reinterpret_cast<uint2*>(dst) = make_uint2(h0, h1);
      *reinterpret_cast<uint2*>(dst + 2 * kD) = make_uint2(l0, l1);
      if (lane == 0) rscale[r] = pow2i(e);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  const uint32_t tl = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);  // this warp's lanes
  if (warp < kM / 32) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {  // columns 0-63 hi, 64-127 lo
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(sm + tid * kQRow + 128 * k + 16 * j);
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
      }
      tc_st32(tl + kColQ + 32 * k, w);
    }
    tc_wait_st();
    tc_fence_before();
  }
  __syncthreads();  // the staged rows are read: the rings are free
  tc_fence_after();

  if (warp < kSoftmax / 32) {
    // ------------------------------------------------------------- softmax
    regs_inc<kRegsSoftmax>();
    const int r = tid & (kM - 1), half = tid / kM;  // row; tokens [32 half, +32) of every stage
    // warps w and w + 4 share rows and meet once a stage at a named barrier;
    // [stage parity][half][row] for what they exchange. The barrier itself
    // has no time limit, so both act on the same view of the abort flag: what
    // either saw before the barrier, told by a word in place of its value
    // (kGone, a NaN that no arithmetic forms), sends both away. (Behind the
    // barrier each might see another state of the flag, and one would go and
    // the other wait at the next meeting.) A warp whose wait runs out says so
    // and arrives at the next meeting, s, without waiting (leave).
    uint32_t* xch = reinterpret_cast<uint32_t*>(sm + kOffMax);
    const int pair = 1 + (warp & 3);
    auto meet = [&](int s, bool gone, float mine, float& other) -> bool {
      xch[((s & 1) * 2 + half) * kM + r] = gone ? kGone : __float_as_uint(mine);
      tc_fence_before();
      asm volatile("bar.sync %0, 64;" ::"r"(pair) : "memory");
      tc_fence_after();
      const uint32_t word = xch[((s & 1) * 2 + (half ^ 1)) * kM + r];
      other = __uint_as_float(word);
      return __all_sync(0xffffffffu, !gone && word != kGone);
    };
    auto leave = [&](int s) {
      xch[((s & 1) * 2 + half) * kM + r] = kGone;
      __syncwarp();
      asm volatile("bar.arrive %0, 64;" ::"r"(pair) : "memory");
    };
    const float kq = rscale[r];
    float m = -INFINITY, l = 0.f;  // O and l are in units of 2^m
    bool ok = true;
    for (int s = 0; s < stages; ++s) {
      const int tile = spt == 1 ? s : s >> 1;
      // PV(s - 2) has completed by then; waiting for it keeps the parity of
      // its barrier in step, since PV(s - 1) is only waited for when O is
      // rescaled
      if (s >= 2 && !wait(B_OF + (s & 1), ((s >> 1) & 1) ^ 1)) {
        ok = false;
        leave(s);
        break;
      }
      // the tile's exponents (their barrier can not have gone on by two
      // phases: eight tiles ahead is further than the copies get)
      if (!wait(B_SF + (s & 1), (s >> 1) & 1) || !wait(B_META + (tile & (kMetaSlots - 1)), (tile / kMetaSlots) & 1)) {
        ok = false;
        leave(s);
        break;
      }
      tc_fence_after();
      const bool gone = *abort_flag != 0;
      const float* meta = reinterpret_cast<const float*>(sm + kOffMeta + (tile & (kMetaSlots - 1)) * kMeta);
      const float k = kq * meta[6 * 128];
      const float ev = meta[6 * 128 + 1];
      uint32_t x[32];
      const uint32_t scol = tl + kColS + 64 * (s & 1);
      tc_ld32(scol + 32 * half, x);
      tc_wait_ld();
      float mx[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        mx[j] = __uint_as_float(x[j]);
#pragma unroll
        for (int i = 1; i < 8; ++i) mx[j] = fmaxf(mx[j], __uint_as_float(x[4 * i + j]));
      }
      const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      float other;
      if (!meet(s, gone, mine, other)) {  // both have read their scores, too: P may take their place
        ok = false;
        break;
      }
      const float mt = fmaf(fmaxf(mine, other), k, ev);
      // a share far above the maximum so far: O and l are brought to the new
      // one. The first stage has nothing to rescale. Half 0 takes O, half 1
      // its small products. l takes the factor's square root twice: after a
      // tile of small values it is as much larger (2^-eV) as the factor is
      // below fp32's range.
      const bool raise = mt > m + kRaise || (m == -INFINITY && mt > m);
      if (__any_sync(0xffffffffu, raise)) {
        const float m_new = raise ? ceilf(mt) : m;
        const float root = m == -INFINITY ? 0.f : fast_exp2(0.5f * (m - m_new)), alpha = root * root;
        if (s > 0) {
          if (!wait(B_OF + ((s - 1) & 1), ((s - 1) >> 1) & 1)) {
            ok = false;
            leave(s + 1);
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < kD / 32; ++q) {
            uint32_t o[32];
            const uint32_t col = tl + (half ? kColL : kColO) + 32 * q;
            tc_ld32(col, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * (raise ? alpha : 1.f));
            tc_st32(col, o);
          }
          tc_wait_st();
        }
        if (raise) {
          l = l * root * root;
          m = m_new;
        }
      }
      const float2 k2 = f2(k), z2 = f2(ev - m);
      float2 sum[2] = {f2(0.f), f2(0.f)};
      uint32_t hi[16], lo[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float2 z = f2fma(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), k2, z2);
        const float2 p = make_float2(fast_exp2(z.x), fast_exp2(z.y));
        sum[i & 1] = f2add(sum[i & 1], p);
        split_hi_lo2(p, hi[i], lo[i]);
      }
      // P over the scores: hi in the first 32 columns (16 a half), lo in the last
      tc_st16(scol + 16 * half, hi);
      tc_st16(scol + 32 + 16 * half, lo);
      const float2 st = f2add(sum[0], sum[1]);
      l = fmaf(st.x + st.y, meta[6 * 128 + 2], l);
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(bar0 + 8 * (B_PF + (s & 1)));
    }
    // ---- this split's partial: maximum, sum, O in the rotated basis
    if (ok) {
      ok = (stages < 2 || wait(B_OF + (stages & 1), ((stages - 2) >> 1) & 1)) &&
           wait(B_OF + ((stages - 1) & 1), ((stages - 1) >> 1) & 1);
      if (!ok) leave(stages);
    }
    float l1;
    if (ok && meet(stages, *abort_flag != 0, l, l1)) {
      tc_fence_after();
      const bool row = r < rows;
      const int pr = kM * blk + (row ? r : 0);
      const int64_t at = static_cast<int64_t>(pr / A.G) * A.Hq + kvh * A.G + pr % A.G;
      float* part = A.ws + (at * A.slots + split) * kPStride(kD);
      // in units that bring the sum to [1, 2), as the other partials of the
      // row have it to within their number of tokens
      l += l1;
      const int el = exponent_of(l);
      const float u0 = pow2i(-(el / 2)), u1 = pow2i(-(el - el / 2));
      if (row && !half) {
        part[0] = m + static_cast<float>(el);
        part[1] = l * u0 * u1;
      }
#pragma unroll 1
      for (int q = 2 * half; q < 2 * half + 2; ++q) {
        uint32_t o[32], small[32];
        tc_ld32(tl + kColO + 32 * q, o);
        tc_ld32(tl + kColL + 32 * q, small);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint((__uint_as_float(o[i]) + __uint_as_float(small[i])) * u0 * u1);
        if (row)
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            *reinterpret_cast<uint4*>(part + 4 + 32 * q + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------ dequantisation
    regs_dec<kRegsDequant>();
    const int w = warp - kSoftmax / 32, p = w & 3, ch = (w >> 2) & 1, kv = w >> 3;  // page of the stage, 64-channel group
    int ring = 0;  // page buffer of the tile, and the parity of its use
    uint32_t use = 0;
    for (int s = 0; s < stages; ++s) {
      const int tile = spt == 1 ? s : s >> 1, sub = spt == 1 ? 0 : s & 1;
      if (sub == 0) {
        if (s > 0 && ++ring == A.ring) {
          ring = 0;
          use ^= 1;
        }
        if (!wait(B_META + (tile & (kMetaSlots - 1)), (tile / kMetaSlots) & 1) || !wait(B_RF + ring, use)) break;
      }
      const float* meta = reinterpret_cast<const float*>(sm + kOffMeta + (tile & (kMetaSlots - 1)) * kMeta);
      const int pg = 4 * sub + p;  // page of the tile
      const unsigned char* page = sm + kOffRaw + ring * A.tile_bytes + pg * A.page_bytes;
      const int slot = s & 1;
      if (s >= 2 && !wait((kv ? B_VE : B_KE) + slot, ((s >> 1) & 1) ^ 1)) break;
      if (kv == 0) {
        unsigned char* kpl = sm + kOffK + slot * 2 * kPlane;
        const float *ka = meta + 256 + 16 * pg, *kb = ka + 128;
        switch (A.k_bits) {
          case 2: dequant_k<2>(page, ka, kb, meta, kpl, ch, 16 * p, lane); break;
          case 3: dequant_k<3>(page, ka, kb, meta, kpl, ch, 16 * p, lane); break;
          case 4: dequant_k<4>(page, ka, kb, meta, kpl, ch, 16 * p, lane); break;
          case 5: dequant_k<5>(page, ka, kb, meta, kpl, ch, 16 * p, lane); break;
          case 6: dequant_k<6>(page, ka, kb, meta, kpl, ch, 16 * p, lane); break;
          default: dequant_k<8>(page, ka, kb, meta, kpl, ch, 16 * p, lane); break;
        }
      } else {
        unsigned char* vpl = sm + kOffV + slot * 2 * kPlane;
        const float *va = meta + 512 + 16 * pg, *vb = va + 128;
        const unsigned char* vpage = page + A.k_part;
        switch (A.v_bits) {
          case 2: dequant_v<2>(vpage, va, vb, meta + 128, vpl, ch, p, lane); break;
          case 3: dequant_v<3>(vpage, va, vb, meta + 128, vpl, ch, p, lane); break;
          case 4: dequant_v<4>(vpage, va, vb, meta + 128, vpl, ch, p, lane); break;
          case 5: dequant_v<5>(vpage, va, vb, meta + 128, vpl, ch, p, lane); break;
          case 6: dequant_v<6>(vpage, va, vb, meta + 128, vpl, ch, p, lane); break;
          default: dequant_v<8>(vpage, va, vb, meta + 128, vpl, ch, p, lane); break;
        }
      }
      fence_proxy_async_smem();  // generic writes -> tensor-core reads
      __syncwarp();
      if (lane == 0) {
        arrive(bar0 + 8 * ((kv ? B_VF : B_KF) + slot));
        if (sub == spt - 1) arrive(bar0 + 8 * (B_RE + ring));
      }
    }
  } else if (warp == kMmaWarp) {
    // ----------------------------------------------------------- MMA issue
    regs_dec<kRegsOther>();
    // descriptors of the first plane of K and of V; offsets are added in
    // units of 16 bytes (shared addresses stay below the field's range)
    const uint64_t kd = tc_desc_sw128(smem_addr(sm + kOffK), 16, 1024), vd = tc_desc_sw128(smem_addr(sm + kOffV), 16, 1024);
    auto qk = [&](int s) -> bool {
      if (!wait(B_KF + (s & 1), (s >> 1) & 1)) return false;
      tc_fence_after();
      const uint64_t b0 = kd + (s & 1) * (2 * kPlane / 16);
      const uint32_t d = tmem + kColS + 64 * (s & 1);
      if (elect_one()) {
        // the small products first: the accumulator is truncated at every
        // step, and while it is small that costs nothing
#pragma unroll
        for (int part = 0; part < 3; ++part)
#pragma unroll
          for (int ks = 0; ks < kD / 16; ++ks)
            mma_ts(d, tmem + kColQ + (part == 0 ? 64 : 0) + 8 * ks,
                   b0 + ((ks / 4) * (kStage * 128) + 32 * (ks % 4) + (part == 1 ? kPlane : 0)) / 16, kIdQK,
                   part > 0 || ks > 0);
        tc_commit(bars + B_SF + (s & 1));
        tc_commit(bars + B_KE + (s & 1));
      }
      __syncwarp();
      return true;
    };
    bool ok = qk(0);
    if (ok && stages > 1) ok = qk(1);
    for (int s = 0; ok && s < stages; ++s) {
      if (!wait(B_VF + (s & 1), (s >> 1) & 1) || !wait(B_PF + (s & 1), (s >> 1) & 1)) break;
      tc_fence_after();
      const uint64_t b0 = vd + (s & 1) * (2 * kPlane / 16);
      const uint32_t a = tmem + kColS + 64 * (s & 1);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kStage / 16; ++ks) {
          const uint64_t hi = b0 + 2 * ks, lo = hi + kPlane / 16;
          mma_ts(tmem + kColO, a + 8 * ks, hi, kIdPV, s > 0 || ks > 0);
          mma_ts(tmem + kColL, a + 32 + 8 * ks, hi, kIdPV, s > 0 || ks > 0);
          mma_ts(tmem + kColL, a + 8 * ks, lo, kIdPV, true);
        }
        tc_commit(bars + B_OF + (s & 1));
        tc_commit(bars + B_VE + (s & 1));
      }
      __syncwarp();
      if (s + 2 < stages) ok = qk(s + 2);
    }
    if (elect_one()) tc_commit(bars + B_FIN);
    __syncwarp();
    mbar_wait_bounded(bars + B_FIN, 0, kMmaWait);  // every MMA issued has completed
  } else {
    // ------------------------------------------- page copies and scales
    regs_dec<kRegsOther>();
    const int kv = warp - kMmaWarp - 1;  // 0: copies and K's scales, 1: V's scales
    const int ring = A.ring;
    auto issue = [&](int tile) {
      const int slot = tile % ring;
      const int32_t* pt = A.table + static_cast<int64_t>(t0 + tile) * ppt;
      if (lane == 0) mbar_arrive_expect_tx(bars + B_RF + slot, A.tile_bytes + A.withhold);
      __syncwarp();
      if (lane < ppt) {
        int phys = pt[lane];
        if (phys < 0 || phys >= A.num_pages) {
          set_error(A.err, KVARN_DEVERR_PAGE_RANGE);
          phys = 0;
        }
        bulk_g2s(sm + kOffRaw + slot * A.tile_bytes + lane * A.page_bytes,
                 A.cache + (static_cast<int64_t>(phys) * A.Hkv + kvh) * A.page_bytes, A.page_bytes, bars + B_RF + slot);
      }
    };
    int issued = 0;
    if (kv == 0)
      for (; issued < min(n, ring); ++issued) issue(issued);
    const int bits = kv ? A.v_bits : A.k_bits;
    const int base = (kv ? A.k_part : 0) + 2 * kD * bits;  // the part's scales within a page
    const float kinv = bits == 2 || bits == 3 ? 2.f : 8.f;  // 1 / code_kappa
    const float ctr = bits == 3 || bits == 5 || bits == 8 ? static_cast<float>(1 << (bits - 1)) : 0.f;
    const float top = static_cast<float>((1 << bits) - 1);
    const int cshift = spt == 1 ? 5 : 4, cmask = (1 << cshift) - 1;  // columns per page: 32 or 16
    int ev = kLeastExp;
    for (int tile = 0; kv < 2 && tile < n; ++tile) {
      if (!wait(B_RF + tile % ring, (tile / ring) & 1)) break;
      const unsigned char* raw = sm + kOffRaw + (tile % ring) * A.tile_bytes + base;
      float* meta = reinterpret_cast<float*>(sm + kOffMeta + (tile & (kMetaSlots - 1)) * kMeta);
      float av[4], bv[4], cv[4];
      auto load = [&](auto sb) {  // this lane's row scales (tokens lane + 32 j) and column scales
        using T = decltype(sb);
        constexpr int SB = sizeof(T);
        auto get = [&](int at) -> float {
          if constexpr (SB == 4) return *reinterpret_cast<const float*>(raw + at);
          else return __half2float(*reinterpret_cast<const __half*>(raw + at));
        };
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = lane + 32 * j;
          const int at = (i / kPageTokens) * A.page_bytes + (i % kPageTokens) * SB;
          av[j] = i < A.N ? get(at) : 0.f;
          bv[j] = i < A.N ? get(at + SB * kPageTokens) : 0.f;
          cv[j] = get((i >> cshift) * A.page_bytes + 2 * SB * kPageTokens + (i & cmask) * SB);
        }
      };
      if (A.scale_bytes == 4) load(0.f);
      else load(__half());
      float row_max = 0.f, col_max = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        meta[256 + 256 * kv + lane + 32 * j] = av[j] * kinv;
        meta[256 + 256 * kv + 128 + lane + 32 * j] = fmaf(av[j], ctr, bv[j]);
        row_max = fmaxf(row_max, fmaxf(fabsf(bv[j]), fabsf(fmaf(av[j], top, bv[j]))));
        col_max = fmaxf(col_max, fabsf(cv[j]));
      }
      row_max = warp_max_xor(row_max, 1, 32);
      col_max = warp_max_xor(col_max, 1, 32);
      int e = exponent_of(row_max) + exponent_of(col_max) + 1;
      if (!kv) e = max(-100, min(100, e));
      else if (row_max * col_max == 0.f) e = max(kLeastZeros, ev - kZeros);
      else e = ev = max(kLeastExp, min(kMostExp, e));
      const float d0 = pow2i(-(e / 2)), d1 = pow2i(-(e - e / 2));
#pragma unroll
      for (int j = 0; j < 4; ++j) meta[128 * kv + lane + 32 * j] = cv[j] * d0 * d1;
      if (lane == 0) {
        if (kv) {
          meta[6 * 128 + 1] = static_cast<float>(e);
          meta[6 * 128 + 2] = pow2i(-e);
        } else {
          meta[6 * 128] = pow2i(e);
        }
      }
      __syncwarp();
      if (lane == 0) arrive(bar0 + 8 * (B_META + (tile & (kMetaSlots - 1))));
      // the tile before this one is converted: its buffer takes the next copy
      if (kv == 0 && tile >= 1 && issued < n) {
        if (!wait(B_RE + (tile - 1) % ring, ((tile - 1) / ring) & 1)) break;
        fence_proxy_async_smem();
        issue(issued++);
      }
    }
    // copies still in flight land before the CTA exits
    for (int tile = max(0, issued - ring); tile < issued; ++tile)
      if (!mbar_wait_bounded(bars + B_RF + tile % ring, (tile / ring) & 1, kDrainWait)) break;
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tc_dealloc(tmem, 512);
  }
  if (tid == 0 && *abort_flag) set_error(A.err, KVARN_DEVERR_TIMEOUT);
  if (blockIdx.x == gridDim.x - 1 && blockIdx.y == gridDim.y - 1) pdl_wait_primary();
}

}  // namespace

int shared_tc_splits(int units, int tiles, int stages_per_tile, int* tps) {
  // A split of t tiles costs its stages and about four stages more (query
  // rows, pipeline fill, partial); one CTA per SM, so the call takes
  // ceil(units x splits / SMs) such rounds: the split length of least cost.
  const int sms = device_sm_count();
  int64_t best = -1;
  for (int k = 1; k <= tiles && k <= 2 * sms; ++k) {
    const int t = (tiles + k - 1) / k;
    const int splits = (tiles + t - 1) / t;
    const int64_t rounds = (static_cast<int64_t>(units) * splits + sms - 1) / sms;
    const int64_t cost = rounds * (t * stages_per_tile + 4);
    if (best < 0 || cost < best) {
      best = cost;
      *tps = t;
    }
  }
  return (tiles + *tps - 1) / *tps;
}

cudaError_t launch_shared_tc(const SharedTcArgs& args, int units, cudaStream_t st) {
  SharedTcArgs A = args;
  A.ring = std::min(kPages, (kSmemMax - 1024 - kOffRaw) / A.tile_bytes);  // two at least: the largest tile has 35840 bytes
  const int smem = kOffRaw + A.ring * A.tile_bytes + 1024;
  auto kern = A.wait_limit < kPollWaitBelow ? shared_tc_kernel<true> : shared_tc_kernel<false>;
  // the limit is the process's, not the call's: one value for calls of every layout, which other threads may be making
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(A.slots, units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, A);
}

}  // namespace kvarn
