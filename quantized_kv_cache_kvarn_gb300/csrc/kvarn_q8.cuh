// The 8-bit block codec: page format, code rounding and operand conversions.
//
// A block is the 16 tokens of a page of one KV head. With A its largest
// magnitude (at least 2^-100) and M the largest code (448 for e4m3, 127 for
// int8), scale = fl(A fl(1 / M)), inverse = fl(fl(1 / A) M) and code =
// rne(fl(x inverse)), every fl an IEEE fp32 operation, so that the codes are
// the same wherever they are formed; the value is code * scale. A block that holds an infinity
// or a NaN has scale NaN and codes 0, and reads as NaN throughout.
#pragma once

#include <cuda_fp8.h>

#include "kvarn_common.cuh"

namespace kvarn {

constexpr int kQ8E4M3 = 0, kQ8Int8 = 1;

// Page of one KV head: K codes, V codes (placements in kvarn.h), the two
// scales, padding to a multiple of 32 bytes (a DRAM sector).
__host__ __device__ constexpr int q8_page(int D) { return 32 * D + 32; }
__host__ __device__ constexpr int q8_scales(int D) { return 32 * D; }

template <int CODE> __host__ __device__ constexpr float q8_top() { return CODE == kQ8Int8 ? 127.f : 448.f; }
constexpr float kQ8Tiny = 0x1p-100f;

// Four values to four code bytes; int8 codes are stored plus 128.
template <int CODE>
__device__ __forceinline__ uint32_t q8_code4(float a, float b, float c, float d, float inv) {
  a = __fmul_rn(a, inv);
  b = __fmul_rn(b, inv);
  c = __fmul_rn(c, inv);
  d = __fmul_rn(d, inv);
  if constexpr (CODE == kQ8E4M3) {
    uint32_t r;
    asm("{ .reg .b16 l, h; cvt.rn.satfinite.e4m3x2.f32 l, %2, %1; cvt.rn.satfinite.e4m3x2.f32 h, %4, %3; mov.b32 %0, {l, h}; }"
        : "=r"(r)
        : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
  } else {
    // adding 1.5 2^23 + 128 rounds to the nearest integer, ties to even, and
    // leaves code + 128 in the low byte
    constexpr float kRound = 12583040.f;
    const uint32_t x = __float_as_uint(__fadd_rn(a, kRound)), y = __float_as_uint(__fadd_rn(b, kRound));
    const uint32_t z = __float_as_uint(__fadd_rn(c, kRound)), w = __float_as_uint(__fadd_rn(d, kRound));
    return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
  }
}

// Code bytes (0, 1) and (2, 3) of a word as exact fp16 pairs.
template <int CODE>
__device__ __forceinline__ void q8_pairs(uint32_t x, uint32_t& p, uint32_t& q) {
  if constexpr (CODE == kQ8E4M3) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(p), "=r"(q)
        : "r"(x));
  } else {
    // byte u behind 0x64 is fp16 1024 + u; 1024 + 128 less leaves the code
    const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));
    p = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(x, 0x64646464u, 0x4140)), off));
    q = h2_as_u32(__hsub2(u32_as_h2(__byte_perm(x, 0x64646464u, 0x4342)), off));
  }
}

}  // namespace kvarn
