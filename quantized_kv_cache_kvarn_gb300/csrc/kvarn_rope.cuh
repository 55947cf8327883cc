// Angles of rotary positions as 64-bit fractions of a turn (kvarn_rope.cu says
// why), and 16-byte vectors of the three element types as fp32 values.
#pragma once

#include "kvarn_common.cuh"

namespace kvarn {

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

}  // namespace kvarn
