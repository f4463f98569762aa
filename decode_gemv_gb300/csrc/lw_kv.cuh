// Layout and element arithmetic of the 4-bit key/value cache (the tile of
// lw_kv_cache in include/lw.h), shared by its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "lw_dev.cuh"

namespace lw {

// Byte offsets of the six parts of a tile of 16 tokens of one head.
template <int D>
struct KvTile {
  static constexpr int G = D / LW_KV_GROUP;
  static constexpr int GP = (G + 1) & ~1;
  static constexpr int kKeyCodes = 0;
  static constexpr int kKeyScale = kKeyCodes + 8 * D;
  static constexpr int kKeyMin = kKeyScale + 32 * G;
  static constexpr int kValCodes = kKeyMin + 32 * GP;
  static constexpr int kValScale = kValCodes + 8 * D;
  static constexpr int kValMin = kValScale + 32 * G;
  static constexpr int kBytes = kValMin + 32 * G;
};
static_assert(KvTile<64>::kBytes % 16 == 0 && KvTile<96>::kBytes % 16 == 0 &&
                  KvTile<128>::kBytes % 16 == 0,
              "tiles are copied in units of 16 bytes");

namespace dev {

template <class T>
__device__ __forceinline__ float kv_float(T x);
template <>
__device__ __forceinline__ float kv_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float kv_float<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float kv_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }

template <class T>
__device__ __forceinline__ T kv_round(float x);
template <>
__device__ __forceinline__ float kv_round<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half kv_round<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 kv_round<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 8 consecutive values, by 16-byte accesses where VEC (the address is then
// 16-byte aligned)
template <class T, bool VEC>
__device__ __forceinline__ void kv_load8(const T* p, float (&x)[8]) {
  if constexpr (VEC) {
    constexpr int kN = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / kN; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(p + kN * i);
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int j = 0; j < kN; ++j) x[kN * i + j] = kv_float<T>(e[j]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = kv_float<T>(p[i]);
  }
}
template <class T, bool VEC>
__device__ __forceinline__ void kv_store8(T* p, const float (&x)[8]) {
  if constexpr (VEC) {
    constexpr int kN = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < 8 / kN; ++i) {
      uint4 u;
      T* e = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int j = 0; j < kN; ++j) e[j] = kv_round<T>(x[kN * i + j]);
      *reinterpret_cast<uint4*>(p + kN * i) = u;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = kv_round<T>(x[i]);
  }
}

// ---- pairs of fp32 and fp16 --------------------------------------------------
// two fp32 operations at once
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)),
        "l"(*reinterpret_cast<unsigned long long*>(&c)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<unsigned long long*>(&a)), "l"(*reinterpret_cast<unsigned long long*>(&b)));
  return *reinterpret_cast<float2*>(&d);
}
__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ float2 h2f(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ uint32_t max_h2(uint32_t x, uint32_t y) {
  return h2bits(__hmax2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y)));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t x, uint32_t y) {
  return h2bits(__hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y)));
}
// x[i] * m + b in fp16 pairs
__device__ __forceinline__ uint32_t fma_h2(uint32_t x, uint32_t m, uint32_t b) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(m), "r"(b));
  return y;
}
// the codes of nibbles 0, 4 and 1, 5 as fp16 integers: 1024 + c less 1024,
// (1024 + 16 c) / 16 less 64
__device__ __forceinline__ uint32_t whole_even(uint32_t w) {
  const uint32_t x = (w & 0x000F000Fu) | 0x64006400u, b = 0xE400E400u;
  return h2bits(__hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&b)));
}
__device__ __forceinline__ uint32_t whole_odd(uint32_t w) {
  return fma_h2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
}

// Scale and minimum of a group of 32 values, 8 of them in each of 4
// neighbouring lanes, and this lane's codes (nibble i = value i).  Every step
// is the definition's, in fp32 and rounded to nearest even (no contraction:
// the written cache is the same whatever compiled this); what the definition
// clamps is clamped where a group of the warp needs it, which is rare.
__device__ __forceinline__ uint32_t kv_quantise8(float (&x)[8], __half& scale, __half& low) {
  float lo = x[0], hi = x[0];
  uint32_t top = 0;   // the largest magnitude: in order as an integer, infinities and NaN last
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo = fminf(lo, x[i]);
    hi = fmaxf(hi, x[i]);
    top = max(top, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  }
  if (__any_sync(0xFFFFFFFFu, top > __float_as_uint(LW_KV_LIMIT))) {
    lo = LW_KV_LIMIT;
    hi = -LW_KV_LIMIT;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = fminf(fmaxf(x[i], -LW_KV_LIMIT), LW_KV_LIMIT);
      lo = fminf(lo, x[i]);
      hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  const bool bad = top >= 0x7F800000u;
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  scale = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), (float)(1.0 / 15.0)));
  low = __float2half_rn(lo);
  const float s = __half2float(scale), m = __half2float(low);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  const float2 nm = make_float2(-m, -m), iv = make_float2(inv, inv);
  float2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = mul2(add2(make_float2(x[2 * i], x[2 * i + 1]), nm), iv);
  // (x - m) * inv never falls as x rises: the codes stay within 0..15 if the
  // lowest's and the highest's do
  const bool out = !(__fmul_rn(__fsub_rn(lo, m), inv) >= -0.5f && __fmul_rn(__fsub_rn(hi, m), inv) < 15.5f);
  if (__any_sync(0xFFFFFFFFu, out)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i].x = fminf(fmaxf(y[i].x, 0.f), 15.f);   // (0 and 15 are whole: rounding after is the same)
      y[i].y = fminf(fmaxf(y[i].y, 0.f), 15.f);
    }
  }
  // rounded by an addition (2^23 + 2^22), then four digits of 4 bits in one exact fp32 number
  const float2 up = make_float2(12582912.f, 12582912.f), dn = make_float2(-12582912.f, -12582912.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = add2(add2(y[i], up), dn);
  const float2 c16 = make_float2(256.f, 256.f);
  const float2 a = fma2(y[1], c16, y[0]), b = fma2(y[3], c16, y[2]);   // digits 0, 2 and 1, 3
  const uint32_t w0 = __float_as_uint(fmaf(a.y, 16.f, a.x) + 8388608.f);
  const uint32_t w1 = __float_as_uint(fmaf(b.y, 16.f, b.x) + 8388608.f);
  uint32_t w = __byte_perm(w0, w1, 0x5410);
  if (bad) {
    scale = low = __ushort_as_half((unsigned short)0x7FFFu);
    w = 0;
  }
  return w;
}

}  // namespace dev
}  // namespace lw
