// Layout and element arithmetic of the 4-bit key/value cache (the tile of
// lw_kv_cache in include/lw.h), shared by its kernels.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include <type_traits>

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

// Smallest and largest of three, a NaN if there is one
__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// 8 consecutive values and their smallest and largest (NaN if one is; 16-bit
// types compared in pairs)
template <class T, bool VEC>
__device__ __forceinline__ void kv_load8_range(const T* p, float (&x)[8], float& lo, float& hi) {
  if constexpr (VEC && sizeof(T) == 2) {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const T2* w = reinterpret_cast<const T2*>(&u);
    const T2 a = __hmin2_nan(__hmin2_nan(w[0], w[1]), __hmin2_nan(w[2], w[3]));
    const T2 b = __hmax2_nan(__hmax2_nan(w[0], w[1]), __hmax2_nan(w[2], w[3]));
    lo = kv_float<T>(__hmin_nan(a.x, a.y));
    hi = kv_float<T>(__hmax_nan(b.x, b.y));
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = kv_float<T>(e[j]);
  } else {
    kv_load8<T, VEC>(p, x);
    lo = min3(min3(min3(x[0], x[1], x[2]), x[3], x[4]), min3(x[5], x[6], x[7]), x[0]);
    hi = max3(max3(max3(x[0], x[1], x[2]), x[3], x[4]), max3(x[5], x[6], x[7]), x[0]);
  }
}

// Scale and minimum of a group of 32 values, 8 of them in each of 4
// neighbouring lanes (lo, hi: the lane's smallest and largest), and this lane's
// codes (nibble i = value i).  Every step is the definition's, in fp32 and
// rounded to nearest even (no contraction: the written cache is the same
// whatever compiled this); what the definition clamps is clamped where a group
// of the warp needs it, which is rare.
__device__ __forceinline__ uint32_t kv_quantise8(float (&x)[8], float lo, float hi, __half& scale, __half& low) {
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    const float a = __shfl_xor_sync(0xFFFFFFFFu, lo, o), b = __shfl_xor_sync(0xFFFFFFFFu, hi, o);
    lo = min3(lo, a, a);
    hi = max3(hi, b, b);
  }
  bool bad = false;
  if (__any_sync(0xFFFFFFFFu, !(lo >= -LW_KV_LIMIT && hi <= LW_KV_LIMIT))) {
    bad = !(lo >= -3.402823466e38f && hi <= 3.402823466e38f);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fminf(fmaxf(x[i], -LW_KV_LIMIT), LW_KV_LIMIT);
    lo = fminf(fmaxf(lo, -LW_KV_LIMIT), LW_KV_LIMIT);
    hi = fminf(fmaxf(hi, -LW_KV_LIMIT), LW_KV_LIMIT);
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
