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

// Scale and minimum of a group of 32 values, 8 of them in each of 4
// neighbouring lanes, and this lane's codes (nibble i = value i).  Every step
// is the definition's, in fp32 and rounded to nearest even (no contraction:
// the written cache is the same whatever compiled this).
__device__ __forceinline__ uint32_t kv_quantise8(const float (&x)[8], __half& scale, __half& low) {
  bool bad = false;
  float lo = LW_KV_LIMIT, hi = -LW_KV_LIMIT;
  float c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    bad |= !(fabsf(x[i]) <= 3.402823466e38f);
    c[i] = fminf(fmaxf(x[i], -LW_KV_LIMIT), LW_KV_LIMIT);
    lo = fminf(lo, c[i]);
    hi = fmaxf(hi, c[i]);
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    bad |= __shfl_xor_sync(0xFFFFFFFFu, (int)bad, o) != 0;
  }
  scale = __float2half_rn(__fmul_rn(__fsub_rn(hi, lo), (float)(1.0 / 15.0)));
  low = __float2half_rn(lo);
  const float s = __half2float(scale), m = __half2float(low);
  const float inv = s > 0.f ? __frcp_rn(s) : 0.f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float r = fminf(fmaxf(rintf(__fmul_rn(__fsub_rn(c[i], m), inv)), 0.f), 15.f);
    w |= (uint32_t)(int)r << (4 * i);
  }
  if (bad) {
    scale = low = __ushort_as_half((unsigned short)0x7FFFu);
    w = 0;
  }
  return w;
}

}  // namespace dev
}  // namespace lw
