// Choosing the largest of many numbers, the lower place first among equals:
// what eviction and sparse attention share.
//
// A number's bits are turned so that whole numbers order as the numbers do
// (every NaN above them, -0 as 0).  The limit -- the key of the last number that
// is chosen -- is found digit by digit from the top: a histogram of the digit
// among the keys that agree with the limit so far, and a scan of it from above.
// Chosen are the keys above the limit and the first so many that equal it.
// Every count is a whole number: the answer depends on no order.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace lw {
namespace dev {

__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);   // -0 + 0 = 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive sum over the threads of a CTA (s: a place a warp), and the total.
template <int NT>
__device__ __forceinline__ uint32_t scan_cta(uint32_t v, uint32_t* s, uint32_t& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  uint32_t inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    before += w < warp ? s[w] : 0;
    total += s[w];
  }
  return before + inc - v;
}

// Clusters: the barrier of all threads (an acquire and a release), a CTA's rank, how many there are, and words of
// another CTA's shared memory.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ float cluster_load(const float* mine, uint32_t rank) {
  float v;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint4 cluster_load4(const void* mine, uint32_t rank) {
  uint4 v;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at)
               : "memory");
  return v;
}

// The digit (of 256) in which the `need`-th largest key lies, by its histogram; need becomes what is left of it
// within that digit.  Whole CTA of at least 256 threads.
template <int NT>
__device__ __forceinline__ uint32_t pick_digit(const uint32_t* hist, uint32_t& need, uint32_t* s, uint32_t* s_pick) {
  uint32_t total;
  const int d = 255 - (int)threadIdx.x;
  const uint32_t mine = threadIdx.x < 256 ? hist[d] : 0;
  const uint32_t above = scan_cta<NT>(mine, s, total);
  if (threadIdx.x < 256 && above < need && above + mine >= need) {
    s_pick[0] = (uint32_t)d;
    s_pick[1] = need - above;
  }
  __syncthreads();
  const uint32_t digit = s_pick[0];
  need = s_pick[1];
  return digit;
}

}  // namespace dev
}  // namespace lw
