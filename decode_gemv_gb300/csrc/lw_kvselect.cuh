// Choosing the largest of many numbers, the lower place first among equals:
// what eviction and sparse attention share.
//
// A number's bits are turned so that whole numbers order as the numbers do
// (every NaN above them, -0 as 0).  A cluster shares the numbers in contiguous
// stretches, a CTA keeps the order keys of its own in shared memory.  The limit
// -- the key of the last number that is chosen -- is found from the top, digit by
// digit: a digit's histogram, among the keys that agree with the limit so far, lies
// in each CTA's shared memory, and every CTA adds the cluster's up, so that all
// find the same digit with one barrier of the cluster a digit.  From the same histograms a CTA knows how many keys above the limit, and
// at it, lie in the stretches before its own: the places follow without another
// exchange.  Chosen are the keys above the limit and the first so many that equal
// it.  Every count is a whole number: the answer depends on no order.
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

#include "lw_kvroom.h"

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

// Clusters: the barrier of all threads (an acquire and a release), a CTA's rank, how many there are, and a word of
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
template <int N>
__device__ __forceinline__ void cluster_load(const uint32_t* mine, uint32_t rank, uint32_t (&v)[N]) {
  static_assert(N == 1 || N == 4, "words");
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(at)
               : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(mine))), "r"(rank));
  if constexpr (N == 1)
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v[0]) : "r"(at) : "memory");
  else
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(at)
                 : "memory");
}
__device__ __forceinline__ float cluster_load(const float* mine, uint32_t rank) {
  uint32_t v[1];
  cluster_load(reinterpret_cast<const uint32_t*>(mine), rank, v);
  return __uint_as_float(v[0]);
}

// Digits of 8 or of 11 bits (the last of 10): four passes, or three over eight times the bins.  64 heads' 65536
// keys, clusters of 4: 46 us and 32; 1200 pages of 64 heads, clusters of 8: 25 us and 78 (every CTA reads the
// others' bins).
template <int BITS>
struct SelectShared {
  static constexpr int kPasses = BITS == 8 ? 4 : 3, kBins = 1 << BITS;
  uint32_t hist[kPasses * kBins];   // zero before select_places
  uint32_t scan[16], pick[2], more[16], same[16];   // (a place a warp)
};

// The `need` (> 0, at most the cluster's count) largest of the cluster's keys: put(place among the chosen, i) for
// each of this CTA's `count` that is one, key(i) being its i-th.  Whole cluster, of CTAs of NT threads (256 to 512).
template <int NT, int BITS, class Key, class Put>
__device__ __forceinline__ void select_places(SelectShared<BITS>& s, int count, uint32_t need, Key key, Put put) {
  constexpr int kWarps = NT / 32, kBins = 1 << BITS, kMine = kBins > NT ? kBins / NT : 1;   // kMine: bins of a thread
  static_assert(NT >= 256 && kWarps <= 16, "threads");
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  const uint32_t ranks = cluster_size(), rank = cluster_rank();
  uint32_t limit = 0, above = 0, equal = 0;   // above, equal: of the stretches before
#pragma unroll 1
  for (int pass = 0; pass < SelectShared<BITS>::kPasses; ++pass) {
    const int shift = max(32 - BITS * (pass + 1), 0), bits = min(BITS, 32 - BITS * pass), bins = 1 << bits;
    const uint32_t mask = pass ? ~0u << (shift + bits) : 0u;
    uint32_t* mine = s.hist + pass * kBins;
#pragma unroll 4
    for (int i = tid; i < count; i += NT) {
      const uint32_t k = key(i);
      if ((k & mask) == limit) atomicAdd(&mine[k >> shift & (uint32_t)(bins - 1)], 1u);
    }
    if (ranks > 1) cluster_sync();
    else __syncthreads();
    // thread t has the kMine bins below bins - kMine t: in all, and in the stretches before
    const int top = bins - kMine * (tid + 1);
    uint32_t sum[kMine] = {}, before[kMine] = {}, all = 0;
    if (top >= 0) {
      for (uint32_t r = 0; r < ranks; ++r) {
        uint32_t x[kMine];
        cluster_load(mine + top, r, x);
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          sum[i] += x[i];
          all += x[i];
          before[i] += r < rank ? x[i] : 0;
        }
      }
    }
    uint32_t total;
    uint32_t over = scan_cta<NT>(all, s.scan, total);
#pragma unroll
    for (int i = kMine - 1; i >= 0; --i) {
      if (over < need && over + sum[i] >= need) {
        s.pick[0] = (uint32_t)(top + i);
        s.pick[1] = need - over;
      }
      over += sum[i];
    }
    __syncthreads();
    const uint32_t digit = s.pick[0];
    need = s.pick[1];
    limit |= digit << shift;
    if (ranks > 1) {
      uint32_t up = 0, at = 0;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        up += top + i > (int)digit ? before[i] : 0;
        at += top + i == (int)digit ? before[i] : 0;
      }
      (void)scan_cta<NT>(up, s.scan, total);
      above += total;
      if (shift == 0) (void)scan_cta<NT>(at, s.scan, equal);
    }
  }
  if (ranks > 1) cluster_sync();   // (no CTA leaves while another reads its histograms)
  // a warp takes a part of the stretch, counts it, and places it
  const int part = ((count + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int i0 = warp * part, i1 = i0 + part < count ? i0 + part : count;
  uint32_t more = 0, same = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i0 + part; i += 32) {
    const uint32_t k = i < i1 ? key(i) : 0u;
    more += __popc(__ballot_sync(0xFFFFFFFFu, i < i1 && k > limit));
    same += __popc(__ballot_sync(0xFFFFFFFFu, i < i1 && k == limit));
  }
  if (lane == 0) {
    s.more[warp] = more;
    s.same[warp] = same;
  }
  __syncthreads();
  for (int v = 0; v < warp; ++v) {
    above += s.more[v];
    equal += s.same[v];
  }
  const uint32_t lower = (1u << lane) - 1;
#pragma unroll 4
  for (int i = i0 + lane; i < i0 + part; i += 32) {
    const uint32_t k = i < i1 ? key(i) : 0u;
    const bool is_more = i < i1 && k > limit, is_same = i < i1 && k == limit;
    const uint32_t bm = __ballot_sync(0xFFFFFFFFu, is_more), bs = __ballot_sync(0xFFFFFFFFu, is_same);
    const uint32_t am = above + __popc(bm & lower), as = equal + __popc(bs & lower);
    if (is_more || (is_same && as < need)) put((int)(am + (as < need ? as : need)), i);
    above += __popc(bm);
    equal += __popc(bs);
  }
}

// This CTA's stretch of [first, last): where it begins, and how many there are
__device__ __forceinline__ int64_t select_stretch(int first, int last, int& count) {
  const uint32_t ranks = cluster_size(), rank = cluster_rank();
  const int stretch = kv_select_stretch((long long)last - first, (int)ranks);
  const int64_t from = first + (int64_t)rank * stretch;
  count = from < last ? (int)(last - from < stretch ? last - from : stretch) : 0;
  return from;
}

}  // namespace dev
}  // namespace lw
