// What the cache attention kernels share: their arguments, the search for a
// CTA's first unit, and the join of an item's partial results.
#pragma once

#include "lw_kv.cuh"
#include "lw_kvplan.h"

namespace lw {

struct AttnArgs {
  lw_kv_attn p;
  const uint8_t* pages;
  int64_t n_pages, page_bytes;
  uint32_t* counters;   // [grid], zero between calls
  float* partials;      // [grid][2] partial results of RT rows
  int32_t page_tokens, heads, group;
  int32_t vec;          // q and out rows are 16-byte aligned
  int32_t parts;        // 0, or the heads of the cache that is seen head by head: see kv_seq
  int32_t* status;
};

namespace dev {

// T and n of sequence b; T = 0 if its query range is not one (LOUD: reported).
// Ordinary loads, here and of the page table: what the work in front writes may
// not be read by way of the read-only path, which the wait for that work does not
// order.
// With `parts` every token and key/value head is a sequence of its own, of one token
// (b = token * parts + head) on kv_len[b] keys, or of none where that is negative.  PARTS: the kernel that takes
// such calls (the other's registers are short: the question alone cost it 4 %).
template <bool LOUD, bool PARTS>
__device__ __forceinline__ void kv_seq(const AttnArgs& a, int b, int& q0, int& T, int& n) {
  if (PARTS && a.parts) {
    q0 = b;
    n = a.p.kv_len[b];
    T = n >= 0;
    n = max(n, 0);
    return;
  }
  q0 = a.p.q_start[b];
  const int q1 = a.p.q_start[b + 1];
  n = a.p.kv_len[b];
  const int most = a.p.table_width * a.page_tokens;
  const bool bad = q0 < 0 || q1 < q0 || q1 > a.p.q_tokens;
  if (LOUD && (bad || n < 0 || n > most)) report(a.status, LW_DEV_BAD_SEQ);
  T = bad ? 0 : q1 - q0;
  n = n < 0 ? 0 : (n > most ? most : n);
}

// Where the rows of packed token i begin
__device__ __forceinline__ int64_t kv_token_at(const AttnArgs& a, int i, int64_t token_stride, int64_t head_stride) {
  if (a.parts <= 1) return i * token_stride;
  const int t = i / a.parts;
  return t * token_stride + (int64_t)(i - t * a.parts) * a.group * head_stride;
}

// Sum over the CTA of one value per thread, and the exclusive sum before
// each thread (s: NT / 32 + 1 places).
template <int NT>
__device__ __forceinline__ long long cta_scan(long long v, long long* s, long long& total) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  long long inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += u;
  }
  __syncthreads();
  if (lane == 31) s[warp] = inc;
  __syncthreads();
  long long before = 0;
  total = 0;
  for (int w = 0; w < NT / 32; ++w) {
    before += w < warp ? s[w] : 0;
    total += s[w];
  }
  return before + inc - v;
}

template <int RT, int PER, int EXTRA>
__device__ __forceinline__ KvShape kv_shape(const AttnArgs& a) {
  return KvShape{a.group, RT, PER, EXTRA, a.p.causal, a.p.window};
}

// On to the next item that has units of this CTA's; false at the end of the
// range.
template <int RT, int PER, int EXTRA, bool PARTS = false>
__device__ __forceinline__ bool kv_advance(const AttnArgs& a, KvWalk& w, int& q0) {
  const KvShape c = kv_shape<RT, PER, EXTRA>(a);
  do {
    const bool same = kv_next(w, a.heads);
    if (w.x >= w.xe) return false;
    if (!same) {
      w.base = w.x;
      w.h = w.rt = 0;
      do {
        ++w.b;
        kv_seq<false, PARTS>(a, w.b, q0, w.T, w.n);
      } while (w.T == 0);
    }
    kv_enter(c, w);
  } while (w.k0 >= w.k1);
  return true;
}

// Row tiles of a sequence up to which one thread counts its weight, and every
// thread walks them; the tiles of longer ones are shared by a warp's lanes (5
// prompts of 2048 tokens, 128 tiles a head: a CTA's start was 90000 to 160000
// cycles of 500000).
constexpr int kKvAlone = 4;

// kv_head_weight of each lane's sequence (0 if T is 0).  Whole warp.
__device__ __forceinline__ long long kv_weight_warp(const KvShape& c, int T, int n) {
  const int lane = threadIdx.x % 32, nrt = T ? kv_row_tiles(T, c.group, c.RT) : 0;
  long long u = nrt && nrt <= kKvAlone ? kv_head_weight(c, T, n) : 0;
  for (uint32_t rest = __ballot_sync(0xFFFFFFFFu, nrt > kKvAlone); rest; rest &= rest - 1) {
    const int l = __ffs(rest) - 1;
    const int t = __shfl_sync(0xFFFFFFFFu, T, l), k = __shfl_sync(0xFFFFFFFFu, n, l);
    const int tiles = __shfl_sync(0xFFFFFFFFu, nrt, l);
    long long s = 0;
    for (int rt = lane; rt < tiles; rt += 32) s += kv_item_weight(c, t, k, rt);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == l) u = s;
  }
  return u;
}

// kv_seek, per_head being the weight of a head.  Whole warp, the same in all lanes.
__device__ __forceinline__ void kv_seek_warp(const KvShape& c, KvWalk& w, long long per_head) {
  w.nrt = kv_row_tiles(w.T, c.group, c.RT);
  if (w.nrt <= kKvAlone) {
    kv_seek(c, w);
    return;
  }
  w.h = (int)((w.x - w.base) / per_head);
  long long begin = w.base + per_head * w.h;
  const int lane = threadIdx.x % 32;
  for (int r0 = 0; r0 < w.nrt; r0 += 32) {
    const long long mine = r0 + lane < w.nrt ? kv_item_weight(c, w.T, w.n, r0 + lane) : 0;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += u;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, w.x < begin + inc);
    if (past) {
      const int l = __ffs(past) - 1;
      w.rt = r0 + l;
      begin += __shfl_sync(0xFFFFFFFFu, inc - mine, l);
      break;
    }
    begin += __shfl_sync(0xFFFFFFFFu, inc, 31);
  }
  kv_item(c, w, begin);
}

// The CTA's range, and its first item.  Whole CTA of NT threads; false if the
// CTA has no units.
template <int NT, int RT, int PER, int EXTRA, bool PARTS = false>
__device__ bool kv_range(const AttnArgs& a, KvWalk& w, int& G, long long& U, int& q0) {
  __shared__ long long s_scan[NT / 32 + 1], s_base, s_head;
  __shared__ int s_b, s_q0, s_T, s_n;
  const KvShape c = kv_shape<RT, PER, EXTRA>(a);
  const int tid = threadIdx.x, batch = a.p.batch;
  long long sum = 0, head = 0;
  int T = 0, n = 0;
  for (int cb = 0; cb < batch; cb += NT) {
    const int b = cb + tid;
    T = n = 0;
    if (b < batch) {
      if (blockIdx.x == 0) kv_seq<true, PARTS>(a, b, q0, T, n);
      else kv_seq<false, PARTS>(a, b, q0, T, n);
    }
    head = kv_weight_warp(c, T, n);
    sum += a.heads * head;
  }
  long long before = cta_scan<NT>(sum, s_scan, U);
  if (U == 0) return false;
  G = (long long)gridDim.x < U ? (int)gridDim.x : (int)U;
  if ((int)blockIdx.x >= G) return false;
  w.x = kv_first(U, blockIdx.x, G);
  w.xe = kv_first(U, blockIdx.x + 1, G);
  const auto take = [&](int b) {   // the sequence at w.x is this thread's
    if (w.x < before || w.x >= before + a.heads * head) return;
    s_b = b;
    s_base = before;
    s_head = head;
    s_q0 = q0;
    s_T = T;
    s_n = n;
  };
  if (batch <= NT) {   // the sums were one sequence each
    take(tid);
  } else {
    long long carry = 0;
    for (int cb = 0; cb < batch && carry <= w.x; cb += NT) {
      const int b = cb + tid;
      long long total;
      T = n = 0;
      if (b < batch) kv_seq<false, PARTS>(a, b, q0, T, n);
      head = kv_weight_warp(c, T, n);
      before = carry + cta_scan<NT>(a.heads * head, s_scan, total);
      take(b);
      carry += total;
    }
  }
  __syncthreads();
  w.b = s_b;
  w.base = s_base;
  q0 = s_q0;
  w.T = s_T;
  w.n = s_n;
  kv_seek_warp(c, w, s_head);
  return w.k0 < w.k1 || kv_advance<RT, PER, EXTRA, PARTS>(a, w, q0);
}

// 4 or 8 consecutive elements of an output row, rounded to its type
template <int N>
__device__ __forceinline__ void store_n(const AttnArgs& a, int64_t at, const float (&f)[N]) {
  if (a.p.dtype == LW_F32) {
    float* o = static_cast<float*>(a.p.out) + at;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      if (a.vec) *reinterpret_cast<float4*>(o + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
      else
        for (int j = 0; j < 4; ++j) o[i + j] = f[i + j];
    }
  } else {
    uint32_t h[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
      h[i] = a.p.dtype == LW_F16
                 ? __half_as_ushort(__float2half_rn(f[2 * i])) | (uint32_t)__half_as_ushort(__float2half_rn(f[2 * i + 1])) << 16
                 : __bfloat16_as_ushort(__float2bfloat16_rn(f[2 * i])) |
                       (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f[2 * i + 1])) << 16;
    uint16_t* o = static_cast<uint16_t*>(a.p.out) + at;
    if (a.vec) {
      if constexpr (N == 8) *reinterpret_cast<uint4*>(o) = make_uint4(h[0], h[1], h[2], h[3]);
      else *reinterpret_cast<uint2*>(o) = make_uint2(h[0], h[1]);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) o[i] = (uint16_t)(h[i / 2] >> (16 * (i % 2)));
    }
  }
}
__device__ __forceinline__ void store4(const AttnArgs& a, int64_t at, const float (&f)[4]) { store_n<4>(a, at, f); }
__device__ __forceinline__ void store8(const AttnArgs& a, int64_t at, const float (&f)[8]) { store_n<8>(a, at, f); }

}  // namespace dev
}  // namespace lw
