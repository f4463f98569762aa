// Accumulated attention weight for few rows: each key's softmax weights summed
// over the rows that share its head.
//
// Mathematics.  With a cached key k_d = sc_g (c_d - 8) + mid_g, mid = mn + 8 sc
// (group g of 32), and q' = q / 2^e (2^e by the row's largest element),
//   q.k = 2^e ( sum_g sc_g sum_{d in g} q'_d (c_d - 8)  +  sum_g mid_g sum_{d in g} q'_d ),
// weight_j += 2^((scale q.k_j - lse) log2 e).  The codes are the matrix operands
// (exact in fp16), the rows' q' the other one: fp16 as 16-bit queries are (their
// own 8 or 11 bits, down to 2^-14 of the row's largest), two parts of 11 bits
// each of fp32 ones.  Scales enter in fp32 after the product.
#pragma once

#include "lw_kvfew.cuh"

namespace lw {

struct WeighArgs {
  lw_kv_weights p;
  const uint8_t* pages;
  int64_t n_pages, page_bytes;
  int32_t page_tokens, heads, group, vec;
  int32_t* status;
};

template <int D, class T>
struct WeighFew {
  static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;   // of an operand
  static constexpr int kWarps = 8, kThreads = 32 * kWarps;
  static constexpr int kBlocks = 8;                        // of 8 rows, staged at once
  static constexpr int kFrag = D / 16 * 2 * 32 * 4;        // bytes of a block's operand part
  static constexpr int kRow = kBlocks * kParts * kFrag;    // then the rows: f, lse, hi, lo, group sums
  static constexpr int kRowWords = 4 + D / 32;
  static constexpr int kRange = kRow + kBlocks * 8 * kRowWords * 4;   // keys that all, and any, rows of a block see
  static constexpr int kBars = kRange + kBlocks * 4 * 4;
  static constexpr int kStages = 4;                        // tiles of a warp on their way
  static constexpr int kRing = (kBars + kWarps * kStages * 8 + 127) / 128 * 128;
  static constexpr int kKeys = KvTile<D>::kValCodes;       // the key half of a tile
  static constexpr int kSmem = kRing + kWarps * kStages * kKeys;
  static constexpr int kPerSm = 2;
};

namespace dev {

// Query range and keys of sequence b (lw_kvattn.cuh's rules).
template <bool LOUD>
__device__ __forceinline__ void weigh_seq(const WeighArgs& a, int b, int& q0, int& T, int& n) {
  q0 = a.p.q_start[b];
  const int q1 = a.p.q_start[b + 1];
  n = a.p.kv_len[b];
  const int most = a.p.table_width * a.page_tokens;
  const bool bad = q0 < 0 || q1 < q0 || q1 > a.p.q_tokens;
  if (LOUD && (bad || n < 0 || n > most || n > a.p.w_keys)) report(a.status, LW_DEV_BAD_SEQ);
  T = bad ? 0 : q1 - q0;
  n = n < 0 ? 0 : (n > most ? most : n);
}

// 8 consecutive elements of a query row
template <class T>
__device__ __forceinline__ void weigh_load8(const WeighArgs& a, int64_t at, float (&x)[8]) {
  const T* p = static_cast<const T*>(a.p.q) + at;
  if (a.vec) kv_load8<T, true>(p, x);
  else kv_load8<T, false>(p, x);
}

// Codes less 8 of nibbles (0, 4), (1, 5), (2, 6), (3, 7) as fp16 pairs
__device__ __forceinline__ void centred(uint32_t w, uint32_t (&h)[4]) {
  const uint32_t b = 0xE408E408u;   // -1032
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = ((w >> (8 * i)) & 0x000F000Fu) | 0x64006400u;
    h[2 * i] = h2bits(__hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&b)));
    h[2 * i + 1] = fma_h2(((w >> (8 * i)) & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD480D480u);   // / 16 - 72
  }
}

// A row of a block into shared memory: lane n * 4 + q has elements 32 g + 8 q .. of row n.
template <int D, class T>
__device__ void weigh_row(const WeighArgs& a, uint8_t* smem, int blk, int r, int q0, int Tq, int n, int h, int lane) {
  using W = WeighFew<D, T>;
  constexpr int G = D / 32;
  const int q = lane % 4;
  const bool live = r < Tq * a.group;
  const int t = live ? r / a.group : 0;
  const int head = h * a.group + r - t * a.group;
  float x[G][8], top = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (live)
      weigh_load8<T>(a, (int64_t)(q0 + t) * a.p.q_token_stride + (int64_t)head * a.p.q_head_stride + 32 * g + 8 * q, x[g]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[g][i]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  // the largest element comes to 2^14 .. 2^15
  int e = (int)(__float_as_uint(top) >> 23) - 127;
  e = e < -100 ? -100 : (e > 127 ? 127 : e);
  const float down = __uint_as_float((uint32_t)(127 - e + 14) << 23);
  uint32_t* frag = reinterpret_cast<uint32_t*>(smem) + blk * W::kParts * (W::kFrag / 4);
  float* row = reinterpret_cast<float*>(smem + W::kRow) + (blk * 8 + lane / 4) * W::kRowWords;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[g][i] *= down;
      z += x[g][i];
    }
    z += __shfl_xor_sync(0xFFFFFFFFu, z, 1);
    z += __shfl_xor_sync(0xFFFFFFFFu, z, 2);
    if (q == 0) row[4 + g] = z;
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (W::kParts == 2) split2<2048>(x[g][i], x[g][i + 4], hi[i], lo[i]);
      else hi[i] = h2bits(__floats2half2_rn(x[g][i], x[g][i + 4]));
    }
    *reinterpret_cast<uint4*>(frag + (g * 32 + lane) * 4) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (W::kParts == 2)
      *reinterpret_cast<uint4*>(frag + W::kFrag / 4 + (g * 32 + lane) * 4) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  int lo = 0, hi = 0;
  if (live) kv_token_keys(Tq, n, t, a.p.causal, a.p.window, lo, hi);
  // what all live rows of the block see, and what any of them does
  int all_lo = live ? lo : 0, all_hi = live ? hi : 0x7FFFFFFF, any_lo = live && hi > lo ? lo : 0x7FFFFFFF, any_hi = live && hi > lo ? hi : 0;
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {
    all_lo = max(all_lo, __shfl_xor_sync(0xFFFFFFFFu, all_lo, o));
    all_hi = min(all_hi, __shfl_xor_sync(0xFFFFFFFFu, all_hi, o));
    any_lo = min(any_lo, __shfl_xor_sync(0xFFFFFFFFu, any_lo, o));
    any_hi = max(any_hi, __shfl_xor_sync(0xFFFFFFFFu, any_hi, o));
  }
  if (q == 0) {
    row[0] = a.p.scale * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
    row[1] = live ? a.p.lse[(int64_t)(q0 + t) * a.p.q_heads + head] : INFINITY;   // a row that is not there weighs 0
    row[2] = __int_as_float(lo);
    row[3] = __int_as_float(hi);
  }
  if (lane == 0) {
    int4* range = reinterpret_cast<int4*>(smem + W::kRange) + blk;
    *range = make_int4(all_lo, all_hi, any_lo, any_hi);
  }
}

// A warp's tiles: first, first + step, ... below `end`, their key halves fetched by bulk copies into a ring of its
// own, in order.  The page table is read 32 tiles at a time, lane i holding the i-th one's place.
template <int D, class T>
struct WeighFetch {
  using W = WeighFew<D, T>;
  uint8_t* ring;
  uint64_t* bars;
  const int32_t* table;
  int64_t head;
  int next, end, step, at, in, out;
  uint32_t there, have, parity;
  const uint8_t* src;

  __device__ __forceinline__ void lookup(const WeighArgs& a, int lane) {
    const int64_t tile = next + (int64_t)lane * step;
    const int tpp = a.page_tokens / LW_KV_TILE;
    const bool mine = tile < end;
    const int page = mine ? table[tile / tpp] : -1;
    const bool ok = page >= 0 && page < a.n_pages;
    if (mine && !ok) report(a.status, LW_DEV_BAD_PAGE);
    there = __ballot_sync(0xFFFFFFFFu, ok);
    src = a.pages + (int64_t)page * a.page_bytes + head + (tile % tpp) * KvTile<D>::kBytes;
    at = 0;
  }
  __device__ __forceinline__ void send(const WeighArgs& a, int lane) {
    if (next >= end) return;
    if (at == 32) lookup(a, lane);
    if (there >> at & 1u) {
      if (lane == at) {
        mbar_arrive_expect_tx(&bars[in], W::kKeys);
        bulk_g2s(ring + in * W::kKeys, src, W::kKeys, &bars[in]);
      }
      have |= 1u << in;
    }
    ++at;
    next += step;
    in = in + 1 == W::kStages ? 0 : in + 1;
  }
  __device__ __forceinline__ void begin(const WeighArgs& a, int first, int lane) {
    next = first;
    in = out = 0;
    have = 0;
    at = 32;
#pragma unroll
    for (int i = 0; i < W::kStages; ++i) send(a, lane);
  }
  // The tile at `out` has come (false: the wait ran out)
  __device__ __forceinline__ bool wait() {
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars[out], parity >> out & 1u));
    if (!ok) return false;
    parity ^= 1u << out;
    have &= ~(1u << out);
    return true;
  }
  // On to the next tile
  __device__ __forceinline__ void pass() { out = out + 1 == W::kStages ? 0 : out + 1; }
  // After a wait that ran out: what is still on its way
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < W::kStages; ++i)
      if (have >> i & 1u) mbar_wait(&bars[i], parity >> i & 1u);
  }
};

template <int D, class T>
__global__ void __launch_bounds__(WeighFew<D, T>::kThreads, WeighFew<D, T>::kPerSm) kv_weigh_few_kernel(const WeighArgs a) {
  using W = WeighFew<D, T>;
  using L = KvTile<D>;
  constexpr int G = L::G;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, t = lane / 4, q = lane % 4;
  const int b = blockIdx.z, h = blockIdx.y;
  WeighFetch<D, T> f;
  f.bars = reinterpret_cast<uint64_t*>(smem + W::kBars) + warp * W::kStages;
  if (lane < W::kStages) mbar_init(&f.bars[lane], 1);
  fence_barrier_init();
  __syncwarp();
  pdl_wait();
  int q0, Tq, n;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) weigh_seq<true>(a, b, q0, Tq, n);
  else weigh_seq<false>(a, b, q0, Tq, n);
  const int keys = n < a.p.w_keys ? n : (int)a.p.w_keys;
  const int tiles = (keys + 15) / 16, first = blockIdx.x * W::kWarps + warp;
  if ((int)blockIdx.x * W::kWarps >= tiles) return;
  const int rows = Tq * a.group;
  const float* add = a.p.add_to ? a.p.add_to + b * a.p.add_seq_stride + h * a.p.add_head_stride : nullptr;
  float* out = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride;
  f.ring = smem + W::kRing + warp * W::kStages * W::kKeys;
  f.table = a.p.page_table + (int64_t)b * a.p.table_stride;
  f.head = (int64_t)h * (a.page_tokens / LW_KV_TILE) * L::kBytes;
  f.end = tiles;
  f.step = gridDim.x * W::kWarps;
  f.parity = 0;
  bool ok = true;
  int r0 = 0;
  do {
    if (ok) f.begin(a, first, lane);
    const int blocks = (min(rows - r0, 8 * W::kBlocks) + 7) / 8;
    if (r0) __syncthreads();
    for (int i = warp; i < blocks; i += W::kWarps) weigh_row<D, T>(a, smem, i, r0 + 8 * i + t, q0, Tq, n, h, lane);
    __syncthreads();
    // what the weights are added to, a tile ahead (what an earlier set of rows left is this thread's own)
    const float* from = r0 ? out : add;
    const auto before = [&](int tile) {
      const int j = 16 * tile + t + 8 * q;
      return q < 2 && from && tile < tiles && j < keys ? from[j] : 0.f;
    };
    float had = before(first);
    for (int tile = first; tile < tiles && ok; tile += f.step) {
      const float had_next = tile < tiles - f.step ? before(tile + f.step) : 0.f;
      const int j0 = 16 * tile + t;
      float sum[2] = {0.f, 0.f};
      if (f.have >> f.out & 1u) {
        ok = f.wait();
        if (!ok) break;
        const uint32_t s = smem_addr(f.ring + f.out * W::kKeys);
        uint32_t c[2][G][4];
        float sc[2][G], mid[2][G];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tk = t + 8 * i;
          uint32_t kc[G], ks[G], km[L::GP / 2];
          lds_words<G>(s + L::kKeyCodes + ((tk * 4 + q) * G) * 4, kc);
          lds_words<G>(s + L::kKeyScale + (tk / 2 * G) * 4, ks);
          lds_words<L::GP / 2>(s + L::kKeyMin + tk * L::GP * 2, km);
#pragma unroll
          for (int g = 0; g < G; ++g) {
            centred(kc[g], c[i][g]);
            const float2 s2 = h2f(ks[g]), m2 = h2f(km[g / 2]);
            sc[i][g] = t % 2 ? s2.y : s2.x;
            mid[i][g] = fmaf(8.f, sc[i][g], g % 2 ? m2.y : m2.x);
          }
        }
        // all lanes have read the place: the next tile may come into it
        fence_proxy_async();
        __syncwarp();
        f.pass();
        f.send(a, lane);
#pragma unroll 1
        for (int k = 0; k < blocks; ++k) {
          const int4 range = *(reinterpret_cast<const int4*>(smem + W::kRange) + k);
          if (16 * tile >= range.w || 16 * tile + 16 <= range.z) continue;
          const uint32_t* frag = reinterpret_cast<const uint32_t*>(smem) + k * W::kParts * (W::kFrag / 4);
          const float* row = reinterpret_cast<const float*>(smem + W::kRow) + (k * 8 + 2 * q) * W::kRowWords;
          float z[2][2] = {};   // [key][row]
#pragma unroll
          for (int g = 0; g < G; ++g) {
            float acc[4];
            const uint4 u = *reinterpret_cast<const uint4*>(frag + (g * 32 + lane) * 4);
            mma_f16_zero(acc, c[0][g][0], c[1][g][0], c[0][g][1], c[1][g][1], u.x, u.y);
            mma_f16(acc, c[0][g][2], c[1][g][2], c[0][g][3], c[1][g][3], u.z, u.w);
            if constexpr (W::kParts == 2) {
              float low[4];
              const uint4 v = *reinterpret_cast<const uint4*>(frag + W::kFrag / 4 + (g * 32 + lane) * 4);
              mma_f16_zero(low, c[0][g][0], c[1][g][0], c[0][g][1], c[1][g][1], v.x, v.y);
              mma_f16(low, c[0][g][2], c[1][g][2], c[0][g][3], c[1][g][3], v.z, v.w);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[i] = fmaf(low[i], 1.f / 2048.f, acc[i]);
            }
            const float qs[2] = {row[4 + g], row[W::kRowWords + 4 + g]};
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                z[i][e] = fmaf(mid[i][g], qs[e], fmaf(sc[i][g], acc[2 * i + e], z[i][e]));
          }
          const bool whole = 16 * tile >= range.x && 16 * tile + 16 <= range.y;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float f = row[e * W::kRowWords], lse = row[e * W::kRowWords + 1];
            const int lo = __float_as_int(row[e * W::kRowWords + 2]), hi = __float_as_int(row[e * W::kRowWords + 3]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float w = ex2(fmaf(z[i][e], f, -lse) * 1.4426950408889634f);
              const int j = j0 + 8 * i;
              if (whole || (j >= lo && j < hi)) sum[i] += w;
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 1);
          sum[i] += __shfl_xor_sync(0xFFFFFFFFu, sum[i], 2);
        }
      } else {
        f.pass();
        f.send(a, lane);
      }
      const int j = j0 + 8 * q;
      if (q < 2 && j < keys) out[j] = had + (q ? sum[1] : sum[0]);
      had = had_next;
    }
    r0 += 8 * W::kBlocks;
  } while (r0 < rows);
  if (!ok) {
    report(a.status, LW_DEV_TIMEOUT);
    f.drain();
  }
}

}  // namespace dev
}  // namespace lw
