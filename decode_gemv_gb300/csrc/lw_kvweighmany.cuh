// Accumulated attention weight for many rows (prompts), on the 5th-generation
// tensor cores.
//
// S = K Q^T has the keys as its first dimension: a key is a lane of tensor
// memory, the thread that owns it adds up its row of exponentials in registers,
// and no reduction crosses threads.  A unit is 128 keys of one head; its rows --
// the packed (token, head of the group) pairs of its sequence -- come 128 at a
// time.  Operands are fp16: a key as two parts, hi + lo (22 bits; restored from
// the codes once a unit), a 16-bit query as itself, an fp32 one as two parts.  So
// S takes two products (three for fp32: hi hi, lo hi, hi lo) into one fp32
// accumulator.  Queries are scaled by a power of two a row, their largest element
// to 2^14; keys by one a unit where all of them are small.
//
// Two kernels.  kv_weigh_rows_kernel writes the rows as operand tiles, once for
// all units (a unit would spend as many instructions on them as on its
// exponentials), with each row's scale and lse in log2 units.  A CTA of
// kv_weigh_many_kernel takes every so many-th unit of a head of a sequence:
//  * warp 0 fetches row tiles by bulk copies (a tile is one contiguous image);
//  * warp 1 issues the products, into three accumulators of 128 columns: the keys are the operand in tensor
//    memory (both in shared memory are 8 KB for 64 cycles of products, all that it gives: 379 us where this takes
//    350);
//  * 8 warps restore the unit's keys and send for the next one's, then two groups of four take the tiles in turn:
//    a thread reads its key's 128 scores and adds 2^(s f - lse) of those that it is
//    seen by.  A key is seen by a contiguous range of rows (causal: from some row
//    on, windowed: up to some row), so only tiles across an end of it are masked.
// 2048 tokens on 14336 keys (8 heads of 128 with 4 query heads each): bf16 369 us, both kernels, 699 TFLOP/s of
// useful products, of which two are carried out for one: 1400, 80 % of what the tensor cores sustain; a tile's
// exponentials take about as long as its products.  fp32, three for one: 492.  8 sequences of 32768 keys, 64 tokens
// each, bf16: 530 us, a unit 4.9 us, of which 1 is products: its start (keys restored, tensor memory written) and its
// end.  The next unit's keys are fetched while this one's rows run (603 -> 553 us at 48 tokens).
// Units are few where keys are: then a cluster shares a unit's row tiles, and rank 0
// adds the ranks' sums in order.
#pragma once

#include "lw_kvmany.cuh"
#include "lw_kvselect.cuh"
#include "lw_kvweigh.cuh"

namespace lw {

template <int D, int PARTS>   // parts of a query operand
struct WeighMany {
  using L = KvTile<D>;
  static constexpr int kRows = 128, kKeys = 128;
  static constexpr int kPart = D * kRows * 2;                  // bytes of one operand part of a row tile
  static constexpr int kImage = PARTS * kPart;
  static constexpr int kParam = kRows * 8;                     // [pair of rows] f, f, -lse, -lse
  static constexpr int kRecord = kImage + kParam;              // of the workspace
  static constexpr int kStages = PARTS == 1 ? 4 : 3;
  static constexpr int kThreads = 320;
  // tensor-memory columns: three accumulators, then the keys' parts
  static constexpr int kBufs = 3, kKeyCol = kBufs * kRows, kKeyCols = D / 2;
  static constexpr int kSlots = 4;   // of barriers and parameters: an even number, so that each is one group's
  static constexpr int kHead = 1024 + 2 * kKeys * 4;           // barriers and flags, the groups' sums
  static constexpr int kParams = kHead;                        // [kSlots]
  static constexpr int kB = kParams + kSlots * kParam;
  // over half an SM's: one CTA an SM, whose tensor memory is all of it
  static constexpr int kNeed = kB + kStages * kImage, kSmem = kNeed > 118784 ? kNeed : 118784;
  static_assert(kSmem <= 232448, "shared memory");
};

struct WeighManyArgs {
  WeighArgs a;
  const uint8_t* rows;    // [heads][row_tiles] records
  int32_t row_tiles;
};
struct WeighRowsArgs {
  WeighArgs a;
  uint8_t* rows;
  int32_t row_tiles;
};

namespace dev {

// One row tile of one head: 4 lanes a row, as weigh_row.
template <int D, class T>
__global__ void __launch_bounds__(512) kv_weigh_rows_kernel(const WeighRowsArgs w) {
  constexpr int PARTS = sizeof(T) == 4 ? 2 : 1, G = D / 32;
  using W = WeighMany<D, PARTS>;
  const WeighArgs& a = w.a;
  const int h = blockIdx.y, row = threadIdx.x / 4, q = threadIdx.x % 4;
  pdl_wait();
  const int64_t r = (int64_t)blockIdx.x * W::kRows + row;
  const bool live = r < a.p.q_tokens * a.group;
  const int64_t tok = live ? r / a.group : 0;
  const int head = h * a.group + (int)(live ? r - tok * a.group : 0);
  float x[G][8], top = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    if (live)
      weigh_load8<T>(a, tok * a.p.q_token_stride + (int64_t)head * a.p.q_head_stride + 32 * g + 8 * q, x[g]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[g][i]));
  }
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
  int e = (int)(__float_as_uint(top) >> 23) - 127;
  e = e < -100 ? -100 : (e > 127 ? 127 : e);
  const float down = __uint_as_float((uint32_t)(127 - e + 14) << 23);
  uint8_t* rec = w.rows + ((int64_t)h * w.row_tiles + blockIdx.x) * W::kRecord;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[g][i] * down, v = x[g][i + 4] * down;
      if constexpr (PARTS == 2) split2<1>(u, v, hi[i], lo[i]);
      else hi[i] = h2bits(__floats2half2_rn(u, v));
    }
    uint8_t* to = rec + (4 * g + q) * (W::kRows * 16) + row * 16;
    *reinterpret_cast<uint4*>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (PARTS == 2) *reinterpret_cast<uint4*>(to + W::kPart) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  if (q == 0) {
    constexpr float kLog2e = 1.4426950408889634f;
    float* p = reinterpret_cast<float*>(rec + W::kImage) + row / 2 * 4 + row % 2;
    p[0] = live ? a.p.scale * __uint_as_float((uint32_t)(e - 14 + 127) << 23) * kLog2e : 0.f;
    p[2] = live ? -a.p.lse[tok * a.p.q_heads + head] * kLog2e : -INFINITY;
  }
}

struct WeighBars {
  uint64_t b_full[4], b_free[4];                    // row tiles
  uint64_t p_full[4], d_full[4], d_free[4];         // their scales and lse; accumulators
  uint64_t last;
};

template <int D, int PARTS>
__global__ void __launch_bounds__(320, 1) kv_weigh_many_kernel(const WeighManyArgs w) {
  using W = WeighMany<D, PARTS>;
  using L = KvTile<D>;
  constexpr int G = L::G, S = W::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  const WeighArgs& a = w.a;
  WeighBars& bar = *reinterpret_cast<WeighBars*>(smem);
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + 512);   // [0] abort
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + 516);
  uint32_t* s_top = reinterpret_cast<uint32_t*>(smem + 520);                      // largest key magnitude, as bits
  float* sums = reinterpret_cast<float*>(smem + 1024);                            // [2][keys]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int h = blockIdx.y, b = blockIdx.z;
  int k0 = (int)(blockIdx.x / ranks) * W::kKeys;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bar.b_full[i], 1);
      mbar_init(&bar.b_free[i], 1);
      mbar_init(&bar.p_full[i], 1);
      mbar_init(&bar.d_full[i], 1);
      mbar_init(&bar.d_free[i], 4);
    }
    mbar_init(&bar.last, 1);
    flags[0] = 0;
    *s_top = 0;
    fence_barrier_init();
  }
  pdl_wait();
  int q0, T, n;
  if (k0 == 0 && rank == 0 && h == 0 && threadIdx.x == 0) weigh_seq<true>(a, b, q0, T, n);
  else weigh_seq<false>(a, b, q0, T, n);
  const int keys = n < a.p.w_keys ? n : (int)a.p.w_keys;
  if (k0 >= keys) return;   // (all of the cluster)
  // rows that see key j of this sequence: [first_row(j), end_row(j)), packed
  const int64_t R0 = (int64_t)q0 * a.group;
  const int past = n - T;   // the first token's position
  const auto first_row = [&](int j) {
    const int64_t t = a.p.causal ? (int64_t)j - past : 0;
    return R0 + (t < 0 ? 0 : t > T ? T : t) * a.group;
  };
  const auto end_row = [&](int j) {
    const int64_t t = a.p.window ? (int64_t)j + a.p.window - past : T;
    return R0 + (t < 0 ? 0 : t > T ? T : t) * a.group;
  };
  if (warp == 1) {
    tmem_alloc(smem_addr(tslot), 512);
    tmem_relinquish();
  }
  __syncthreads();   // (barriers)
  bool ok = true;
  int done = 0, sent = 0;   // row tiles of the units before (the barriers' phases go on), and (thread 0) sent for
  uint32_t unit = 0;
  const int step = (int)(gridDim.x / ranks) * W::kKeys;
  const float* add = a.p.add_to ? a.p.add_to + b * a.p.add_seq_stride + h * a.p.add_head_stride : nullptr;
  float* out = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride;
  // Keys: a lane of tensor memory each, half of their elements a group of four warps (2 ..)
  const int kw = warp - 2, group = kw / 4, quarter = warp % 4, key = 32 * quarter + lane;
  constexpr int kOct = D / 16;   // 8-element columns of a thread: words of codes
  uint32_t kc[kOct];
  __half sc[kOct], mn[kOct];
  bool next_real = false;
  const auto fetch = [&](int k0) {
    next_real = false;
    if (warp < 2 || k0 >= keys) return;
    const int j = k0 + key, tile = j / 16, tpp = a.page_tokens / LW_KV_TILE, tk = j % 16;
    const bool seen = j < keys && first_row(j) < end_row(j);   // (else its page is not needed)
    const int page = seen ? a.p.page_table[(int64_t)b * a.p.table_stride + tile / tpp] : -1;
    next_real = page >= 0 && page < a.n_pages;
    if (!next_real && seen) report(a.status, LW_DEV_BAD_PAGE);
    if (!next_real) return;
    const uint8_t* s = a.pages + page * a.page_bytes + ((int64_t)h * tpp + tile % tpp) * L::kBytes;
#pragma unroll
    for (int i = 0; i < kOct; ++i) {
      const int o = kOct * group + i, g = o / 4;   // column o: elements 32 g + 8 (o % 4) ..
      kc[i] = *reinterpret_cast<const uint32_t*>(s + L::kKeyCodes + ((tk * 4 + o % 4) * G + g) * 4);
      sc[i] = *reinterpret_cast<const __half*>(s + L::kKeyScale + 2 * ((tk / 2 * G + g) * 2 + tk % 2));
      mn[i] = *reinterpret_cast<const __half*>(s + L::kKeyMin + 2 * (tk * L::GP + g));
    }
  };
  fetch(k0);
  for (int next; k0 < keys; k0 = next) {
    next = k0 < keys - step ? k0 + step : keys;
    const int k1 = min(k0 + W::kKeys, keys);
    const int64_t ra = first_row(k0), rb = end_row(k1 - 1);
    // what the sums are added to
    const int at = k0 + (int)threadIdx.x;
    const bool last = rank == 0 && threadIdx.x < W::kKeys && at < keys;
    const float had = last && add ? add[at] : 0.f;
    if (ra >= rb) {   // no row sees these keys (the same in all of the cluster)
      fetch(next);
      if (last) out[at] = had;
      continue;
    }
    // this rank's row tiles
    const int first_tile = (int)(ra / W::kRows), all = (int)((rb - 1) / W::kRows) - first_tile + 1;
    const int t0 = first_tile + (int)((int64_t)all * rank / ranks);
    const int nt = first_tile + (int)((int64_t)all * (rank + 1) / ranks) - t0;
    // (thread 0) The next row tile, where its places are free: the first ones while the keys come
    const auto send = [&] {
      const int s = sent % S, d = sent % W::kSlots;
      ok = many_wait(&bar.b_free[s], (uint32_t)(sent / S & 1) ^ 1u, flags) &&
           many_wait(&bar.d_free[d], (uint32_t)(sent / W::kSlots & 1) ^ 1u, flags);
      if (!ok) return;
      const uint8_t* src = w.rows + ((int64_t)h * w.row_tiles + t0 + sent - done) * W::kRecord;
      mbar_arrive_expect_tx(&bar.p_full[d], W::kParam);
      bulk_g2s(smem + W::kParams + d * W::kParam, src + W::kImage, W::kParam, &bar.p_full[d]);
      mbar_arrive_expect_tx(&bar.b_full[s], W::kImage);
      bulk_g2s(smem + W::kB + s * W::kImage, src, W::kImage, &bar.b_full[s]);
      ++sent;
    };
    if (threadIdx.x == 0)
      for (int i = 0; i < S && i < nt && ok; ++i) send();
    // ---- the keys, which have been sent for
    const int j = k0 + key;
    const bool real = next_real;   // (a key past the end, or of a page that is not there, is seen by no row)
    if (warp >= 2) {
      float top = 0.f;
      if (real)
#pragma unroll
        for (int i = 0; i < kOct; ++i) {
          const float m = __half2float(mn[i]);
          top = fmaxf(top, fmaxf(fabsf(m), fabsf(fmaf(15.f, __half2float(sc[i]), m))));
        }
      top = top <= 3.402823466e38f ? top : 65504.f;
      const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top));
      if (lane == 0) atomicMax(s_top, most);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    // all keys below 2^-4: brought up to there (lo parts would have too few bits as fp16); a power of two
    const int ke = (int)(*s_top >> 23) - 127, lift = ke < -4 ? min(-4 - ke, 24) : 0;
    const float up = __uint_as_float((uint32_t)(127 + lift) << 23);
    if (warp >= 2) {
      const uint32_t to = tmem + ((uint32_t)(32 * quarter) << 16) + W::kKeyCol + 4 * kOct * group;
#pragma unroll
      for (int i = 0; i < kOct; i += 2) {
        uint32_t hi[8] = {}, lo[8] = {};
        if (real) {
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t c = e % 2 ? whole_odd(kc[i + x] >> (8 * (e / 2))) : whole_even(kc[i + x] >> (8 * (e / 2)));
              const float s1 = __half2float(sc[i + x]), m1 = __half2float(mn[i + x]);
              const float2 y = mul2(fma2(h2f(c), make_float2(s1, s1), make_float2(m1, m1)), make_float2(up, up));
              split2<1>(y.x, y.y, hi[4 * x + e], lo[4 * x + e]);
            }
        }
        __syncwarp();
        tmem_st8(to + 4 * i, hi);
        tmem_st8(to + W::kKeyCols + 4 * i, lo);
      }
      tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0) *s_top = 0;   // (all have read it)
    fetch(next);   // the next unit's, while this one's rows run
    if (warp == 0) {   // ---- row tiles
      if (lane == 0) {
        for (; sent < done + nt && ok;) send();
        if (!ok) {
          flags[0] = 1;
          report(a.status, LW_DEV_TIMEOUT);
          for (int x = max(0, sent - 4); x < sent; ++x) {   // no copy may be in flight when the CTA ends
            mbar_wait(&bar.p_full[x % W::kSlots], (uint32_t)(x / W::kSlots & 1));
            if (x >= sent - S) mbar_wait(&bar.b_full[x % S], (uint32_t)(x / S & 1));
          }
          sent = done + nt;
        }
      }
    } else if (warp == 1) {   // ---- products
      const auto wait = [&](uint64_t* x, uint32_t parity) { return __all_sync(0xFFFFFFFFu, many_wait(x, parity, flags)) != 0; };
      const uint32_t base = smem_addr(smem), tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const int count = __shfl_sync(0xFFFFFFFFu, nt, 0);
      const uint32_t kh = tm + W::kKeyCol, kl = kh + W::kKeyCols;
      const int first = __shfl_sync(0xFFFFFFFFu, done, 0);
      for (int i = first; i < first + count && ok; ++i) {
        const int s = i % S, d = i % W::kBufs, was = i - W::kBufs;   // (the tile that had the accumulators before)
        ok = (was < 0 || wait(&bar.d_free[was % W::kSlots], (uint32_t)(was / W::kSlots & 1))) && wait(&bar.b_full[s], (uint32_t)(i / S & 1));
        if (!ok) break;
        tc_fence_after();
        const uint64_t qh = sdesc(base + W::kB + s * W::kImage, W::kRows * 16, 128), ql = qh + (W::kPart >> 4);
        const uint32_t to = tm + W::kRows * d;
        if (elect_one()) {
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            umma_bf16_ta(to, kl + 8 * x, qh + (2 * x * W::kRows * 16 >> 4), idesc_f16(W::kRows), x > 0);
          if constexpr (PARTS == 2) {
#pragma unroll
            for (int x = 0; x < D / 16; ++x)
              umma_bf16_ta(to, kh + 8 * x, ql + (2 * x * W::kRows * 16 >> 4), idesc_f16(W::kRows), 1);
          }
#pragma unroll
          for (int x = 0; x < D / 16; ++x)
            umma_bf16_ta(to, kh + 8 * x, qh + (2 * x * W::kRows * 16 >> 4), idesc_f16(W::kRows), 1);
          umma_commit(&bar.b_free[s]);
          umma_commit(&bar.d_full[i % W::kSlots]);
        }
        __syncwarp();
      }
      if (!ok) {
        flags[0] = 1;
        if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
      }
      __syncwarp();
      if (elect_one()) umma_commit(&bar.last);   // no product may be in flight when the tensor memory goes
      __syncwarp();
      mbar_wait(&bar.last, unit & 1u);
    } else {   // ---- exponentials
      const uint32_t mine = tmem + ((uint32_t)(32 * quarter) << 16);
      const int64_t from = real ? first_row(j) : 0, to = real ? end_row(j) : 0;
      const float down = __uint_as_float((uint32_t)(127 - lift) << 23);
      float2 total = make_float2(0.f, 0.f);
      for (int i = done + ((group ^ done) & 1); i < done + nt && ok; i += 2) {   // (tile i is group i % 2's)
        const int d = i % W::kBufs, slot = i % W::kSlots;
        const int64_t r0 = (int64_t)(t0 + i - done) * W::kRows;
        ok = __all_sync(0xFFFFFFFFu, many_wait(&bar.p_full[slot], (uint32_t)(i / W::kSlots & 1), flags) &&
                                         many_wait(&bar.d_full[slot], (uint32_t)(i / W::kSlots & 1), flags));
        if (!ok) break;
        tc_fence_after();
        const uint32_t params = smem_addr(smem) + W::kParams + slot * W::kParam;
        const bool whole = __all_sync(0xFFFFFFFFu, lift == 0 && from <= r0 && to >= r0 + W::kRows);
        const int lo = (int)(from - r0 < 0 ? 0 : from - r0 > W::kRows ? W::kRows : from - r0);
        const int hi = (int)(to - r0 < 0 ? 0 : to - r0 > W::kRows ? W::kRows : to - r0);
        float2 part[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t z[2][32];
        tmem_ld32(mine + W::kRows * d, z[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait();
          if (c < 3) tmem_ld32(mine + W::kRows * d + 32 * (c + 1), z[(c + 1) & 1]);
          const uint32_t(&y)[32] = z[c & 1];
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 p = lds_f4(params + (16 * c + e) * 16);
              const float2 x = fma2(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), make_float2(p.x, p.y),
                                    make_float2(p.z, p.w));
              part[e & 1] = add2(part[e & 1], make_float2(ex2(x.x), ex2(x.y)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float4 p = lds_f4(params + (16 * c + e) * 16);
              const float2 s = mul2(make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])), make_float2(down, down));
              const float2 x = fma2(s, make_float2(p.x, p.y), make_float2(p.z, p.w));
              const int col = 32 * c + 2 * e;
              part[e & 1] = add2(part[e & 1], make_float2(col >= lo && col < hi ? ex2(x.x) : 0.f,
                                                          col + 1 >= lo && col + 1 < hi ? ex2(x.y) : 0.f));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.d_free[slot]);
        total = add2(total, add2(part[0], part[1]));
      }
      if (!ok) {
        flags[0] = 1;
        if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
      }
      sums[group * W::kKeys + key] = total.x + total.y;
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    done += nt;
    // the groups' sums, then the ranks', in order
    if (threadIdx.x < W::kKeys) sums[threadIdx.x] += sums[W::kKeys + threadIdx.x];
    if (ranks > 1) cluster_sync();
    if (last) {
      float sum = sums[threadIdx.x];
      for (int r = 1; r < ranks; ++r) sum += cluster_load(sums + threadIdx.x, (uint32_t)r);
      out[at] = had + sum;
    }
    if (ranks > 1) cluster_sync();   // (a rank's sums stay until they are read)
    ++unit;
  }
  __syncthreads();
  if (warp == 1) tmem_dealloc(*tslot, 512);
}

}  // namespace dev
}  // namespace lw
