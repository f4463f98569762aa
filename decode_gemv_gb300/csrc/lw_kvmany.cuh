// Cache attention for many rows: chunks of prompts, on the 5th-generation
// tensor cores.
//
// An item is 128 rows (token, head) of one key/value head; keys come 64 at a
// time.  S = Q K^T and O += P V are tcgen05.mma with the first operand (Q, P)
// and the accumulators in tensor memory, the second (K, V, restored to fp16
// from their codes) in shared memory:
//  * 4 loader warps, one per 16-key tile of the 64: fetch their tile by bulk
//    copies (a ring of their own), restore k = sc c + mn and v = sc c + mn by
//    one rounded fp16 fma each, and store them as operand tiles (two buffers);
//  * 4 row warps, one thread per row: put the row of Q into tensor memory
//    (scaled by a power of two: the fp16 range), then for every 64 keys read
//    the row of S, take p = 2^(s - m), store it as fp16 over S, and add the
//    row's sum.  m is raised, and O rescaled, only where a score passes it by
//    2^8 (p stays below 2^8, in fp16 range and precision).  One of their
//    threads issues the products (a ninth warp would take the registers of
//    three).
// Two CTAs share an SM: one's products run while the other's rows are at
// work.  Operands of 11 bits (fp16) under outputs of 8 (bf16).
//
// The operand tiles are K-major core matrices of 8 x 16 bytes.  A key code
// word holds 8 elements of one key: its fp16 pairs are elements (0,4), (1,5),
// (2,6), (3,7), stored in that order, and Q in the same.  A value code word
// holds 4 elements of two keys: pairs along the keys, as P needs them; column
// nu = 32 g + 8 i + n of the product is element 32 g + 4 n + i (eight lanes
// then store 128 consecutive bytes).
#pragma once

#include "lw_btc.cuh"
#include "lw_kvfew.cuh"

namespace lw {

constexpr int kManyRows = 128, kManyKeys = 64;
constexpr int kManyUnit = kManyKeys / LW_KV_TILE;   // 16-key tiles of a unit = loader warps
constexpr int kManyThreads = 32 * 8;                // 4 row warps, 4 loader warps
constexpr int kManyPerSm = 2;
constexpr int kManyStages = 4;                      // tiles of a loader's ring

template <int D>
struct Many {
  using L = KvTile<D>;
  static constexpr int kKLbo = kManyKeys * 16 + 32;   // bytes between 8-element columns (32: bank offset)
  static constexpr int kKBytes = D / 8 * kKLbo;
  static constexpr int kVLbo = D * 16;                // bytes between 8-key columns
  static constexpr int kVBytes = kManyKeys / 8 * kVLbo;
  static constexpr int kHead = 1024;                  // barriers and flags
  static constexpr int kK = kHead, kV = kK + 2 * kKBytes;
  static constexpr int kRing = kV + 2 * kVBytes;
  static constexpr int kSmem = kRing + kManyUnit * kManyStages * L::kBytes;
  static constexpr int kPartial = kManyRows * (D + 2);   // floats: m, l, then [D / 4][rows][4]
  // tensor-memory columns: S (and P over it), O, Q
  static constexpr uint32_t kS = 0, kO = kManyKeys, kQ = kO + D;
  static constexpr uint32_t kCols = 256;
  static_assert(kQ + D / 2 <= kCols, "tensor memory");
};

namespace dev {

__host__ __device__ constexpr uint32_t idesc_f16(uint32_t n) {   // F16 operands, FP32 sums, M = 128
  return (1u << 4) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void sts_u4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint32_t pair_lo(uint32_t w) { return __byte_perm(w, w, 0x1010); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t w) { return __byte_perm(w, w, 0x3232); }
// the codes of nibbles 0, 4 and 1, 5 as fp16 integers: 1024 + c less 1024
__device__ __forceinline__ uint32_t whole_even(uint32_t w) {
  const uint32_t x = (w & 0x000F000Fu) | 0x64006400u, b = 0xE400E400u;
  return h2bits(__hadd2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&b)));
}
__device__ __forceinline__ uint32_t whole_odd(uint32_t w) {   // 1024 + 16 c
  return fma_h2((w & 0x00F000F0u) | 0x64006400u, 0x2C002C00u, 0xD400D400u);
}

// A wait that gives up when another role has
__device__ __forceinline__ bool many_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) return false;
  }
}

// The row warps' barrier: whether `ok` holds in all of them
__device__ __forceinline__ bool rows_agree(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}

// Barriers of a CTA
struct ManyBars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];   // per operand buffer
  uint64_t s_full, o_full;                               // a product is complete
  uint64_t last;                                         // everything issued has completed
  uint64_t ring[kManyUnit][kManyStages];
};

template <int D>
__global__ void __launch_bounds__(kManyThreads, kManyPerSm) kv_many_kernel(const AttnArgs a) {
  using F = Many<D>;
  using L = KvTile<D>;
  constexpr int G = L::G;
  extern __shared__ __align__(128) uint8_t smem[];
  ManyBars& bar = *reinterpret_cast<ManyBars*>(smem);
  static_assert(sizeof(ManyBars) <= 512, "barriers");
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + 512);   // [0] abort, [1] last part,
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + 528);                     // tensor memory
  // [unit % 4][tile]: the tile's keys are there (written before k_full, read
  // after s_full; four units on, the rows have long answered)
  volatile uint8_t* present = smem + 544;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.k_full[i], kManyUnit);
      mbar_init(&bar.v_full[i], kManyUnit);
      mbar_init(&bar.k_free[i], 1);
      mbar_init(&bar.v_free[i], 1);
    }
    mbar_init(&bar.s_full, 1);
    mbar_init(&bar.o_full, 1);
    mbar_init(&bar.last, 1);
    for (int i = 0; i < kManyUnit; ++i)
      for (int j = 0; j < kManyStages; ++j) mbar_init(&bar.ring[i][j], 1);
    flags[0] = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_addr(tslot), F::kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();
  KvWalk w;
  int Gc, q0;
  long long U;
  const bool any = kv_range<kManyThreads, kManyRows, kManyUnit>(a, w, Gc, U, q0);
  bool ok = true;   // no wait ran out

  if (any && warp >= 4 && warp < 8) {   // ---- loaders
    const int lw = warp - 4;
    FewFetch<D, kManyUnit, 1, kManyStages> t;
    t.bars = bar.ring[lw];
    t.ring = smem + F::kRing + lw * kManyStages * L::kBytes;
    t.parity = t.have = 0;
    uint32_t it = 0;
    for (bool more = true; more && ok;) {
      t.begin(a, w, lw, lane);
      // rows of the item all see the keys [all_lo, all_hi)
      int all_lo, all_hi, x;
      {
        int t1 = (w.rt * kManyRows + kManyRows - 1) / a.group;
        if (t1 > w.T - 1) t1 = w.T - 1;
        kv_token_keys(w.T, w.n, w.rt * kManyRows / a.group, a.p.causal, a.p.window, x, all_hi);
        kv_token_keys(w.T, w.n, t1, a.p.causal, a.p.window, all_lo, x);
      }
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        const int tile = w.span.lo + k * kManyUnit + lw, buf = it & 1;
        const uint32_t par = (it >> 1 & 1u) ^ 1u;
        const bool there = tile < w.span.hi && (t.have >> t.out & 1u);
        if (there && !t.wait()) { ok = false; mbar_wait(&t.bars[t.out], (t.parity >> t.out & 1u) ^ 1u); break; }
        const uint32_t s = smem_addr(t.ring) + t.out * L::kBytes;
        const int kb = tile * LW_KV_TILE;
        const bool edge = kb < all_lo || kb + LW_KV_TILE > all_hi;
        if (!__all_sync(0xFFFFFFFFu, many_wait(&bar.k_free[buf], par, flags))) { ok = false; break; }
        if (there) {
          const int q = lane & 3;
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // key 8 h + lane / 4, elements 32 g + 8 q + 0..7
            const int tk = 8 * h + lane / 4;
            uint32_t cw[G], sw[G];
            lds_words<G>(s + L::kKeyCodes + (uint32_t)((tk * 4 + q) * G) * 4, cw);
            lds_words<G>(s + L::kKeyScale + (uint32_t)(tk / 2 * G) * 4, sw);
            bool nan = false;
            if (edge) {   // rows that do not see a key must not get its NaN through V (0 x NaN): let it come by S
#pragma unroll
              for (int g = 0; g < G; ++g) {
                const uint32_t z = lds_u16(s + L::kValScale + (uint32_t)((tk / 2 * G + g) * 2 + tk % 2) * 2);
                nan |= (z & 0x7FFFu) > 0x7C00u;
              }
            }
            const uint32_t to = smem_addr(smem) + F::kK + buf * F::kKBytes + (uint32_t)((lw * 2 + h) * 128 + (lane / 4) * 16);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              uint32_t sc = tk & 1 ? pair_hi(sw[g]) : pair_lo(sw[g]);
              const uint32_t m1 = lds_u16(s + L::kKeyMin + (uint32_t)(tk * L::GP + g) * 2);
              const uint32_t mn = pair_lo(m1);
              if (nan) sc = 0x7FFF7FFFu;
              const uint32_t w0 = cw[g], w1 = cw[g] >> 8;
              sts_u4(to + (uint32_t)((4 * g + q) * F::kKLbo), fma_h2(whole_even(w0), sc, mn),
                     fma_h2(whole_odd(w0), sc, mn), fma_h2(whole_even(w1), sc, mn), fma_h2(whole_odd(w1), sc, mn));
            }
          }
        }
        if (lane == 0) present[it % 4 * kManyUnit + lw] = there;
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.k_full[buf]);
        if (!__all_sync(0xFFFFFFFFu, many_wait(&bar.v_free[buf], par, flags))) { ok = false; break; }
        {
          const int n = lane & 7, gh = lane >> 3 & 1, h = lane >> 4;   // 8 keys 8 h.., groups gh, gh + 2
          const uint32_t to = smem_addr(smem) + F::kV + buf * F::kVBytes + (uint32_t)((lw * 2 + h) * F::kVLbo + n * 16);
#pragma unroll
          for (int gg = 0; gg < (G + 1) / 2; ++gg) {
            const int g = 2 * gg + gh;
            if (g >= G) continue;
            uint32_t e[4], o[4], e2[4], o2[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int p = 4 * h + j;   // pair of keys
              uint32_t cw = 0, sc = 0, mn = 0;
              if (there) {
                cw = lds_u32(s + L::kValCodes + (uint32_t)((p * 8 + n) * G + g) * 4);
                sc = lds_u32(s + L::kValScale + (uint32_t)(p * G + g) * 4);
                mn = lds_u32(s + L::kValMin + (uint32_t)(p * G + g) * 4);
                if (edge) {
                  const int key = kb + 2 * p;
                  const uint32_t keep = (key < w.n && (sc & 0x7FFFu) <= 0x7C00u ? 0xFFFFu : 0u) |
                                        (key + 1 < w.n && (sc & 0x7FFF0000u) <= 0x7C000000u ? 0xFFFF0000u : 0u);
                  sc &= keep;
                  mn &= keep;
                }
              }
              e[j] = fma_h2(whole_even(cw), sc, mn);
              o[j] = fma_h2(whole_odd(cw), sc, mn);
              e2[j] = fma_h2(whole_even(cw >> 8), sc, mn);
              o2[j] = fma_h2(whole_odd(cw >> 8), sc, mn);
            }
            sts_u4(to + (4 * g + 0) * 128, e[0], e[1], e[2], e[3]);
            sts_u4(to + (4 * g + 1) * 128, o[0], o[1], o[2], o[3]);
            sts_u4(to + (4 * g + 2) * 128, e2[0], e2[1], e2[2], e2[3]);
            sts_u4(to + (4 * g + 3) * 128, o2[0], o2[1], o2[2], o2[3]);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_full[buf]);
        if (tile < w.span.hi) {
          t.out = t.out + 1 == kManyStages ? 0 : t.out + 1;
          t.send(a, lane);
        }
      }
      if (ok) more = kv_advance<kManyRows, kManyUnit>(a, w, q0);
    }
    if (!ok) {
      flags[0] = 1;
      if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
      for (int i = 0; i < kManyStages; ++i)   // no copy may be in flight when the CTA ends
        if (t.have >> i & 1u) mbar_wait(&t.bars[i], t.parity >> i & 1u);
    }
  } else if (any && warp < 4) {   // ---- rows
    const uint32_t mine = tmem + ((uint32_t)(32 * warp) << 16);   // this warp's quarter
    const int row = threadIdx.x;
    const uint32_t kbase = smem_addr(smem) + F::kK, vbase = smem_addr(smem) + F::kV;
    // the issuing thread's: S of unit u, once its keys are there; O of unit u
    const auto issue_s = [&](uint32_t u) {
      const uint32_t at = kbase + (u & 1) * F::kKBytes;
      if (!many_wait(&bar.k_full[u & 1], u >> 1 & 1u, flags)) return false;
      tc_fence_after();
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        umma_bf16_ta(tmem + F::kS, tmem + F::kQ + 8 * s, sdesc(at + 2 * s * F::kKLbo, F::kKLbo, 128),
                     idesc_f16(kManyKeys), s > 0);
      umma_commit(&bar.s_full);
      umma_commit(&bar.k_free[u & 1]);
      return true;
    };
    const auto issue_o = [&](uint32_t u, bool first) {
      const uint32_t at = vbase + (u & 1) * F::kVBytes;
      if (!many_wait(&bar.v_full[u & 1], u >> 1 & 1u, flags)) return false;
      tc_fence_after();
#pragma unroll
      for (int s = 0; s < kManyKeys / 16; ++s)
        umma_bf16_ta(tmem + F::kO, tmem + F::kS + 8 * s, sdesc(at + 2 * s * F::kVLbo, F::kVLbo, 128),
                     idesc_f16(D), !first || s > 0);
      umma_commit(&bar.o_full);
      umma_commit(&bar.v_free[u & 1]);
      return true;
    };
    uint32_t it = 0;
    bool stop = false;   // rows_agree said no
    for (bool more = true; more && ok;) {
      const int r = w.rt * kManyRows + row;
      const bool live = r < w.T * a.group;
      const int tok = live ? r / a.group : w.T - 1, hq = w.h * a.group + (live ? r - tok * a.group : 0);
      int lo, hi, all_lo, all_hi, x;
      kv_token_keys(w.T, w.n, tok, a.p.causal, a.p.window, lo, hi);
      {
        int t1 = (w.rt * kManyRows + kManyRows - 1) / a.group;
        if (t1 > w.T - 1) t1 = w.T - 1;
        kv_token_keys(w.T, w.n, w.rt * kManyRows / a.group, a.p.causal, a.p.window, x, all_hi);
        kv_token_keys(w.T, w.n, t1, a.p.causal, a.p.window, all_lo, x);
      }
      // the row of Q, scaled by 2^-e
      float f;
      {
        const int64_t at = (int64_t)(q0 + tok) * a.p.q_token_stride + (int64_t)hq * a.p.q_head_stride;
        float top = 0.f, y[8];
        for (int o = 0; o < D / 8; ++o) {
          load_q8(a, at + 8 * o, y);
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
        }
        int e = (int)(__float_as_uint(top) >> 23) - 127;
        e = e < -100 ? -100 : (e > 126 ? 126 : e);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        f = a.p.scale * 1.4426950408889634f * __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 1
        for (int o = 0; o < D / 16; ++o) {
          uint32_t z[8];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            load_q8(a, at + 16 * o + 8 * j, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[4 * j + i] = h2bits(__floats2half2_rn(y[i] * down, y[i + 4] * down));
          }
          tmem_st8(mine + F::kQ + 8 * o, z);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      ok = rows_agree(ok);   // (every Q row is in place; all four warps go on, or none)
      if (!ok) break;
      if (row == 0) ok = issue_s(it);
      float m = -INFINITY, mu = 0.f, l = 0.f;
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        const int kb = (w.span.lo + k * kManyUnit) * LW_KV_TILE;
        __syncwarp();
        if (ok) ok = many_wait(&bar.s_full, it & 1u, flags);
        tc_fence_after();
        const uint32_t there = *reinterpret_cast<const volatile uint32_t*>(present + it % 4 * kManyUnit);
        uint32_t s0[32], s1[32];
        tmem_ld32(mine + F::kS, s0);
        tmem_ld32(mine + F::kS + 32, s1);
        tmem_ld_wait();
        float2 t[32];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          t[j] = mul2(make_float2(__uint_as_float(s0[2 * j]), __uint_as_float(s0[2 * j + 1])), make_float2(f, f));
          t[16 + j] = mul2(make_float2(__uint_as_float(s1[2 * j]), __uint_as_float(s1[2 * j + 1])), make_float2(f, f));
        }
        if (kb < all_lo || kb + kManyKeys > all_hi || there != 0x01010101u) {
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const bool in = there >> (8 * (j / 8)) & 1u;
            const int key = kb + 2 * j;
            if (!(in && key >= lo && key < hi)) t[j].x = -INFINITY;
            if (!(in && key + 1 >= lo && key + 1 < hi)) t[j].y = -INFINITY;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) top = fmaxf(top, fmaxf(t[j].x, t[j].y));
        if (__any_sync(0xFFFFFFFFu, top > m + 8.f)) {
          const float mx = fmaxf(m, top);
          mu = mx == -INFINITY ? 0.f : mx;
          const float al = ex2(m - mu);
          m = mx;
          l *= al;
          if (k > w.k0) {   // (the product of the keys before is complete: S came after it)
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t z[32];
              tmem_ld32(mine + F::kO + c, z);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) z[j] = __float_as_uint(__uint_as_float(z[j]) * al);
              tmem_st32(mine + F::kO + c, z);
            }
          }
        }
        float2 sum = make_float2(0.f, 0.f);
        uint32_t p[32];
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float2 y = make_float2(ex2(t[j].x - mu), ex2(t[j].y - mu));
          sum.x += y.x;
          sum.y += y.y;
          p[j] = h2bits(__floats2half2_rn(y.x, y.y));
        }
        l += sum.x + sum.y;
        tmem_st32(mine + F::kS, p);
        tmem_st_wait();
        tc_fence_before();
        ok = rows_agree(ok);
        if (!ok) { stop = true; break; }
        if (row == 0) {
          ok = issue_o(it, k == w.k0);
          // S lies over P: the next S once the sum over P is complete
          if (ok && k + 1 < w.k1) ok = many_wait(&bar.o_full, it & 1u, flags) && issue_s(it + 1);
        }
      }
      if (stop) break;
      const KvWalk v = w;
      const int vq0 = q0;
      more = kv_advance<kManyRows, kManyUnit>(a, w, q0);
      __syncwarp();
      if (ok) ok = many_wait(&bar.o_full, (it - 1) & 1u, flags);
      ok = rows_agree(ok);
      if (!ok) break;
      tc_fence_after();
      const bool whole = v.k0 == 0 && v.k1 == v.units;
      float* part = a.partials + ((size_t)blockIdx.x * 2 + (v.k0 == 0)) * F::kPartial;
      const auto give = [&](int g, float l, const float (&z)[32]) {   // 32 elements of the row, [i][n]
        if (!live) return;
        const float inv = 1.f / l;
        const int64_t at = (int64_t)(vq0 + tok) * a.p.out_token_stride + (int64_t)hq * a.p.out_head_stride + 32 * g;
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = l == 0.f ? 0.f : z[8 * (i % 4) + n + i / 4] * inv;
          store8(a, at + 4 * n, y);
        }
      };
      const auto give_lse = [&](float m, float l) {
        if (live && a.p.lse)
          a.p.lse[(int64_t)(vq0 + tok) * a.p.q_heads + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      };
#pragma unroll 1
      for (int g = 0; g < G; ++g) {
        uint32_t u[32];
        float z[32];
        tmem_ld32(mine + F::kO + 32 * g, u);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(u[j]);
        if (whole) {
          give(g, l, z);
        } else {
#pragma unroll
          for (int n = 0; n < 8; ++n)
            *reinterpret_cast<float4*>(part + 2 * kManyRows + ((8 * g + n) * kManyRows + row) * 4) =
                make_float4(z[n], z[8 + n], z[16 + n], z[24 + n]);
        }
      }
      tc_fence_before();
      if (whole) {
        give_lse(m, l);
      } else {
        part[row] = m;
        part[kManyRows + row] = l;
        const long long x0 = v.x - v.k0;
        const int c0 = tc_owner(x0, U, Gc), parts = tc_owner(x0 + v.units - 1, U, Gc) - c0 + 1;
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (threadIdx.x == 0) {
          const bool last = atomicAdd(a.counters + c0, 1u) == (uint32_t)parts - 1u;
          if (last) a.counters[c0] = 0;
          flags[1] = last;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (flags[1]) {
          __threadfence();
          const auto from = [&](int i) {
            return a.partials + (i ? (size_t)(c0 + i) * 2 : (size_t)c0 * 2 + 1) * F::kPartial;
          };
          float M = -INFINITY, S = 0.f;
          for (int i = 0; i < parts; ++i) M = fmaxf(M, __ldcg(from(i) + row));
          const float Mu = M == -INFINITY ? 0.f : M;
          for (int i = 0; i < parts; ++i) S = fmaf(__ldcg(from(i) + kManyRows + row), ex2(__ldcg(from(i) + row) - Mu), S);
#pragma unroll 1
          for (int g = 0; g < G; ++g) {
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = 0.f;
#pragma unroll 1
            for (int i = 0; i < parts; ++i) {
              const float* p = from(i);
              const float e = ex2(__ldcg(p + row) - Mu);
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(p + 2 * kManyRows + ((8 * g + n) * kManyRows + row) * 4));
                z[n] = fmaf(y.x, e, z[n]);
                z[8 + n] = fmaf(y.y, e, z[8 + n]);
                z[16 + n] = fmaf(y.z, e, z[16 + n]);
                z[24 + n] = fmaf(y.w, e, z[24 + n]);
              }
            }
            give(g, S, z);
          }
          give_lse(M, S);
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
      }
    }
    if (!ok) {
      flags[0] = 1;
      if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
    }
    if (row == 0) {   // no product may be in flight when the tensor memory goes
      umma_commit(&bar.last);
      mbar_wait(&bar.last, 0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, F::kCols);
}

}  // namespace dev
}  // namespace lw
