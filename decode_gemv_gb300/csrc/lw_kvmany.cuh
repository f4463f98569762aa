// Cache attention for many rows: chunks of prompts, on the 5th-generation
// tensor cores.
//
// An item is up to 256 rows (token, head) of one key/value head, two tiles of
// 128; keys come 64 at a time.  S = Q K^T and O += P V are tcgen05.mma: Q, K
// and V (fp16, restored from the codes) are operand tiles in shared memory, P
// and the accumulators lie in tensor memory.
//  * 6 loader warps take the 16-key tiles in turn: bulk copies bring the next
//    ones while the last, in registers, is restored -- k = sc c + mn and v = sc c +
//    mn by one rounded fp16 fma each -- and stored as operand tiles (four
//    buffers), once for both row tiles;
//  * 8 row warps, one thread per row: put Q into shared memory (each row scaled
//    by a power of two: the fp16 range), then for every 64 keys read the row of
//    S, take p = 2^(s - m), store p 2^11 as fp16 over S, and add the row's sum.  m
//    is raised, and O rescaled, only where a score passes it by 2^4: p 2^11 stays
//    within 2^15, below fp16's largest number, and a p of 2^-25 still has 11 bits
//    (in units of 1 all of the keys beside one that dominates its row were lost);
//  * 2 warps issue the products, one per row tile: the queue of products is
//    short (an issue takes as long as the product before it), so that while one
//    waits for its rows the other keeps the tensor cores at work.  All lanes
//    walk along and one is elected to issue (descriptors are warp-uniform then:
//    from divergent code an issue took 80 cycles, more than its product).  S has
//    two buffers a tile: the next S is computed while the rows work on this one.
// That is for bf16 calls: operands of 11 bits (fp16) under outputs of 8.
//
// WIDE (fp16 and fp32 calls): every operand is two fp16 parts, x = hi + lo 2^-11,
// an item is one tile of 128 rows, and what the second tile had holds the lo
// parts: S = Qh Kh + 2^-11 (Qh Kl + Ql Kh), O likewise from P and V, the two sums
// in accumulators of their own (issuer 0 the first, issuer 1 the second; fp16
// queries are their hi parts).  Two threads share a row, 32 keys of a unit each
// (one a row had the loaders and the tensor cores wait: 2 x 1024 tokens on 4096
// keys 537 -> 443 us when it was changed), and agree through shared memory on the row's maximum where
// it is raised.  Restoring an element is five times the work, so there are 8
// loaders (64 wide: 6 of more registers); the buffers are what fits.
//
// Measured (8 heads of 128 with 4 query heads each), us and useful TFLOP/s, two
// products a (row, key) pair:
//   bf16  2048 tokens on 16384 keys 398, 1295    4096 on 4096 152, 906
//         8 x 64 on 8192 82, 835                 8 x 512 on 512 73, 237
//   fp16  2 x 1024 on 4096 405, 297 (five products for two)
//   fp32  2 x 90 on 2400 51, 136; 2048 on 6000 559, 298 (six products for two)
// Long bf16 chunks are bound by the row warps' softmax and the loaders' restoring
// together (issue 63 %, tensor cores 53 %): two row warps and one and a half
// loaders share a scheduler, a unit takes 2000 cycles, its products 1250 and its
// exponentials 1000.  The registers are short: a bf16 thread spills 94 to 142 bytes,
// one of WIDE 96 and 128 wide (96 registers) 396 to 466.  Short items are bound by their starts and ends: reading Q
// 7000 cycles, writing out 4000 to 9000, joining a cut item's parts 10000.
//
// The operand tiles are K-major core matrices of 8 x 16 bytes.  A key code
// word holds 8 elements of one key: its fp16 pairs are elements (0,4), (1,5),
// (2,6), (3,7), stored in that order, and Q in the same.  A value code word
// holds 4 elements of two keys: pairs along the keys, as P needs them; column
// nu = 32 g + 8 i + n of the product is element 32 g + 4 n + i (eight lanes
// then store 128 consecutive bytes).
#pragma once

#include <type_traits>

#include "lw_btc.cuh"
#include "lw_kvfew.cuh"

namespace lw {

constexpr int kManyTile = 128, kManyKeys = 64;
constexpr int kManyUnit = kManyKeys / LW_KV_TILE;   // 16-key tiles of a unit
constexpr int kManyPerSm = 1;

template <int D, bool WIDE>
struct Many {
  using L = KvTile<D>;
  static constexpr int kRows = WIDE ? kManyTile : 2 * kManyTile;   // of an item
  // an item's start and end, in units' time: some 20000 cycles of 2100 (WIDE: 4000 a unit, 2500 where 64
  // wide).  4096 tokens on 4096 keys: 6 175 us, 8 156, 10 152, 12 155, 16 157
  static constexpr int kExtra = WIDE ? (D == 64 ? 8 : 4) : 10;
  static constexpr int kBufs = !WIDE || D == 64 ? 4 : D == 96 ? 3 : 2;   // restored units
  // With two buffers a key tile is free after its S, not after its O: the keys two units on are
  // restored while the rows work (with the pair as one, O(i) - restore - S(i + 2) - O(i + 1) were
  // a chain of 5000 cycles a unit).
  static constexpr bool kSplit = kBufs == 2;
  static constexpr int kLoaders = WIDE && D > 64 ? 8 : 6, kStages = WIDE && D > 64 ? 1 : 2;   // loader warps, places of a loader's ring
  static constexpr int kRowWarps = 8, kWarps = kRowWarps + kLoaders + 2, kThreads = 32 * kWarps;
  static constexpr int kTileWarps = WIDE ? 8 : 4;     // row warps of a row tile
  static constexpr int kQLbo = kManyTile * 16 + 16;   // bytes between 8-element columns (16, 32: bank offset)
  static constexpr int kQBytes = D / 8 * kQLbo;
  static constexpr int kKLbo = kManyKeys * 16 + 32;
  static constexpr int kKBytes = D / 8 * kKLbo;
  static constexpr int kVLbo = D * 16;                // bytes between 8-key columns
  static constexpr int kVBytes = kManyKeys / 8 * kVLbo;
  static constexpr int kHead = WIDE ? 3584 : 1024;    // barriers, flags, what the halves of a row exchange
  static constexpr int kQ = kHead, kKv = kQ + 2 * kQBytes;   // a buffer: K, V (WIDE: and their lo parts)
  static constexpr int kKvBytes = kKBytes + kVBytes;
  static constexpr int kBufBytes = WIDE ? 2 * kKvBytes : kKvBytes;
  static constexpr int kRing = kKv + kBufs * kBufBytes;   // tiles as they are stored
  static constexpr int kSmem = kRing + kLoaders * kStages * L::kBytes;
  static constexpr int kPartial = kManyTile * (D + 2);   // of a tile, floats: m, l, then [D / 4][rows][4]
  // tensor-memory columns: S of tile x, buffer i (and P over it); O of tile x (WIDE: of part x; both parts
  // of P over the first S)
  __host__ __device__ static constexpr uint32_t s_col(int x, int i) { return 128 * x + 64 * i; }
  __host__ __device__ static constexpr uint32_t o_col(int x) { return 256 + D * x; }
  static constexpr uint32_t kCols = 512;
  // log2 units: p is carried as p 2^kUp, and m raised where a score passes it by kSlack
  static constexpr float kUp = 11.f, kSlack = 4.f;
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
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void sts_u4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// A wait that gives up when another role has
__device__ __forceinline__ bool many_wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
  const auto passed = [&] {   // sleeps up to 2 us in the barrier
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(2000u)
        : "memory");
    return ok != 0;
  };
  if (mbar_try_wait(bar, parity)) return true;   // (the form without a time is the faster)
  const long long t0 = clock64();
  for (;;) {
    if (passed()) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitCycles) return false;
  }
}

// The barrier of a tile's row warps: whether `ok` holds in all of them
template <int THREADS>
__device__ __forceinline__ bool rows_agree(int tile, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok), "r"(1 + tile), "n"(THREADS)
      : "memory");
  return r != 0;
}
// The barrier of the two warps that share 32 rows: how many of their lanes say yes
__device__ __forceinline__ uint32_t pair_count(int quarter, bool yes) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.popc.u32 %0, %2, 64, p;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)yes), "r"(3 + quarter)
      : "memory");
  return r;
}

// Rows 2 p0 .. 2 p1 - 1 of a warp's 32 rows of Q into rows 32 quarter .. of the
// operand tile, each scaled by 2^-e and given the sign of `scale` (so that the
// largest product is the largest score); WIDE: lo 2^11 goes to the tile at
// `to_lo` (fp16 queries are their hi parts, and e = 0).  Two rows at a time, a
// lane eight elements (whole lines: a lane per row took 16 times the tag lookups
// and bounded an item's start).  q + row_at is this lane's row, 0 where row_at
// < 0.  Returns 2^e of this lane's row, if it is one of these.
template <int D, class T, bool VEC, bool WIDE>
__device__ __forceinline__ float many_query(const T* q, int64_t row_at, float scale, uint32_t to, uint32_t to_lo,
                                            int quarter, int lane, int p0, int p1) {
  constexpr bool kHalf = std::is_same_v<T, __half>;
  constexpr int kW = sizeof(T) * 2;                                          // words of 8 elements
  constexpr int kBatch = sizeof(T) == 4 ? 4 : 8;   // rows on their way at once
  const int half = lane >> 4, o = lane & 15;
  const uint32_t sign = __float_as_uint(scale) & 0x80000000u;
  float mine = 1.f;
#pragma unroll 1
  for (int i0 = p0; i0 < p1; i0 += kBatch) {
    uint32_t y[kBatch][kW];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t at = __shfl_sync(0xFFFFFFFFu, row_at, 2 * (i0 + i) + half);
#pragma unroll
      for (int j = 0; j < kW; ++j) y[i][j] = 0u;
      if (at >= 0 && o < D / 8) {
        const T* p = q + at + 8 * o;
        if constexpr (VEC) {
#pragma unroll
          for (int j = 0; j < kW; j += 4) {
            const uint4 u = *reinterpret_cast<const uint4*>(p + j * (4 / sizeof(T)));
            y[i][j] = u.x; y[i][j + 1] = u.y; y[i][j + 2] = u.z; y[i][j + 3] = u.w;
          }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
          for (int j = 0; j < 8; ++j) y[i][j] = __float_as_uint(p[j]);
        } else {
          const uint16_t* e = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = e[2 * j] | (uint32_t)e[2 * j + 1] << 16;
        }
      }
    }
    // the rows' largest magnitudes, by their bits, side by side (bf16: two at once)
    uint32_t top[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      top[i] = 0;
#pragma unroll
      for (int j = 0; j < kW && !kHalf; ++j)
        top[i] = sizeof(T) == 4 ? max(top[i], y[i][j] & 0x7FFFFFFFu) : __vmaxu2(top[i], y[i][j] & 0x7FFF7FFFu);
    }
#pragma unroll
    for (int d = 8; d && !kHalf; d >>= 1)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t z = __shfl_xor_sync(0xFFFFFFFFu, top[i], d);
        top[i] = sizeof(T) == 4 ? max(top[i], z) : __vmaxu2(top[i], z);
      }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // pair j: elements j and j + 4
      uint32_t hi[4], lo[4];
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int j = 0; j < 4; ++j) hi[j] = __byte_perm(y[i][j / 2], y[i][2 + j / 2], j % 2 ? 0x7632 : 0x5410);
      }
      if constexpr (kHalf) {
#pragma unroll
        for (int j = 0; j < 4; ++j) hi[j] ^= sign | sign >> 16;
      } else {
        const uint32_t m = sizeof(T) == 4 ? top[i] : max(top[i] << 16, top[i] & 0xFFFF0000u);
        int e = (int)(m >> 23) - 127;
        e = e < -100 ? -100 : (e > 126 ? 126 : e);
        const float up = __shfl_sync(0xFFFFFFFFu, __uint_as_float((uint32_t)(127 + e) << 23), (lane & 1) << 4);
        if (lane >> 1 == i0 + i) mine = up;
        const float down = __uint_as_float((uint32_t)(127 - e) << 23 | sign);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 z;
          if constexpr (sizeof(T) == 4) z = make_float2(__uint_as_float(y[i][j]), __uint_as_float(y[i][j + 4]));
          else z = make_float2(__uint_as_float(hi[j] << 16), __uint_as_float(hi[j] & 0xFFFF0000u));
          z = mul2(z, make_float2(down, down));
          if constexpr (WIDE) split2<2048>(z.x, z.y, hi[j], lo[j]);
          else hi[j] = h2bits(__floats2half2_rn(z.x, z.y));
        }
      }
      const int row = 2 * (i0 + i) + half;
      const uint32_t at = (uint32_t)(o * Many<D, WIDE>::kQLbo + (4 * quarter + row / 8) * 128 + (row % 8) * 16);
      if (o < D / 8) {
        sts_u4(to + at, hi[0], hi[1], hi[2], hi[3]);
        if constexpr (WIDE && !kHalf) sts_u4(to_lo + at, lo[0], lo[1], lo[2], lo[3]);
      }
    }
  }
  return mine;
}

// sc c + mn of a pair of codes, as one rounded fp16 pair or as two parts
template <bool WIDE>
__device__ __forceinline__ void restore(uint32_t c, uint32_t sc, uint32_t mn, uint32_t& hi, uint32_t& lo) {
  if constexpr (WIDE) {
    const float2 x = fma2(h2f(c), h2f(sc), h2f(mn));
    split2<2048>(x.x, x.y, hi, lo);
  } else {
    hi = fma_h2(c, sc, mn);
  }
}

// One lane of a converged warp
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A loader lane's share of a 16-key tile as it is stored: keys lane / 4 and 8
// more, elements 32 g + 8 (lane % 4) + 0..7; values of keys 8 h .. 8 h + 7
// (h = lane / 16), groups g0 .. g0 + GW - 1, elements 32 g + 4 (lane % 8) + 0..3.
template <int D>
struct ManyRaw {
  using L = KvTile<D>;
  static constexpr int G = L::G, GW = (G + 1) / 2;
  uint32_t kc[2][G], ks[2][G], km[2][L::GP / 2], vc[4][GW], vs[4][GW], vm[4][GW];

  __device__ __forceinline__ void read(uint32_t s, int lane) {
    const int q = lane & 3, n = lane & 7, h = lane >> 4, g0 = GW * (lane >> 3 & 1);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tk = 8 * i + lane / 4;
      lds_words<G>(s + L::kKeyCodes + ((tk * 4 + q) * G) * 4, kc[i]);
      lds_words<G>(s + L::kKeyScale + (tk / 2 * G) * 4, ks[i]);
      lds_words<L::GP / 2>(s + L::kKeyMin + (tk * L::GP) * 2, km[i]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int p = 4 * h + j;   // pair of keys
      if constexpr (G % 2 == 0) {
        lds_words<GW>(s + L::kValCodes + ((p * 8 + n) * G + g0) * 4, vc[j]);
        lds_words<GW>(s + L::kValScale + (p * G + g0) * 4, vs[j]);
        lds_words<GW>(s + L::kValMin + (p * G + g0) * 4, vm[j]);
      } else {
#pragma unroll
        for (int i = 0; i < GW; ++i) {
          const int g = g0 + i < G ? g0 + i : G - 1;   // (the group past the last is not stored)
          vc[j][i] = lds_u32(s + L::kValCodes + ((p * 8 + n) * G + g) * 4);
          vs[j][i] = lds_u32(s + L::kValScale + (p * G + g) * 4);
          vm[j][i] = lds_u32(s + L::kValMin + (p * G + g) * 4);
        }
      }
    }
  }
};

// Groups (a bit each) with a NaN under one of a unit's keys from kb on that a row of
// keys [lo, hi) sees; keys: [tile][group], a bit a key.  Rare, and kept out of the
// row warps' loop, whose registers are short.
template <int G>
__device__ __noinline__ uint8_t many_nan_groups(const volatile uint16_t* keys, uint32_t tiles, int kb, int lo, int hi) {
  uint32_t groups = 0;
#pragma unroll 1
  for (int i = 0; i < 4 * kManyUnit; ++i) {
    const int key = kb + i / 4 * LW_KV_TILE;
    if (i % 4 >= G || !(tiles >> (8 * (i / 4)) & 2u)) continue;
    uint32_t bits = keys[i];
    bits &= lo <= key ? 0xFFFFu : lo >= key + 16 ? 0u : 0xFFFFu << (lo - key);
    bits &= hi >= key + 16 ? 0xFFFFu : hi <= key ? 0u : (1u << (hi - key)) - 1u;
    if (bits) groups |= 1u << (i % 4);
  }
  return (uint8_t)groups;
}

// Barriers of a CTA.  Those of a row tile are one per S buffer, so that the use
// before the one waited for is always complete (a parity names one of two).
struct ManyBars {
  uint64_t kv_full[4], kv_free[4];                       // per operand buffer (kSplit: k full, v free)
  uint64_t v_full[2], k_free[2];                         // kSplit
  uint64_t q_full[2], s_full[2][2], p_full[2][2], o_done[2][2];   // per row tile (and S buffer)
  uint64_t last[2];                                      // everything issued has completed
  uint64_t ring[12];                                     // [loader][place]
};

template <int D, bool WIDE>
__global__ void __launch_bounds__(Many<D, WIDE>::kThreads, kManyPerSm) kv_many_kernel(const AttnArgs a) {
  using F = Many<D, WIDE>;
  constexpr int kRows = F::kRows, kBufs = F::kBufs, kLoaders = F::kLoaders, kStages = F::kStages;
  constexpr bool kSplit = F::kSplit;
  static_assert(!kSplit || WIDE, "a tile without rows lets its buffers go as pairs");
  static_assert(kLoaders * kStages <= 12, "ring barriers");
  using L = KvTile<D>;
  constexpr int G = L::G;
  extern __shared__ __align__(128) uint8_t smem[];
  ManyBars& bar = *reinterpret_cast<ManyBars*>(smem);
  static_assert(sizeof(ManyBars) <= 512, "barriers");
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(smem + 512);   // [0] abort, [1], [2] last part of a tile's item
  uint32_t* tslot = reinterpret_cast<uint32_t*>(smem + 528);   // tensor memory
  // [unit % 4][tile]: 1: the tile's keys are there, 2: some of them have a NaN in a value group that
  // is masked here (written before kv_full, read after s_full; four units on, the rows have answered)
  volatile uint8_t* present = smem + 544;
  // [unit % 4][tile][group]: those keys, a bit each.  A row that does not see such a key must not get
  // its NaN by way of V (0 x NaN), so V has zeros there and the rows that do see it set the group's
  // outputs at the end.
  volatile uint16_t* nan_keys = reinterpret_cast<volatile uint16_t*>(smem + 576);
  volatile uint8_t* nan_row = smem + 704 + threadIdx.x;   // a row thread's groups with a NaN under a key that it sees
  float* xch = reinterpret_cast<float*>(smem + 1024);   // WIDE: [2][rows], [rows] 2^e of Q, [2][rows] sums
  constexpr int kIssuer = F::kRowWarps + kLoaders;      // the first of the two
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&bar.kv_full[i], kLoaders);
      mbar_init(&bar.kv_free[i], 2);   // both tiles' products
      if (kSplit) {
        mbar_init(&bar.v_full[i], kLoaders);
        mbar_init(&bar.k_free[i], 2);
      }
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bar.last[x], 1);
      mbar_init(&bar.q_full[x], F::kTileWarps);
      mbar_init(&bar.s_full[x][0], 1);
      mbar_init(&bar.s_full[x][1], 1);
      mbar_init(&bar.p_full[x][0], F::kTileWarps);
      mbar_init(&bar.p_full[x][1], F::kTileWarps);
      mbar_init(&bar.o_done[x][0], 1);
      mbar_init(&bar.o_done[x][1], 1);
    }
    for (int i = 0; i < 12; ++i) mbar_init(&bar.ring[i], 1);
    flags[0] = 0;
    fence_barrier_init();
  }
  if (warp == kIssuer) {
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
  const bool any = kv_range<F::kThreads, kRows, kManyUnit, F::kExtra>(a, w, Gc, U, q0);
  bool ok = true;   // no wait ran out

  if (any && warp >= F::kRowWarps && warp < kIssuer) {   // ---- loaders
    const int lw = warp - F::kRowWarps;
    constexpr int GW = ManyRaw<D>::GW;
    uint32_t it0 = 0;                 // units before this item
    FewFetch<D, kLoaders, 1, kStages> t;
    t.bars = bar.ring + lw * kStages;
    t.ring = smem + F::kRing + lw * kStages * L::kBytes;
    t.parity = t.have = 0;
    for (bool more = true; more && ok;) {
      const int base = w.span.lo + w.k0 * kManyUnit, count = (w.k1 - w.k0) * kManyUnit;
      t.begin(a, w, base + lw, base + count, lane);
      // rows of the item all see the keys [all_lo, all_hi)
      int all_lo, all_hi, x;
      {
        int t1 = (w.rt * kRows + kRows - 1) / a.group;
        if (t1 > w.T - 1) t1 = w.T - 1;
        kv_token_keys(w.T, w.n, w.rt * kRows / a.group, a.p.causal, a.p.window, x, all_hi);
        kv_token_keys(w.T, w.n, t1, a.p.causal, a.p.window, all_lo, x);
      }
      // Every loader takes its turn in every unit, also in one without a tile of its own: the unit
      // is full when all have, so that none is ever a phase of a barrier ahead or behind.
      int o = lw;   // this warp's next tile (the last unit may run past the span)
      for (int i = 0; ok && i < count / kManyUnit; ++i) {
        const uint32_t it = it0 + i, buf = it % kBufs;
        const uint32_t turn = (it / kBufs & 1u) ^ 1u;   // the buffer is free
        if (o >= (i + 1) * kManyUnit) {
          if (kSplit) {
            ok = __all_sync(0xFFFFFFFFu, many_wait(&bar.k_free[buf], turn, flags));
            if (lane == 0) mbar_arrive(&bar.kv_full[buf]);
            if (!ok) break;
          }
          ok = __all_sync(0xFFFFFFFFu, many_wait(&bar.kv_free[buf], turn, flags));
          if (lane == 0) mbar_arrive(kSplit ? &bar.v_full[buf] : &bar.kv_full[buf]);
          continue;
        }
        const int sub = o - i * kManyUnit;
        const bool there = t.have >> t.out & 1u;
        const int kb = (base + o) * LW_KV_TILE;
        const bool edge = kb < all_lo || kb + LW_KV_TILE > all_hi;
        const int q = lane & 3, n = lane & 7, h = lane >> 4, g0 = GW * (lane >> 3 & 1);
        ManyRaw<D> r;
        if (there) {
          if (!t.wait()) { ok = false; mbar_wait(&t.bars[t.out], (t.parity >> t.out & 1u) ^ 1u); break; }
          r.read(smem_addr(t.ring) + t.out * L::kBytes, lane);
          fence_proxy_async();   // (these reads before the copy that follows)
          __syncwarp();
        }
        if (base + o < w.span.hi) {
          t.out = t.out + 1 == kStages ? 0 : t.out + 1;
          t.send(a, lane);
        }
        if (!there) {   // no keys: S is masked, and V has to be finite
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < GW; ++i) r.vc[j][i] = r.vs[j][i] = r.vm[j][i] = 0;
        }
        ok = __all_sync(0xFFFFFFFFu, many_wait(kSplit ? &bar.k_free[buf] : &bar.kv_free[buf], turn, flags));
        if (!ok) break;
        const uint32_t kto = smem_addr(smem) + F::kKv + buf * F::kBufBytes + (uint32_t)(sub * 256 + (lane / 4) * 16 + q * F::kKLbo);
        const uint32_t vto = smem_addr(smem) + F::kKv + buf * F::kBufBytes + F::kKBytes +
                             (uint32_t)((sub * 2 + h) * F::kVLbo + n * 16 + g0 * 512);
        if (there) {
          const uint32_t half = lane & 4 ? 0x3232u : 0x1010u;   // key 2 j or 2 j + 1
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              const uint32_t sc = __byte_perm(r.ks[i][g], 0, half);
              const uint32_t mn = __byte_perm(r.km[i][g / 2], 0, g % 2 ? 0x3232u : 0x1010u);
              const uint32_t w0 = r.kc[i][g], w1 = r.kc[i][g] >> 8, to = kto + (uint32_t)(i * 128 + 4 * g * F::kKLbo);
              uint32_t hi[4], lo[4];
              restore<WIDE>(whole_even(w0), sc, mn, hi[0], lo[0]);
              restore<WIDE>(whole_odd(w0), sc, mn, hi[1], lo[1]);
              restore<WIDE>(whole_even(w1), sc, mn, hi[2], lo[2]);
              restore<WIDE>(whole_odd(w1), sc, mn, hi[3], lo[3]);
              sts_u4(to, hi[0], hi[1], hi[2], hi[3]);
              if (WIDE) sts_u4(to + F::kKvBytes, lo[0], lo[1], lo[2], lo[3]);
            }
        }
        bool nans = false;
        if (there && edge) {
          uint32_t bad[GW] = {}, some = 0;   // keys with a NaN scale, as bits of the tile
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int key = kb + 2 * (4 * h + j);
#pragma unroll
            for (int i = 0; i < GW; ++i) {
              const uint32_t z = r.vs[j][i];
              const bool n0 = (z & 0x7FFFu) > 0x7C00u, n1 = (z & 0x7FFF0000u) > 0x7C000000u;
              const uint32_t keep = (key < w.n && !n0 ? 0xFFFFu : 0u) | (key + 1 < w.n && !n1 ? 0xFFFF0000u : 0u);
              r.vs[j][i] &= keep;
              r.vm[j][i] &= keep;
              bad[i] |= ((uint32_t)(key < w.n && n0) | (uint32_t)(key + 1 < w.n && n1) << 1) << (2 * (4 * h + j));
              some |= bad[i];
            }
          }
          nans = __any_sync(0xFFFFFFFFu, some != 0);
          if (nans) {
#pragma unroll
            for (int i = 0; i < GW; ++i) {   // the two halves of the warp have 8 keys each of the same groups
              bad[i] |= __shfl_xor_sync(0xFFFFFFFFu, bad[i], 16);
              if (lane < 16 && lane % 8 == 0 && g0 + i < G)
                nan_keys[(it % 4 * kManyUnit + sub) * 4 + g0 + i] = (uint16_t)bad[i];
            }
            __syncwarp();
          }
        }
        if (lane == 0) present[it % 4 * kManyUnit + sub] = nans ? 3 : there;
        if (kSplit) {
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.kv_full[buf]);
          ok = __all_sync(0xFFFFFFFFu, many_wait(&bar.kv_free[buf], turn, flags));
          if (!ok) break;
        }
#pragma unroll
        for (int i = 0; i < GW; ++i) {
          if (G % 2 && g0 + i >= G) continue;
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            uint32_t e[4], o[4], el[4], ol[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              restore<WIDE>(whole_even(r.vc[j][i] >> (8 * st)), r.vs[j][i], r.vm[j][i], e[j], el[j]);
              restore<WIDE>(whole_odd(r.vc[j][i] >> (8 * st)), r.vs[j][i], r.vm[j][i], o[j], ol[j]);
            }
            const uint32_t to = vto + (uint32_t)(i * 512 + (2 * st) * 128);
            sts_u4(to, e[0], e[1], e[2], e[3]);
            sts_u4(to + 128, o[0], o[1], o[2], o[3]);
            if (WIDE) {
              sts_u4(to + F::kKvBytes, el[0], el[1], el[2], el[3]);
              sts_u4(to + F::kKvBytes + 128, ol[0], ol[1], ol[2], ol[3]);
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(kSplit ? &bar.v_full[buf] : &bar.kv_full[buf]);
        o += kLoaders;
      }
      it0 += w.k1 - w.k0;
      if (ok) more = kv_advance<kRows, kManyUnit, F::kExtra>(a, w, q0);
    }
    if (!ok) {
      flags[0] = 1;
      if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
      for (int i = 0; i < kStages; ++i)   // no copy may be in flight when the CTA ends
        if (t.have >> i & 1u) mbar_wait(&t.bars[i], t.parity >> i & 1u);
    }
  } else if (any && warp >= kIssuer) {   // ---- issuers
    const auto uniform = [](int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); };
    const auto wait = [&](uint64_t* b, bool parity) { return __all_sync(0xFFFFFFFFu, many_wait(b, parity, flags)) != 0; };
    const int x = uniform(warp - kIssuer);   // row tile (WIDE: 0 the hi products, 1 the lo ones)
    const int xr = WIDE ? 0 : x;                      // whose rows
    const uint32_t tm = uniform(tmem), base = smem_addr(smem);
    const uint64_t qd = sdesc(base + F::kQ + x * F::kQBytes, F::kQLbo, 128);
    int buf = 0, sbuf = 0;   // operand and S buffer of the item's first unit
    uint32_t kvph = 0, vph = 0, qph = 0;    // phases of kv_full and v_full (a bit a buffer) and q_full
    uint32_t pph = 0, oph = 0, used = 0;    // of p_full and o_done, and whether the place has held a P (a bit an S buffer)
    const bool q_lo = WIDE && a.p.dtype == LW_F32;   // (fp16 queries are their hi parts)
    for (bool more = true; more && ok;) {
      const bool mine = WIDE || uniform(w.T * a.group - w.rt * kRows > x * kManyTile);
      const int n = uniform(w.k1 - w.k0);
      // S for the item's i-th unit, over the P of two units before
      const auto issue_s = [&](int i) {
        const int kv = (buf + i) % kBufs, sb = (sbuf + i) & 1;
        if (!wait(&bar.kv_full[kv], kvph >> kv & 1u)) return false;
        kvph ^= 1u << kv;
        if (i == 0) {
          if (!wait(&bar.q_full[xr], qph)) return false;
          qph ^= 1u;
        }
        if (used >> sb & 1u) {
          if (!wait(&bar.o_done[x][sb], oph >> sb & 1u)) return false;
          if (WIDE && x == 0 && !wait(&bar.o_done[1][sb], oph >> sb & 1u)) return false;   // (reads P too)
          oph ^= 1u << sb;
        }
        used |= 1u << sb;
        tc_fence_after();
        const uint64_t kd = sdesc(base + F::kKv + kv * F::kBufBytes, F::kKLbo, 128);
        const uint32_t d = tm + F::s_col(x, sb);
        if (elect_one()) {
          if (!WIDE || x == 0) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              umma_bf16(d, qd + (2 * s * F::kQLbo >> 4), kd + (2 * s * F::kKLbo >> 4), idesc_f16(kManyKeys), s > 0);
          } else {
            const uint64_t qh = qd - (F::kQBytes >> 4), kl = kd + (F::kKvBytes >> 4);
#pragma unroll
            for (int s = 0; s < D / 16; ++s)
              umma_bf16(d, qh + (2 * s * F::kQLbo >> 4), kl + (2 * s * F::kKLbo >> 4), idesc_f16(kManyKeys), s > 0);
            if (q_lo) {
#pragma unroll
              for (int s = 0; s < D / 16; ++s)
                umma_bf16(d, qd + (2 * s * F::kQLbo >> 4), kd + (2 * s * F::kKLbo >> 4), idesc_f16(kManyKeys), 1);
            }
          }
          umma_commit(&bar.s_full[x][sb]);
          if (kSplit) umma_commit(&bar.k_free[kv]);
        }
        __syncwarp();
        return true;
      };
      const auto issue_o = [&](int i) {   // O += P V
        const int kv = (buf + i) % kBufs, sb = (sbuf + i) & 1;
        if (kSplit) {
          if (!wait(&bar.v_full[kv], vph >> kv & 1u)) return false;
          vph ^= 1u << kv;
        }
        if (!wait(&bar.p_full[xr][sb], pph >> sb & 1u)) return false;
        pph ^= 1u << sb;
        tc_fence_after();
        const uint64_t vd = sdesc(base + F::kKv + kv * F::kBufBytes + F::kKBytes, F::kVLbo, 128);
        const uint32_t d = tm + F::o_col(x), p = tm + F::s_col(xr, sb);
        if (elect_one()) {
          const uint64_t v = vd + (WIDE && x ? F::kKvBytes >> 4 : 0);
#pragma unroll
          for (int s = 0; s < kManyKeys / 16; ++s)
            umma_bf16_ta(d, p + 8 * s, v + (2 * s * F::kVLbo >> 4), idesc_f16(D), i > 0 || s > 0);
          if (WIDE && x) {
#pragma unroll
            for (int s = 0; s < kManyKeys / 16; ++s)
              umma_bf16_ta(d, p + 32 + 8 * s, vd + (2 * s * F::kVLbo >> 4), idesc_f16(D), 1);
          }
          umma_commit(&bar.o_done[x][sb]);
          umma_commit(&bar.kv_free[kv]);
        }
        __syncwarp();
        return true;
      };
      if (mine) {
        ok = issue_s(0) && (n == 1 || issue_s(1));
#pragma unroll 1
        for (int i = 0; ok && i < n; ++i) ok = issue_o(i) && (i + 2 >= n || issue_s(i + 2));
      } else {   // no rows here: only let the buffers go
#pragma unroll 1
        for (int i = 0; ok && i < n; ++i) {
          const int kv = (buf + i) % kBufs;
          ok = wait(&bar.kv_full[kv], kvph >> kv & 1u);
          kvph ^= 1u << kv;
          if (lane == 0) mbar_arrive(&bar.kv_free[kv]);
          __syncwarp();
        }
      }
      buf = (buf + n) % kBufs;
      sbuf = (sbuf + n) & 1;
      if (ok) more = uniform(kv_advance<kRows, kManyUnit, F::kExtra>(a, w, q0));
    }
    if (!ok) {
      flags[0] = 1;
      if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
    }
    __syncwarp();
    if (elect_one()) umma_commit(&bar.last[x]);   // no product may be in flight when the tensor memory goes
    __syncwarp();
    mbar_wait(&bar.last[x], 0);
  } else if (any) {   // ---- rows
    // Tile and row of this thread.  WIDE: two threads a row, this one has keys 32 hf .. 32 hf + 31 of a unit.
    const int x = WIDE ? 0 : warp / 4, hf = WIDE ? warp / 4 : 0, quarter = warp % 4, row = threadIdx.x % kManyTile;
    constexpr int kMine = WIDE ? 32 : 64;   // keys of a unit
    constexpr int kTileThreads = 32 * F::kTileWarps;
    const uint32_t mine = tmem + ((uint32_t)(32 * quarter) << 16);   // this warp's quarter
    uint32_t it = 0;     // units of the CTA; S lies in buffer it % 2
    uint32_t used = 0;   // a bit an S buffer: how often this tile has used it, mod 2 (the phase of its
                         // next s_full; its last o_done has the other)
    struct Row { int tok, hq, lo, hi; bool live; };
    const auto find = [&](const KvWalk& v) {
      const int r = v.rt * kRows + x * kManyTile + row;
      Row y;
      y.live = r < v.T * a.group;
      y.tok = y.live ? r / a.group : v.T - 1;
      y.hq = v.h * a.group + (y.live ? r - y.tok * a.group : 0);
      kv_token_keys(v.T, v.n, y.tok, a.p.causal, a.p.window, y.lo, y.hi);
      return y;
    };
    const auto tile_there = [&](const KvWalk& v) { return v.rt * kRows + x * kManyTile < v.T * a.group; };
    float f = 0.f;   // log2 units per unit of S
    const auto load_q = [&](const Row& y, int s0) {
      const int64_t at = y.live ? (int64_t)(s0 + y.tok) * a.p.q_token_stride + (int64_t)y.hq * a.p.q_head_stride : -1;
      const uint32_t to = smem_addr(smem) + F::kQ + x * F::kQBytes;
      const auto read = [&](auto* q) {   // the rows, by their type
        using T = std::remove_const_t<std::remove_pointer_t<decltype(q)>>;
        const int p0 = WIDE ? 8 * hf : 0, p1 = WIDE ? p0 + 8 : 16;
        return a.vec ? many_query<D, T, true, WIDE>(q, at, a.p.scale, to, to + F::kQBytes, quarter, lane, p0, p1)
                     : many_query<D, T, false, WIDE>(q, at, a.p.scale, to, to + F::kQBytes, quarter, lane, p0, p1);
      };
      float e2;
      if constexpr (!WIDE) e2 = read(static_cast<const __nv_bfloat16*>(a.p.q));
      else e2 = a.p.dtype == LW_F16 ? read(static_cast<const __half*>(a.p.q)) : read(static_cast<const float*>(a.p.q));
      if constexpr (WIDE) {   // the other half's rows
        if (lane / 16 == hf) xch[2 * kManyTile + row] = e2;
        pair_count(quarter, true);
        e2 = xch[2 * kManyTile + row];
      }
      // (never 0: a masked score times it stays -inf)
      f = fmaxf(fabsf(a.p.scale) * 1.4426950408889634f * e2, 1e-37f);
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full[x]);
    };
    Row y = find(w);
    if (tile_there(w)) load_q(y, q0);
    for (bool more = true; more;) {
      const KvWalk v = w;
      const int vq0 = q0;
      more = kv_advance<kRows, kManyUnit, F::kExtra>(a, w, q0);
      if (!tile_there(v)) {   // a short row tile: the other warps' alone
        it += v.k1 - v.k0;
        if (more) {
          y = find(w);
          if (tile_there(w)) load_q(y, q0);
        }
        continue;
      }
      // keys that every row of the tile sees
      int all_lo, all_hi, u0;
      {
        const int r0 = v.rt * kRows + x * kManyTile;
        int t1 = (r0 + kManyTile - 1) / a.group;
        if (t1 > v.T - 1) t1 = v.T - 1;
        kv_token_keys(v.T, v.n, r0 / a.group, a.p.causal, a.p.window, u0, all_hi);
        kv_token_keys(v.T, v.n, t1, a.p.causal, a.p.window, all_lo, u0);
      }
      float m = -INFINITY, mu = -F::kUp, l = 0.f;   // the maximum, the same (or 0) less kUp, sum of p 2^kUp
      *nan_row = 0;
      for (int k = v.k0; k < v.k1; ++k, ++it) {
        const int kb = (v.span.lo + k * kManyUnit) * LW_KV_TILE;
        const int b = it & 1;
        const uint32_t sc = mine + F::s_col(x, b) + 32 * hf;
        if (ok) ok = many_wait(&bar.s_full[x][b], used >> b & 1u, flags);
        if (WIDE && ok) ok = many_wait(&bar.s_full[1][b], used >> b & 1u, flags);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!WIDE && !ok) break;
        tc_fence_after();
        const uint32_t tiles = *reinterpret_cast<const volatile uint32_t*>(present + it % 4 * kManyUnit);
        const uint32_t there = tiles >> (16 * hf) & (WIDE ? 0xFFFFu : 0xFFFFFFFFu);
        if (tiles & 0x02020202u)   // (both halves of a row look at all of its keys)
          *nan_row |= many_nan_groups<G>(nan_keys + it % 4 * 4 * kManyUnit, tiles, kb, y.lo, y.hi);
        uint32_t s0[32], s1[32];   // WIDE: the scores are s0 (s1 brings the lo parts' sum)
        tmem_ld32(sc, s0);
        if constexpr (!WIDE) tmem_ld32(sc + 32, s1);
        else tmem_ld32(mine + F::s_col(1, b) + 32 * hf, s1);
        tmem_ld_wait();
        if constexpr (WIDE) {   // and the lo parts' sum
          const float2 down = make_float2(4.8828125e-4f, 4.8828125e-4f);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 t = fma2(make_float2(__uint_as_float(s1[j]), __uint_as_float(s1[j + 1])), down,
                                  make_float2(__uint_as_float(s0[j]), __uint_as_float(s0[j + 1])));
            s0[j] = __float_as_uint(t.x);
            s0[j + 1] = __float_as_uint(t.y);
          }
        }
        const int ka = kb + 32 * hf;   // this thread's first key
        if (ka < all_lo || ka + kMine > all_hi || there != (WIDE ? 0x0101u : 0x01010101u)) {
#pragma unroll
          for (int j = 0; j < kMine; ++j) {
            const bool in = there >> (8 * (j / 16)) & 1u;
            if (!(in && ka + j >= y.lo && ka + j < y.hi)) (j < 32 ? s0[j % 32] : s1[j % 32]) = 0xFF800000u;
          }
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          top = fmaxf(top, __uint_as_float(s0[j]));
          if (!WIDE) top = fmaxf(top, __uint_as_float(s1[j]));
        }
        top *= f;
        bool raise = __any_sync(0xFFFFFFFFu, top > m + F::kSlack);
        if constexpr (WIDE) {   // Both halves or none, also of an end: a wait that ran out counts 32, a raise 1.
          // (And both have read S, so that P may go over it.)
          const uint32_t say = pair_count(quarter, !ok || (raise && lane == 0));
          if (say >= 32) {
            ok = false;
            break;
          }
          raise = say != 0;
          if (raise) {
            xch[hf * kManyTile + row] = top;
            pair_count(quarter, true);
            top = fmaxf(top, xch[(hf ^ 1) * kManyTile + row]);
          }
        }
        if (raise) {
          const float mx = fmaxf(m, top);
          mu = mx == -INFINITY ? 0.f : mx;
          const float al = ex2(m - mu);
          mu -= F::kUp;
          m = mx;
          l *= al;
          if (k > v.k0) {   // once the sum over the keys before is complete
            const bool ph = (used >> (b ^ 1) & 1u) ^ 1u;
            ok = many_wait(&bar.o_done[x][b ^ 1], ph, flags) && (!WIDE || many_wait(&bar.o_done[1][b ^ 1], ph, flags));
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!WIDE && !ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int d = 0; ok && d < D; d += 32) {   // (WIDE: the hi parts' sum one half, the lo parts' the other)
              uint32_t z[32];
              tmem_ld32(mine + F::o_col(x + hf) + d, z);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) z[j] = __float_as_uint(__uint_as_float(z[j]) * al);
              tmem_st32(mine + F::o_col(x + hf) + d, z);
            }
          }
        }
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 f2 = make_float2(f, f), mu2 = make_float2(-mu, -mu);
        // (the parts of p go where the scores were)
#pragma unroll
        for (int j = 0; j < kMine / 2; ++j) {
          uint32_t* s = j < 16 ? s0 + 2 * j : s1 + 2 * (j - 16);
          const float2 t = fma2(make_float2(__uint_as_float(s[0]), __uint_as_float(s[1])), f2, mu2);
          const float2 z = make_float2(ex2(t.x), ex2(t.y));
          sum[j % 2] = add2(sum[j % 2], z);
          if constexpr (WIDE) split2<2048>(z.x, z.y, s[0], s[1]);
          else s[0] = h2bits(__floats2half2_rn(z.x, z.y));
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if constexpr (!WIDE) {
          uint32_t p[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) p[j] = j < 16 ? s0[2 * j] : s1[2 * (j - 16)];
          tmem_st32(sc, p);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // hi parts, lo parts
            uint32_t p[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) p[j] = s0[2 * j + h];
            tmem_st16(mine + F::s_col(x, b) + 32 * h + 16 * hf, p);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[x][b]);
        used ^= 1u << b;
      }
      // (every S of this item is complete: Q's place is free)
      const Row o = y;
      if constexpr (WIDE) {   // (the halves stay together; and their sums)
        float* sums = xch + 3 * kManyTile;
        sums[hf * kManyTile + row] = l;
        ok = pair_count(quarter, ok) == 64;
        l = sums[row] + sums[kManyTile + row];
      }
      if (more) {
        y = find(w);
        if (ok && tile_there(w)) load_q(y, q0);
      }
      {
        const int b = (it - 1) & 1;
        if (ok) ok = many_wait(&bar.o_done[x][b], (used >> b & 1u) ^ 1u, flags);
        if (WIDE && ok) ok = many_wait(&bar.o_done[1][b], (used >> b & 1u) ^ 1u, flags);
      }
      ok = rows_agree<kTileThreads>(x, ok);   // all warps of the tile go on to the barriers below, or none
      if (!ok) break;
      tc_fence_after();
      const bool whole = v.k0 == 0 && v.k1 == v.units;
      float* part = a.partials + (((size_t)blockIdx.x * 2 + (v.k0 == 0)) * 2 + x) * F::kPartial;
      const auto give = [&](int g, float l, const float (&z)[32]) {   // 32 elements of the row, [i][n]
        if (!o.live) return;
        const float inv = 1.f / l;
        const int64_t at = (int64_t)(vq0 + o.tok) * a.p.out_token_stride + (int64_t)o.hq * a.p.out_head_stride + 32 * g;
#pragma unroll
        for (int n = 0; n < 8; n += 2) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = l == 0.f ? 0.f : z[8 * (i % 4) + n + i / 4] * inv;
          store8(a, at + 4 * n, y);
        }
      };
      const auto give_lse = [&](float m, float l) {
        if (hf == 0 && o.live && a.p.lse)
          a.p.lse[(int64_t)(vq0 + o.tok) * a.p.q_heads + o.hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
      };
#pragma unroll 1
      for (int g = hf; g < G; g += F::kTileWarps / 4) {
        uint32_t u[32];
        float z[32];
        tmem_ld32(mine + F::o_col(x) + 32 * g, u);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(u[j]);
        if constexpr (WIDE) {
          tmem_ld32(mine + F::o_col(1) + 32 * g, u);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = fmaf(__uint_as_float(u[j]), 4.8828125e-4f, z[j]);
        }
        if (*nan_row >> g & 1) {
#pragma unroll
          for (int j = 0; j < 32; ++j) z[j] = __uint_as_float(0x7FFFFFFFu);
        }
        if (whole) {
          give(g, l, z);
        } else if (o.live) {
#pragma unroll
          for (int n = 0; n < 8; ++n)
            *reinterpret_cast<float4*>(part + 2 * kManyTile + ((8 * g + n) * kManyTile + row) * 4) =
                make_float4(z[n], z[8 + n], z[16 + n], z[24 + n]);
        }
      }
      tc_fence_before();
      if (whole) {
        give_lse(m - F::kUp, l);
      } else {
        if (hf == 0) {
          part[row] = m - F::kUp;   // (the parts' sums are relative to this)
          part[kManyTile + row] = l;
        }
        const int c0 = kv_owner(v.first, U, Gc), parts = kv_owner(v.first + v.units - 1, U, Gc) - c0 + 1;
        __threadfence();
        rows_agree<kTileThreads>(x, true);
        if (row == 0 && hf == 0) {
          const bool last = atomicAdd(a.counters + 2 * c0 + x, 1u) == (uint32_t)parts - 1u;
          if (last) a.counters[2 * c0 + x] = 0;
          flags[1 + x] = last;
        }
        rows_agree<kTileThreads>(x, true);
        if (flags[1 + x]) {
          __threadfence();
          const auto from = [&](int i) {
            return a.partials + ((i ? (size_t)(c0 + i) * 2 : (size_t)c0 * 2 + 1) * 2 + x) * F::kPartial;
          };
          float M = -INFINITY, S = 0.f;
          for (int i = 0; i < parts; ++i) M = fmaxf(M, __ldcg(from(i) + row));
          const float Mu = M == -INFINITY ? 0.f : M;
          for (int i = 0; i < parts; ++i) S = fmaf(__ldcg(from(i) + kManyTile + row), ex2(__ldcg(from(i) + row) - Mu), S);
#pragma unroll 1
          for (int g = hf; o.live && g < G; g += F::kTileWarps / 4) {
            float z[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) z[j] = 0.f;
#pragma unroll 1
            for (int i = 0; i < parts; ++i) {
              const float* p = from(i);
              const float e = ex2(__ldcg(p + row) - Mu);
#pragma unroll
              for (int n = 0; n < 8; ++n) {
                const float4 y = __ldcg(reinterpret_cast<const float4*>(p + 2 * kManyTile + ((8 * g + n) * kManyTile + row) * 4));
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
        rows_agree<kTileThreads>(x, true);
      }
    }
    if (!ok) {
      flags[0] = 1;
      if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kIssuer) tmem_dealloc(tmem, F::kCols);
}

}  // namespace dev
}  // namespace lw
