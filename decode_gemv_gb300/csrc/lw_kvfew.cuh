// Cache attention for few rows: the query tokens of a sequence times the
// heads that share a key/value head fit one row tile of a warp-wide matrix
// instruction (single tokens, drafted tokens).
//
// Mathematics.  With a cached key k_d = sc_g c_d + mn_g (group g of 32) and
// q' = q / 2^e (2^e the row's magnitude),
//   q.k = 2^e ( sum_g sc_g sum_{d in g} q'_d c_d  +  sum_g mn_g sum_{d in g} q'_d ),
// and with v_jd = sc_jg (c_jd - 8) + mid_jg, mid = mn + 8 sc,
//   sum_j p_j v_jd = sum_j (p_j sc_jg) (c_jd - 8) + sum_j p_j mid_jg.
// So the codes themselves are the matrix operands (exact: a 4-bit integer is
// a subnormal fp16, c 2^-24, by masking alone; MODE 0 makes it normal first,
// because the instruction aligns a subnormal's products by its least exponent
// and drops what falls below: 1e-5 of the result), the scales enter in fp32
// after the key product and in p before the value product, and the minimums
// take one further matrix instruction each.  The values' codes are centred
// because both sums would otherwise be some 2 sqrt(n) times their difference:
// the matrix instruction's accumulation truncates, and 9000 keys lost 1.3e-4 to
// that.  The middles, not fp16 any more, go in as two parts in MODE 0 (hi, lo).
//
// The key product has the rows as its first dimension (16 places), the value
// product as its second (8 columns a step): the first one's accumulator
// fragment is then the second one's operand fragment, and the accumulators of
// 8 rows of 128 values take 32 registers.  The operands q', its group sums,
// p sc and p are fp16: in MODE 0 (fp32 and fp16 calls, 8 rows) as two parts of
// 11 bits each -- q' = hi + lo 2^-11 in rows 0..7 and 8..15 of one instruction,
// p and p sc as hi + lo in two -- in MODE 1 (16 rows) and MODE 2 (8 rows) one part,
// for bf16 calls: q is exact there (down to 2^-13 of the row's largest element),
// its group sums are in two parts (the lower ones in the instruction's other 8 places,
// against the same minimums: one part moved a score by 2e-3 where minimums are large),
// and p and p sc rounded to 11 bits are 8 times finer than the output's 8.  p is
// carried as p 2^15 and p sc as p sc 2^(15 + x) with x by the largest scale so
// far, so that both end just below fp16's largest number: a p of 2^-29 of the
// row's largest then still has 11 bits (in units of 1 all of the keys beside one
// that dominates its row were lost: 1e-2 of the result).  Products
// accumulate in fp32, in MODE 0 for kFewFlush tiles before they are added to
// shared memory rounded to nearest (the truncation of many steps is a drift,
// not a scatter).
//
// Structure.  A CTA walks its range of units (lw_kvplan.h).  Its warps take the
// 16-key tiles in turn, fetched by bulk copies into a ring of their own, and each
// keeps its own running maximum, sum and accumulators (one pass over the data)
// until the item ends; then the next item's first tiles are sent for, and the
// warps' states are joined in shared memory.  An item cut between CTAs leaves
// partial states in the workspace, and the CTA that brings the item's count to
// its end joins them, in CTA order (the answer does not depend on the order of
// arrival).
//
// Bound by instruction issue where keys are many: a tile of 16 keys is 250
// instructions, and they issue in 53 % of the slots (waits on the matrix
// instructions' results, 4 warps a scheduler).  8 sequences of 65536 keys, 8 heads
// of 128 with 4 query heads each: bf16 157 us (0.67 GB of cache, 4.3 TB/s), fp32
// 205 us.  At 128 registers a thread the 128-wide forms spill: 40 to 124 bytes with
// items of 8 rows, 720 with 16 (253 us where 8 rows take 157; two items of 8 are no
// faster).  Bound by latency where they are few: 37 keys 7.5 us, 4097 keys of one
// sequence 15 us (a launch, the search of the range, a tile a warp, the join of up to
// 32 parts a head: each a chain of loads; 8 heads of weight 39 on 304 CTAs leave
// 48 CTAs an item's front alone, without a unit).
#pragma once

#include "lw_kvattn.cuh"

namespace lw {

constexpr int kFewFlush = 32;                       // tiles between two additions (MODE 0)
constexpr int kFewExtra = 6;                        // an item's start and end, in units' time (lw_kvplan.h)

template <int D, int MODE>
struct Few {
  using L = KvTile<D>;
  // 16 warps an SM, as the registers allow.  Four CTAs of 4 warps instead of two
  // of 8: 256 sequences of 100 keys 43 -> 36 us, but 38 of 8192 94 -> 104 us and
  // one of 4097 15 -> 18 us (more items cut, more parts to join); 20 warps of 96
  // registers: 8 of 65536 159 -> 264 us (spills).
  static constexpr int kWarps = 8, kPerSm = 2, kThreads = 32 * kWarps;
  // tiles a warp takes at once: two where their operands fit the registers
  // (8 sequences of 65536 keys, 64 wide: 104 -> 93 us; 128 wide 157 -> 196 us)
  static constexpr int kPair = D == 64 ? 2 : 1;
  static constexpr int kStages = D == 64 ? 2 : 3;    // places of a warp's ring
  static constexpr int kUnit = kWarps * kPair;       // tiles of a unit
  static constexpr int kRows = MODE == 1 ? 16 : 8;   // rows of an item
  static constexpr int kJoin = MODE == 0 ? 8 : 4;    // of them joined at a time
  static constexpr int kRing = 256;                  // after the barriers and the flag
  static constexpr int kSums = kRing + kWarps * kStages * kPair * L::kBytes;   // [warps][kJoin][D]
  static constexpr int kState = kSums + kWarps * kJoin * D * 4;           // m, l [warps][8]
  static constexpr int kNeed = kState + 2 * kWarps * 8 * 4;
  // above the limit that holds without an attribute (static shared memory counts towards it)
  static constexpr int kSmem = kNeed > 49168 ? kNeed : 49168;
  static constexpr int kPartial = kRows * (D + 2);   // floats: m, l, then the rows
};

namespace dev {

// Place of element d (a multiple of 4) of row r among a warp's 8 rows in shared
// memory: the four rows that a quarter of a warp stores at once fall on
// different banks.
template <int D>
__device__ __forceinline__ int few_place(int r, int d) { return r * D + (d ^ ((r & 6) * 4)); }

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// the same with a zero accumulator
__device__ __forceinline__ void mma_f16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x = hi + lo / up: the fp16 pairs of two values
template <int UP>
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 up = make_float2(UP, UP), f = mul2(__half22float2(h), make_float2(-UP, -UP));
  const float2 d = fma2(make_float2(x, y), up, f);   // exact
  hi = h2bits(h);
  lo = h2bits(__floats2half2_rn(d.x, d.y));
}
template <int N>
__device__ __forceinline__ void lds_words(uint32_t at, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 u = lds_u4(at);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else if constexpr (N == 2) {
    const uint2 u = lds_u2(at);
    w[0] = u.x; w[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = lds_u32(at + 4 * i);   // 3 words, or one
  }
}
// the value operands: (c - 8) 2^-10 of the nibbles 0, 4 and 1, 5
__device__ __forceinline__ uint32_t centre_even(uint32_t w) { return fma_h2(w & 0x000F000Fu, 0x74007400u, 0xA000A000u); }
__device__ __forceinline__ uint32_t centre_odd(uint32_t w) { return fma_h2(w & 0x00F000F0u, 0x64006400u, 0xA000A000u); }
// the key operands: c 2^-10 in MODE 0, else c 2^-24 and c 2^-20
template <int MODE>
__device__ __forceinline__ uint32_t code_even(uint32_t w) {
  return MODE == 0 ? fma_h2(w & 0x000F000Fu, 0x74007400u, 0u) : w & 0x000F000Fu;
}
template <int MODE>
__device__ __forceinline__ uint32_t code_odd(uint32_t w) {
  return MODE == 0 ? fma_h2(w & 0x00F000F0u, 0x64006400u, 0u) : w & 0x00F000F0u;
}

// 8 consecutive elements of a query row, fp32
__device__ __forceinline__ void load_q8(const AttnArgs& a, int64_t at, float (&x)[8]) {
  if (a.p.dtype == LW_F32) {
    const float* p = static_cast<const float*>(a.p.q) + at;
    if (a.vec) kv_load8<float, true>(p, x); else kv_load8<float, false>(p, x);
  } else if (a.p.dtype == LW_F16) {
    const __half* p = static_cast<const __half*>(a.p.q) + at;
    if (a.vec) kv_load8<__half, true>(p, x); else kv_load8<__half, false>(p, x);
  } else {
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.p.q) + at;
    if (a.vec) kv_load8<__nv_bfloat16, true>(p, x); else kv_load8<__nv_bfloat16, false>(p, x);
  }
}

// One row's operands and running state in a lane (quad lane q holds the
// elements 32 g + 8 q + 0..7).
struct FewRow {
  float f;          // log2 units per unit of the scaled product
  int lo, hi;       // keys it sees
  float m, mu, l;   // running maximum (log2 units), the same (or 0) less 15, sum of p 2^15
};

template <int D, int MODE>
struct FewWarp {
  using L = KvTile<D>;
  static constexpr int G = L::G, NR = MODE == 1 ? 2 : 1;
  static constexpr float kUp = 15.f, kDown = 3.0517578125e-5f;   // 2^-15
  uint32_t aq[G][2][MODE == 2 ? 2 : 4];   // query operands: step, (a0, a2) or a0..a3
  uint32_t am[2];   // group sums, two parts (MODE 1: [part][row] in shared memory, registers are short)
  FewRow row[NR];
  // value sums: [g][s]: elements 32 g + 4 (lane / 4) + 2 s, + 1 (registers 0, 1
  // and 2, 3) of rows 2 q, 2 q + 1 (and 8 more for the second NR); om: sums of
  // the middles of group lane / 4 (hi parts; lane / 4 - 4: lo parts)
  float o[NR][G][2][4], om[NR][4];
  float unit;       // 2^(-15 - x): om and l are of p 2^15, o of p sc 2^(15 + x)
  uint32_t limit;   // largest scale that x covers, twice (fp16)
  float fm;         // row[0].m when the sums last went to shared memory (MODE 0)

  // Row r of the row tile (lane / 4, and lane / 4 + 8 in MODE 1)
  __device__ void load_row(const AttnArgs& a, const KvWalk& w, int q0, int rt_rows, int which, int lane,
                           uint32_t* sums) {
    const int q = lane % 4, r = w.rt * rt_rows + lane / 4 + 8 * which;
    float x[G][8], top = 0.f;
    const bool live = r < w.T * a.group;
    const int t = live ? r / a.group : w.T - 1;
    if (live) {
      const int64_t at = (int64_t)(q0 + t) * a.p.q_token_stride +
                         (int64_t)(w.h * a.group + r - t * a.group) * a.p.q_head_stride + 8 * q;
#pragma unroll
      for (int g = 0; g < G; ++g) load_q8(a, at + 32 * g, x[g]);
    } else {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[g][i] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[g][i]));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    int e = (int)(__float_as_uint(top) >> 23) - 127;
    e = e < -100 ? -100 : (e > 126 ? 126 : e);
    // 2^-e, with the sign of the scale: the largest product is the largest score
    const float down = __uint_as_float((uint32_t)(127 - e) << 23 | (__float_as_uint(a.p.scale) & 0x80000000u));
    FewRow& s = row[which];
    // products carry the codes' power of two and 2^-e
    // (never 0: a masked score times it stays -inf)
    s.f = fmaxf(fabsf(a.p.scale) * 1.4426950408889634f * (MODE == 0 ? 1024.f : 16777216.f) *
                    __uint_as_float((uint32_t)(127 + e) << 23), 1e-37f);
    kv_token_keys(w.T, w.n, t, a.p.causal, a.p.window, s.lo, s.hi);
    s.m = -INFINITY;
    s.mu = -kUp;
    s.l = 0.f;
    float sum[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[g][i] *= down;
        z += x[g][i];
      }
      z += __shfl_xor_sync(0xFFFFFFFFu, z, 1);
      sum[g] = z + __shfl_xor_sync(0xFFFFFFFFu, z, 2);
#pragma unroll
      for (int st = 0; st < 2; ++st) {   // nibbles 2 st, 2 st + 4; then 2 st + 1, 2 st + 5
        constexpr float kOdd = MODE == 0 ? 1.f : 0.0625f;
        const float u0 = x[g][2 * st], u1 = x[g][2 * st + 4];
        const float v0 = x[g][2 * st + 1] * kOdd, v1 = x[g][2 * st + 5] * kOdd;
        if constexpr (MODE == 0) {
          split2<2048>(u0, u1, aq[g][st][0], aq[g][st][1]);
          split2<2048>(v0, v1, aq[g][st][2], aq[g][st][3]);
        } else if constexpr (MODE == 1) {
          aq[g][st][which] = h2bits(__floats2half2_rn(u0, u1));
          aq[g][st][2 + which] = h2bits(__floats2half2_rn(v0, v1));
        } else {
          aq[g][st][0] = h2bits(__floats2half2_rn(u0, u1));
          aq[g][st][1] = h2bits(__floats2half2_rn(v0, v1));
        }
      }
    }
    float s0 = 0.f, s1 = 0.f;   // groups 2 q, 2 q + 1
#pragma unroll
    for (int g = 0; g < G; ++g) {
      if (g == 2 * q) s0 = sum[g];
      if (g == 2 * q + 1) s1 = sum[g];
    }
    if constexpr (MODE == 0) split2<2048>(s0, s1, am[0], am[1]);
    else if constexpr (MODE == 1) split2<1>(s0, s1, sums[4 * lane + which], sums[4 * lane + 2 + which]);
    else split2<1>(s0, s1, am[0], am[1]);
  }

  // sums: MODE 1: 512 bytes of shared memory, the warp's until its first put
  __device__ void start(const AttnArgs& a, const KvWalk& w, int q0, int rt_rows, int lane, uint32_t* sums) {
#pragma unroll
    for (int i = 0; i < NR; ++i) load_row(a, w, q0, rt_rows, i, lane, sums);
    clear();
    follow(0);
    fm = -INFINITY;
  }
  // x for scales up to `top` (fp16 bits): p sc 2^(15 + x) below 2^15, and above 2^14 for the largest.
  // With one part x = 0 does where that is above 2^9 (scales from 2^-6 to 1, as a rule): the floor of
  // fp16 then lies at 2^-34 of the row's largest p.
  __device__ __forceinline__ void follow(uint32_t top) {
    top = min(top, 0x7BFFu);
    const int bit = 31 - __clz(top | 1u);
    int e = top < 0x400u ? bit - 24 : (int)(top >> 10) - 15;   // top in [2^e, 2^(e + 1))
    uint32_t most = top < 0x400u ? (2u << bit) - 1u : top | 0x3FFu;
    if constexpr (MODE != 0) {
      if (e >= -6 && e < 0) {
        e = -1;
        most = 0x3BFFu;
      }
      e = e < -16 ? -16 : e;   // (2^x is an fp16)
    }
    unit = __uint_as_float((uint32_t)(127 - 15 + 1 + e) << 23);   // x = -1 - e
    limit = most * 0x10001u;
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < NR; ++i) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[i][g][0][j] = o[i][g][1][j] = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) om[i][j] = 0.f;
    }
  }

  // NT tiles of 16 keys, keys kb .. kb + 16 NT - 1.  EDGE: some row does not see
  // some of them (those may hold any bits).
  template <bool EDGE, int NT>
  __device__ __forceinline__ void tiles(uint32_t s, int kb, int n, int lane, uint32_t sums) {
    const int q = lane % 4, r = lane / 4;
    uint4 m4;
    if constexpr (MODE == 1) m4 = lds_u4(sums + 16 * lane);
    float2 t[NT][NR][2];   // scores: keys 2 q, 2 q + 1 of the tile, and 8 more
    uint32_t see[NT][NR];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {   // 8 keys each
        const uint32_t at = s + (uint32_t)(i * L::kBytes);
        float c[4];
        uint32_t mn = 0;
        if (2 * q < L::GP) mn = lds_u32(at + L::kKeyMin + (uint32_t)((8 * h + r) * L::GP + 2 * q) * 2);
        if (G % 2 && q == G / 2) mn &= 0xFFFFu;
        if constexpr (MODE == 0) mma_f16_zero(c, am[0], am[1], 0u, 0u, mn, 0u);
        else if constexpr (MODE == 1) mma_f16_zero(c, m4.x, m4.y, m4.z, m4.w, mn, mn);
        else mma_f16_zero(c, am[0], 0u, am[1], 0u, mn, mn);
        constexpr float kUnit = MODE == 0 ? 9.765625e-4f : 5.9604644775390625e-8f;   // as the codes' products
        float2 x = mul2(make_float2(c[0], c[1]), make_float2(kUnit, kUnit));
        float2 y = mul2(make_float2(c[2], c[3]), make_float2(kUnit, kUnit));
        uint32_t kw[G], sw[G];
        lds_words<G>(at + L::kKeyCodes + (uint32_t)(((8 * h + r) * 4 + q) * G) * 4, kw);
        lds_words<G>(at + L::kKeyScale + (uint32_t)((4 * h + q) * G) * 4, sw);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          float d[4];
          const uint32_t w = kw[g] >> 8;
          if constexpr (MODE == 2) {
            mma_f16_zero(d, aq[g][0][0], 0u, aq[g][0][1], 0u, code_even<MODE>(kw[g]), code_odd<MODE>(kw[g]));
            mma_f16(d, aq[g][1][0], 0u, aq[g][1][1], 0u, code_even<MODE>(w), code_odd<MODE>(w));
          } else {
            mma_f16_zero(d, aq[g][0][0], aq[g][0][1], aq[g][0][2], aq[g][0][3], code_even<MODE>(kw[g]),
                         code_odd<MODE>(kw[g]));
            mma_f16(d, aq[g][1][0], aq[g][1][1], aq[g][1][2], aq[g][1][3], code_even<MODE>(w), code_odd<MODE>(w));
          }
          const float2 sc = h2f(sw[g]);
          x = fma2(sc, make_float2(d[0], d[1]), x);
          if constexpr (MODE != 2) y = fma2(sc, make_float2(d[2], d[3]), y);
        }
        if constexpr (MODE == 0) x = fma2(y, make_float2(4.8828125e-4f, 4.8828125e-4f), x);   // 2^-11
        t[i][0][h] = x;
        if constexpr (NR == 2) t[i][NR - 1][h] = y;
      }
    bool up = false;
    float top[NR];
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      top[j] = -INFINITY;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if constexpr (EDGE) {
          see[i][j] = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int key = kb + 16 * i + 8 * (u / 2) + 2 * q + u % 2;
            float& z = u % 2 ? t[i][j][u / 2].y : t[i][j][u / 2].x;
            if (key >= row[j].lo && key < row[j].hi) see[i][j] |= 1u << u;
            else z = -INFINITY;
          }
        }
        top[j] = fmaxf(fmaxf(top[j], t[i][j][0].x), t[i][j][0].y);
        top[j] = fmaxf(fmaxf(top[j], t[i][j][1].x), t[i][j][1].y);
      }
      top[j] *= row[j].f;
      up |= top[j] > row[j].m;
    }
    // the value operands' unit covers the largest scale so far (a NaN is none: the maximum leaves it out)
    uint32_t big = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t at = s + (uint32_t)(i * L::kBytes + L::kValScale);
      uint32_t s0[G], s1[G];
      lds_words<G>(at + (uint32_t)(q * G) * 4, s0);
      lds_words<G>(at + (uint32_t)((q + 4) * G) * 4, s1);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if constexpr (EDGE) {
          s0[g] = cut(s0[g], kb + 16 * i + 2 * q, n);
          s1[g] = cut(s1[g], kb + 16 * i + 8 + 2 * q, n);
        }
        big = max_h2(big, max_h2(s0[g], s1[g]));
      }
    }
    up |= max_h2(big, limit) != limit;
    if (__any_sync(0xFFFFFFFFu, up)) {   // a new maximum: rescale
      float al[NR];
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        float x = top[j];
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
        x = fmaxf(x, row[j].m);
        const float mu = x == -INFINITY ? 0.f : x;
        al[j] = ex2(row[j].m - mu);
        row[j].m = x;
      }
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) big = max_h2(big, __shfl_xor_sync(0xFFFFFFFFu, big, d));
      big = max_h2(big, limit);
      const float before = unit;
      follow(max(big & 0x7FFFu, big >> 16));
      const float down = before * __uint_as_float(0x7F000000u - __float_as_uint(unit));
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        row[j].l *= al[j];
        // (p 2^15 comes out of the exponential)
        row[j].mu = (row[j].m == -INFINITY ? 0.f : row[j].m) - kUp;
        // to the lanes that hold the rows' sums
        const float a0 = __shfl_sync(0xFFFFFFFFu, al[j], 8 * q), a1 = __shfl_sync(0xFFFFFFFFu, al[j], 8 * q + 4);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float x = u % 2 ? a1 : a0;
          om[j][u] *= x;
          const float y = x * down;
#pragma unroll
          for (int g = 0; g < G; ++g) {
            o[j][g][0][u] *= y;
            o[j][g][1][u] *= y;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t at = s + (uint32_t)(i * L::kBytes);
      float2 p[NR][2];        // p 2^15
      uint32_t ph[NR][2];     // the same in fp16
#pragma unroll
      for (int j = 0; j < NR; ++j) {
        const float2 f2 = make_float2(row[j].f, row[j].f), mu2 = make_float2(-row[j].mu, -row[j].mu);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float2 z = fma2(t[i][j][h], f2, mu2);
          p[j][h] = make_float2(ex2(z.x), ex2(z.y));
          ph[j][h] = h2bits(__floats2half2_rn(p[j][h].x, p[j][h].y));
        }
        row[j].l += (p[j][0].x + p[j][0].y) + (p[j][1].x + p[j][1].y);
      }
      if constexpr (MODE == 0) {   // middles: rows of this instruction are groups, hi parts, then lo parts
        uint32_t a0 = 0, a2 = 0;
        if (r % 4 < G) {
          const auto middle = [&](int pair, int key) {
            const float2 mn = h2f(lds_u32(at + L::kValMin + (uint32_t)(pair * G + r % 4) * 4));
            const float2 sc = h2f(lds_u32(at + L::kValScale + (uint32_t)(pair * G + r % 4) * 4));
            float x = fmaf(8.f, sc.x, mn.x), y = fmaf(8.f, sc.y, mn.y);
            if constexpr (EDGE) {   // 0 x a masked key's bits has to be 0; a NaN group's scale shows it
              if (key >= n || isnan(x)) x = 0.f;
              if (key + 1 >= n || isnan(y)) y = 0.f;
            }
            uint32_t hi, lo;
            split2<2048>(x, y, hi, lo);
            return r < 4 ? hi : lo;
          };
          a0 = middle(q, kb + 16 * i + 2 * q);
          a2 = middle(q + 4, kb + 16 * i + 8 + 2 * q);
        }
        uint32_t b0, b1, c0, c1;
        split2<1>(p[0][0].x, p[0][0].y, b0, c0);
        split2<1>(p[0][1].x, p[0][1].y, b1, c1);
        mma_f16(om[0], a0, 0u, a2, 0u, c0, c1);
        mma_f16(om[0], a0, 0u, a2, 0u, b0, b1);
      } else {   // minimums and scales: rows 0..3 and 4..7; joined in fp32 tile by tile (their sums cancel)
        uint32_t a0 = 0, a2 = 0;
        if (r % 4 < G) {
          const uint32_t from = at + (r < 4 ? L::kValMin : L::kValScale) + (uint32_t)(r % 4) * 4;
          a0 = lds_u32(from + (uint32_t)(q * G) * 4);
          a2 = lds_u32(from + (uint32_t)((q + 4) * G) * 4);
          if constexpr (EDGE) {
            a0 = clean(cut(a0, kb + 16 * i + 2 * q, n));
            a2 = clean(cut(a2, kb + 16 * i + 8 + 2 * q, n));
          }
        }
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          float c[4];
          mma_f16_zero(c, a0, 0u, a2, 0u, ph[j][0], ph[j][1]);
          om[j][0] += fmaf(8.f, __shfl_down_sync(0xFFFFFFFFu, c[0], 16), c[0]);
          om[j][1] += fmaf(8.f, __shfl_down_sync(0xFFFFFFFFu, c[1], 16), c[1]);
        }
      }
      uint32_t v0[G], v1[G], s0[G], s1[G];
      lds_words<G>(at + L::kValScale + (uint32_t)(q * G) * 4, s0);
      lds_words<G>(at + L::kValScale + (uint32_t)((q + 4) * G) * 4, s1);
      lds_words<G>(at + L::kValCodes + (uint32_t)((q * 8 + r) * G) * 4, v0);
      lds_words<G>(at + L::kValCodes + (uint32_t)(((q + 4) * 8 + r) * G) * 4, v1);
      if (MODE == 0 || unit != kDown) {   // p 2^(15 + x)
        const float by = __uint_as_float(0x77800000u - __float_as_uint(unit));   // 2^x
        if constexpr (MODE == 0) {
          p[0][0] = mul2(p[0][0], make_float2(by, by));
          p[0][1] = mul2(p[0][1], make_float2(by, by));
        } else {
          const uint32_t by2 = h2bits(__float2half2_rn(by));
          if (by < 1.f) {
#pragma unroll
            for (int j = 0; j < NR; ++j) {
              ph[j][0] = mul_h2(ph[j][0], by2);
              ph[j][1] = mul_h2(ph[j][1], by2);
            }
          } else {   // (p has no room: the scales, exactly)
#pragma unroll
            for (int g = 0; g < G; ++g) {
              s0[g] = mul_h2(s0[g], by2);
              s1[g] = mul_h2(s1[g], by2);
            }
          }
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if constexpr (EDGE) {   // what lies past the end may be anything
          s0[g] = cut(s0[g], kb + 16 * i + 2 * q, n);
          s1[g] = cut(s1[g], kb + 16 * i + 8 + 2 * q, n);
        }
        uint32_t b0[NR], b1[NR], c0[NR], c1[NR];
#pragma unroll
        for (int j = 0; j < NR; ++j) {
          if constexpr (MODE == 0) {
            const float2 ux = mul2(p[j][0], h2f(s0[g])), uy = mul2(p[j][1], h2f(s1[g]));
            float u[4] = {ux.x, ux.y, uy.x, uy.y};
            if constexpr (EDGE) {   // a NaN that this row does not see
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (!(see[i][j] >> k & 1u)) u[k] = 0.f;
            }
            split2<1>(u[0], u[1], b0[j], c0[j]);
            split2<1>(u[2], u[3], b1[j], c1[j]);
          } else {
            b0[j] = mul_h2(ph[j][0], s0[g]);
            b1[j] = mul_h2(ph[j][1], s1[g]);
            if constexpr (EDGE) {
              b0[j] &= (see[i][j] & 1u ? 0xFFFFu : 0u) | (see[i][j] & 2u ? 0xFFFF0000u : 0u);
              b1[j] &= (see[i][j] & 4u ? 0xFFFFu : 0u) | (see[i][j] & 8u ? 0xFFFF0000u : 0u);
            }
          }
        }
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint32_t w0 = v0[g] >> (8 * st), w1 = v1[g] >> (8 * st);
          const uint32_t a0 = centre_even(w0), a1 = centre_odd(w0), a2 = centre_even(w1), a3 = centre_odd(w1);
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            if constexpr (MODE == 0) mma_f16(o[j][g][st], a0, a1, a2, a3, c0[j], c1[j]);
            mma_f16(o[j][g][st], a0, a1, a2, a3, b0[j], b1[j]);
          }
        }
      }
    }
  }

  // A pair of keys' halves, 0 past the end; the same without NaN
  static __device__ __forceinline__ uint32_t cut(uint32_t w, int key, int n) {
    return (key < n ? w & 0xFFFFu : 0u) | (key + 1 < n ? w & 0xFFFF0000u : 0u);
  }
  static __device__ __forceinline__ uint32_t clean(uint32_t w) {
    return ((w & 0x7FFFu) > 0x7C00u ? 0u : w & 0xFFFFu) | ((w & 0x7FFF0000u) > 0x7C000000u ? 0u : w & 0xFFFF0000u);
  }

  // This lane's elements 32 g + 4 (lane / 4) + 0..3 of row 2 q + e (and 8 which),
  // in true units
  __device__ __forceinline__ float4 finish(int which, int g, int e, int lane) const {
    // the lanes with this group's sums (MODE 0: and their lo parts) for rows 2 q, 2 q + 1
    float mn = __shfl_sync(0xFFFFFFFFu, om[which][e], 4 * g + lane % 4);
    if constexpr (MODE == 0)
      mn = fmaf(__shfl_sync(0xFFFFFFFFu, om[which][e], 16 + 4 * g + lane % 4), 4.8828125e-4f, mn);
    mn *= kDown;
    const float up = 1024.f * unit;
    return make_float4(fmaf(o[which][g][0][e], up, mn), fmaf(o[which][g][0][2 + e], up, mn),
                       fmaf(o[which][g][1][e], up, mn), fmaf(o[which][g][1][2 + e], up, mn));
  }

  // Put the sums of the 8 rows (8 `which` ..) into shared memory, or add them to
  // what it holds of them (MODE 0, after a flush); outside MODE 0 rows 4 part ..
  // 4 part + 3 alone.  at: the warp's rows there.
  __device__ __forceinline__ void put(int which, int part, int lane, float* at) const {
    const int q = lane % 4;
    const float held = MODE == 0 ? (fm == -INFINITY ? 0.f : ex2(fm - (row[0].m == -INFINITY ? 0.f : row[0].m))) : 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float h = MODE == 0 ? __shfl_sync(0xFFFFFFFFu, held, 8 * q + 4 * e) : 0.f;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int r = MODE == 0 ? 2 * q + e : 2 * (q & 1) + e;
        float4* to = reinterpret_cast<float4*>(at + few_place<D>(r, 32 * g + 4 * (lane / 4)));
        float4 x = finish(which, g, e, lane);
        if (MODE == 0 && h != 0.f) {
          const float4 y = *to;
          x = make_float4(fmaf(y.x, h, x.x), fmaf(y.y, h, x.y), fmaf(y.z, h, x.z), fmaf(y.w, h, x.w));
        }
        if (MODE == 0 || q / 2 == part) *to = x;
      }
    }
  }
  __device__ __forceinline__ void flush(int lane, float* at) {
    put(0, 0, lane, at);
    clear();
    fm = row[0].m;
  }
};

// Output rows r0..r0+7 of the item from unnormalised sums
template <int RT>
__device__ __forceinline__ void few_out(const AttnArgs& a, const KvWalk& w, int q0, int r, int d, float m,
                                        float l, float (&f)[4]) {
  const int rr = w.rt * RT + r;
  if (rr >= w.T * a.group) return;
  const int t = rr / a.group, hq = w.h * a.group + rr - t * a.group;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = l == 0.f ? 0.f : f[i] * inv;
  store4(a, (int64_t)(q0 + t) * a.p.out_token_stride + (int64_t)hq * a.p.out_head_stride + d, f);
  if (d == 0 && a.p.lse)
    a.p.lse[(int64_t)(q0 + t) * a.p.q_heads + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// A warp's tiles, N (1 or 2) neighbours at a time: sent for in order, STAGES
// ahead.  The table is read 32 tiles at a time, lane i holding where the i-th
// lies and sending for it.  STEP: tiles to the warp's next.
template <int D, int STEP, int N, int STAGES>
struct FewFetch {
  static constexpr int kTile = KvTile<D>::kBytes;
  static constexpr uint32_t kAll = (1u << N) - 1;
  uint8_t* ring;
  uint64_t* bars;
  const int32_t* table;    // the sequence's pages
  const uint8_t* src;      // this lane's tile, of the 32
  int64_t head;            // first byte of the head in a page
  int first, last;         // the item's tiles of this warp: first .. first + N - 1, then STEP on, below last
  int next, at;            // tile to send for; its place among the 32
  uint32_t there;          // which of the 32 have a page
  int in, out;             // ring places to fill and to use
  uint32_t have, parity;   // tiles sent for (N bits a place); phase per place

  __device__ __forceinline__ void lookup(const AttnArgs& a, int lane) {
    const int tile = next + lane / N * STEP + lane % N, tpp = a.page_tokens / LW_KV_TILE;
    const bool mine = tile < last;
    const int page = mine ? table[tile / tpp] : -1;
    const bool ok = page >= 0 && page < a.n_pages;
    if (mine && !ok) report(a.status, LW_DEV_BAD_PAGE);
    there = __ballot_sync(0xFFFFFFFFu, ok);
    src = a.pages + (int64_t)page * a.page_bytes + head + (tile % tpp) * kTile;
    at = 0;
  }
  // The warp's tiles of an item: from, from + STEP, ... below `to`
  __device__ __forceinline__ void begin(const AttnArgs& a, const KvWalk& w, int from, int to, int lane) {
    table = a.p.page_table + (int64_t)w.b * a.p.table_stride;
    head = (int64_t)w.h * (a.page_tokens / LW_KV_TILE) * kTile;
    next = first = from;
    last = to < w.span.hi ? to : w.span.hi;
    in = out = 0;
    have = 0;
    at = 32;
#pragma unroll
    for (int i = 0; i < STAGES; ++i) send(a, lane);
  }
  __device__ __forceinline__ void send(const AttnArgs& a, int lane) {
    if (next >= last) return;
    if (at == 32) lookup(a, lane);
    const uint32_t some = there >> at & kAll;
    if (some) {
      if (lane == at) mbar_arrive_expect_tx(&bars[in], (uint32_t)__popc(some) * kTile);
      __syncwarp();
      if ((lane ^ at) < N && (there >> lane & 1u))
        bulk_g2s(ring + (N * in + lane % N) * kTile, src, kTile, &bars[in]);
      have |= some << (N * in);
    }
    at += N;
    next += STEP;
    in = in + 1 == STAGES ? 0 : in + 1;
  }
  // The tiles at `out` have come (false: the wait ran out)
  __device__ __forceinline__ bool wait() {
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars[out], parity >> out & 1u));
    parity ^= 1u << out;
    have &= ~(kAll << (N * out));
    return ok;
  }
};

template <int D, int MODE>
__global__ void __launch_bounds__(Few<D, MODE>::kThreads, Few<D, MODE>::kPerSm) kv_few_kernel(const AttnArgs a) {
  using F = Few<D, MODE>;
  using L = KvTile<D>;
  constexpr int RT = F::kRows, W = F::kWarps, NT = F::kThreads, J = F::kJoin;
  extern __shared__ __align__(128) uint8_t smem[];
  // the current item and the next: one thread walks (registers are short)
  __shared__ KvWalk s_walk[2];
  __shared__ long long s_U;
  __shared__ int s_q0[2], s_more, s_G, s_last;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  FewFetch<D, F::kUnit, F::kPair, F::kStages> t;
  t.bars = reinterpret_cast<uint64_t*>(smem) + warp * F::kStages;
  t.ring = smem + F::kRing + warp * F::kStages * F::kPair * L::kBytes;
  t.parity = t.have = 0;
  if (lane == 0) {
    for (int i = 0; i < F::kStages; ++i) mbar_init(&t.bars[i], 1);
    fence_barrier_init();
  }
  __syncwarp();
  pdl_wait();
  {
    KvWalk w;
    int G, q0;
    long long U;
    if (!kv_range<NT, RT, F::kUnit, kFewExtra>(a, w, G, U, q0)) return;
    if (threadIdx.x == 0) {
      s_walk[0] = w;
      s_q0[0] = q0;
      s_G = G;
      s_U = U;
    }
    __syncthreads();
  }
  const auto begin = [&](const KvWalk& w) {
    t.begin(a, w, w.span.lo + w.k0 * F::kUnit + F::kPair * warp, w.span.lo + w.k1 * F::kUnit, lane);
  };

  FewWarp<D, MODE> f;
  bool dead = false;   // a wait ran out: reported, and only the barriers are kept up
  float* s_o = reinterpret_cast<float*>(smem + F::kSums);
  float* s_m = reinterpret_cast<float*>(smem + F::kState);
  float* s_l = s_m + W * 8;
  float* mine = s_o + warp * J * D;
  begin(s_walk[0]);
  for (int cur = 0;; cur ^= 1) {
    const KvWalk& w = s_walk[cur];
    if (threadIdx.x == NT - 32) {   // the item after, while this one's first tiles come
      KvWalk x = w;
      int q0 = s_q0[cur];
      s_more = kv_advance<RT, F::kUnit, kFewExtra>(a, x, q0);
      s_walk[cur ^ 1] = x;
      s_q0[cur ^ 1] = q0;
    }
    __syncwarp();
    f.start(a, w, s_q0[cur], RT, lane, reinterpret_cast<uint32_t*>(mine));
    // keys that every row of the item sees
    int all_lo, all_hi, x;
    {
      int t1 = (w.rt * RT + RT - 1) / a.group;
      if (t1 > w.T - 1) t1 = w.T - 1;
      kv_token_keys(w.T, w.n, w.rt * RT / a.group, a.p.causal, a.p.window, x, all_hi);
      kv_token_keys(w.T, w.n, t1, a.p.causal, a.p.window, all_lo, x);
    }
    int held = 0;
    for (int tile = t.first; tile < t.last && !dead; tile += F::kUnit) {
      const uint32_t some = t.have >> (F::kPair * t.out) & ((1u << F::kPair) - 1);
      if (some) {   // else their pages are missing
        if (!t.wait()) {
          dead = true;
          if (lane == 0) report(a.status, LW_DEV_TIMEOUT);
          mbar_wait(&t.bars[t.out], (t.parity >> t.out & 1u) ^ 1u);
          break;
        }
        if (MODE == 0 && held >= kFewFlush) {
          f.flush(lane, mine);
          held = 0;
        }
        const uint32_t at = smem_addr(t.ring) + F::kPair * t.out * L::kBytes;
        const int kb = tile * LW_KV_TILE;
        if (some == (1u << F::kPair) - 1 && kb >= all_lo && kb + F::kPair * LW_KV_TILE <= all_hi) {
          f.template tiles<false, F::kPair>(at, kb, w.n, lane, smem_addr(mine));
        } else {
#pragma unroll 1
          for (int i = 0; i < F::kPair; ++i)
            if (some >> i & 1u) f.template tiles<true, 1>(at + i * L::kBytes, kb + i * LW_KV_TILE, w.n, lane, smem_addr(mine));
        }
        held += F::kPair;
        fence_proxy_async();   // (this lane's reads before the copy that takes the place next, also the next item's)
        __syncwarp();
      }
      t.out = t.out + 1 == F::kStages ? 0 : t.out + 1;
      t.send(a, lane);
    }

    // join the warps, J rows at a time
    const bool whole = w.k0 == 0 && w.k1 == w.units;
    float* part = a.partials + ((size_t)blockIdx.x * 2 + (w.k0 == 0)) * F::kPartial;
#pragma unroll
    for (int i = 0; i < RT / J; ++i) {
      const int which = i * J / 8;
      if (i * J % 8 == 0) {
        float l = f.row[which].l * f.kDown;
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        if (lane % 4 == 0) {
          s_m[warp * 8 + lane / 4] = f.row[which].m;
          s_l[warp * 8 + lane / 4] = l;
        }
      }
      f.put(which, i * J % 8 / 4, lane, mine);
      __syncthreads();
      // the next item's first tiles, before this one's join
      if (i == 0 && s_more && !dead) begin(s_walk[cur ^ 1]);
      for (int j = threadIdx.x; j < J * (D / 4); j += NT) {
        const int r = j / (D / 4), d = 4 * (j % (D / 4)), r8 = i * J % 8 + r;
        float m = -INFINITY, sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < W; ++u) m = fmaxf(m, s_m[u * 8 + r8]);
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int u = 0; u < W; ++u) {
          const float e = ex2(s_m[u * 8 + r8] - mu);
          sum = fmaf(s_l[u * 8 + r8], e, sum);
          const float4 z = *reinterpret_cast<const float4*>(s_o + u * J * D + few_place<D>(r, d));
          y[0] = fmaf(z.x, e, y[0]);
          y[1] = fmaf(z.y, e, y[1]);
          y[2] = fmaf(z.z, e, y[2]);
          y[3] = fmaf(z.w, e, y[3]);
        }
        const int rr = i * J + r;
        if (whole) {
          few_out<RT>(a, w, s_q0[cur], rr, d, m, sum, y);
        } else {
          if (d == 0) {
            part[rr] = m;
            part[RT + rr] = sum;
          }
          *reinterpret_cast<float4*>(part + 2 * RT + rr * D + d) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
      __syncthreads();
    }
    if (!whole) {
      const int c0 = kv_owner(w.first, s_U, s_G), parts = kv_owner(w.first + w.units - 1, s_U, s_G) - c0 + 1;
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) {
        const bool last = atomicAdd(a.counters + c0, 1u) == (uint32_t)parts - 1u;
        if (last) a.counters[c0] = 0;
        s_last = last;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        const auto from = [&](int i) { return a.partials + (i ? (size_t)(c0 + i) * 2 : (size_t)c0 * 2 + 1) * F::kPartial; };
        // the parts' maxima and sums by way of shared memory, as far as they fit
        constexpr int kFit = W * J * D / (2 * RT);
        const bool fit = parts <= kFit;
        if (fit)
          for (int j = threadIdx.x; j < parts * 2 * RT; j += NT) s_o[j] = __ldcg(from(j / (2 * RT)) + j % (2 * RT));
        __syncthreads();
        for (int j = threadIdx.x; j < RT * (D / 4); j += NT) {
          const int r = j / (D / 4), d = 4 * (j % (D / 4));
          if (w.rt * RT + r >= w.T * a.group) continue;
          const auto state = [&](int i, int k) { return fit ? s_o[i * 2 * RT + k] : __ldcg(from(i) + k); };
          float m = -INFINITY, sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
          for (int i = 0; i < parts; ++i) m = fmaxf(m, state(i, r));
          const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 8
          for (int i = 0; i < parts; ++i) {
            const float4 z = __ldcg(reinterpret_cast<const float4*>(from(i) + 2 * RT + r * D + d));
            const float e = ex2(state(i, r) - mu);
            sum = fmaf(state(i, RT + r), e, sum);
            y[0] = fmaf(z.x, e, y[0]);
            y[1] = fmaf(z.y, e, y[1]);
            y[2] = fmaf(z.z, e, y[2]);
            y[3] = fmaf(z.w, e, y[3]);
          }
          few_out<RT>(a, w, s_q0[cur], r, d, m, sum, y);
        }
      }
      __syncthreads();
    }
    if (!s_more) break;
    __syncthreads();   // (all have read s_more and the item)
  }
  if (dead)   // no copy may be in flight when the CTA ends
    for (int i = 0; i < F::kStages; ++i)
      if (t.have >> (F::kPair * i) & ((1u << F::kPair) - 1)) mbar_wait(&t.bars[i], t.parity >> i & 1u);
}

}  // namespace dev
}  // namespace lw
