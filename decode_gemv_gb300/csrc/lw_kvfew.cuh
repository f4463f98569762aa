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
// and drops what falls below: 1e-5 of the result), the scales enter in fp32 after
// the key product and in p before the value product, and the minimums take one
// further matrix instruction each.  The values' codes are centred because both
// sums would otherwise be some 2 sqrt(n) times their difference: the matrix
// instruction's accumulation truncates, and 9000 keys lost 1.3e-4 to that.  The
// middles, not fp16 any more, take two columns each (hi, lo).  The other
// operands (q', its group sums, p sc, p) are fp16: in MODE 0 (fp32 and fp16
// calls) as two parts x = hi + lo 2^-11 of 11 bits each, hi in rows 0..7 and
// lo in rows 8..15 of the same instruction, which the rows of a single token
// leave free; in MODE 1 (16 rows) and MODE 2 (8 rows) hi alone, for bf16
// calls: q is exact there, and p rounded to 11 bits is 8 times finer than the
// output's 8.  Products accumulate in fp32, in MODE 0 for kFewFlush tiles
// before they are added to shared memory rounded to nearest (the truncation
// of many steps is a drift, not a scatter).
//
// Structure.  A CTA walks its range of units (lw_kvplan.h); a producer warp
// fills a ring of shared-memory stages with a unit's 16-key tiles by bulk
// copies, tile w for consumer warp w, which keeps its own running maximum,
// sum and accumulators (one pass over the data) until the item ends; then the
// warps' states are joined in shared memory.  An item cut between CTAs leaves
// partial states in the workspace, and the CTA that brings the item's count
// to its end joins them, in CTA order (the answer does not depend on the
// order of arrival).
#pragma once

#include "lw_kvattn.cuh"

namespace lw {

constexpr int kFewWarps = 8;                        // consumer warps = tiles of a unit
constexpr int kFewThreads = 32 * (kFewWarps + 1);
constexpr int kFewStages = 4;
constexpr int kFewFlush = 32;                       // tiles between two additions (MODE 0)

template <int D, int MODE>
struct Few {
  using L = KvTile<D>;
  static constexpr int kRows = MODE == 1 ? 16 : 8;   // rows of an item
  static constexpr int kStage = kFewWarps * L::kBytes;
  static constexpr int kPitch = D + 4;               // floats: conflict-free row writes
  static constexpr int kRing = 256;
  static constexpr int kJoin = kRing + kFewStages * kStage;
  static constexpr int kState = kJoin + kFewWarps * 8 * kPitch * 4;   // m, l [warps][8]
  static constexpr int kSmem = kState + 2 * kFewWarps * 8 * 4;
  static constexpr int kPartial = kRows * (D + 2);   // floats: m, l, then the rows
};

namespace dev {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t h2bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ float2 h2f(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
// x = hi + lo 2^-11: the fp16 pairs of two values
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = h2bits(h);
  lo = h2bits(__floats2half2_rn((x - f.x) * 2048.f, (y - f.y) * 2048.f));
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
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
    for (int i = 0; i < N; ++i) w[i] = lds_u32(at + 4 * i);
  }
}
__device__ __forceinline__ void few_bar() {   // the consumer warps
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kFewWarps) : "memory");
}

// x[i] * m + b in fp16 pairs; the operands are exact here
__device__ __forceinline__ uint32_t fma_h2(uint32_t x, uint32_t m, uint32_t b) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(x), "r"(m), "r"(b));
  return y;
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
  float m, mu, l;   // running maximum (log2 units), the same or 0, sum
};

template <int D, int MODE>
struct FewWarp {
  using L = KvTile<D>;
  static constexpr int G = L::G, NR = MODE == 1 ? 2 : 1;
  uint32_t aq[G][2][MODE == 2 ? 2 : 4];   // query operands: step, (a0, a2) or a0..a3
  uint32_t am[MODE == 2 ? 1 : 2];         // group sums
  FewRow row[NR];
  float o[G][4][4], om[4];
  float fm;         // row[0].m when the sums last went to shared memory (MODE 0)

  // Row r of the row tile (lane / 4, and lane / 4 + 8 in MODE 1)
  __device__ void load_row(const AttnArgs& a, const KvWalk& w, int q0, int rt_rows, int which, int lane) {
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
    const float down = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e
    FewRow& s = row[which];
    // products carry the codes' power of two and 2^-e
    s.f = a.p.scale * 1.4426950408889634f * (MODE == 0 ? 1024.f : 16777216.f) * __uint_as_float((uint32_t)(127 + e) << 23);
    kv_token_keys(w.T, w.n, t, a.p.causal, a.p.window, s.lo, s.hi);
    s.m = -INFINITY;
    s.mu = s.l = 0.f;
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
          split2(u0, u1, aq[g][st][0], aq[g][st][1]);
          split2(v0, v1, aq[g][st][2], aq[g][st][3]);
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
    if constexpr (MODE == 0) split2(s0, s1, am[0], am[1]);
    else am[which] = h2bits(__floats2half2_rn(s0, s1));
  }

  __device__ void start(const AttnArgs& a, const KvWalk& w, int q0, int rt_rows, int lane) {
#pragma unroll
    for (int i = 0; i < NR; ++i) load_row(a, w, q0, rt_rows, i, lane);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[g][i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) om[j] = 0.f;
    fm = -INFINITY;
  }

  // One tile of 16 keys, keys kb..kb+15.  EDGE: some row does not see some of
  // them (those may hold any bits).
  template <bool EDGE>
  __device__ __forceinline__ void tile(uint32_t s, int kb, int n, int lane) {
    const int q = lane % 4, r = lane / 4;
    float t[NR][4];
    uint32_t see[NR];
#pragma unroll
    for (int h = 0; h < 2; ++h) {   // 8 keys each
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      uint32_t mn = 0;
      if (2 * q < L::GP) mn = lds_u32(s + L::kKeyMin + (uint32_t)((8 * h + r) * L::GP + 2 * q) * 2);
      if (G % 2 && q == G / 2) mn &= 0xFFFFu;
      mma_f16(c, am[0], MODE == 2 ? 0u : am[MODE == 2 ? 0 : 1], 0u, 0u, mn, 0u);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] *= MODE == 0 ? 9.765625e-4f : 5.9604644775390625e-8f;   // as the codes' products
      uint32_t kw[G], sw[G];
      lds_words<G>(s + L::kKeyCodes + (uint32_t)(((8 * h + r) * 4 + q) * G) * 4, kw);
      lds_words<G>(s + L::kKeyScale + (uint32_t)((4 * h + q) * G) * 4, sw);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          const uint32_t w = kw[g] >> (8 * st);
          if constexpr (MODE == 2) mma_f16(d, aq[g][st][0], 0u, aq[g][st][1], 0u, code_even<MODE>(w), code_odd<MODE>(w));
          else mma_f16(d, aq[g][st][0], aq[g][st][1], aq[g][st][2], aq[g][st][3], code_even<MODE>(w), code_odd<MODE>(w));
        }
        const float2 sc = h2f(sw[g]);
        c[0] = fmaf(sc.x, d[0], c[0]);
        c[1] = fmaf(sc.y, d[1], c[1]);
        if constexpr (MODE != 2) {
          c[2] = fmaf(sc.x, d[2], c[2]);
          c[3] = fmaf(sc.y, d[3], c[3]);
        }
      }
      if constexpr (MODE == 0) {
        c[0] = fmaf(c[2], 4.8828125e-4f, c[0]);   // 2^-11
        c[1] = fmaf(c[3], 4.8828125e-4f, c[1]);
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        t[i][2 * h] = c[2 * i] * row[i].f;
        t[i][2 * h + 1] = c[2 * i + 1] * row[i].f;
      }
    }
    bool up = false;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if constexpr (EDGE) {
        see[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = kb + 8 * (j / 2) + 2 * q + j % 2;
          if (key >= row[i].lo && key < row[i].hi) see[i] |= 1u << j;
          else t[i][j] = -INFINITY;
        }
      }
      up |= fmaxf(fmaxf(t[i][0], t[i][1]), fmaxf(t[i][2], t[i][3])) > row[i].m;
    }
    if (__any_sync(0xFFFFFFFFu, up)) {   // some row has a new maximum: rescale
      float al[2];
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float x = fmaxf(fmaxf(t[i][0], t[i][1]), fmaxf(t[i][2], t[i][3]));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
        x = fmaxf(x, row[i].m);
        row[i].mu = x == -INFINITY ? 0.f : x;
        al[i] = ex2(row[i].m - row[i].mu);
        row[i].m = x;
        row[i].l *= al[i];
      }
      if (NR == 1) al[1] = al[0];
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < (MODE == 2 ? 2 : 4); ++j) o[g][i][j] *= al[j / 2];
#pragma unroll
      for (int j = 0; j < (MODE == 2 ? 2 : 4); ++j) om[j] *= al[j / 2];
    }
    float p[NR][4];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i][j] = ex2(t[i][j] - row[i].mu);
      row[i].l += (p[i][0] + p[i][1]) + (p[i][2] + p[i][3]);
    }
    // middles: columns of this instruction are groups, their hi parts, then their lo parts
    {
      uint32_t b0 = 0, b1 = 0, a0, a1 = 0, a2, a3 = 0;
      if (r % 4 < G) {
        auto middle = [&](int pair, int key) {
          const float2 mn = h2f(lds_u32(s + L::kValMin + (uint32_t)(pair * G + r % 4) * 4));
          const float2 sc = h2f(lds_u32(s + L::kValScale + (uint32_t)(pair * G + r % 4) * 4));
          float x = fmaf(8.f, sc.x, mn.x), y = fmaf(8.f, sc.y, mn.y);
          if constexpr (EDGE) {   // 0 x a masked key's bits has to be 0; a NaN group's scale shows it
            if (key >= n || isnan(x)) x = 0.f;
            if (key + 1 >= n || isnan(y)) y = 0.f;
          }
          uint32_t hi, lo;
          split2(x, y, hi, lo);
          return r < 4 ? hi : lo;
        };
        b0 = middle(q, kb + 2 * q);
        b1 = middle(q + 4, kb + 8 + 2 * q);
      }
      if constexpr (MODE == 0) {
        split2(p[0][0], p[0][1], a0, a1);
        split2(p[0][2], p[0][3], a2, a3);
      } else {
        a0 = h2bits(__floats2half2_rn(p[0][0], p[0][1]));
        a2 = h2bits(__floats2half2_rn(p[0][2], p[0][3]));
        if constexpr (MODE == 1) {
          a1 = h2bits(__floats2half2_rn(p[NR - 1][0], p[NR - 1][1]));
          a3 = h2bits(__floats2half2_rn(p[NR - 1][2], p[NR - 1][3]));
        }
      }
      mma_f16(om, a0, a1, a2, a3, b0, b1);
    }
    uint32_t v0[G], v1[G], s0[G], s1[G];
    lds_words<G>(s + L::kValCodes + (uint32_t)((q * 8 + r) * G) * 4, v0);
    lds_words<G>(s + L::kValCodes + (uint32_t)(((q + 4) * 8 + r) * G) * 4, v1);
    lds_words<G>(s + L::kValScale + (uint32_t)(q * G) * 4, s0);
    lds_words<G>(s + L::kValScale + (uint32_t)((q + 4) * G) * 4, s1);
#pragma unroll
    for (int i = 0; i < NR; ++i)   // p sc 4 stays below 2^16: scales are at most 8192
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i][j] *= 4.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float2 x = h2f(s0[g]), y = h2f(s1[g]);
      const float sc[4] = {x.x, x.y, y.x, y.y};
      float u[NR][4];
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          u[i][j] = p[i][j] * sc[j];
          if constexpr (EDGE)
            if (!(see[i] >> j & 1u)) u[i][j] = 0.f;
        }
      uint32_t a0, a1 = 0, a2, a3 = 0;
      if constexpr (MODE == 0) {
        split2(u[0][0], u[0][1], a0, a1);
        split2(u[0][2], u[0][3], a2, a3);
      } else {
        a0 = h2bits(__floats2half2_rn(u[0][0], u[0][1]));
        a2 = h2bits(__floats2half2_rn(u[0][2], u[0][3]));
        if constexpr (MODE == 1) {
          a1 = h2bits(__floats2half2_rn(u[NR - 1][0], u[NR - 1][1]));
          a3 = h2bits(__floats2half2_rn(u[NR - 1][2], u[NR - 1][3]));
        }
      }
      mma_f16(o[g][0], a0, a1, a2, a3, centre_even(v0[g]), centre_even(v1[g]));
      mma_f16(o[g][1], a0, a1, a2, a3, centre_odd(v0[g]), centre_odd(v1[g]));
      mma_f16(o[g][2], a0, a1, a2, a3, centre_even(v0[g] >> 8), centre_even(v1[g] >> 8));
      mma_f16(o[g][3], a0, a1, a2, a3, centre_odd(v0[g] >> 8), centre_odd(v1[g] >> 8));
    }
  }

  // This lane's 8 elements (32 g + 8 q + 0..7) of row `which`, in true units
  __device__ __forceinline__ void finish(int which, int g, int lane, float (&x)[8]) const {
    float m0 = om[2 * which], m1 = om[2 * which + 1];
    if constexpr (MODE == 0) {
      m0 = fmaf(om[2], 4.8828125e-4f, m0);
      m1 = fmaf(om[3], 4.8828125e-4f, m1);
    }
    const int src = (lane & ~3) + g / 2;   // the lane with columns g & ~1, g | 1; their lo parts two on
    const float mx = g % 2 ? m1 : m0;
    const float mn = fmaf(__shfl_sync(0xFFFFFFFFu, mx, src + 2), 4.8828125e-4f,
                          __shfl_sync(0xFFFFFFFFu, mx, src));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y0 = o[g][i][2 * which], y1 = o[g][i][2 * which + 1];
      if constexpr (MODE == 0) {
        y0 = fmaf(o[g][i][2], 4.8828125e-4f, y0);
        y1 = fmaf(o[g][i][3], 4.8828125e-4f, y1);
      }
      constexpr float up = 256.f;   // 2^10 / 4
      x[i] = fmaf(y0, up, mn);
      x[4 + i] = fmaf(y1, up, mn);
    }
  }

  // The same with what went to shared memory before (at: this lane's 8
  // elements of group 0 there)
  __device__ __forceinline__ void gather(int which, int g, int lane, const float* at, float (&x)[8]) const {
    finish(which, g, lane, x);
    if (MODE == 0 && __any_sync(0xFFFFFFFFu, fm != -INFINITY)) {
      const float e = ex2(fm - row[0].mu);
      const float4 u = *reinterpret_cast<const float4*>(at + 32 * g);
      const float4 v = *reinterpret_cast<const float4*>(at + 32 * g + 4);
      const float y[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (fm != -INFINITY) x[i] = fmaf(y[i], e, x[i]);
    }
  }
  __device__ __forceinline__ void put(int which, int g, int lane, float* at) const {
    float x[8];
    gather(which, g, lane, at, x);
    *reinterpret_cast<float4*>(at + 32 * g) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(at + 32 * g + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
  __device__ __forceinline__ void flush(int lane, float* at) {
#pragma unroll
    for (int g = 0; g < G; ++g) put(0, g, lane, at);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[g][i][j] = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) om[j] = 0.f;
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

template <int D, int MODE>
__global__ void __launch_bounds__(kFewThreads, 1) kv_few_kernel(const AttnArgs a) {
  using F = Few<D, MODE>;
  using L = KvTile<D>;
  constexpr int RT = F::kRows, G = L::G, W = kFewWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* full = reinterpret_cast<uint64_t*>(smem);
  uint64_t* empty = full + kFewStages;
  volatile uint32_t* mask = reinterpret_cast<volatile uint32_t*>(smem + 128);   // tiles copied, per stage
  volatile uint32_t* flag = mask + kFewStages;   // [0] a wait ran out, [1] last part of an item
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kFewStages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], W);
    }
    flag[0] = 0;
    fence_barrier_init();
  }
  pdl_wait();
  KvWalk w;
  int G_, q0;
  long long U;
  if (!kv_range<kFewThreads, RT, W>(a, w, G_, U, q0)) return;   // (its barriers order the set-up above)

  if (warp == W) {   // producer
    const int tpp = a.page_tokens / LW_KV_TILE;
    auto entry = [&](const KvWalk& v, int k) {   // this lane's page of unit k
      const int tile = v.span.lo + k * W + lane;
      if (lane >= W || tile >= v.span.hi) return -2;
      return __ldg(a.p.page_table + (int64_t)v.b * a.p.table_stride + tile / tpp);
    };
    uint32_t it = 0;
    bool dead = false;
    int page = entry(w, w.k0), k = w.k0;
    KvWalk nx = w;
    int nq0;
    for (bool more = true; more;) {
      const KvWalk cur = nx;
      const int ck = k, cpage = page;
      if (++k == nx.k1) {
        more = kv_advance<RT, W>(a, nx, nq0);
        k = nx.k0;
      }
      if (more) page = entry(nx, k);   // one unit ahead
      const int s = it % kFewStages;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], (it / kFewStages & 1u) ^ 1u))) {
        dead = true;
        break;
      }
      const bool use = cpage >= 0 && cpage < a.n_pages;
      if (!use && cpage != -2) report(a.status, LW_DEV_BAD_PAGE);
      else if (cpage == -2 && lane < W && cur.span.lo + ck * W + lane < cur.span.hi) report(a.status, LW_DEV_BAD_PAGE);
      const uint32_t got = __ballot_sync(0xFFFFFFFFu, use);
      if (lane == 0) {
        mask[s] = got;
        mbar_arrive_expect_tx(&full[s], (uint32_t)__popc(got) * L::kBytes);
      }
      __syncwarp();
      if (use) {
        const int tile = cur.span.lo + ck * W + lane;
        bulk_g2s(smem + F::kRing + s * F::kStage + lane * L::kBytes,
                 a.pages + cpage * a.page_bytes + ((int64_t)cur.h * tpp + tile % tpp) * L::kBytes, L::kBytes,
                 &full[s]);
      }
      ++it;
    }
    if (dead) {   // no copy may be in flight when the CTA ends
      flag[0] = 1;
      report(a.status, LW_DEV_TIMEOUT);
      for (uint32_t i = it > kFewStages ? it - kFewStages : 0; i < it; ++i)
        mbar_wait(&full[i % kFewStages], i / kFewStages & 1u);
    }
    return;
  }

  FewWarp<D, MODE> f;
  uint32_t it = 0;
  bool dead = false;
  float* s_o = reinterpret_cast<float*>(smem + F::kJoin);
  float* s_m = reinterpret_cast<float*>(smem + F::kState);
  float* s_l = s_m + W * 8;
  for (bool more = true; more;) {
    f.start(a, w, q0, RT, lane);
    // keys that every row of the item sees
    int all_lo, all_hi, x;
    {
      int t1 = (w.rt * RT + RT - 1) / a.group;
      if (t1 > w.T - 1) t1 = w.T - 1;
      kv_token_keys(w.T, w.n, w.rt * RT / a.group, a.p.causal, a.p.window, x, all_hi);
      kv_token_keys(w.T, w.n, t1, a.p.causal, a.p.window, all_lo, x);
    }
    float* mine = s_o + (warp * 8 + lane / 4) * F::kPitch + 8 * (lane % 4);
    int held = 0;
    for (int k = w.k0; k < w.k1; ++k, ++it) {
      if (MODE == 0 && held == kFewFlush) {
        f.flush(lane, mine);
        held = 0;
      }
      const int s = it % kFewStages;
      if (!dead && (flag[0] || !__all_sync(0xFFFFFFFFu, mbar_wait(&full[s], it / kFewStages & 1u)))) {
        dead = true;
        flag[0] = 1;
        report(a.status, LW_DEV_TIMEOUT);
      }
      dead = __any_sync(0xFFFFFFFFu, dead);
      if (!dead && (mask[s] >> warp & 1u)) {
        const uint32_t at = smem_addr(smem + F::kRing) + s * F::kStage + warp * L::kBytes;
        const int kb = (w.span.lo + k * W + warp) * LW_KV_TILE;
        if (kb >= all_lo && kb + LW_KV_TILE <= all_hi) f.template tile<false>(at, kb, w.n, lane);
        else f.template tile<true>(at, kb, w.n, lane);
        ++held;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    // join the warps, 8 rows at a time
    const bool whole = w.k0 == 0 && w.k1 == w.units;
    float* part = a.partials + ((size_t)blockIdx.x * 2 + (w.k0 == 0)) * F::kPartial;
#pragma unroll
    for (int i = 0; i < FewWarp<D, MODE>::NR; ++i) {
      float l = f.row[i].l;
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
      l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
      if (lane % 4 == 0) {
        s_m[warp * 8 + lane / 4] = f.row[i].m;
        s_l[warp * 8 + lane / 4] = l;
      }
#pragma unroll
      for (int g = 0; g < G; ++g) f.put(i, g, lane, mine);
      few_bar();
      for (int j = threadIdx.x; j < 8 * (D / 4); j += 32 * W) {
        const int r = j / (D / 4), d = 4 * (j % (D / 4));
        float m = -INFINITY, sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int v = 0; v < W; ++v) m = fmaxf(m, s_m[v * 8 + r]);
        const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int v = 0; v < W; ++v) {
          const float e = ex2(s_m[v * 8 + r] - mu);
          sum = fmaf(s_l[v * 8 + r], e, sum);
          const float4 z = *reinterpret_cast<const float4*>(s_o + (v * 8 + r) * F::kPitch + d);
          y[0] = fmaf(z.x, e, y[0]);
          y[1] = fmaf(z.y, e, y[1]);
          y[2] = fmaf(z.z, e, y[2]);
          y[3] = fmaf(z.w, e, y[3]);
        }
        if (whole) {
          few_out<RT>(a, w, q0, 8 * i + r, d, m, sum, y);
        } else {
          if (d == 0) {
            part[8 * i + r] = m;
            part[RT + 8 * i + r] = sum;
          }
          *reinterpret_cast<float4*>(part + 2 * RT + (8 * i + r) * D + d) = make_float4(y[0], y[1], y[2], y[3]);
        }
      }
      few_bar();
    }
    if (!whole) {
      const long long x0 = w.x - w.k0;
      const int c0 = tc_owner(x0, U, G_), parts = tc_owner(x0 + w.units - 1, U, G_) - c0 + 1;
      __threadfence();
      few_bar();
      if (threadIdx.x == 0) {
        const bool last = atomicAdd(a.counters + c0, 1u) == (uint32_t)parts - 1u;
        if (last) a.counters[c0] = 0;
        flag[1] = last;
      }
      few_bar();
      if (flag[1]) {
        __threadfence();
        for (int j = threadIdx.x; j < RT * (D / 4); j += 32 * W) {
          const int r = j / (D / 4), d = 4 * (j % (D / 4));
          float m = -INFINITY, sum = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
          const float* p0 = a.partials + ((size_t)c0 * 2 + 1) * F::kPartial;
          auto at = [&](int i) { return i ? a.partials + (size_t)(c0 + i) * 2 * F::kPartial : p0; };
          for (int i = 0; i < parts; ++i) m = fmaxf(m, __ldcg(at(i) + r));
          const float mu = m == -INFINITY ? 0.f : m;
#pragma unroll 4
          for (int i = 0; i < parts; ++i) {
            const float* p = at(i);
            const float e = ex2(__ldcg(p + r) - mu);
            sum = fmaf(__ldcg(p + RT + r), e, sum);
            const float4 z = __ldcg(reinterpret_cast<const float4*>(p + 2 * RT + r * D + d));
            y[0] = fmaf(z.x, e, y[0]);
            y[1] = fmaf(z.y, e, y[1]);
            y[2] = fmaf(z.z, e, y[2]);
            y[3] = fmaf(z.w, e, y[3]);
          }
          few_out<RT>(a, w, q0, r, d, m, sum, y);
        }
      }
      few_bar();
    }
    more = kv_advance<RT, W>(a, w, q0);
  }
}

}  // namespace dev
}  // namespace lw
