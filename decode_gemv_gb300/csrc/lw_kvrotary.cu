// Rotary positions: the table of cosines and sines, and the cache write that
// rotates the tokens' keys and queries as they pass.
#include "lw_kv.cuh"
#include "lw_kv.h"

#include <cmath>

namespace lw {

namespace {

// ---- the table ---------------------------------------------------------------
constexpr int kMostPairs = 64;
struct TableArgs {
  double f[kMostPairs];
  double gain;
  float* table;
  int64_t first, n;
  int32_t pairs;
};

// A thread an angle, in fp64: 2^31 positions leave 2^-22 of a turn, a million 2^-33.  Once a model, not once
// a step (131072 positions of 64 pairs: 8.4 million sincos).
__global__ void __launch_bounds__(256) rotary_table_kernel(const TableArgs a) {
  dev::pdl_wait();
  const int64_t all = a.n * a.pairs;
  for (int64_t x = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; x < all; x += (int64_t)gridDim.x * blockDim.x) {
    const int64_t row = x / a.pairs;
    const int i = (int)(x - row * a.pairs);
    double s, c;
    sincos((double)(a.first + row) * a.f[i], &s, &c);
    a.table[row * 2 * a.pairs + i] = (float)(c * a.gain);
    a.table[row * 2 * a.pairs + a.pairs + i] = (float)(s * a.gain);
  }
}

// ---- the write ---------------------------------------------------------------
struct RotaryArgs {
  CacheArgs c;
  RowsArgs q, q_out;
  const int64_t* positions;
  const float* table;
  int64_t table_rows;
  int64_t write_blocks;      // blocks of the first role; the others rotate queries
  int32_t rot, q_heads;
  int32_t splits, per_split, kv_splits, kv_per_split;   // shares of the heads, and heads of a share
};

// The table's row of a token's position; NULL if the token is skipped (a position past the table is reported
// where `first`).
__device__ __forceinline__ const float* table_row(const RotaryArgs& a, int64_t tok, bool first) {
  const int64_t p = a.positions[tok];
  if (p < 0 || p >= a.table_rows) {
    if (p >= 0 && first) dev::report(a.c.status, LW_DEV_BAD_POSITION);
    return nullptr;
  }
  return a.table + p * a.rot;
}
__device__ __forceinline__ void load8f(const float* p, float (&x)[8]) {
  const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
  x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
  x[4] = v.x; x[5] = v.y; x[6] = v.z; x[7] = v.w;
}

// 8 elements as they lie in memory, by 16-byte accesses
template <class T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    const T* e = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = dev::kv_float<T>(e[i]);
  }
};

// ---- keys and values -----------------------------------------------------------
// What a thread does to elements 8 ch .. 8 ch + 7 of every key head of its token.  WIDE (rot a multiple of 16,
// rows and table on 16-byte boundaries): all of them are rotated, on one side of their pairs, or none is.
template <class T, bool WIDE, bool NEAR>
struct KeyTurn {
  float c[8], s[8];       // !NEAR: of elements 8 ch + i, the sine with the sign that its product enters with;
                          // NEAR: of pairs 4 ch + i, i < 4
  const float* row;
  int d0, other, half, rot;
  bool turned;

  __device__ __forceinline__ void begin(const float* r, int ch, int rot_) {
    row = r;
    rot = rot_;
    half = rot / 2;
    d0 = 8 * ch;
    turned = d0 < rot;
    other = d0 < half ? d0 + half : d0 - half;
    if constexpr (WIDE) {
      if (!turned) return;
      if constexpr (NEAR) {
        const float4 u = *reinterpret_cast<const float4*>(row + d0 / 2), v = *reinterpret_cast<const float4*>(row + half + d0 / 2);
        c[0] = u.x; c[1] = u.y; c[2] = u.z; c[3] = u.w;
        s[0] = v.x; s[1] = v.y; s[2] = v.z; s[3] = v.w;
      } else {
        const bool low = d0 < half;
        load8f(row + (low ? d0 : d0 - half), c);
        load8f(row + half + (low ? d0 : d0 - half), s);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = low ? -s[i] : s[i];
      }
    }
  }
  // k: the head's elements as they are; far: their partners' (WIDE, !NEAR)
  __device__ __forceinline__ void turn(const T* key, const Raw8<T>& far, float (&k)[8]) const {
    if constexpr (WIDE) {
      if (!turned) return;
      if constexpr (NEAR) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = k[2 * i], y = k[2 * i + 1];
          k[2 * i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
          k[2 * i + 1] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
        }
      } else {
        float y[8];
        far.values(y);
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = __fadd_rn(__fmul_rn(k[i], c[i]), __fmul_rn(y[i], s[i]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d < rot) {
          const bool low = NEAR ? d % 2 == 0 : d < half;
          const int pair = NEAR ? d / 2 : (low ? d : d - half);
          const float z = __fmul_rn(dev::kv_float<T>(key[NEAR ? d ^ 1 : (low ? d + half : d - half)]), row[half + pair]);
          k[i] = __fadd_rn(__fmul_rn(k[i], row[pair]), low ? -z : z);
        }
      }
    }
  }
};

// Key and value heads [h0, h1) of one token into its slot.  Whole warps: a group's four lanes agree on its range.
template <class T, int D, bool WIDE, bool NEAR>
__device__ __forceinline__ void write_heads(const RotaryArgs& a, int64_t tok, int ch, int h0, int h1) {
  using L = KvTile<D>;
  int64_t at = -1, slot = -1;
  KeyTurn<T, WIDE, NEAR> turn;
  const T *k = static_cast<const T*>(a.c.k.ptr), *v = static_cast<const T*>(a.c.v.ptr);
  if (tok < a.c.n) {
    slot = a.c.slots[tok];
    const float* row = table_row(a, tok, h0 == 0 && ch == 0);
    if (row) {
      at = dev::slot_tile(a.c, slot, L::kBytes, h0 == 0 && ch == 0);
      turn.begin(row, ch, a.rot);
    }
    k += tok * a.c.k.token_stride;
    v += tok * a.c.v.token_stride;
  }
  const int t = (int)(slot % LW_KV_TILE);
  Raw8<T> rk, rv, rf;
  const auto load = [&](int h) {
    if constexpr (WIDE) {
      rk.load(k + h * a.c.k.head_stride + 8 * ch);
      rv.load(v + h * a.c.v.head_stride + 8 * ch);
      if (!NEAR && turn.turned) rf.load(k + h * a.c.k.head_stride + turn.other);
    }
  };
  if (at >= 0) load(h0);
#pragma unroll 1
  for (int h = h0; h < h1; ++h) {
    float x[8] = {}, y[8] = {}, lo[2] = {}, hi[2] = {};
    if (at >= 0) {
      if constexpr (WIDE) {
        rk.values(x);
        rv.values(y);
        turn.turn(nullptr, rf, x);
        if (h + 1 < h1) load(h + 1);
      } else {
        dev::kv_load8<T, false>(k + h * a.c.k.head_stride + 8 * ch, x);
        dev::kv_load8<T, false>(v + h * a.c.v.head_stride + 8 * ch, y);
        turn.turn(k + h * a.c.k.head_stride, rf, x);
      }
      lo[0] = dev::min3(dev::min3(dev::min3(x[0], x[1], x[2]), x[3], x[4]), dev::min3(x[5], x[6], x[7]), x[0]);
      hi[0] = dev::max3(dev::max3(dev::max3(x[0], x[1], x[2]), x[3], x[4]), dev::max3(x[5], x[6], x[7]), x[0]);
      lo[1] = dev::min3(dev::min3(dev::min3(y[0], y[1], y[2]), y[3], y[4]), dev::min3(y[5], y[6], y[7]), y[0]);
      hi[1] = dev::max3(dev::max3(dev::max3(y[0], y[1], y[2]), y[3], y[4]), dev::max3(y[5], y[6], y[7]), y[0]);
    }
    __half ks, km, vs, vm;
    const uint32_t kw = dev::kv_quantise8(x, lo[0], hi[0], ks, km), vw = dev::kv_quantise8(y, lo[1], hi[1], vs, vm);
    if (at >= 0)
      dev::kv_put8<D>(a.c.pages + at + (int64_t)h * a.c.page_tiles * L::kBytes, t, ch, kw, ks, km, vw, vs, vm);
  }
}

// ---- queries -------------------------------------------------------------------
// Query heads [h0, h1) of one token: thread `part` of D / 16 holds 8 pairs' cosines and sines and takes those
// pairs of every head (it alone reads and writes them: q_out may be q), or 16 of the elements that stay.
template <class T, int D, bool WIDE, bool NEAR>
__device__ __forceinline__ void rotate_queries(const RotaryArgs& a, const float* row, int64_t tok, int part, int h0,
                                               int h1) {
  const T* q = static_cast<const T*>(a.q.ptr) + tok * a.q.token_stride;
  T* out = static_cast<T*>(a.q_out.ptr) + tok * a.q_out.token_stride;
  const int half = a.rot / 2;
  const bool same = q == out;
  if constexpr (WIDE) {
    constexpr int kAhead = sizeof(T) == 4 ? 2 : 4;   // heads on their way at once
    const bool turned = 16 * part < a.rot;
    if (!turned && same) return;
    const int x0 = turned && !NEAR ? 8 * part : 16 * part, y0 = turned && !NEAR ? half + 8 * part : x0 + 8;
    float c[8], s[8];
    if (turned) {
      load8f(row + 8 * part, c);
      load8f(row + half + 8 * part, s);
    }
#pragma unroll 1
    for (int h = h0; h < h1; h += kAhead) {
      Raw8<T> rx[kAhead], ry[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < h1) {
          rx[i].load(q + (h + i) * a.q.head_stride + x0);
          ry[i].load(q + (h + i) * a.q.head_stride + y0);
        }
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (h + i < h1) {
          float x[8], y[8];
          rx[i].values(x);
          ry[i].values(y);
          if (turned) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              // (pair j: elements j of x and y, or neighbours, the first four pairs in x)
              float& u = NEAR ? (j < 4 ? x[(2 * j) & 7] : y[(2 * j) & 7]) : x[j];
              float& v = NEAR ? (j < 4 ? x[(2 * j + 1) & 7] : y[(2 * j + 1) & 7]) : y[j];
              const float nu = __fsub_rn(__fmul_rn(u, c[j]), __fmul_rn(v, s[j]));
              v = __fadd_rn(__fmul_rn(v, c[j]), __fmul_rn(u, s[j]));
              u = nu;
            }
          }
          dev::kv_store8<T, true>(out + (h + i) * a.q_out.head_stride + x0, x);
          dev::kv_store8<T, true>(out + (h + i) * a.q_out.head_stride + y0, y);
        }
    }
  } else {
#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
      const T* p = q + h * a.q.head_stride;
      T* o = out + h * a.q_out.head_stride;
#pragma unroll 1
      for (int j = part; j < half; j += D / 16) {
        const int x0 = NEAR ? 2 * j : j, y0 = NEAR ? 2 * j + 1 : j + half;
        const float u = dev::kv_float<T>(p[x0]), v = dev::kv_float<T>(p[y0]), c = row[j], s = row[half + j];
        o[x0] = dev::kv_round<T>(__fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s)));
        o[y0] = dev::kv_round<T>(__fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s)));
      }
      if (!same)
#pragma unroll 1
        for (int d = a.rot + part; d < D; d += D / 16) o[d] = p[d];
    }
  }
}

constexpr int kTokens = 16;   // of a writing block; twice as many of a rotating one

// Measured, 65536 tokens of 32 query and 8 key/value heads of 128 in bf16: 254 us, 5.4 TB/s of the 1.37 GB that
// have to move (a copy reaches 6.8); in fp32 464 us.  A block a head, each with its tokens' angles and slots read anew,
// took 577 us: a chain of three reads for 4 KB of keys and values.  One token: 2.4 us, the same chain.
// Not WIDE (rot no multiple of 16, or rows off 16-byte boundaries): element by element, angles and partners read anew
// for each head.  96 wide, bf16: 48 elements rotated 209 us, 24 of them 657.
template <class T, int D, bool WIDE, bool NEAR>
__global__ void __launch_bounds__(kTokens * D / 8, 3) kv_write_rotary_kernel(const RotaryArgs a) {
  dev::pdl_wait();
  if (blockIdx.x < a.write_blocks) {
    constexpr int kChunks = D / 8;
    const int64_t block = blockIdx.x / a.kv_splits;
    const int h0 = (int)(blockIdx.x - block * a.kv_splits) * a.kv_per_split;
    const int h1 = h0 + a.kv_per_split < a.c.heads ? h0 + a.kv_per_split : a.c.heads;
    write_heads<T, D, WIDE, NEAR>(a, block * kTokens + threadIdx.x / kChunks, threadIdx.x % kChunks, h0, h1);
  } else {
    constexpr int kParts = D / 16;
    const int64_t b = blockIdx.x - a.write_blocks, block = b / a.splits;
    const int h0 = (int)(b - block * a.splits) * a.per_split;
    const int h1 = h0 + a.per_split < a.q_heads ? h0 + a.per_split : a.q_heads;
    const int64_t tok = block * (2 * kTokens) + threadIdx.x / kParts;
    if (tok >= a.c.n) return;
    const float* row = table_row(a, tok, false);
    if (row) rotate_queries<T, D, WIDE, NEAR>(a, row, tok, threadIdx.x % kParts, h0, h1);
  }
}

template <class T, int D>
lw_status launch_d(const RotaryArgs& a, bool wide, bool near, dim3 grid, cudaStream_t st) {
  auto k = wide ? (near ? kv_write_rotary_kernel<T, D, true, true> : kv_write_rotary_kernel<T, D, true, false>)
                : (near ? kv_write_rotary_kernel<T, D, false, true> : kv_write_rotary_kernel<T, D, false, false>);
  return kv_launch("lw_kv_write_rotary", k, grid, kTokens * D / 8, 0, 1, st, a);
}
template <class T>
lw_status launch_t(const RotaryArgs& a, int dim, bool wide, bool near, dim3 grid, cudaStream_t st) {
  return dim == 64   ? launch_d<T, 64>(a, wide, near, grid, st)
         : dim == 96 ? launch_d<T, 96>(a, wide, near, grid, st)
                     : launch_d<T, 128>(a, wide, near, grid, st);
}

}  // namespace
}  // namespace lw

using namespace lw;

extern "C" lw_status lw_rotary_table(const lw_rotary* r, int64_t first, int64_t n, float* table, void* stream) {
  clear_error();
  if (!r) return fail(LW_ERR_INVALID_ARG, "NULL rotary");
  if (r->rot < 2 || r->rot > 2 * kMostPairs || r->rot % 2)
    return fail(LW_ERR_SHAPE, "rot %d: an even number from 2 to %d", r->rot, 2 * kMostPairs);
  if (r->scaling < LW_ROTARY_PLAIN || r->scaling > LW_ROTARY_YARN)
    return fail(LW_ERR_UNSUPPORTED, "scaling %d", r->scaling);
  const auto finite = [](double x) { return x >= -1e300 && x <= 1e300; };
  if (!(r->base > 1.0) || !finite(r->base)) return fail(LW_ERR_INVALID_ARG, "base %g", r->base);
  if (r->scaling != LW_ROTARY_PLAIN && (!(r->factor > 0.0) || !finite(r->factor)))
    return fail(LW_ERR_INVALID_ARG, "factor %g", r->factor);
  const bool bands = r->scaling == LW_ROTARY_BANDS, yarn = r->scaling == LW_ROTARY_YARN;
  const double low = r->low != 0.0 ? r->low : 1.0, high = r->high != 0.0 ? r->high : (yarn ? 32.0 : 4.0);
  if ((bands || yarn) && (!(r->old_length > 0.0) || !finite(r->old_length) || !(low > 0.0) || !(high > low) || !finite(high)))
    return fail(LW_ERR_INVALID_ARG, "old_length %g, low %g, high %g", r->old_length, low, high);
  if (!finite(r->gain)) return fail(LW_ERR_INVALID_ARG, "gain %g", r->gain);
  if (first < 0 || n < 0 || first > (1ll << 31) || n > (1ll << 31) || first + n > (1ll << 31))
    return fail(LW_ERR_SHAPE, "positions %lld .. + %lld", (long long)first, (long long)n);
  if (n == 0) return LW_OK;
  if (!table || reinterpret_cast<uintptr_t>(table) % 4) return fail(LW_ERR_INVALID_ARG, "table missing or misaligned");
  constexpr double kTurn = 6.283185307179586476925286766559;
  TableArgs a{};
  a.pairs = r->rot / 2;
  a.table = table;
  a.first = first;
  a.n = n;
  a.gain = r->gain != 0.0 ? r->gain : (yarn ? 0.1 * std::log(r->factor) + 1.0 : 1.0);
  double base = r->base;
  if (r->scaling == LW_ROTARY_NTK && r->rot > 2) base *= std::pow(r->factor, (double)r->rot / (r->rot - 2));
  const auto pair = [&](double turns) {
    return r->rot * std::log(r->old_length / (turns * kTurn)) / (2.0 * std::log(base));
  };
  double from = 0.0, to = 0.0;
  if (yarn) {
    from = std::fmax(0.0, std::floor(pair(high)));
    to = std::fmin(r->rot - 1.0, std::ceil(pair(low)));
  }
  for (int i = 0; i < a.pairs; ++i) {
    const double f = std::pow(base, -2.0 * i / r->rot);
    double keep = r->scaling == LW_ROTARY_LINEAR ? 0.0 : 1.0;
    if (bands) keep = (r->old_length * f / kTurn - low) / (high - low);
    if (yarn) keep = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - from) / std::fmax(to - from, 0.001)));
    keep = std::fmin(1.0, std::fmax(0.0, keep));
    a.f[i] = keep == 1.0 ? f : f * (keep + (1.0 - keep) / r->factor);
  }
  const int64_t blocks = (n * a.pairs + 255) / 256, most = 32ll * device_sm_count();
  return kv_launch("lw_rotary_table", rotary_table_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, 0, 1,
                   static_cast<cudaStream_t>(stream), a);
}

extern "C" lw_status lw_kv_write_rotary(const lw_kv_cache* c, const lw_kv_rotated* p, int32_t* d_status,
                                        void* stream) {
  const char* fn = "lw_kv_write_rotary";
  clear_error();
  lw_status s = check_kv_cache(c);
  if (s != LW_OK) return s;
  if (!p) return fail(LW_ERR_INVALID_ARG, "NULL arguments");
  if (p->n < 0) return fail(LW_ERR_INVALID_ARG, "%s: %lld tokens", fn, (long long)p->n);
  if (!kv_type_ok(p->k.dtype) || !kv_type_ok(p->v.dtype))
    return fail(LW_ERR_UNSUPPORTED, "%s: unknown type %d / %d", fn, p->k.dtype, p->v.dtype);
  if (p->k.dtype != p->v.dtype)
    return fail(LW_ERR_INVALID_ARG, "%s: keys of type %d, values of type %d", fn, p->k.dtype, p->v.dtype);
  const bool queries = p->q.ptr != nullptr;
  if (queries) {
    if (!kv_type_ok(p->q.dtype)) return fail(LW_ERR_UNSUPPORTED, "%s: unknown type %d", fn, p->q.dtype);
    if (p->q.dtype != p->k.dtype || p->q_out.dtype != p->q.dtype)
      return fail(LW_ERR_INVALID_ARG, "%s: keys of type %d, queries of type %d go to type %d", fn, p->k.dtype,
                  p->q.dtype, p->q_out.dtype);
    if (p->q_heads < 1 || p->q_heads > 65535) return fail(LW_ERR_SHAPE, "%s: %d query heads", fn, p->q_heads);
  }
  if (p->rot < 2 || p->rot > c->head_dim || p->rot % 2)
    return fail(LW_ERR_SHAPE, "%s: rot %d of %d", fn, p->rot, c->head_dim);
  if (p->interleaved != 0 && p->interleaved != 1)
    return fail(LW_ERR_INVALID_ARG, "%s: interleaved %d", fn, p->interleaved);
  if (p->table_rows < 0 || p->table_rows > (1ll << 31))
    return fail(LW_ERR_SHAPE, "%s: a table of %lld rows", fn, (long long)p->table_rows);
  if (p->n == 0) return LW_OK;
  if (!p->k.ptr || !p->v.ptr || !p->slots || !p->positions || (p->table_rows && !p->table) || (queries && !p->q_out.ptr))
    return fail(LW_ERR_INVALID_ARG, "%s: NULL keys, values, slots, positions, table or q_out", fn);
  const auto off = [](const void* x, uintptr_t n) { return reinterpret_cast<uintptr_t>(x) % n != 0; };
  const uintptr_t es = (uintptr_t)kv_type_bytes(p->k.dtype);
  if (off(p->k.ptr, es) || off(p->v.ptr, es) || off(p->slots, 8) || off(p->positions, 8) || off(p->table, 4) ||
      (queries && (off(p->q.ptr, es) || off(p->q_out.ptr, es))))
    return fail(LW_ERR_INVALID_ARG, "%s: an address is not aligned to its type", fn);
  RotaryArgs a{};
  a.c = kv_cache_args(c, &p->k, &p->v, p->slots, p->n, d_status);
  a.q = {p->q.ptr, p->q.token_stride, p->q.head_stride};
  a.q_out = {p->q_out.ptr, p->q_out.token_stride, p->q_out.head_stride};
  a.positions = p->positions;
  a.table = p->table;
  a.table_rows = p->table_rows;
  a.rot = p->rot;
  a.q_heads = queries ? p->q_heads : 0;
  // A block takes all heads of its tokens (16 that are written, 32 that are rotated), or a share of them where
  // tokens are few: some blocks an SM
  const auto share = [](int64_t groups, int heads, int32_t& splits, int32_t& per) {
    int64_t n = (6ll * device_sm_count() + groups - 1) / groups;
    if (n > heads) n = heads;
    if (n < 1) n = 1;
    per = (int32_t)((heads + n - 1) / n);
    splits = per ? (heads + per - 1) / per : 1;
  };
  const int64_t groups = (p->n + 2 * kTokens - 1) / (2 * kTokens), writes = (p->n + kTokens - 1) / kTokens;
  share(groups, a.q_heads, a.splits, a.per_split);
  share(writes, c->kv_heads, a.kv_splits, a.kv_per_split);
  a.write_blocks = writes * a.kv_splits;
  const int64_t blocks = a.write_blocks + (queries ? groups * a.splits : 0);
  if (blocks > (1ll << 31) - 1) return fail(LW_ERR_SHAPE, "%s: %lld tokens", fn, (long long)p->n);
  const bool wide = p->rot % 16 == 0 && !off(p->table, 16) &&
                    kv_rows_aligned(p->k.ptr, p->k.token_stride, p->k.head_stride, p->k.dtype) &&
                    kv_rows_aligned(p->v.ptr, p->v.token_stride, p->v.head_stride, p->v.dtype) &&
                    (!queries || (kv_rows_aligned(p->q.ptr, p->q.token_stride, p->q.head_stride, p->q.dtype) &&
                                  kv_rows_aligned(p->q_out.ptr, p->q_out.token_stride, p->q_out.head_stride, p->q.dtype)));
  const bool near = p->interleaved != 0;
  const dim3 grid((unsigned)blocks);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return p->k.dtype == LW_F32   ? launch_t<float>(a, c->head_dim, wide, near, grid, st)
         : p->k.dtype == LW_F16 ? launch_t<__half>(a, c->head_dim, wide, near, grid, st)
                        : launch_t<__nv_bfloat16>(a, c->head_dim, wide, near, grid, st);
}
