// Accumulated attention weight for few rows: each key's softmax weights summed
// over the rows that share its head.
//
// Mathematics.  With a cached key k_d = sc_g c_d + mn_g (group g of 32) and
// q' = q / 2^e (2^e by the row's largest element),
//   q.k = 2^e ( sum_g sc_g sum_{d in g} q'_d c_d  +  sum_g mn_g sum_{d in g} q'_d ),
// weight_j += 2^((scale q.k_j - lse) log2 e).  The codes are the matrix operands
// (exact in fp16, the keys as the instruction's 16 rows), q' the other one (8
// columns): fp16 as 16-bit queries are (their own 8 or 11 bits, down to 2^-23 of
// the row's largest), two parts of 11 bits each of fp32 ones.  Scales enter in
// fp32 after the product; the minimums, fp16 as they are, take one more matrix
// instruction against the group sums in two parts.
//
// Structure.  A warp takes 32 keys at a time, their halves of the tiles fetched
// by bulk copies into a ring of its own; the sum over the rows is a sum over 4
// lanes and the row blocks.  ONE: a block of 8 rows whose operands stay in
// registers (one token of a group of up to 8 heads; more rows take the keys once
// a block); else up to 64 rows in shared memory.
//
// Where keys are many: 250 instructions a tile of 16 keys (a third restores the codes) in 60 % of the issue slots; the
// rest are waits on the matrix instructions' results, 4 warps a scheduler (6 warps of 80 registers spill: 142 us
// where this takes 129).  8 sequences of 20000 to 131072 keys (8 heads of 128 with 4 query heads each): bf16 130
// us, 0.47 GB of keys and weights, 3.6 TB/s; fp32 161.  Under a window of 129 keys 44, the weights of 32 keys a warp at a
// time.  4097 keys of one sequence: 5.5 us, a chain of reads.
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

template <int D, class T, bool ONE>
struct WeighFew {
  static constexpr int kParts = sizeof(T) == 4 ? 2 : 1;   // of an operand
  static constexpr int kWarps = 8, kThreads = 32 * kWarps, kPerSm = 2;
  static constexpr int kBlocks = ONE ? 1 : 8;              // of 8 rows, staged at once
  static constexpr int kFrag = D / 32 * 32 * 16;           // bytes of a block's operand part: a uint4 a lane and group
  static constexpr int kSum = kBlocks * kParts * kFrag;    // group sums: a uint2 a lane and block
  static constexpr int kRow = kSum + kBlocks * 256;        // rows: f, lse, lo, hi
  static constexpr int kRange = kRow + kBlocks * 8 * 16;   // keys that all, and any, rows of a block see
  static constexpr int kBars = kRange + kBlocks * 16;
  static constexpr int kPair = 2, kStages = 3;             // tiles fetched at once, and places of a warp's ring
  static constexpr int kRing = (kBars + kWarps * kStages * 8 + 127) / 128 * 128;
  static constexpr int kKeys = KvTile<D>::kValCodes;       // bytes of the key half of a tile
  static constexpr int kSmem = kRing + kWarps * kStages * kPair * kKeys;
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

// The first key that a row of a sequence of T > 0 query tokens sees (the last one is the sequence's)
__device__ __forceinline__ int weigh_first(const WeighArgs& a, int T, int n) {
  const int64_t lo = a.p.window ? (int64_t)n - T - a.p.window + 1 : 0;
  return lo > 0 ? (int)lo : 0;
}

// 8 consecutive elements of a query row
template <class T>
__device__ __forceinline__ void weigh_load8(const WeighArgs& a, int64_t at, float (&x)[8]) {
  const T* p = static_cast<const T*>(a.p.q) + at;
  if (a.vec) kv_load8<T, true>(p, x);
  else kv_load8<T, false>(p, x);
}

// A row of a block into shared memory: lane n * 4 + q has elements 32 g + 8 q .. of row n.
template <int D, class T, bool ONE>
__device__ void weigh_row(const WeighArgs& a, uint8_t* smem, int blk, int r, int q0, int Tq, int n, int h, int lane) {
  using W = WeighFew<D, T, ONE>;
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
  // the largest element comes to 2^9 .. 2^10: a group's sum of magnitudes stays below 2^15
  int e = (int)(__float_as_uint(top) >> 23) - 127;
  e = e < -100 ? -100 : (e > 127 ? 127 : e);
  const float down = __uint_as_float((uint32_t)(127 - e + 9) << 23);
  uint8_t* frag = smem + blk * W::kParts * W::kFrag;
  float sum[4] = {};
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
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (W::kParts == 2) split2<1>(x[g][i], x[g][i + 4], hi[i], lo[i]);
      else hi[i] = h2bits(__floats2half2_rn(x[g][i], x[g][i + 4]));
    }
    *reinterpret_cast<uint4*>(frag + (g * 32 + lane) * 16) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    if constexpr (W::kParts == 2)
      *reinterpret_cast<uint4*>(frag + W::kFrag + (g * 32 + lane) * 16) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  uint32_t sh = 0, sl = 0;   // groups 2 q, 2 q + 1
  if (q < 2) split2<1>(q ? sum[2] : sum[0], q ? sum[3] : sum[1], sh, sl);
  *reinterpret_cast<uint2*>(smem + W::kSum + blk * 256 + lane * 8) = make_uint2(sh, sl);
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
  if (q == 0)   // (a row that is not there weighs 0: its lse is infinite)
    *reinterpret_cast<float4*>(smem + W::kRow + (blk * 8 + lane / 4) * 16) =
        make_float4(a.p.scale * __uint_as_float((uint32_t)(e - 9 + 127) << 23),
                    live ? a.p.lse[(int64_t)(q0 + t) * a.p.q_heads + head] : INFINITY, __int_as_float(lo), __int_as_float(hi));
  if (lane == 0) *reinterpret_cast<int4*>(smem + W::kRange + blk * 16) = make_int4(all_lo, all_hi, any_lo, any_hi);
}

// A warp's pairs of neighbouring tiles: first, first + step, ... below `end` (in tiles), their key halves fetched by
// bulk copies into a ring of its own, in order.  Tiles below `seen` hold no key that a row sees: they need no page.
// The page table is read 32 tiles at a time: lanes 2 i and 2 i + 1 hold the i-th pair's places.
template <int D, class T, bool ONE>
struct WeighFetch {
  using W = WeighFew<D, T, ONE>;
  uint8_t* ring;
  uint64_t* bars;
  const int32_t* table;
  int64_t head;
  int next, seen, end, step, at, in, out;
  uint32_t there, have, parity;   // tiles that have a page; tiles sent for (2 bits a place); phase per place
  const uint8_t* src;

  __device__ __forceinline__ void lookup(const WeighArgs& a, int lane) {
    const int64_t tile = next + (int64_t)(lane / 2) * step + lane % 2;
    const int tpp = a.page_tokens / LW_KV_TILE;
    const bool mine = tile >= seen && tile < end;
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
    const uint32_t some = there >> at & 3u;
    if (some) {
      if (lane == at) mbar_arrive_expect_tx(&bars[in], (uint32_t)__popc(some) * W::kKeys);
      __syncwarp();
      if ((lane ^ at) < 2 && (there >> lane & 1u)) bulk_g2s(ring + (2 * in + lane % 2) * W::kKeys, src, W::kKeys, &bars[in]);
      have |= some << (2 * in);
    }
    at += 2;
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
  // The tiles at `out` have come (false: the wait ran out)
  __device__ __forceinline__ bool wait() {
    const bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&bars[out], parity >> out & 1u));
    if (!ok) return false;
    parity ^= 1u << out;
    have &= ~(3u << (2 * out));
    return true;
  }
  // On to the next pair
  __device__ __forceinline__ void pass() { out = out + 1 == W::kStages ? 0 : out + 1; }
  // After a wait that ran out: what is still on its way
  __device__ __forceinline__ void drain() {
    for (int i = 0; i < W::kStages; ++i)
      if (have >> (2 * i) & 3u) mbar_wait(&bars[i], parity >> i & 1u);
  }
};

// A lane's share of a tile's keys t and t + 8: codes as fp16 pairs, scales, and minimums as an operand
template <int D>
struct WeighTile {
  using L = KvTile<D>;
  static constexpr int G = L::G;
  uint32_t kc[2][G], ks[2][G], mn[2];
  __device__ __forceinline__ void read(uint32_t s, int lane) {
    const int t = lane / 4, q = lane % 4;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int tk = t + 8 * i;
      lds_words<G>(s + L::kKeyCodes + ((tk * 4 + q) * G) * 4, kc[i]);
      lds_words<G>(s + L::kKeyScale + (tk / 2 * G) * 4, ks[i]);
      mn[i] = 2 * q < G ? lds_u32(s + L::kKeyMin + (tk * (L::GP / 2) + q) * 4) : 0u;
      if (G % 2 && q == G / 2) mn[i] &= 0xFFFFu;   // (the last minimum's neighbour is not one)
    }
  }
  // Group g: operands of the two matrix instructions, and the keys' scales
  __device__ __forceinline__ void group(int g, int lane, uint32_t (&c)[2][4], float2& sc) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      c[i][0] = whole_even(kc[i][g]);
      c[i][1] = whole_odd(kc[i][g]);
      c[i][2] = whole_even(kc[i][g] >> 8);
      c[i][3] = whole_odd(kc[i][g] >> 8);
    }
    sc = h2f(__byte_perm(ks[0][g], ks[1][g], lane & 4 ? 0x7632 : 0x5410));   // by the parity of t
  }
};

template <int D, class T, bool ONE>
__global__ void __launch_bounds__(WeighFew<D, T, ONE>::kThreads, WeighFew<D, T, ONE>::kPerSm)
    kv_weigh_few_kernel(const WeighArgs a) {
  using W = WeighFew<D, T, ONE>;
  using L = KvTile<D>;
  constexpr int G = L::G, P = W::kParts;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, t = lane / 4, q = lane % 4;
  const int b = blockIdx.z, h = blockIdx.y;
  WeighFetch<D, T, ONE> f;
  f.bars = reinterpret_cast<uint64_t*>(smem + W::kBars) + warp * W::kStages;
  if (lane < W::kStages) mbar_init(&f.bars[lane], 1);
  fence_barrier_init();
  __syncwarp();
  pdl_wait();
  int q0, Tq, n;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) weigh_seq<true>(a, b, q0, Tq, n);
  else weigh_seq<false>(a, b, q0, Tq, n);
  const int keys = n < a.p.w_keys ? n : (int)a.p.w_keys;
  const int tiles = (keys + 15) / 16, first = 2 * (blockIdx.x * W::kWarps + warp);
  if (2 * (int)blockIdx.x * W::kWarps >= tiles) return;
  const int rows = Tq * a.group;
  const float* add = a.p.add_to ? a.p.add_to + b * a.p.add_seq_stride + h * a.p.add_head_stride : nullptr;
  float* out = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride;
  f.ring = smem + W::kRing + warp * W::kStages * 2 * W::kKeys;
  f.table = a.p.page_table + (int64_t)b * a.p.table_stride;
  f.head = (int64_t)h * (a.page_tokens / LW_KV_TILE) * L::kBytes;
  f.seen = Tq ? weigh_first(a, Tq, n) / 16 : tiles;
  f.end = tiles;
  f.step = gridDim.x * W::kWarps * 2;
  f.parity = 0;
  bool ok = true;
  int r0 = 0;
  do {
    if (ok) f.begin(a, first, lane);
    const int blocks = (min(rows - r0, 8 * W::kBlocks) + 7) / 8;
    if (r0) __syncthreads();
    for (int i = warp; i < blocks; i += W::kWarps) weigh_row<D, T, ONE>(a, smem, i, r0 + 8 * i + t, q0, Tq, n, h, lane);
    __syncthreads();
    // the block's operands (ONE: for good)
    uint4 fr[P][G];
    uint2 qs;
    float4 row[2];
    int4 range;
    const auto load_block = [&](int k) {
#pragma unroll
      for (int x = 0; x < P; ++x)
#pragma unroll
        for (int g = 0; g < G; ++g) fr[x][g] = *reinterpret_cast<const uint4*>(smem + (k * P + x) * W::kFrag + (g * 32 + lane) * 16);
      qs = *reinterpret_cast<const uint2*>(smem + W::kSum + k * 256 + lane * 8);
      row[0] = *reinterpret_cast<const float4*>(smem + W::kRow + (k * 8 + 2 * q) * 16);
      row[1] = *reinterpret_cast<const float4*>(smem + W::kRow + (k * 8 + 2 * q + 1) * 16);
      range = *reinterpret_cast<const int4*>(smem + W::kRange + k * 16);
    };
    if (ONE && blocks) load_block(0);
    // Lane (t, q) writes keys t + 8 (q % 2) of tile q / 2 of a pair.  What is added to comes a pair ahead (what an
    // earlier set of rows left is this thread's own).
    const float* from = r0 ? out : add;
    const auto key_of = [&](int tile) { return 16 * (tile + q / 2) + t + 8 * (q % 2); };
    const auto before = [&](int tile) { return from && tile < tiles && key_of(tile) < keys ? from[key_of(tile)] : 0.f; };
    float had = before(first);
    for (int tile = first; tile < tiles && ok; tile += f.step) {
      const float had_next = tile < tiles - f.step ? before(tile + f.step) : 0.f;
      const uint32_t some = blocks ? f.have >> (2 * f.out) & 3u : 0u;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};   // [tile of the pair][key t, t + 8]
      if (f.have >> (2 * f.out) & 3u) {
        ok = f.wait();
        if (!ok) break;
        const uint32_t s = smem_addr(f.ring + 2 * f.out * W::kKeys);
        WeighTile<D> x[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) x[u].read(s + u * W::kKeys, lane);
        // all lanes have read the place: the next pair may come into it
        fence_proxy_async();
        __syncwarp();
        f.pass();
        f.send(a, lane);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // (ONE: without a branch, so that the two tiles' chains interleave; what is not there is dropped below)
          if (!ONE && !(some >> u & 1u)) continue;
          const int j0 = 16 * (tile + u);
          // (ONE: the codes become operands group by group; else once for all blocks)
          uint32_t c[ONE ? 1 : G][2][4];
          float2 sc[ONE ? 1 : G];
          if constexpr (!ONE)
#pragma unroll
            for (int g = 0; g < G; ++g) x[u].group(g, lane, c[g], sc[g]);
#pragma unroll 1
          for (int k = 0; k < (ONE ? 1 : blocks); ++k) {
            if constexpr (!ONE) {
              range = *reinterpret_cast<const int4*>(smem + W::kRange + k * 16);
              if (j0 >= range.w || j0 + 16 <= range.z) continue;
              load_block(k);
            }
            float z[4];   // [key][row]
            mma_f16_zero(z, x[u].mn[0], x[u].mn[1], x[u].mn[0], x[u].mn[1], qs.x, qs.y);
#pragma unroll
            for (int g = 0; g < G; ++g) {
              constexpr int kNone = 0;
              const int at = ONE ? kNone : g;
              if constexpr (ONE) x[u].group(g, lane, c[0], sc[0]);
              float acc[4];
              const auto& y = c[at];
              mma_f16_zero(acc, y[0][0], y[1][0], y[0][1], y[1][1], fr[0][g].x, fr[0][g].y);
              mma_f16(acc, y[0][2], y[1][2], y[0][3], y[1][3], fr[0][g].z, fr[0][g].w);
              if constexpr (P == 2) {
                mma_f16(acc, y[0][0], y[1][0], y[0][1], y[1][1], fr[P - 1][g].x, fr[P - 1][g].y);
                mma_f16(acc, y[0][2], y[1][2], y[0][3], y[1][3], fr[P - 1][g].z, fr[P - 1][g].w);
              }
              z[0] = fmaf(sc[at].x, acc[0], z[0]);
              z[1] = fmaf(sc[at].x, acc[1], z[1]);
              z[2] = fmaf(sc[at].y, acc[2], z[2]);
              z[3] = fmaf(sc[at].y, acc[3], z[3]);
            }
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ex2(fmaf(z[i], row[i % 2].x, -row[i % 2].y) * 1.4426950408889634f);
            if (j0 < range.x || j0 + 16 > range.y || (ONE && !(some >> u & 1u))) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int j = j0 + t + 8 * (i / 2);
                if (j < __float_as_int(row[i % 2].z) || j >= __float_as_int(row[i % 2].w) || !(some >> u & 1u)) w[i] = 0.f;
              }
            }
            sum[2 * u] += w[0] + w[1];
            sum[2 * u + 1] += w[2] + w[3];
          }
        }
        // over the four lanes; lane q keeps the q-th: two exchanges
        const float s0 = q & 1 ? sum[0] : sum[1], s1 = q & 1 ? sum[2] : sum[3];
        sum[0] = (q & 1 ? sum[1] : sum[0]) + __shfl_xor_sync(0xFFFFFFFFu, s0, 1);
        sum[1] = (q & 1 ? sum[3] : sum[2]) + __shfl_xor_sync(0xFFFFFFFFu, s1, 1);
        sum[0] = (q & 2 ? sum[1] : sum[0]) + __shfl_xor_sync(0xFFFFFFFFu, q & 2 ? sum[0] : sum[1], 2);
      } else {
        f.pass();
        f.send(a, lane);
      }
      if (key_of(tile) < keys) out[key_of(tile)] = had + sum[0];
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
