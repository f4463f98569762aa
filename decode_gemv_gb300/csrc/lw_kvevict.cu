// Eviction from the 4-bit cache by accumulated attention weight.
#include "lw_kv.cuh"
#include "lw_kv.h"
#include "lw_kvselect.cuh"

namespace lw {
namespace {

struct EvictArgs {
  lw_kv_eviction p;
  uint8_t* pages;
  int64_t n_pages, page_bytes;
  int32_t page_tokens, heads, most_keys;
  int32_t* status;
};

template <bool LOUD>
__device__ __forceinline__ int evict_keys(const EvictArgs& a, int b) {
  const int n = a.p.kv_len[b];
  int64_t most = (int64_t)a.p.table_width * a.page_tokens;
  if (a.p.w_keys < most) most = a.p.w_keys;
  if (LOUD && (n < 0 || n > most)) dev::report(a.status, LW_DEV_BAD_SEQ);
  return n < 0 ? 0 : (n > most ? (int)most : n);
}

// ---- the choice ----------------------------------------------------------------
// A cluster a head (lw_kvselect.cuh); a stretch that is too long for shared memory is read again instead.  64 heads'
// 65536 keys some 32 us, where 17 MB have to come: after the load a CTA walks its keys five times (three digits by
// atomics in shared memory, the count, the places), with barriers between.
constexpr int kMostSelect = 40960;   // order keys a CTA keeps
constexpr int kSelect = 512;
using EvictShared = dev::SelectShared<11>;

__global__ void __launch_bounds__(kSelect) kv_evict_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t smem[];
  EvictShared& s = *reinterpret_cast<EvictShared*>(smem);
  uint32_t* keys = smem + sizeof(EvictShared) / 4;     // [a.most_keys]
  const int h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int rank = (int)dev::cluster_rank();
  for (int i = tid; i < EvictShared::kPasses * EvictShared::kBins; i += kSelect) s.hist[i] = 0;
  dev::pdl_wait();
  const int n = h == 0 && rank == 0 && tid == 0 ? evict_keys<true>(a, b) : evict_keys<false>(a, b);
  const int m = n < a.p.keep ? n : a.p.keep;
  if (h == 0 && rank == 0 && tid == 0) a.p.out_len[b] = m;
  int32_t* kept = a.p.kept + ((int64_t)b * a.heads + h) * a.p.keep;
  const int self = rank * kSelect + tid, all = (int)dev::cluster_size() * kSelect;
  for (int64_t i = (int64_t)m + self; i < a.p.keep; i += all) kept[i] = -1;
  if (n <= a.p.keep) {   // (the same in all of the cluster)
    for (int64_t i = self; i < n; i += all) kept[i] = (int)i;
    return;
  }
  // keys [first, last) compete for `need` places
  const int first = a.p.first, last = n - a.p.recent;
  for (int64_t i = self; i < first; i += all) kept[i] = (int)i;
  for (int64_t i = (int64_t)last + self; i < n; i += all) kept[m - n + i] = (int)i;
  const uint32_t need = (uint32_t)(m - first - a.p.recent);
  if (need == 0) return;
  int count;
  const int64_t from = dev::select_stretch(first, last, count);
  const float* w = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride + from;
  const bool here = count <= a.most_keys;
  if (here) {
    constexpr int kAhead = 8;
    for (int i0 = tid; i0 < count; i0 += kAhead * kSelect) {
      float x[kAhead];
#pragma unroll
      for (int e = 0; e < kAhead; ++e) x[e] = i0 + e * kSelect < count ? w[i0 + e * kSelect] : 0.f;
#pragma unroll
      for (int e = 0; e < kAhead; ++e)
        if (i0 + e * kSelect < count) keys[i0 + e * kSelect] = dev::order_key(x[e]);
    }
  }
  __syncthreads();
  dev::select_places<kSelect, 11>(s, count, need, [&](int i) { return here ? keys[i] : dev::order_key(w[i]); },
                     [&](int place, int i) { kept[first + place] = (int)(from + i); });
}

// ---- the move ------------------------------------------------------------------
// A cluster a head; every warp assembles one tile of 16 kept tokens a round,
// while the next round's tokens are looked up.  In place a round's tokens are all
// read before any is written (a barrier of the cluster between), and later
// rounds' tokens lie behind its places (kept[i] >= i); into other pages, the
// warps need not wait for one another.
// 64 heads' 8192 of 65536 keys: the call 88 us into other pages, 97 in place (the choice among them some 32: keeping one
// key takes 35).  The 84 MB that move are read as some 235: a token of 160 bytes lies in ten sectors (its pair's value
// codes, scales and minimums beside its own), and memory gives 64 bytes at a time: 47 us at a copy's rate.
constexpr int kMoveWarps = 16, kMove = 32 * kMoveWarps;

// The tokens of a tile: lane i (and i + 16) has the i-th.
struct MoveTokens {
  int64_t src;   // its tile, -1 if there is none
  int j;         // its key, -1 if there is none
  float weight;
};

template <int D>
struct MoveTile {
  using L = KvTile<D>;
  static constexpr int G = L::G;
  static constexpr int kCodes = 2 * D / 32;   // words of key codes a lane; of value codes as many
  uint32_t kc[kCodes], vc[kCodes], km, ks, vs, vm;

  // tile and place of the token in lane t (all lanes ask)
  static __device__ __forceinline__ const uint8_t* token(const uint8_t* pages, const MoveTokens& x, int t, int& tt) {
    const int64_t s = __shfl_sync(0xFFFFFFFFu, x.src, t);
    tt = __shfl_sync(0xFFFFFFFFu, x.j, t) & 15;
    return pages + (s < 0 ? 0 : s);   // (what is not there is read from the first tile, and not written)
  }
  __device__ __forceinline__ void read(const uint8_t* pages, const MoveTokens& x, int lane) {
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const int at = lane + 32 * i;
      int tt;
      const uint8_t* s = token(pages, x, at / (D / 8), tt);
      kc[i] = *reinterpret_cast<const uint32_t*>(s + L::kKeyCodes + 4 * (tt * (D / 8) + at % (D / 8)));
    }
    {
      constexpr int kPer = L::GP / 2;
      const int at = lane % (16 * kPer);
      int tt;
      const uint8_t* s = token(pages, x, at / kPer, tt);
      km = *reinterpret_cast<const uint32_t*>(s + L::kKeyMin + 4 * (tt * kPer + at % kPer));
    }
    // words of two tokens
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const int at = lane + 32 * i, p = at / (8 * G), r = at % (8 * G);
      uint32_t v = 0;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        int tt;
        const uint8_t* s = token(pages, x, 2 * p + e, tt);
        v |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kValCodes + 4 * (tt / 2 * 8 * G + r) + 2 * (tt % 2)) << (16 * e);
      }
      vc[i] = v;
    }
    const int at = lane % (8 * G), p = at / G, g = at % G;
    ks = vs = vm = 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      int tt;
      const uint8_t* s = token(pages, x, 2 * p + e, tt);
      const int o = 4 * (tt / 2 * G + g) + 2 * (tt % 2);
      ks |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kKeyScale + o) << (16 * e);
      vs |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kValScale + o) << (16 * e);
      vm |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kValMin + o) << (16 * e);
    }
  }
  // `have`: which tokens there are
  __device__ __forceinline__ void write(uint8_t* dst, uint32_t have, int lane) const {
    const auto put = [&](uint8_t* at, uint32_t v, int t) {   // a word of tokens t and t + 1
      if ((have >> t & 3u) == 3u) *reinterpret_cast<uint32_t*>(at) = v;
      else if (have >> t & 1u) *reinterpret_cast<uint16_t*>(at) = (uint16_t)v;
      else if (have >> (t + 1) & 1u) *reinterpret_cast<uint16_t*>(at + 2) = (uint16_t)(v >> 16);
    };
#pragma unroll
    for (int i = 0; i < kCodes; ++i) {
      const int at = lane + 32 * i;
      if (have >> (at / (D / 8)) & 1u) *reinterpret_cast<uint32_t*>(dst + L::kKeyCodes + 4 * at) = kc[i];
      put(dst + L::kValCodes + 4 * at, vc[i], 2 * (at / (8 * G)));
    }
    constexpr int kPer = L::GP / 2;
    if (lane < 16 * kPer && (have >> (lane / kPer) & 1u)) *reinterpret_cast<uint32_t*>(dst + L::kKeyMin + 4 * lane) = km;
    if (lane < 8 * G) {
      put(dst + L::kKeyScale + 4 * lane, ks, 2 * (lane / G));
      put(dst + L::kValScale + 4 * lane, vs, 2 * (lane / G));
      put(dst + L::kValMin + 4 * lane, vm, 2 * (lane / G));
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kMove, 2) kv_evict_move_kernel(const EvictArgs a) {
  using L = KvTile<D>;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ranks = (int)dev::cluster_size(), rank = (int)dev::cluster_rank();
  const int h = blockIdx.y, b = blockIdx.z, tpp = a.page_tokens / LW_KV_TILE;
  dev::pdl_wait();
  const int n = evict_keys<false>(a, b);
  const int m = n < a.p.keep ? n : a.p.keep;
  const int32_t* kept = a.p.kept + ((int64_t)b * a.heads + h) * a.p.keep;
  const int32_t *from = a.p.page_table + (int64_t)b * a.p.table_stride, *to = a.p.out_table + (int64_t)b * a.p.out_stride;
  const float* w = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride;
  float* ow = a.p.out_weights ? a.p.out_weights + b * a.p.ow_seq_stride + h * a.p.ow_head_stride : nullptr;
  const int tiles = (m + 15) / 16, step = ranks * kMoveWarps;
  // places that are read as well (the same in all of the cluster)
  const bool in_place = tiles > 0 && (from[0] == to[0] || w == ow);
  const auto key_of = [&](int tile) {   // this lane's kept key
    const int i = 16 * tile + lane % 16;
    return tile < tiles && i < m ? kept[i] : -1;
  };
  const auto look = [&](int j) {
    MoveTokens x{-1, j, 0.f};
    if (j >= 0) {
      const int page = from[j / a.page_tokens];
      if (page >= 0 && page < a.n_pages)
        x.src = page * a.page_bytes + ((int64_t)h * tpp + (j / LW_KV_TILE) % tpp) * L::kBytes;
      else dev::report(a.status, LW_DEV_BAD_PAGE);
      if (ow) x.weight = w[j];
    }
    return x;
  };
  const auto place = [&](int tile) -> uint8_t* {
    if (tile >= tiles) return nullptr;
    const int page = to[tile / tpp];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) dev::report(a.status, LW_DEV_BAD_PAGE);
      return nullptr;
    }
    return a.pages + page * a.page_bytes + ((int64_t)h * tpp + tile % tpp) * L::kBytes;
  };
  int tile = rank * kMoveWarps + warp;
  MoveTokens x = look(key_of(tile));
  int next_key = key_of(tile + step);
  for (int t0 = 0; t0 < tiles; t0 += step, tile += step) {
    uint8_t* const dst = place(tile);
    // a tile whose tokens are all in their places already is left as it is
    const bool stay = __all_sync(0xFFFFFFFFu, x.src < 0 || (a.pages + x.src == dst && x.j % 16 == lane % 16));
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, x.src >= 0) & 0xFFFFu;
    const bool move = dst && !stay;
    MoveTile<D> z;
    if (move) z.read(a.pages, x, lane);
    const MoveTokens y = look(next_key);   // (behind this round's places)
    next_key = key_of(tile + 2 * step);
    if (in_place) dev::cluster_sync();
    if (ow && lane < 16 && x.j >= 0) ow[16 * tile + lane] = x.weight;
    if (move) z.write(dst, have, lane);
    x = y;
  }
  if (!ow) return;
  if (in_place) dev::cluster_sync();   // (weights behind the kept ones' places have been read by then)
  const int64_t end = n < a.p.ow_keys ? n : a.p.ow_keys;
  for (int64_t i = m + rank * kMove + (int)threadIdx.x; i < end; i += ranks * kMove) ow[i] = 0.f;
}

}  // namespace
}  // namespace lw

using namespace lw;

extern "C" lw_status lw_kv_evict(const lw_kv_cache* c, const lw_kv_eviction* p, int32_t* d_status, void* stream) {
  const char* fn = "lw_kv_evict";
  clear_error();
  lw_status s = check_kv_cache(c);
  if (s != LW_OK) return s;
  if (!p) return fail(LW_ERR_INVALID_ARG, "NULL arguments");
  if (p->batch < 1 || p->batch > 65535) return fail(LW_ERR_SHAPE, "%s: batch %d (1..65535)", fn, p->batch);
  if (p->keep < 1 || p->first < 0 || p->recent < 0 || (int64_t)p->first + p->recent > p->keep)
    return fail(LW_ERR_INVALID_ARG, "%s: keep %d, first %d, recent %d", fn, p->keep, p->first, p->recent);
  if (p->table_width < 0 || p->table_stride < 0 || (int64_t)p->table_width * c->page_tokens > kKvMost)
    return fail(LW_ERR_SHAPE, "%s: page table of %d pages of %d tokens", fn, p->table_width, c->page_tokens);
  if (p->out_width < 0 || p->out_stride < 0 || (int64_t)p->out_width * c->page_tokens > kKvMost ||
      (int64_t)p->out_width * c->page_tokens < p->keep)
    return fail(LW_ERR_SHAPE, "%s: %d pages of %d tokens for %d keys", fn, p->out_width, c->page_tokens, p->keep);
  if (p->w_keys < 0 || (p->out_weights && p->ow_keys < p->keep))
    return fail(LW_ERR_SHAPE, "%s: rows of %lld weights, of %lld that are kept", fn, (long long)p->w_keys,
                (long long)p->ow_keys);
  if (!p->kv_len || !p->out_table || !p->out_len || !p->kept || (p->table_width && !p->page_table) ||
      (p->w_keys && !p->weights))
    return fail(LW_ERR_INVALID_ARG, "%s: NULL weights, kv_len, out_len, kept or a page table", fn);
  const auto off = [](const void* x) { return reinterpret_cast<uintptr_t>(x) % 4 != 0; };
  if (off(p->weights) || off(p->kv_len) || off(p->page_table) || off(p->out_table) || off(p->out_len) ||
      off(p->out_weights) || off(p->kept))
    return fail(LW_ERR_INVALID_ARG, "%s: an address is not aligned to its type", fn);
  if (p->out_len == p->kv_len) return fail(LW_ERR_INVALID_ARG, "%s: out_len is kv_len", fn);
  EvictArgs a{};
  a.p = *p;
  a.pages = static_cast<uint8_t*>(c->pages);
  a.n_pages = c->n_pages;
  a.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  a.page_tokens = c->page_tokens;
  a.heads = c->kv_heads;
  a.status = d_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // CTAs of a head.  The choice: some 4096 keys each, as far as three an SM have room
  const int64_t pairs = (int64_t)p->batch * c->kv_heads, sms = device_sm_count();
  int64_t keys = (int64_t)p->table_width * c->page_tokens;
  if (p->w_keys < keys) keys = p->w_keys;
  int ranks = 1;
  while (ranks < 8 && 2 * ranks * pairs <= 3 * sms && keys > 4096ll * ranks) ranks *= 2;
  int64_t most = kv_select_room(keys, ranks);
  if (most > kMostSelect) most = kMostSelect;
  a.most_keys = (int32_t)most;
  const size_t smem = sizeof(EvictShared) + (size_t)most * 4;
  if (resident_blocks(reinterpret_cast<const void*>(kv_evict_select_kernel), kSelect, smem) < 1)
    return fail(LW_ERR_CUDA, "%s: the kernel does not fit this device", fn);
  s = kv_launch(fn, kv_evict_select_kernel, dim3((unsigned)ranks, (unsigned)c->kv_heads, (unsigned)p->batch), kSelect,
                smem, ranks, st, a);
  if (s != LW_OK) return s;
  // The move: until the device is full (two an SM)
  const int64_t rounds = (p->keep + 16 * kMoveWarps - 1) / (16 * kMoveWarps);
  ranks = 1;
  while (ranks < 8 && ranks < rounds && 2 * ranks * pairs <= 2 * sms) ranks *= 2;
  const dim3 grid((unsigned)ranks, (unsigned)c->kv_heads, (unsigned)p->batch);
  return c->head_dim == 64   ? kv_launch(fn, kv_evict_move_kernel<64>, grid, kMove, 0, ranks, st, a)
         : c->head_dim == 96 ? kv_launch(fn, kv_evict_move_kernel<96>, grid, kMove, 0, ranks, st, a)
                             : kv_launch(fn, kv_evict_move_kernel<128>, grid, kMove, 0, ranks, st, a);
}
