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
  int32_t page_tokens, heads;
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
constexpr int kSelect = 1024;

// A CTA a head: kept[b][h], ascending.
__global__ void __launch_bounds__(kSelect) kv_evict_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[256], s_scan[32], s_pick[2];
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  dev::pdl_wait();
  const int n = h == 0 && tid == 0 ? evict_keys<true>(a, b) : evict_keys<false>(a, b);
  const int m = n < a.p.keep ? n : a.p.keep;
  if (h == 0 && tid == 0) a.p.out_len[b] = m;
  int32_t* kept = a.p.kept + ((int64_t)b * a.heads + h) * a.p.keep;
  for (int i = m + tid; i < a.p.keep; i += kSelect) kept[i] = -1;
  if (n <= a.p.keep) {
    for (int i = tid; i < n; i += kSelect) kept[i] = i;
    return;
  }
  // keys [first, last) compete for `need` places
  const int first = a.p.first, last = n - a.p.recent;
  const float* w = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride;
  uint32_t need = (uint32_t)(m - a.p.first - a.p.recent), limit = 0;
  const bool some = need > 0;
  if (some) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0 : ~0u << (shift + 8);
      for (int i = first + tid; i < last; i += kSelect) {
        const uint32_t k = dev::order_key(w[i]);
        if ((k & mask) == limit) atomicAdd(&hist[k >> shift & 255], 1u);
      }
      __syncthreads();
      limit |= dev::pick_digit<kSelect>(hist, need, s_scan, s_pick) << shift;
    }
  }
  for (int i = tid; i < first; i += kSelect) kept[i] = i;
  for (int i = last + tid; i < n; i += kSelect) kept[m - n + i] = i;
  if (!some) return;
  uint32_t above = 0, equal = 0;   // before this stretch of keys
  for (int i0 = first; i0 < last; i0 += kSelect) {
    const int i = i0 + tid;
    const uint32_t k = i < last ? dev::order_key(w[i]) : 0;
    const bool more = i < last && k > limit, same = i < last && k == limit;
    uint32_t total;
    const uint32_t pos = dev::scan_cta<kSelect>((uint32_t)more | (uint32_t)same << 16, s_scan, total);
    const uint32_t ab = above + (pos & 0xFFFFu), eq = equal + (pos >> 16);
    if (more || (same && eq < need)) kept[first + ab + (eq < need ? eq : need)] = i;
    above += total & 0xFFFFu;
    equal += total >> 16;
  }
}

// ---- the move ------------------------------------------------------------------
// A cluster a head; every warp assembles one tile of 16 kept tokens a round.  A
// round's tokens are all read before any is written (a barrier of the cluster
// between), and later rounds' tokens lie behind its places (kept[i] >= i): the
// places may be the source's own.
constexpr int kMoveWarps = 16, kMove = 32 * kMoveWarps;

__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

template <int D>
__global__ void __launch_bounds__(kMove, 2) kv_evict_move_kernel(const EvictArgs a) {
  using L = KvTile<D>;
  constexpr int G = L::G;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int ranks = (int)cluster_size(), rank = (int)cluster_rank();
  const int h = blockIdx.y, b = blockIdx.z, tpp = a.page_tokens / LW_KV_TILE;
  dev::pdl_wait();
  const int n = evict_keys<false>(a, b);
  const int m = n < a.p.keep ? n : a.p.keep;
  const int32_t* kept = a.p.kept + ((int64_t)b * a.heads + h) * a.p.keep;
  const int32_t *from = a.p.page_table + (int64_t)b * a.p.table_stride, *to = a.p.out_table + (int64_t)b * a.p.out_stride;
  const float* w = a.p.weights + b * a.p.w_seq_stride + h * a.p.w_head_stride;
  float* ow = a.p.out_weights ? a.p.out_weights + b * a.p.ow_seq_stride + h * a.p.ow_head_stride : nullptr;
  const int tiles = (m + 15) / 16, step = ranks * kMoveWarps;
  for (int t0 = 0; t0 < tiles; t0 += step) {
    const int tile = t0 + rank * kMoveWarps + warp;
    const bool mine = tile < tiles;
    uint8_t* dst = nullptr;
    float weight = 0.f;
    uint32_t have = 0;
    bool stay = false;
    constexpr int kCodes = 2 * D / 32;   // words of key codes a lane; of value codes as many
    uint32_t kc[kCodes], vc[kCodes], km = 0, ks = 0, vs = 0, vm = 0;
    if (mine) {
      const int page_to = to[tile / tpp];
      const bool dst_ok = page_to >= 0 && page_to < a.n_pages;
      if (!dst_ok && lane == 0) dev::report(a.status, LW_DEV_BAD_PAGE);
      if (dst_ok) dst = a.pages + page_to * a.page_bytes + ((int64_t)h * tpp + tile % tpp) * L::kBytes;
      // lanes 0..15: a token each
      const int i = 16 * tile + lane % 16;
      const int j = i < m ? kept[i] : -1;
      int64_t src = -1;   // the token's tile
      if (j >= 0) {
        const int page = from[j / a.page_tokens];
        if (page >= 0 && page < a.n_pages)
          src = page * a.page_bytes + ((int64_t)h * tpp + (j / LW_KV_TILE) % tpp) * L::kBytes;
        else dev::report(a.status, LW_DEV_BAD_PAGE);
        if (ow) weight = w[j];
      }
      have = __ballot_sync(0xFFFFFFFFu, src >= 0) & 0xFFFFu;
      // all in their places already
      stay = __all_sync(0xFFFFFFFFu, src < 0 || (a.pages + src == dst && j % 16 == lane % 16));
      const auto tok = [&](int t, int& tt) -> const uint8_t* {   // tile and place of the t-th token (all lanes)
        const int64_t s = __shfl_sync(0xFFFFFFFFu, src, t);
        tt = __shfl_sync(0xFFFFFFFFu, j, t) & 15;
        return a.pages + (s < 0 ? 0 : s);
      };
      if (!stay) {
#pragma unroll
        for (int x = 0; x < kCodes; ++x) {
          const int i = lane + 32 * x, t = i / (D / 8);
          int tt;
          const uint8_t* s = tok(t, tt);
          kc[x] = *reinterpret_cast<const uint32_t*>(s + L::kKeyCodes + 4 * (tt * (D / 8) + i % (D / 8)));
        }
        {
          constexpr int kPer = L::GP / 2;
          const int i = lane % (16 * kPer), t = i / kPer;
          int tt;
          const uint8_t* s = tok(t, tt);
          km = *reinterpret_cast<const uint32_t*>(s + L::kKeyMin + 4 * (tt * kPer + i % kPer));
        }
        // words of two tokens: halves of token 2 p and 2 p + 1
#pragma unroll
        for (int x = 0; x < kCodes; ++x) {
          const int i = lane + 32 * x, p = i / (8 * G), r = i % (8 * G);
          uint32_t v = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int tt;
            const uint8_t* s = tok(2 * p + e, tt);
            v |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kValCodes + 4 * (tt / 2 * 8 * G + r) + 2 * (tt % 2)) << (16 * e);
          }
          vc[x] = v;
        }
        {
          const int i = lane % (8 * G), p = i / G, g = i % G;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            int tt;
            const uint8_t* s = tok(2 * p + e, tt);
            const int at = 4 * (tt / 2 * G + g) + 2 * (tt % 2);
            ks |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kKeyScale + at) << (16 * e);
            vs |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kValScale + at) << (16 * e);
            vm |= (uint32_t) * reinterpret_cast<const uint16_t*>(s + L::kValMin + at) << (16 * e);
          }
        }
      }
    }
    cluster_sync();
    if (mine) {
      const int i = 16 * tile + lane;
      if (ow && lane < 16 && i < m) ow[i] = weight;
      if (dst && !stay) {
        const auto put = [&](uint8_t* at, uint32_t v, int t) {   // a word of tokens t and t + 1
          if ((have >> t & 3u) == 3u) *reinterpret_cast<uint32_t*>(at) = v;
          else if (have >> t & 1u) *reinterpret_cast<uint16_t*>(at) = (uint16_t)v;
          else if (have >> (t + 1) & 1u) *reinterpret_cast<uint16_t*>(at + 2) = (uint16_t)(v >> 16);
        };
#pragma unroll
        for (int x = 0; x < kCodes; ++x) {
          const int i = lane + 32 * x;
          if (have >> (i / (D / 8)) & 1u) *reinterpret_cast<uint32_t*>(dst + L::kKeyCodes + 4 * i) = kc[x];
          put(dst + L::kValCodes + 4 * i, vc[x], 2 * (i / (8 * G)));
        }
        constexpr int kPer = L::GP / 2;
        if (lane < 16 * kPer && (have >> (lane / kPer) & 1u)) *reinterpret_cast<uint32_t*>(dst + L::kKeyMin + 4 * lane) = km;
        if (lane < 8 * G) {
          put(dst + L::kKeyScale + 4 * lane, ks, 2 * (lane / G));
          put(dst + L::kValScale + 4 * lane, vs, 2 * (lane / G));
          put(dst + L::kValMin + 4 * lane, vm, 2 * (lane / G));
        }
      }
    }
  }
  if (!ow) return;
  cluster_sync();   // (weights behind the kept ones' places were read by then)
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
  s = kv_launch(fn, kv_evict_select_kernel, dim3((unsigned)c->kv_heads, (unsigned)p->batch), kSelect, 0, 1, st, a);
  if (s != LW_OK) return s;
  // CTAs of a head, until the device is full twice over (two fit an SM)
  const int64_t pairs = (int64_t)p->batch * c->kv_heads, rounds = (p->keep + 16 * kMoveWarps - 1) / (16 * kMoveWarps);
  int ranks = 1;
  while (ranks < 8 && ranks < rounds && 2 * ranks * pairs <= 2 * device_sm_count()) ranks *= 2;
  const dim3 grid((unsigned)ranks, (unsigned)c->kv_heads, (unsigned)p->batch);
  return c->head_dim == 64   ? kv_launch(fn, kv_evict_move_kernel<64>, grid, kMove, 0, ranks, st, a)
         : c->head_dim == 96 ? kv_launch(fn, kv_evict_move_kernel<96>, grid, kMove, 0, ranks, st, a)
                             : kv_launch(fn, kv_evict_move_kernel<128>, grid, kMove, 0, ranks, st, a);
}
