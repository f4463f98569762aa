// Accumulated attention weight over the 4-bit cache.
#include "lw_kvweighmany.cuh"
#include "lw_kv.h"

namespace lw {
namespace {

template <int D, class T, bool ONE>
lw_status launch_few(const WeighArgs& a, dim3 grid, cudaStream_t st) {
  using W = WeighFew<D, T, ONE>;
  const auto kernel = dev::kv_weigh_few_kernel<D, T, ONE>;
  if (resident_blocks(reinterpret_cast<const void*>(kernel), W::kThreads, W::kSmem) < 1)
    return fail(LW_ERR_CUDA, "lw_kv_weigh: the kernel does not fit this device");
  return kv_launch("lw_kv_weigh", kernel, grid, W::kThreads, W::kSmem, 1, st, a);
}
template <int D, bool ONE>
lw_status launch_few_t(const WeighArgs& a, dim3 grid, cudaStream_t st) {
  return a.p.dtype == LW_F32   ? launch_few<D, float, ONE>(a, grid, st)
         : a.p.dtype == LW_F16 ? launch_few<D, __half, ONE>(a, grid, st)
                               : launch_few<D, __nv_bfloat16, ONE>(a, grid, st);
}
template <int D>
lw_status launch_few_d(const WeighArgs& a, bool one, dim3 grid, cudaStream_t st) {
  return one ? launch_few_t<D, true>(a, grid, st) : launch_few_t<D, false>(a, grid, st);
}

// The variant, by the rows of a sequence on a key/value head.  us, 8 sequences of 32768 keys | 64 of 512, 8 heads of
// 128: a block of 8 rows in registers, 64 rows in shared memory, kv_weigh_many_kernel
//   bf16   8 rows   57  71        |  12  13        fp32   8 rows   71  81        |  14  15
//         16 rows  110  89        |  22  16              16 rows  138 107        |  25  19
//        128 rows  855 397  455   | 157  59  73         128 rows 1076 542  464   | 185  79  83
//        160 rows      519  554   |      77  87         160 rows      705  603   |     102 104
//        192 rows      594  550   |      87  88
// One sequence of 8192 keys alone: bf16 256 rows 35 and 24, fp32 192 rows 35 and 28.  (kv_weigh_many_kernel takes
// rows 128 at a time, and a unit of 128 keys starts slowly.  Between 64 and 128 rows in fp32 the first 64 cost 271
// and the next ones as much.)
constexpr int kOneMost = 8, kFewMost16 = 160, kFewMost32 = 112;

inline int64_t row_tiles(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens) {
  return (q_tokens * (q_heads / c->kv_heads) + 127) / 128;
}
inline size_t record_bytes(int D, int parts) { return (size_t)parts * D * 256 + 1024; }

template <int D, class T>
lw_status launch_many(const WeighArgs& a, void* ws, int64_t tiles, int64_t key_tiles, cudaStream_t st) {
  constexpr int kParts = sizeof(T) == 4 ? 2 : 1;
  using W = WeighMany<D, kParts>;
  const auto kernel = dev::kv_weigh_many_kernel<D, kParts>;
  if (resident_blocks(reinterpret_cast<const void*>(kernel), W::kThreads, W::kSmem) < 1)
    return fail(LW_ERR_CUDA, "lw_kv_weigh: the kernel does not fit this device");
  const WeighRowsArgs r{a, static_cast<uint8_t*>(ws), (int32_t)tiles};
  const lw_status s = kv_launch("lw_kv_weigh", dev::kv_weigh_rows_kernel<D, T>, dim3((unsigned)tiles, (unsigned)a.heads),
                                512, 0, 1, st, r);
  if (s != LW_OK) return s;
  const WeighManyArgs w{a, static_cast<const uint8_t*>(ws), (int32_t)tiles};
  // CTAs of a sequence's head: each takes every so many-th unit, and fetches the next one's keys meanwhile.  One
  // sequence's units are alike: as many CTAs as the device takes at once, if that many fit its heads; several
  // sequences may not be: some rounds of CTAs, of 4 to 8 the one that wastes least (a table may also be far wider
  // than its sequences are long: a CTA without keys costs 2 us).
  const int64_t pairs = (int64_t)a.heads * a.p.batch, sms = device_sm_count();
  int64_t x = 1;
  double best = 0.0;
  for (int k = a.p.batch == 1 ? 1 : 4; k <= 8 && best < 0.95; ++k) {
    const int64_t n = k * sms / pairs > 1 ? k * sms / pairs : 1;
    const double use = (double)(n * pairs) / (double)((n * pairs + sms - 1) / sms * sms);
    if (use > best) {
      best = use;
      x = n;
    }
  }
  if (x > key_tiles) x = key_tiles;
  // CTAs of a unit, until the device is full
  int ranks = 1;
  while (ranks < 8 && 2 * ranks * key_tiles * pairs <= device_sm_count()) ranks *= 2;
  return kv_launch("lw_kv_weigh", kernel, dim3((unsigned)(x * ranks), (unsigned)a.heads, (unsigned)a.p.batch),
                   W::kThreads, W::kSmem, ranks, st, w);
}
template <int D>
lw_status launch_many_t(const WeighArgs& a, void* ws, int64_t tiles, int64_t key_tiles, cudaStream_t st) {
  return a.p.dtype == LW_F32   ? launch_many<D, float>(a, ws, tiles, key_tiles, st)
         : a.p.dtype == LW_F16 ? launch_many<D, __half>(a, ws, tiles, key_tiles, st)
                               : launch_many<D, __nv_bfloat16>(a, ws, tiles, key_tiles, st);
}

}  // namespace
}  // namespace lw

using namespace lw;

extern "C" size_t lw_kv_weigh_workspace_bytes(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens) {
  if (!c || !lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens) || q_heads < 1 || q_heads % c->kv_heads ||
      q_tokens < 0 || q_tokens > kKvMost / q_heads)
    return 0;
  // none for few rows in all: whatever sequences they are of, kv_weigh_few_kernel takes them, in every type
  if (q_tokens * (q_heads / c->kv_heads) <= kFewMost32) return 0;
  return kv_counter_bytes() + (size_t)c->kv_heads * row_tiles(c, q_heads, q_tokens) * record_bytes(c->head_dim, 2);
}

extern "C" lw_status lw_kv_weigh(const lw_kv_cache* c, const lw_kv_weights* a, void* ws, size_t ws_bytes,
                                 int32_t* d_status, void* stream) {
  const char* fn = "lw_kv_weigh";
  clear_error();
  lw_status s = check_kv_cache(c);
  if (s != LW_OK) return s;
  if (!a) return fail(LW_ERR_INVALID_ARG, "NULL arguments");
  if (!kv_type_ok(a->dtype)) return fail(LW_ERR_UNSUPPORTED, "%s: unknown type %d", fn, a->dtype);
  if (a->q_heads < 1 || a->q_heads > 65535 || a->q_heads % c->kv_heads)
    return fail(LW_ERR_SHAPE, "%s: %d query heads on %d key/value heads", fn, a->q_heads, c->kv_heads);
  if (a->batch < 1 || a->batch > 65535) return fail(LW_ERR_SHAPE, "%s: batch %d (1..65535)", fn, a->batch);
  if (a->q_tokens < 0 || a->q_tokens > (1ll << 31) - 1 || a->q_tokens * a->q_heads > kKvMost ||
      (int64_t)a->max_q * a->q_heads > kKvMost)
    return fail(LW_ERR_SHAPE, "%s: %lld query tokens of %d heads", fn, (long long)a->q_tokens, a->q_heads);
  if (a->max_q < 0) return fail(LW_ERR_INVALID_ARG, "%s: max_q %d", fn, a->max_q);
  if (a->window < 0) return fail(LW_ERR_INVALID_ARG, "%s: window %d", fn, a->window);
  if (a->causal != 0 && a->causal != 1) return fail(LW_ERR_INVALID_ARG, "%s: causal %d", fn, a->causal);
  if (!(a->scale >= -3.402823466e38f && a->scale <= 3.402823466e38f))
    return fail(LW_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  if (a->table_width < 0 || a->table_stride < 0 || (int64_t)a->table_width * c->page_tokens > kKvMost)
    return fail(LW_ERR_SHAPE, "%s: page table of %d pages of %d tokens", fn, a->table_width, c->page_tokens);
  if (a->w_keys < 0) return fail(LW_ERR_INVALID_ARG, "%s: rows of %lld weights", fn, (long long)a->w_keys);
  if (a->table_width == 0 || a->w_keys == 0) return LW_OK;   // no key has a place
  if (!a->q_start || !a->kv_len || !a->page_table || !a->weights || (a->q_tokens && (!a->q || !a->lse)))
    return fail(LW_ERR_INVALID_ARG, "%s: NULL q, lse, q_start, kv_len, page_table or weights", fn);
  const auto off = [](const void* x, uintptr_t n) { return reinterpret_cast<uintptr_t>(x) % n != 0; };
  if (off(a->q, (uintptr_t)kv_type_bytes(a->dtype)) || off(a->lse, 4) || off(a->q_start, 4) || off(a->kv_len, 4) ||
      off(a->page_table, 4) || off(a->add_to, 4) || off(a->weights, 4))
    return fail(LW_ERR_INVALID_ARG, "%s: an address is not aligned to its type", fn);
  const size_t need = lw_kv_weigh_workspace_bytes(c, a->q_heads, a->q_tokens);
  if (need && (!ws || ws_bytes < need || off(ws, 16)))
    return fail(LW_ERR_INVALID_ARG, "%s: workspace missing, misaligned or %zu bytes of %zu", fn, ws_bytes, need);
  WeighArgs w{};
  w.p = *a;
  w.pages = static_cast<const uint8_t*>(c->pages);
  w.n_pages = c->n_pages;
  w.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  w.page_tokens = c->page_tokens;
  w.heads = c->kv_heads;
  w.group = a->q_heads / c->kv_heads;
  w.vec = kv_rows_aligned(a->q, a->q_token_stride, a->q_head_stride, a->dtype);
  w.status = d_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int64_t keys = (int64_t)a->table_width * c->page_tokens;
  if (a->w_keys < keys) keys = a->w_keys;
  const int64_t rows = (a->max_q < a->q_tokens ? a->max_q : a->q_tokens) * w.group;
  if (rows > (a->dtype == LW_F32 ? kFewMost32 : kFewMost16)) {
    const int64_t tiles = row_tiles(c, a->q_heads, a->q_tokens), key_tiles = (keys + 127) / 128;
    ws = static_cast<uint8_t*>(ws) + kv_counter_bytes();   // (which may be attention's workspace)
    return c->head_dim == 64   ? launch_many_t<64>(w, ws, tiles, key_tiles, st)
           : c->head_dim == 96 ? launch_many_t<96>(w, ws, tiles, key_tiles, st)
                               : launch_many_t<128>(w, ws, tiles, key_tiles, st);
  }
  // CTAs of a sequence's head: some 32 tiles a warp (a CTA's start, its rows and first copies, is 2 us), but
  // enough CTAs for the device to be full, if a warp has a pair of tiles to do
  const int64_t pairs = (int64_t)a->batch * c->kv_heads;
  const int64_t tiles = (keys + 15) / 16;
  const int64_t fill = (2 * device_sm_count() + pairs - 1) / pairs;
  int64_t x = (tiles + 15) / 16 < fill ? (tiles + 15) / 16 : fill;
  if (x < (tiles + 255) / 256) x = (tiles + 255) / 256;
  const int64_t most = (32 * device_sm_count() + pairs - 1) / pairs;   // (tables far wider than the sequences are long)
  if (x > most) x = most;
  const dim3 grid((unsigned)x, (unsigned)c->kv_heads, (unsigned)a->batch);
  return c->head_dim == 64   ? launch_few_d<64>(w, rows <= kOneMost, grid, st)
         : c->head_dim == 96 ? launch_few_d<96>(w, rows <= kOneMost, grid, st)
                             : launch_few_d<128>(w, rows <= kOneMost, grid, st);
}
