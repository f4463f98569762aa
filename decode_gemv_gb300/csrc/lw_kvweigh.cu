// Accumulated attention weight over the 4-bit cache.
#include "lw_kvweigh.cuh"
#include "lw_kv.h"

namespace lw {
namespace {

template <int D, class T>
lw_status launch_few(const WeighArgs& a, dim3 grid, cudaStream_t st) {
  using W = WeighFew<D, T>;
  if (resident_blocks(reinterpret_cast<const void*>(dev::kv_weigh_few_kernel<D, T>), W::kThreads, W::kSmem) < 1)
    return fail(LW_ERR_CUDA, "lw_kv_weigh: the kernel does not fit this device");
  return kv_launch("lw_kv_weigh", dev::kv_weigh_few_kernel<D, T>, grid, W::kThreads, W::kSmem, 1, st, a);
}
template <int D>
lw_status launch_few_t(const WeighArgs& a, dim3 grid, cudaStream_t st) {
  return a.p.dtype == LW_F32   ? launch_few<D, float>(a, grid, st)
         : a.p.dtype == LW_F16 ? launch_few<D, __half>(a, grid, st)
                               : launch_few<D, __nv_bfloat16>(a, grid, st);
}

}  // namespace
}  // namespace lw

using namespace lw;

extern "C" size_t lw_kv_weigh_workspace_bytes(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens) {
  (void)c;
  (void)q_heads;
  (void)q_tokens;
  return 0;
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
  // CTAs of a sequence's head: some 32 tiles a warp (a CTA's start, its rows and first copies, is 2 us), but
  // enough CTAs for the device to be full, if a warp has a tile to do
  const int64_t pairs = (int64_t)a->batch * c->kv_heads;
  const int64_t tiles = ((int64_t)a->table_width * c->page_tokens + 15) / 16;
  const int64_t fill = (2 * device_sm_count() + pairs - 1) / pairs;
  int64_t x = (tiles + 7) / 8 < fill ? (tiles + 7) / 8 : fill;
  if (x < (tiles + 255) / 256) x = (tiles + 255) / 256;
  if (x > 65535) x = 65535;
  const dim3 grid((unsigned)x, (unsigned)c->kv_heads, (unsigned)a->batch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c->head_dim == 64   ? launch_few_t<64>(w, grid, st)
         : c->head_dim == 96 ? launch_few_t<96>(w, grid, st)
                             : launch_few_t<128>(w, grid, st);
}
