// The 4-bit key/value cache: argument checks of its calls, and the kernels
// that write tokens into it and read them back.
#include "lw_kv.cuh"
#include "lw_kv.h"

namespace lw {

lw_status check_kv_cache(const lw_kv_cache* c) {
  if (!c) return fail(LW_ERR_INVALID_ARG, "NULL cache");
  if (!lw_kv_tile_bytes(c->head_dim))
    return fail(LW_ERR_UNSUPPORTED, "head_dim %d: 64, 96 and 128 are supported", c->head_dim);
  if (!lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens))
    return fail(LW_ERR_SHAPE, "kv_heads %d, page_tokens %d (a positive multiple of %d)", c->kv_heads,
                c->page_tokens, LW_KV_TILE);
  if (c->n_pages < 1 || c->n_pages > ((1ll << 32) - 1) / c->page_tokens)
    return fail(LW_ERR_SHAPE, "%lld pages of %d tokens", (long long)c->n_pages, c->page_tokens);
  if (!c->pages || (reinterpret_cast<uintptr_t>(c->pages) & 15u))
    return fail(LW_ERR_INVALID_ARG, "pages missing or not 16-byte aligned");
  return LW_OK;
}

namespace {

struct RowsArgs {
  void* ptr;
  int64_t token_stride, head_stride;
};
struct CacheArgs {
  RowsArgs k, v;
  uint8_t* pages;
  const int64_t* slots;
  int64_t n, n_slots, page_bytes;
  int32_t page_tiles, page_shift, heads;   // page_tiles = 2^page_shift, or page_shift < 0
  int32_t* status;
};

// The tile of a slot (head 0: its place in the pages; -1 if the slot is not
// stored).  A slot past the pages is reported where `first`.
__device__ __forceinline__ int64_t slot_tile(const CacheArgs& a, int64_t slot, int tile_bytes, bool first) {
  if (slot < 0 || slot >= a.n_slots) {
    if (slot >= 0 && first) dev::report(a.status, LW_DEV_BAD_SLOT);
    return -1;
  }
  const uint32_t tile = (uint32_t)(slot / LW_KV_TILE);   // (slots are below 2^32)
  const uint32_t page = a.page_shift >= 0 ? tile >> a.page_shift : tile / (uint32_t)a.page_tiles;
  return page * a.page_bytes + (int64_t)(tile - page * (uint32_t)a.page_tiles) * tile_bytes;
}

// Both kernels: a block takes 16 tokens of one head (a tile of the cache, if they
// are consecutive, whose lines it completes), a thread 8 consecutive keys and the
// same 8 values of one of them (4 neighbouring lanes a group).  The bytes that
// have to move are 2 in or out a bf16 element and 0.625 for the cache.
// Measured, 65536 tokens of 8 heads of 128 in bf16: write 87 us, 4.05 TB/s
// (issue-bound: 84 % of the slots, 21 instructions a value: a third of them the
// definition's steps on each value, the rest a group's scale, minimum, reciprocal
// and limits, done in all four lanes of the group, and a token's slot, tile and
// addresses, for every 8 + 8 values), read 68 us, 5.2 TB/s.  A copy reaches 6.8.
constexpr int kTokens = 16;

template <class T, int D, bool VEC>
__global__ void __launch_bounds__(kTokens * D / 8) kv_write_kernel(const CacheArgs a) {
  using L = KvTile<D>;
  constexpr int kChunks = D / 8;
  const int64_t tok = (int64_t)blockIdx.x * kTokens + threadIdx.x / kChunks;
  const int ch = threadIdx.x % kChunks, h = blockIdx.y;
  dev::pdl_wait();
  int64_t at = -1, slot = -1;
  float k[8] = {}, v[8] = {}, lo[2] = {}, hi[2] = {};
  if (tok < a.n) {
    slot = a.slots[tok];
    dev::kv_load8_range<T, VEC>(static_cast<const T*>(a.k.ptr) + tok * a.k.token_stride + h * a.k.head_stride + 8 * ch,
                                k, lo[0], hi[0]);
    dev::kv_load8_range<T, VEC>(static_cast<const T*>(a.v.ptr) + tok * a.v.token_stride + h * a.v.head_stride + 8 * ch,
                                v, lo[1], hi[1]);
    at = slot_tile(a, slot, L::kBytes, h == 0 && ch == 0);
  }
  __half ks, km, vs, vm;
  const uint32_t kw = dev::kv_quantise8(k, lo[0], hi[0], ks, km), vw = dev::kv_quantise8(v, lo[1], hi[1], vs, vm);
  if (at < 0) return;
  const int t = (int)(slot % LW_KV_TILE), g = ch >> 2, q = ch & 3;
  uint8_t* tile = a.pages + at + (int64_t)h * a.page_tiles * L::kBytes;
  const int par = 2 * ((t / 2 * L::G + g) * 2 + t % 2);
  *reinterpret_cast<uint32_t*>(tile + L::kKeyCodes + 4 * ((t * 4 + q) * L::G + g)) = kw;
  uint8_t* u = tile + L::kValCodes + 4 * ((t / 2 * 8 + 2 * q) * L::G + g) + 2 * (t % 2);
  *reinterpret_cast<uint16_t*>(u) = (uint16_t)vw;
  *reinterpret_cast<uint16_t*>(u + 4 * L::G) = (uint16_t)(vw >> 16);
  // a lane of the group each
  if (q == 0) *reinterpret_cast<__half*>(tile + L::kKeyScale + par) = ks;
  if (q == 1) *reinterpret_cast<__half*>(tile + L::kKeyMin + 2 * (t * L::GP + g)) = km;
  if (q == 2) *reinterpret_cast<__half*>(tile + L::kValScale + par) = vs;
  if (q == 3) *reinterpret_cast<__half*>(tile + L::kValMin + par) = vm;
}

// scale * code + min of 8 codes
__device__ __forceinline__ void restore8(uint32_t w, __half scale, __half low, float (&x)[8]) {
  const float s = __half2float(scale), m = __half2float(low);
  const float2 s2 = make_float2(s, s), m2 = make_float2(m, m);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = i % 2 ? dev::whole_odd(w >> (8 * (i / 2))) : dev::whole_even(w >> (8 * (i / 2)));
    const float2 y = dev::fma2(dev::h2f(c), s2, m2);
    x[i] = y.x;
    x[i + 4] = y.y;
  }
}

template <class T, int D, bool VEC>
__global__ void __launch_bounds__(kTokens * D / 8) kv_read_kernel(const CacheArgs a) {
  using L = KvTile<D>;
  constexpr int kChunks = D / 8;
  const int64_t tok = (int64_t)blockIdx.x * kTokens + threadIdx.x / kChunks;
  const int ch = threadIdx.x % kChunks, h = blockIdx.y;
  dev::pdl_wait();
  if (tok >= a.n) return;
  const int64_t slot = a.slots[tok];
  const int64_t at = slot_tile(a, slot, L::kBytes, h == 0 && ch == 0);
  float k[8] = {}, v[8] = {};
  if (at >= 0) {
    const int t = (int)(slot % LW_KV_TILE), g = ch >> 2, q = ch & 3;
    const uint8_t* tile = a.pages + at + (int64_t)h * a.page_tiles * L::kBytes;
    const int par = 2 * ((t / 2 * L::G + g) * 2 + t % 2);
    const uint32_t kw = *reinterpret_cast<const uint32_t*>(tile + L::kKeyCodes + 4 * ((t * 4 + q) * L::G + g));
    const __half ks = *reinterpret_cast<const __half*>(tile + L::kKeyScale + par);
    const __half km = *reinterpret_cast<const __half*>(tile + L::kKeyMin + 2 * (t * L::GP + g));
    const uint8_t* u = tile + L::kValCodes + 4 * ((t / 2 * 8 + 2 * q) * L::G + g) + 2 * (t % 2);
    const uint32_t vw = *reinterpret_cast<const uint16_t*>(u) |
                        (uint32_t) * reinterpret_cast<const uint16_t*>(u + 4 * L::G) << 16;
    const __half vs = *reinterpret_cast<const __half*>(tile + L::kValScale + par);
    const __half vm = *reinterpret_cast<const __half*>(tile + L::kValMin + par);
    restore8(kw, ks, km, k);
    restore8(vw, vs, vm, v);
  }
  dev::kv_store8<T, VEC>(static_cast<T*>(a.k.ptr) + tok * a.k.token_stride + h * a.k.head_stride + 8 * ch, k);
  dev::kv_store8<T, VEC>(static_cast<T*>(a.v.ptr) + tok * a.v.token_stride + h * a.v.head_stride + 8 * ch, v);
}

template <class T, int D>
cudaError_t launch_rows(const CacheArgs& a, bool write, bool vec, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((a.n + kTokens - 1) / kTokens), (unsigned)a.heads);
  cfg.blockDim = dim3(kTokens * D / 8);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (write)
    return vec ? cudaLaunchKernelEx(&cfg, kv_write_kernel<T, D, true>, a)
               : cudaLaunchKernelEx(&cfg, kv_write_kernel<T, D, false>, a);
  return vec ? cudaLaunchKernelEx(&cfg, kv_read_kernel<T, D, true>, a)
             : cudaLaunchKernelEx(&cfg, kv_read_kernel<T, D, false>, a);
}

template <class T>
cudaError_t launch_rows_d(const CacheArgs& a, int dim, bool write, bool vec, cudaStream_t st) {
  if (dim == 64) return launch_rows<T, 64>(a, write, vec, st);
  if (dim == 96) return launch_rows<T, 96>(a, write, vec, st);
  return launch_rows<T, 128>(a, write, vec, st);
}

lw_status kv_rows_call(const char* fn, const lw_kv_cache* c, const int64_t* slots, int64_t n,
                       const lw_kv_rows* k, const lw_kv_rows* v, bool write, int32_t* d_status,
                       void* stream) {
  clear_error();
  lw_status s = check_kv_cache(c);
  if (s != LW_OK) return s;
  if (!k || !v) return fail(LW_ERR_INVALID_ARG, "%s: NULL rows", fn);
  if (n < 0) return fail(LW_ERR_INVALID_ARG, "%s: %lld tokens", fn, (long long)n);
  if (!kv_type_ok(k->dtype) || !kv_type_ok(v->dtype))
    return fail(LW_ERR_UNSUPPORTED, "%s: unknown type %d / %d", fn, k->dtype, v->dtype);
  if (k->dtype != v->dtype)
    return fail(LW_ERR_INVALID_ARG, "%s: keys of type %d, values of type %d", fn, k->dtype, v->dtype);
  if (n == 0) return LW_OK;
  if (!k->ptr || !v->ptr || !slots) return fail(LW_ERR_INVALID_ARG, "%s: NULL keys, values or slots", fn);
  const uintptr_t es = (uintptr_t)kv_type_bytes(k->dtype);
  if (reinterpret_cast<uintptr_t>(k->ptr) % es || reinterpret_cast<uintptr_t>(v->ptr) % es ||
      reinterpret_cast<uintptr_t>(slots) % 8)
    return fail(LW_ERR_INVALID_ARG, "%s: an address is not aligned to its type", fn);
  if ((n + kTokens - 1) / kTokens > (1ll << 31) - 1)
    return fail(LW_ERR_SHAPE, "%s: %lld tokens", fn, (long long)n);
  CacheArgs a{};
  a.k = {k->ptr, k->token_stride, k->head_stride};
  a.v = {v->ptr, v->token_stride, v->head_stride};
  a.pages = static_cast<uint8_t*>(c->pages);
  a.slots = slots;
  a.n = n;
  a.n_slots = c->n_pages * c->page_tokens;
  a.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  a.page_tiles = c->page_tokens / LW_KV_TILE;
  a.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (a.page_tiles == 1 << i) a.page_shift = i;
  a.heads = c->kv_heads;
  a.status = d_status;
  const bool vec = kv_rows_aligned(k->ptr, k->token_stride, k->head_stride, k->dtype) &&
                   kv_rows_aligned(v->ptr, v->token_stride, v->head_stride, v->dtype);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = k->dtype == LW_F32   ? launch_rows_d<float>(a, c->head_dim, write, vec, st)
                        : k->dtype == LW_F16 ? launch_rows_d<__half>(a, c->head_dim, write, vec, st)
                                             : launch_rows_d<__nv_bfloat16>(a, c->head_dim, write, vec, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LW_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
  }
  return LW_OK;
}

}  // namespace
}  // namespace lw

using namespace lw;

extern "C" size_t lw_kv_tile_bytes(int32_t head_dim) {
  return head_dim == 64    ? KvTile<64>::kBytes
         : head_dim == 96  ? KvTile<96>::kBytes
         : head_dim == 128 ? KvTile<128>::kBytes
                           : 0;
}

extern "C" size_t lw_kv_page_bytes(int32_t kv_heads, int32_t head_dim, int32_t page_tokens) {
  if (kv_heads < 1 || kv_heads > 65535 || page_tokens < 1 || page_tokens % LW_KV_TILE ||
      page_tokens > (1 << 20))
    return 0;
  return lw_kv_tile_bytes(head_dim) * (size_t)(page_tokens / LW_KV_TILE) * (size_t)kv_heads;
}

extern "C" lw_status lw_kv_write(const lw_kv_cache* c, const lw_kv_rows* k, const lw_kv_rows* v,
                                 const int64_t* slots, int64_t n, int32_t* d_status, void* stream) {
  return kv_rows_call("lw_kv_write", c, slots, n, k, v, true, d_status, stream);
}

extern "C" lw_status lw_kv_read(const lw_kv_cache* c, const int64_t* slots, int64_t n,
                                const lw_kv_rows* k, const lw_kv_rows* v, int32_t* d_status,
                                void* stream) {
  return kv_rows_call("lw_kv_read", c, slots, n, k, v, false, d_status, stream);
}

extern "C" size_t lw_kv_workspace_bytes(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens,
                                        int32_t batch) {
  if (!c || !lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens) || q_heads < 1 ||
      q_heads % c->kv_heads || q_tokens < 0 || batch < 1)
    return 0;
  return kv_attention_workspace(c, q_heads, q_tokens);
}

extern "C" lw_status lw_kv_attention(const lw_kv_cache* c, const lw_kv_attn* a, void* ws,
                                     size_t ws_bytes, int32_t* d_status, void* stream) {
  clear_error();
  lw_status s = check_kv_cache(c);
  if (s != LW_OK) return s;
  if (!a) return fail(LW_ERR_INVALID_ARG, "NULL arguments");
  if (!kv_type_ok(a->dtype)) return fail(LW_ERR_UNSUPPORTED, "unknown type %d", a->dtype);
  if (a->q_heads < 1 || a->q_heads > 65535 || a->q_heads % c->kv_heads)
    return fail(LW_ERR_SHAPE, "%d query heads on %d key/value heads", a->q_heads, c->kv_heads);
  if (a->batch < 1 || a->batch > 65535) return fail(LW_ERR_SHAPE, "batch %d (1..65535)", a->batch);
  if (a->q_tokens < 0 || a->q_tokens > (1ll << 31) - 1)
    return fail(LW_ERR_SHAPE, "%lld query tokens", (long long)a->q_tokens);
  // (rows and keys are counted in 32 bits, to the end of the last item or unit)
  if (a->q_tokens * a->q_heads > kKvMost || (int64_t)a->max_q * a->q_heads > kKvMost)
    return fail(LW_ERR_SHAPE, "%lld query tokens of %d heads", (long long)a->q_tokens, a->q_heads);
  if (a->max_q < 0) return fail(LW_ERR_INVALID_ARG, "max_q %d", a->max_q);
  if (a->window < 0) return fail(LW_ERR_INVALID_ARG, "window %d", a->window);
  if (a->causal != 0 && a->causal != 1) return fail(LW_ERR_INVALID_ARG, "causal %d", a->causal);
  if (!(a->scale >= -3.402823466e38f && a->scale <= 3.402823466e38f))
    return fail(LW_ERR_INVALID_ARG, "scale is not finite");
  if (a->table_width < 0 || a->table_stride < 0 ||
      (int64_t)a->table_width * c->page_tokens > kKvMost)
    return fail(LW_ERR_SHAPE, "page table of %d pages of %d tokens", a->table_width, c->page_tokens);
  if (a->q_tokens == 0) return LW_OK;
  if (!a->q || !a->out || !a->q_start || !a->kv_len || (a->table_width && !a->page_table))
    return fail(LW_ERR_INVALID_ARG, "NULL q, out, q_start, kv_len or page_table");
  const uintptr_t es = (uintptr_t)kv_type_bytes(a->dtype);
  if (reinterpret_cast<uintptr_t>(a->q) % es || reinterpret_cast<uintptr_t>(a->out) % es ||
      reinterpret_cast<uintptr_t>(a->lse) % 4 || reinterpret_cast<uintptr_t>(a->q_start) % 4 ||
      reinterpret_cast<uintptr_t>(a->kv_len) % 4 || reinterpret_cast<uintptr_t>(a->page_table) % 4)
    return fail(LW_ERR_INVALID_ARG, "an address is not aligned to its type");
  const size_t need = lw_kv_workspace_bytes(c, a->q_heads, a->q_tokens, a->batch);
  if (!ws || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15u))
    return fail(LW_ERR_INVALID_ARG, "workspace missing, misaligned or %zu bytes of %zu", ws_bytes, need);
  return launch_kv_attention(c, a, ws, d_status, static_cast<cudaStream_t>(stream));
}
