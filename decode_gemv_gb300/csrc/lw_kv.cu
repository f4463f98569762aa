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
  if (c->n_pages < 1 || c->n_pages > (1ll << 31) - 1)
    return fail(LW_ERR_SHAPE, "%lld pages", (long long)c->n_pages);
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
  int32_t page_tokens, heads;
  int32_t* status;
};

// Where token t of a slot's tile starts: the tile's address (head 0), -1 if
// the slot is not stored.  A slot past the pages is reported by lane `first`.
__device__ __forceinline__ int64_t slot_tile(const CacheArgs& a, int64_t slot, int tile_bytes,
                                             bool first) {
  if (slot < 0) return -1;
  if (slot >= a.n_slots) {
    if (first) dev::report(a.status, LW_DEV_BAD_SLOT);
    return -1;
  }
  const int64_t page = slot / a.page_tokens;
  const int in = (int)(slot - page * a.page_tokens);
  return page * a.page_bytes + (int64_t)(in / LW_KV_TILE) * tile_bytes;
}

constexpr int kCacheThreads = 256;

// One thread quantises 8 consecutive values of one head of one token (4
// neighbouring lanes a group); blockIdx.y = 0 for keys, 1 for values.
template <class T, int D, bool VEC>
__global__ void __launch_bounds__(kCacheThreads) kv_write_kernel(const CacheArgs a) {
  using L = KvTile<D>;
  constexpr int kChunks = D / 8;
  const int64_t i = (int64_t)blockIdx.x * kCacheThreads + threadIdx.x;
  const int64_t row = i / kChunks;
  const int ch = (int)(i - row * kChunks);
  const int64_t tok = row / a.heads;
  const int h = (int)(row - tok * a.heads);
  const bool val = blockIdx.y == 1;
  const RowsArgs& r = val ? a.v : a.k;
  int64_t at = -1, slot = -1;
  float x[8] = {};
  if (tok < a.n) {
    slot = a.slots[tok];
    at = slot_tile(a, slot, L::kBytes, !val && h == 0 && ch == 0);
    if (at >= 0)
      dev::kv_load8<T, VEC>(static_cast<const T*>(r.ptr) + tok * r.token_stride + h * r.head_stride + 8 * ch, x);
  }
  __half scale, low;
  const uint32_t w = dev::kv_quantise8(x, scale, low);
  if (at < 0) return;
  const int t = (int)(slot % LW_KV_TILE), g = ch >> 2, q = ch & 3;
  uint8_t* tile = a.pages + at + (int64_t)h * (a.page_tokens / LW_KV_TILE) * L::kBytes;
  if (!val) {
    *reinterpret_cast<uint32_t*>(tile + L::kKeyCodes + 4 * ((t * 4 + q) * L::G + g)) = w;
    if (q == 0) {
      *reinterpret_cast<__half*>(tile + L::kKeyScale + 2 * ((t / 2 * L::G + g) * 2 + t % 2)) = scale;
      *reinterpret_cast<__half*>(tile + L::kKeyMin + 2 * (t * L::GP + g)) = low;
    }
  } else {
    uint8_t* u = tile + L::kValCodes + 4 * ((t / 2 * 8 + 2 * q) * L::G + g) + 2 * (t % 2);
    *reinterpret_cast<uint16_t*>(u) = (uint16_t)w;
    *reinterpret_cast<uint16_t*>(u + 4 * L::G) = (uint16_t)(w >> 16);
    if (q == 0) {
      *reinterpret_cast<__half*>(tile + L::kValScale + 2 * ((t / 2 * L::G + g) * 2 + t % 2)) = scale;
      *reinterpret_cast<__half*>(tile + L::kValMin + 2 * ((t / 2 * L::G + g) * 2 + t % 2)) = low;
    }
  }
}

template <class T, int D, bool VEC>
__global__ void __launch_bounds__(kCacheThreads) kv_read_kernel(const CacheArgs a) {
  using L = KvTile<D>;
  constexpr int kChunks = D / 8;
  const int64_t i = (int64_t)blockIdx.x * kCacheThreads + threadIdx.x;
  const int64_t row = i / kChunks;
  const int ch = (int)(i - row * kChunks);
  const int64_t tok = row / a.heads;
  if (tok >= a.n) return;
  const int h = (int)(row - tok * a.heads);
  const bool val = blockIdx.y == 1;
  const RowsArgs& r = val ? a.v : a.k;
  const int64_t slot = a.slots[tok];
  const int64_t at = slot_tile(a, slot, L::kBytes, !val && h == 0 && ch == 0);
  float x[8] = {};
  if (at >= 0) {
    const int t = (int)(slot % LW_KV_TILE), g = ch >> 2, q = ch & 3;
    const uint8_t* tile = a.pages + at + (int64_t)h * (a.page_tokens / LW_KV_TILE) * L::kBytes;
    uint32_t w;
    __half scale, low;
    if (!val) {
      w = *reinterpret_cast<const uint32_t*>(tile + L::kKeyCodes + 4 * ((t * 4 + q) * L::G + g));
      scale = *reinterpret_cast<const __half*>(tile + L::kKeyScale + 2 * ((t / 2 * L::G + g) * 2 + t % 2));
      low = *reinterpret_cast<const __half*>(tile + L::kKeyMin + 2 * (t * L::GP + g));
    } else {
      const uint8_t* u = tile + L::kValCodes + 4 * ((t / 2 * 8 + 2 * q) * L::G + g) + 2 * (t % 2);
      w = *reinterpret_cast<const uint16_t*>(u) |
          (uint32_t) * reinterpret_cast<const uint16_t*>(u + 4 * L::G) << 16;
      scale = *reinterpret_cast<const __half*>(tile + L::kValScale + 2 * ((t / 2 * L::G + g) * 2 + t % 2));
      low = *reinterpret_cast<const __half*>(tile + L::kValMin + 2 * ((t / 2 * L::G + g) * 2 + t % 2));
    }
    const float s = __half2float(scale), m = __half2float(low);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(s, (float)((w >> (4 * j)) & 15u), m);
  }
  dev::kv_store8<T, VEC>(static_cast<T*>(r.ptr) + tok * r.token_stride + h * r.head_stride + 8 * ch, x);
}

template <class T, int D>
void launch_rows(const CacheArgs& a, bool write, bool vec, cudaStream_t st) {
  const int64_t threads = a.n * a.heads * (D / 8);
  const dim3 grid((unsigned)((threads + kCacheThreads - 1) / kCacheThreads), 2);
  if (write) {
    if (vec) kv_write_kernel<T, D, true><<<grid, kCacheThreads, 0, st>>>(a);
    else kv_write_kernel<T, D, false><<<grid, kCacheThreads, 0, st>>>(a);
  } else {
    if (vec) kv_read_kernel<T, D, true><<<grid, kCacheThreads, 0, st>>>(a);
    else kv_read_kernel<T, D, false><<<grid, kCacheThreads, 0, st>>>(a);
  }
}

template <class T>
void launch_rows_d(const CacheArgs& a, int dim, bool write, bool vec, cudaStream_t st) {
  if (dim == 64) launch_rows<T, 64>(a, write, vec, st);
  else if (dim == 96) launch_rows<T, 96>(a, write, vec, st);
  else launch_rows<T, 128>(a, write, vec, st);
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
  if (n > (1ll << 40) / ((int64_t)c->kv_heads * c->head_dim))
    return fail(LW_ERR_SHAPE, "%s: %lld tokens", fn, (long long)n);
  CacheArgs a{};
  a.k = {k->ptr, k->token_stride, k->head_stride};
  a.v = {v->ptr, v->token_stride, v->head_stride};
  a.pages = static_cast<uint8_t*>(c->pages);
  a.slots = slots;
  a.n = n;
  a.n_slots = c->n_pages * c->page_tokens;
  a.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  a.page_tokens = c->page_tokens;
  a.heads = c->kv_heads;
  a.status = d_status;
  const bool vec = kv_rows_aligned(k->ptr, k->token_stride, k->head_stride, k->dtype) &&
                   kv_rows_aligned(v->ptr, v->token_stride, v->head_stride, v->dtype);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (k->dtype == LW_F32) launch_rows_d<float>(a, c->head_dim, write, vec, st);
  else if (k->dtype == LW_F16) launch_rows_d<__half>(a, c->head_dim, write, vec, st);
  else launch_rows_d<__nv_bfloat16>(a, c->head_dim, write, vec, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(LW_ERR_CUDA, "%s: %s", fn, cudaGetErrorString(e));
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
  return kv_attention_workspace(c);
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
  if (a->q_tokens * a->q_heads > (1ll << 31) - 1 || (int64_t)a->max_q * a->q_heads > (1ll << 31) - 1)
    return fail(LW_ERR_SHAPE, "%lld query tokens of %d heads", (long long)a->q_tokens, a->q_heads);
  if (a->max_q < 0) return fail(LW_ERR_INVALID_ARG, "max_q %d", a->max_q);
  if (a->window < 0) return fail(LW_ERR_INVALID_ARG, "window %d", a->window);
  if (a->causal != 0 && a->causal != 1) return fail(LW_ERR_INVALID_ARG, "causal %d", a->causal);
  if (!(a->scale >= -3.402823466e38f && a->scale <= 3.402823466e38f))
    return fail(LW_ERR_INVALID_ARG, "scale is not finite");
  if (a->table_width < 0 || a->table_stride < 0 ||
      (int64_t)a->table_width * c->page_tokens > (1ll << 31) - 1)
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
