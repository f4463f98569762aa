// Attention over the 4-bit key/value cache: the launches.
#include "lw_kvfew.cuh"
#include "lw_kvmany.cuh"
#include "lw_kv.h"

namespace lw {
namespace {

using AttnKernel = void (*)(const AttnArgs);

struct Variant {
  AttnKernel kernel;
  int threads, per_sm, smem;
};
template <int D>
Variant variant(int mode) {
  if (mode == 0) return {dev::kv_few_kernel<D, 0>, Few<D, 0>::kThreads, Few<D, 0>::kPerSm, Few<D, 0>::kSmem};
  if (mode == 1) return {dev::kv_few_kernel<D, 1>, Few<D, 1>::kThreads, Few<D, 1>::kPerSm, Few<D, 1>::kSmem};
  if (mode == 2) return {dev::kv_few_kernel<D, 2>, Few<D, 2>::kThreads, Few<D, 2>::kPerSm, Few<D, 2>::kSmem};
  if (mode == 3) return {dev::kv_many_kernel<D, false>, Many<D, false>::kThreads, kManyPerSm, Many<D, false>::kSmem};
  return {dev::kv_many_kernel<D, true>, Many<D, true>::kThreads, kManyPerSm, Many<D, true>::kSmem};
}

// The workspace: counters and partial results of the most resident CTAs of a
// launch (counts of either kernel: a counter, and two parts of an item, a CTA;
// twice that for the two row tiles of kv_many_kernel).
constexpr int kMostPerSm = 2;
static_assert(Few<64, 0>::kPerSm <= kMostPerSm && Few<64, 1>::kPerSm <= kMostPerSm && Few<64, 2>::kPerSm <= kMostPerSm &&
                  2 * kManyPerSm <= kMostPerSm,
              "workspace places");

// Rows of a sequence on a key/value head up to which kv_few_kernel takes a call (the crossings at the rule below)
constexpr int kFewMostBf16 = 24, kFewMost = 32;

}  // namespace

size_t kv_counter_bytes() { return ((size_t)kMostPerSm * device_sm_count() * 4 + 255) / 256 * 256; }

// A call whose tokens, were they all one sequence's, are few rows is kv_few_kernel's in every type.
size_t kv_attention_workspace(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens) {
  const size_t few = (size_t)kMostPerSm * 2 * 16, many = (size_t)2 * 2 * kManyTile;   // rows an SM
  const bool all_few = q_tokens * (q_heads / c->kv_heads) <= kFewMostBf16;
  return kv_counter_bytes() + (size_t)device_sm_count() * (all_few ? few : many) * (size_t)(c->head_dim + 2) * 4;
}

lw_status launch_kv_attention(const lw_kv_cache* c, const lw_kv_attn* p, int parts, void* ws, int32_t* status,
                              cudaStream_t st) {
  AttnArgs a{};
  a.p = *p;
  a.pages = static_cast<const uint8_t*>(c->pages);
  a.n_pages = c->n_pages;
  a.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  a.counters = static_cast<uint32_t*>(ws);
  a.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kv_counter_bytes());
  a.page_tokens = c->page_tokens;
  a.heads = c->kv_heads;
  a.group = p->q_heads / c->kv_heads;
  a.vec = kv_rows_aligned(p->q, p->q_token_stride, p->q_head_stride, p->dtype) &&
          kv_rows_aligned(p->out, p->out_token_stride, p->out_head_stride, p->dtype);
  a.parts = parts;
  a.status = status;
  // The variant, by the rows of a sequence on a key/value head.  us, kv_few_kernel (items of 8 rows, or
  // of 16) against kv_many_kernel, at 8 sequences of 32768 keys | 64 of 512, 8 heads of 128:
  //   bf16  8 rows    90, 138 : 197 |  26,  39 : 70      fp32  16 rows  210 : 422 |  53 : 123
  //        12 rows   161, 143 : 198 |  46,  40 : 69            32 rows  399 : 423 |  90 : 124
  //        16 rows   161, 146 : 198 |  47,  41 : 69            48 rows  590 : 423 | 144 : 126
  //        24 rows   233, 251 : 199 |  67,  81 : 69            64 rows  779 : 425 | 182 : 129
  //        32 rows   303, 256 : 199 |  80,  82 : 70
  // One sequence of 8192 keys alone, bf16: 16 rows 19, 26 : 49, 32 rows 25, 28 : 50, 48 rows 30, 33 : 50;
  // fp32: 32 rows 29 : 51, 64 rows 40 : 55 (kv_many_kernel's items start and end slowly); the lengths are
  // not known here, so the rule is the full device's.  At 24 rows in bf16 each side wins one column, and
  // one sequence alone decides.  (Items of 16 rows at 128 wide, 720 bytes a thread of which are spilled:
  // they read the cache once where items of 8 read it twice.)
  const long long rows = (p->max_q < p->q_tokens ? p->max_q : p->q_tokens) * a.group;
  // (A token that reads pages of its own is the rows of one group: kv_few_kernel's.)
  const int mode = p->dtype != LW_BF16 ? (rows > kFewMost && !parts ? 4 : 0)
                                       : (rows > kFewMostBf16 && !parts ? 3 : rows > 8 && rows <= 16 ? 1 : 2);
  const Variant v = c->head_dim == 64 ? variant<64>(mode) : c->head_dim == 96 ? variant<96>(mode) : variant<128>(mode);
  if (resident_blocks(reinterpret_cast<const void*>(v.kernel), v.threads, v.smem) < 1)
    return fail(LW_ERR_CUDA, "lw_kv_attention: the kernel does not fit this device");
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(v.per_sm * device_sm_count()));
  cfg.blockDim = dim3(v.threads);
  cfg.dynamicSmemBytes = v.smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, v.kernel, a);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(LW_ERR_CUDA, "lw_kv_attention: %s", cudaGetErrorString(e));
  }
  return LW_OK;
}

}  // namespace lw
