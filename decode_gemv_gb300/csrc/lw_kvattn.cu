// Attention over the 4-bit key/value cache.
#include "lw_kv.cuh"
#include "lw_kv.h"

namespace lw {
namespace {

struct AttnArgs {
  lw_kv_attn p;
  const uint8_t* pages;
  int64_t n_pages, page_bytes;
  int32_t page_tokens, heads, group;
  int32_t* status;
};

constexpr int kAttnWarps = 8;

// One CTA per (query token, query head): its warps take every kAttnWarps-th
// key, lane l holding the elements 32 g + l of the head; scores by a warp
// sum, an online softmax per warp, the warps' states joined at the end.
template <class T, int D>
__global__ void __launch_bounds__(32 * kAttnWarps) kv_attn_kernel(const AttnArgs a) {
  using L = KvTile<D>;
  constexpr int G = L::G;
  __shared__ float s_m[kAttnWarps], s_l[kAttnWarps], s_o[kAttnWarps][D];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int64_t tok = blockIdx.x;
  const int hq = blockIdx.y, h = hq / a.group;
  // the token's sequence: the last with q_start <= tok
  int b = 0;
  for (int lo = 0, hi = a.p.batch - 1; lo <= hi;) {
    const int mid = (lo + hi) / 2;
    if (a.p.q_start[mid] <= tok) { b = mid; lo = mid + 1; } else hi = mid - 1;
  }
  const int64_t q0 = a.p.q_start[b], q1 = a.p.q_start[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > a.p.q_tokens) {
    if (threadIdx.x == 0) dev::report(a.status, LW_DEV_BAD_SEQ);
    return;
  }
  if (tok < q0 || tok >= q1) return;
  int64_t n = a.p.kv_len[b];
  const int64_t most = (int64_t)a.p.table_width * a.page_tokens;
  if (n < 0 || n > most) {
    if (threadIdx.x == 0) dev::report(a.status, LW_DEV_BAD_SEQ);
    n = n < 0 ? 0 : most;
  }
  const int64_t pos = n - (q1 - q0) + (tok - q0);
  int64_t hi = a.p.causal && pos + 1 < n ? pos + 1 : n;
  int64_t lo = a.p.window && pos - a.p.window + 1 > 0 ? pos - a.p.window + 1 : 0;
  const T* qp = static_cast<const T*>(a.p.q) + tok * a.p.q_token_stride + hq * a.p.q_head_stride;
  float q[G], o[G], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int g = 0; g < G; ++g) {
    q[g] = dev::kv_float<T>(qp[32 * g + lane]) * a.p.scale;
    o[g] = 0.f;
  }
  const int sh = 4 * (lane % 4);
  for (int64_t j = lo + warp; j < hi; j += kAttnWarps) {
    const int page = a.p.page_table[b * a.p.table_stride + j / a.page_tokens];
    if (page < 0 || page >= a.n_pages) {
      if (lane == 0) dev::report(a.status, LW_DEV_BAD_PAGE);
      continue;
    }
    const int in = (int)(j % a.page_tokens), t = in % LW_KV_TILE;
    const uint8_t* tile = a.pages + page * a.page_bytes +
                          ((int64_t)h * (a.page_tokens / LW_KV_TILE) + in / LW_KV_TILE) * L::kBytes;
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t c = *reinterpret_cast<const uint16_t*>(
          tile + L::kKeyCodes + 4 * ((t * 4 + lane / 8) * G + g) + 2 * (lane / 4 % 2));
      const float sc = __half2float(*reinterpret_cast<const __half*>(
          tile + L::kKeyScale + 2 * ((t / 2 * G + g) * 2 + t % 2)));
      const float mn = __half2float(*reinterpret_cast<const __half*>(tile + L::kKeyMin + 2 * (t * L::GP + g)));
      s = fmaf(q[g], fmaf(sc, (float)((c >> sh) & 15u), mn), s);
    }
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float mx = fmaxf(m, s);
    const float base = mx == -INFINITY ? 0.f : mx;
    const float w = expf(m - base), p = expf(s - base);
    m = mx;
    l = l * w + p;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const uint32_t c = *reinterpret_cast<const uint16_t*>(
          tile + L::kValCodes + 4 * ((t / 2 * 8 + lane / 4) * G + g) + 2 * (t % 2));
      const int par = 2 * ((t / 2 * G + g) * 2 + t % 2);
      const float sc = __half2float(*reinterpret_cast<const __half*>(tile + L::kValScale + par));
      const float mn = __half2float(*reinterpret_cast<const __half*>(tile + L::kValMin + par));
      o[g] = fmaf(p, fmaf(sc, (float)((c >> sh) & 15u), mn), o[g] * w);
    }
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int g = 0; g < G; ++g) s_o[warp][32 * g + lane] = o[g];
  __syncthreads();
  if (warp) return;
  float top = -INFINITY;
  for (int w = 0; w < kAttnWarps; ++w) top = fmaxf(top, s_m[w]);
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f, f[G] = {};
  for (int w = 0; w < kAttnWarps; ++w) {
    const float e = expf(s_m[w] - base);
    sum += s_l[w] * e;
#pragma unroll
    for (int g = 0; g < G; ++g) f[g] += s_o[w][32 * g + lane] * e;
  }
  T* op = static_cast<T*>(a.p.out) + tok * a.p.out_token_stride + hq * a.p.out_head_stride;
#pragma unroll
  for (int g = 0; g < G; ++g) op[32 * g + lane] = dev::kv_round<T>(sum == 0.f ? 0.f : f[g] / sum);
  if (lane == 0 && a.p.lse) a.p.lse[tok * a.p.q_heads + hq] = sum == 0.f ? -INFINITY : top + logf(sum);
}

template <class T>
void launch_t(const AttnArgs& a, int dim, cudaStream_t st) {
  const dim3 grid((unsigned)a.p.q_tokens, (unsigned)a.p.q_heads);
  if (dim == 64) kv_attn_kernel<T, 64><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  else if (dim == 96) kv_attn_kernel<T, 96><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  else kv_attn_kernel<T, 128><<<grid, 32 * kAttnWarps, 0, st>>>(a);
}

}  // namespace

lw_status launch_kv_attention(const lw_kv_cache* c, const lw_kv_attn* p, void* ws, int32_t* status,
                              cudaStream_t st) {
  (void)ws;
  AttnArgs a{};
  a.p = *p;
  a.pages = static_cast<const uint8_t*>(c->pages);
  a.n_pages = c->n_pages;
  a.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  a.page_tokens = c->page_tokens;
  a.heads = c->kv_heads;
  a.group = p->q_heads / c->kv_heads;
  a.status = status;
  if (p->dtype == LW_F32) launch_t<float>(a, c->head_dim, st);
  else if (p->dtype == LW_F16) launch_t<__half>(a, c->head_dim, st);
  else launch_t<__nv_bfloat16>(a, c->head_dim, st);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(LW_ERR_CUDA, "lw_kv_attention: %s", cudaGetErrorString(e));
  return LW_OK;
}

}  // namespace lw
