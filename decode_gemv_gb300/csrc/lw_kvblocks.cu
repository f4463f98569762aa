// Sparse attention over the 4-bit cache: summaries of pages, and the choice of
// the pages that each query reads.
#include "lw_kv.cuh"
#include "lw_kv.h"
#include "lw_kvselect.cuh"

namespace lw {
namespace {

constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100

// A page's record of one head: int8 hi[D], lo[D], fp32 step, 12 bytes unused
__host__ __device__ constexpr int record_bytes(int D) { return 2 * D + 16; }

// ---- summaries -----------------------------------------------------------------
struct SummaryArgs {
  lw_kv_summaries p;
  const uint8_t* pages;
  int64_t n_pages, page_bytes;
  int32_t page_tokens, heads;
  int32_t* status;
};
constexpr int kSumWarps = 8;

// Bound by instruction issue: 519 instructions for 16 keys (measured with pages of 64: a sixth is the page's reduction
// over lanes, the rest restores codes and compares) in 68 % of the slots, two CTAs an SM.  8 sequences of 20000 to
// 131072 tokens, 8 heads of 128: 168 us, 0.38 GB of keys, 2.3 TB/s; one page of each of 16 sequences' 16 heads 7 us.
// A warp a page and head: lanes hold keys lane / 4 and 8 more of a tile, elements 32 g + 8 (lane % 4) + 0..7.
template <int D>
__global__ void __launch_bounds__(32 * kSumWarps, 2) kv_summarise_kernel(const SummaryArgs a) {
  using L = KvTile<D>;
  constexpr int G = L::G, GX = G == 2 ? 2 : 4;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, t = lane / 4, q = lane % 4;
  const int h = blockIdx.y, b = blockIdx.z, tpp = a.page_tokens / LW_KV_TILE;
  dev::pdl_wait();
  const int len = a.p.kv_len[b], most = a.p.table_width * a.page_tokens;
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0 && (len < 0 || len > most)) dev::report(a.status, LW_DEV_BAD_SEQ);
  const int n = len < 0 ? 0 : (len > most ? most : len);
  const int start = max(a.p.start[b], 0);
  if (start >= n) return;
  const int last = (n - 1) / a.page_tokens, step = gridDim.x * kSumWarps;
  const int32_t* table = a.p.page_table + (int64_t)b * a.p.table_stride;
  int blk = start / a.page_tokens + blockIdx.x * kSumWarps + warp;
  // what is read next: a tile ahead, over the ends of pages too
  const auto page_of = [&](int x) { return x <= last ? table[x] : -1; };
  const auto keys_of = [&](int x) { return min(n - x * a.page_tokens, a.page_tokens); };
  const auto there = [&](int page) { return page >= 0 && page < a.n_pages; };
  struct Raw {
    uint32_t kc[2][G], ks[2][G], km[2][L::GP / 2];
  };
  const auto read = [&](Raw& r, int page, int tile, int keys) {
    // (a key past the end: the lane's other one once more, or the first)
    const uint8_t* s = a.pages + page * a.page_bytes + ((int64_t)h * tpp + tile) * L::kBytes;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int left = keys - 16 * tile, tk = t + 8 * e < left ? t + 8 * e : (t < left ? t : 0);
      dev::ldg_words<G>(s + L::kKeyCodes + ((tk * 4 + q) * G) * 4, r.kc[e]);
      dev::ldg_words<G>(s + L::kKeyScale + (tk / 2 * G) * 4, r.ks[e]);
      dev::ldg_words<L::GP / 2>(s + L::kKeyMin + tk * L::GP * 2, r.km[e]);
    }
  };
  Raw now;
  int page = page_of(blk), next_page = page_of(blk + step);
  if (blk <= last && there(page)) read(now, page, 0, keys_of(blk));
  for (; blk <= last; blk += step, page = next_page, next_page = page_of(blk + step)) {
    if (!there(page)) {
      if (lane == 0) dev::report(a.status, LW_DEV_BAD_PAGE);
      if (there(next_page)) read(now, next_page, 0, keys_of(blk + step));
      continue;
    }
    const int keys = keys_of(blk), tiles = (keys + 15) / 16;
    float lo[GX][8], hi[GX][8];
#pragma unroll
    for (int g = 0; g < GX; ++g)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        lo[g][i] = INFINITY;
        hi[g][i] = -INFINITY;
      }
#pragma unroll 1
    for (int tile = 0; tile < tiles; ++tile) {
      const Raw r = now;
      if (tile + 1 < tiles) read(now, page, tile + 1, keys);
      else if (there(next_page)) read(now, next_page, 0, keys_of(blk + step));
      // (which of a pair of scales: by the key that was read)
      const bool odd = t < keys - 16 * tile && t % 2;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        float2 y[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 s2 = dev::h2f(r.ks[e][g]), m2 = dev::h2f(r.km[e][g / 2]);
          const float sc = odd ? s2.y : s2.x, mn = g % 2 ? m2.y : m2.x;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t c = i % 2 ? dev::whole_odd(r.kc[e][g] >> (8 * (i / 2))) : dev::whole_even(r.kc[e][g] >> (8 * (i / 2)));
            y[e][i] = dev::fma2(dev::h2f(c), make_float2(sc, sc), make_float2(mn, mn));
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[g][i] = dev::min3(lo[g][i], y[0][i].x, y[1][i].x);
          hi[g][i] = dev::max3(hi[g][i], y[0][i].x, y[1][i].x);
          lo[g][i + 4] = dev::min3(lo[g][i + 4], y[0][i].y, y[1][i].y);
          hi[g][i + 4] = dev::max3(hi[g][i + 4], y[0][i].y, y[1][i].y);
        }
      }
    }
    // over the keys: lane t of a channel's 8 ends up with the 4 channels of group t / 2, half t % 2 (64 wide:
    // of group t / 2 % 2)
    float l4[4], h4[4];
    {
      constexpr int kHalf = GX / 2;
#pragma unroll
      for (int x = 0; x < kHalf; ++x)   // a lane keeps half the groups
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool up = GX == 4 ? lane & 16 : lane & 8;
          const int o = GX == 4 ? 16 : 8;
          const float gl = __shfl_xor_sync(0xFFFFFFFFu, up ? lo[x][i] : lo[x + kHalf][i], o);
          const float gh = __shfl_xor_sync(0xFFFFFFFFu, up ? hi[x][i] : hi[x + kHalf][i], o);
          const float ol = up ? lo[x + kHalf][i] : lo[x][i], oh = up ? hi[x + kHalf][i] : hi[x][i];
          lo[x][i] = dev::min3(ol, gl, gl);
          hi[x][i] = dev::max3(oh, gh, gh);
        }
      if constexpr (GX == 4) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool up = lane & 8;
          const float gl = __shfl_xor_sync(0xFFFFFFFFu, up ? lo[0][i] : lo[1][i], 8);
          const float gh = __shfl_xor_sync(0xFFFFFFFFu, up ? hi[0][i] : hi[1][i], 8);
          const float ol = up ? lo[1][i] : lo[0][i], oh = up ? hi[1][i] : hi[0][i];
          lo[0][i] = dev::min3(ol, gl, gl);
          hi[0][i] = dev::max3(oh, gh, gh);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float gl = __shfl_xor_sync(0xFFFFFFFFu, lo[0][i], 16), gh = __shfl_xor_sync(0xFFFFFFFFu, hi[0][i], 16);
          lo[0][i] = dev::min3(lo[0][i], gl, gl);
          hi[0][i] = dev::max3(hi[0][i], gh, gh);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool up = lane & 4;
        const float gl = __shfl_xor_sync(0xFFFFFFFFu, up ? lo[0][i] : lo[0][i + 4], 4);
        const float gh = __shfl_xor_sync(0xFFFFFFFFu, up ? hi[0][i] : hi[0][i + 4], 4);
        const float ol = up ? lo[0][i + 4] : lo[0][i], oh = up ? hi[0][i + 4] : hi[0][i];
        l4[i] = dev::min3(ol, gl, gl);
        h4[i] = dev::max3(oh, gh, gh);
      }
    }
    const int g = GX == 4 ? t / 2 : t / 2 % 2;
    const bool real = g < G;   // (96 wide: the fourth group is not there)
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (real) top = dev::max3(top, fabsf(l4[i]), fabsf(h4[i]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float x = __shfl_xor_sync(0xFFFFFFFFu, top, o);
      top = dev::max3(top, x, x);
    }
    const bool zero = !(top > kTiny);   // (or a NaN)
    const float inv = zero ? 0.f : __fmul_rn(127.f, __frcp_rn(top));
    uint32_t wl = 0, wh = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int cl = zero ? 0 : __float2int_rn(__fmul_rn(l4[i], inv)), ch = zero ? 0 : __float2int_rn(__fmul_rn(h4[i], inv));
      wl |= (uint32_t)(cl & 255) << (8 * i);
      wh |= (uint32_t)(ch & 255) << (8 * i);
    }
    uint8_t* r = static_cast<uint8_t*>(a.p.summary) + ((int64_t)page * a.heads + h) * record_bytes(D);
    if (real && (GX == 4 || lane < 16)) {
      const int at = 32 * g + 8 * q + 4 * (t % 2);
      *reinterpret_cast<uint32_t*>(r + at) = wh;
      *reinterpret_cast<uint32_t*>(r + D + at) = wl;
    }
    if (lane == 0) *reinterpret_cast<float*>(r + 2 * D) = __fmul_rn(top, (float)(1.0 / 127.0));
  }
}

// ---- scores and choice ---------------------------------------------------------
struct BlockArgs {
  lw_kv_attn p;
  lw_kv_blocks s;
  int32_t* pages;        // [q_tokens * heads][blocks]: pages of the cache seen head by head
  int32_t* lens;         // [q_tokens * heads]: keys in them, -1 for a token of no sequence
  int64_t n_pages;
  int32_t page_tokens, heads, group, most_pages;   // most_pages: room for a CTA's stretch
  int32_t* status;
};

constexpr int kMostGroup = 128, kChoose = 256;
using ChooseShared = dev::SelectShared<8>;

// The pages of one query token and key/value head, ascending.  A cluster a token and head: its CTAs score stretches of
// the pages and choose together (lw_kvselect.cuh).
// Scores.  The codes of the group's query heads have their positive and negative parts apart, so that the larger of
// c hi and c lo is picked by a product: sum c+ hi + c- lo, in whole numbers (dp4a).  8 lanes take a record.
// 64 tokens and heads on up to 2048 pages 25 us (17 MB of records), 768 on up to 563 20 us (of calls of 51 and 61):
// chains of reads (ranges, page table, records, page table) and the choice's barriers; two kernels, the scores by way
// of memory, took 28 and 22.
template <int D, class T>
__global__ void __launch_bounds__(kChoose) kv_choose_kernel(const BlockArgs a) {
  constexpr int W = D / 32, NT = kChoose, kWarps = NT / 32;   // W: words of a part of a record a lane
  extern __shared__ __align__(16) uint32_t smem[];
  ChooseShared& s = *reinterpret_cast<ChooseShared*>(smem);
  uint32_t* keys = smem + sizeof(ChooseShared) / 4;      // [a.most_pages]
  uint32_t* codes = keys + a.most_pages;                      // [group][2][8][W]
  float* units = reinterpret_cast<float*>(codes + a.group * (D / 2));
  __shared__ int s_seq, s_pos;
  const int h = blockIdx.y, tok = blockIdx.z, tid = threadIdx.x, warp = tid / 32, lane = tid % 32, r = lane % 8;
  const int rank = (int)dev::cluster_rank(), self = rank * NT + tid, all = (int)dev::cluster_size() * NT;
  for (int i = tid; i < ChooseShared::kPasses * ChooseShared::kBins; i += NT) s.hist[i] = 0;
  if (tid == 0) s_seq = 0x7FFFFFFF;
  dev::pdl_wait();
  // the sequences' ranges, a thread one: sent for before the queries are, so that their ways overlap
  int q0 = -1, q1 = -1, len = 0;
  const auto sequence = [&](int i) {
    q0 = i < a.p.batch ? a.p.q_start[i] : -1;
    q1 = i < a.p.batch ? a.p.q_start[i + 1] : -1;
    len = i < a.p.batch ? a.p.kv_len[i] : 0;
  };
  sequence(tid);
  // ---- the queries' codes, four heads a warp at a time
  for (int g0 = 4 * warp; g0 < a.group; g0 += 4 * kWarps) {
    const int g = g0 + lane / 8;
    const T* q = static_cast<const T*>(a.p.q) + (int64_t)tok * a.p.q_token_stride +
                 (int64_t)(h * a.group + (g < a.group ? g : 0)) * a.p.q_head_stride + r * (D / 8);
    float x[D / 8], top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      x[i] = dev::kv_float<T>(q[i]);
      top = dev::max3(top, fabsf(x[i]), top);
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float y = __shfl_xor_sync(0xFFFFFFFFu, top, o);
      top = dev::max3(top, y, y);
    }
    const bool zero = !(top > kTiny && top <= 3.402823466e38f);
    const float inv = zero ? 0.f : __fmul_rn(127.f, __frcp_rn(top));
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint32_t plus = 0, minus = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = zero ? 0 : __float2int_rn(__fmul_rn(x[4 * w + i], inv));
        plus |= (uint32_t)(max(c, 0) & 255) << (8 * i);
        minus |= (uint32_t)(min(c, 0) & 255) << (8 * i);
      }
      if (g < a.group) {
        codes[((g * 2) * 8 + r) * W + w] = plus;
        codes[((g * 2 + 1) * 8 + r) * W + w] = minus;
      }
    }
    if (g < a.group && r == 0) units[g] = zero ? 0.f : __fmul_rn(top, (float)(1.0 / 127.0));
  }
  __syncthreads();
  // ---- the sequence that has the token, and the token's key position
  const int most = a.p.table_width * a.page_tokens;
  for (int i0 = 0; i0 < a.p.batch; i0 += NT) {
    const int i = i0 + tid;
    if (i0) sequence(i);
    if (i < a.p.batch && h == 0 && tok == 0 && rank == 0 && (q0 < 0 || q1 < q0 || q1 > a.p.q_tokens || len < 0 || len > most))
      dev::report(a.status, LW_DEV_BAD_SEQ);
    const bool has = q0 >= 0 && q1 <= a.p.q_tokens && q0 <= tok && tok < q1;
    if (has) atomicMin(&s_seq, i);   // (ranges that overlap: the first)
    __syncthreads();
    if (has && s_seq == i) s_pos = (int)((int64_t)min(max(len, 0), most) - q1 + tok);
  }
  __syncthreads();
  const int64_t row = (int64_t)tok * a.heads + h;
  const int b = s_seq, pos = s_pos;
  if (b == 0x7FFFFFFF) {   // of none (the same in all of the cluster)
    if (self == 0) a.lens[row] = -1;
    return;
  }
  const int nb = pos < 0 ? 0 : pos / a.page_tokens + 1, count = nb < a.s.blocks ? nb : a.s.blocks;
  const int32_t* table = a.p.page_table + (int64_t)b * a.p.table_stride;
  int32_t* pages = a.pages + row * a.s.blocks;
  int32_t* chosen = a.s.chosen ? a.s.chosen + row * a.s.blocks : nullptr;
  const auto put = [&](int i, int blk) {
    const int page = table[blk];
    const bool ok = page >= 0 && page < a.n_pages;
    pages[i] = ok ? page * a.heads + h : -1;
    if (chosen) chosen[i] = blk;
  };
  if (chosen)
    for (int i = count + self; i < a.s.blocks; i += all) chosen[i] = -1;
  if (self == 0) a.lens[row] = nb ? (count - 1) * a.page_tokens + pos - (nb - 1) * a.page_tokens + 1 : 0;
  if (nb <= a.s.blocks) {
    for (int i = self; i < nb; i += all) put(i, i);
    return;
  }
  const int first = a.s.first, last = nb - a.s.recent;
  for (int i = self; i < first; i += all) put(i, i);
  for (int i = last + self; i < nb; i += all) put(count - nb + i, i);
  const uint32_t need = (uint32_t)(count - first - a.s.recent);
  if (need == 0) return;
  // ---- this CTA's stretch of the pages that compete
  int mine;
  const int from = (int)dev::select_stretch(first, last, mine);
  for (int i0 = 0; i0 < mine; i0 += 8 * 4 * kWarps) {
    // eight rounds of a page an eight lanes: lane r knows the r-th one's
    const int ir = i0 + r * 4 * kWarps + 4 * warp + lane / 8;
    const int page_r = ir < mine ? table[from + ir] : -1;
#pragma unroll 4
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e * 4 * kWarps + 4 * warp + lane / 8;
      if (i0 + e * 4 * kWarps + 4 * warp >= mine) break;   // (the same in all of the warp)
      const int page = __shfl_sync(0xFFFFFFFFu, page_r, (lane & 24) + e);
      const bool ok = page >= 0 && page < a.n_pages;
      const uint8_t* rec = static_cast<const uint8_t*>(a.s.summary) + ((int64_t)(ok ? page : 0) * a.heads + h) * record_bytes(D);
      uint32_t hi[W], lo[W];
      dev::ldg_words<W>(rec + 4 * W * r, hi);
      dev::ldg_words<W>(rec + D + 4 * W * r, lo);
      const float step = *reinterpret_cast<const float*>(rec + 2 * D);
      float best = -INFINITY;
      for (int g = 0; g < a.group; ++g) {
        int dot = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          dot = __dp4a((int)codes[((g * 2) * 8 + r) * W + w], (int)hi[w], dot);
          dot = __dp4a((int)codes[((g * 2 + 1) * 8 + r) * W + w], (int)lo[w], dot);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        best = fmaxf(best, __fmul_rn(units[g], (float)dot));
      }
      // (a page outside the cache is read by nobody: the attention leaves it out)
      if (r == 0 && i < mine) keys[i] = dev::order_key(ok ? __fmul_rn(step, best) : -INFINITY);
    }
  }
  __syncthreads();
  dev::select_places<NT, 8>(s, mine, need, [&](int i) { return keys[i]; }, [&](int place, int i) { put(first + place, from + i); });
}

constexpr int kMostWidth = 40960;   // order keys of a page table in one CTA's shared memory

template <int D, class T>
lw_status launch_choose(BlockArgs a, cudaStream_t st) {
  const char* fn = "lw_kv_attention_blocks";
  // CTAs of a token and head: some 256 pages each, as far as six an SM have room
  const int64_t pairs = a.p.q_tokens * a.heads;
  int ranks = 1;
  while (ranks < 8 && 2 * ranks * pairs <= 6 * device_sm_count() && a.p.table_width > 256 * ranks) ranks *= 2;
  a.most_pages = (int32_t)kv_select_room(a.p.table_width, ranks);
  const size_t smem = sizeof(ChooseShared) + (size_t)a.most_pages * 4 + (size_t)a.group * (2 * D + 4);
  if (resident_blocks(reinterpret_cast<const void*>(kv_choose_kernel<D, T>), kChoose, smem) < 1)
    return fail(LW_ERR_CUDA, "%s: the kernel does not fit this device", fn);
  return kv_launch(fn, kv_choose_kernel<D, T>, dim3((unsigned)ranks, (unsigned)a.heads, (unsigned)a.p.q_tokens),
                   kChoose, smem, ranks, st, a);
}
template <int D>
lw_status launch_choose_t(const BlockArgs& a, cudaStream_t st) {
  return a.p.dtype == LW_F32   ? launch_choose<D, float>(a, st)
         : a.p.dtype == LW_F16 ? launch_choose<D, __half>(a, st)
                               : launch_choose<D, __nv_bfloat16>(a, st);
}

// The cache with a head's share of a page as a page: what a query that reads pages of its own attends to
lw_kv_cache by_head(const lw_kv_cache* c) {
  lw_kv_cache v = *c;
  v.n_pages = c->n_pages * c->kv_heads;
  v.kv_heads = 1;
  return v;
}

// Workspace: attention's, then page numbers and lengths of each token and head
struct BlockSpace {
  size_t pages, lens, bytes;
};
BlockSpace block_space(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens, int32_t blocks) {
  const lw_kv_cache v = by_head(c);
  const size_t rows = (size_t)q_tokens * c->kv_heads;
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  BlockSpace s{};
  s.pages = up(kv_attention_workspace(&v, q_heads / c->kv_heads, q_tokens * c->kv_heads));
  s.lens = s.pages + up(rows * blocks * 4);
  s.bytes = s.lens + up(rows * 4);
  return s;
}

}  // namespace
}  // namespace lw

using namespace lw;

extern "C" size_t lw_kv_summary_bytes(const lw_kv_cache* c) {
  if (!c || !lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens) || c->n_pages < 1) return 0;
  return (size_t)c->n_pages * c->kv_heads * record_bytes(c->head_dim);
}

extern "C" lw_status lw_kv_summarise(const lw_kv_cache* c, const lw_kv_summaries* p, int32_t* d_status, void* stream) {
  const char* fn = "lw_kv_summarise";
  clear_error();
  lw_status s = check_kv_cache(c);
  if (s != LW_OK) return s;
  if (!p) return fail(LW_ERR_INVALID_ARG, "NULL arguments");
  if (p->batch < 1 || p->batch > 65535) return fail(LW_ERR_SHAPE, "%s: batch %d (1..65535)", fn, p->batch);
  if (p->table_width < 0 || p->table_stride < 0 || (int64_t)p->table_width * c->page_tokens > kKvMost)
    return fail(LW_ERR_SHAPE, "%s: page table of %d pages of %d tokens", fn, p->table_width, c->page_tokens);
  const auto off = [](const void* x, uintptr_t n) { return reinterpret_cast<uintptr_t>(x) % n != 0; };
  if (!p->summary || !p->start || !p->kv_len || (p->table_width && !p->page_table))
    return fail(LW_ERR_INVALID_ARG, "%s: NULL summary, start, kv_len or page_table", fn);
  if (off(p->summary, 16) || off(p->start, 4) || off(p->kv_len, 4) || off(p->page_table, 4))
    return fail(LW_ERR_INVALID_ARG, "%s: an address is not aligned to its type", fn);
  SummaryArgs a{};
  a.p = *p;
  a.pages = static_cast<const uint8_t*>(c->pages);
  a.n_pages = c->n_pages;
  a.page_bytes = (int64_t)lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens);
  a.page_tokens = c->page_tokens;
  a.heads = c->kv_heads;
  a.status = d_status;
  // CTAs of a sequence's head: what there may be to do, or what fills the device a few times over
  const int64_t pairs = (int64_t)p->batch * c->kv_heads;
  int64_t x = (p->table_width + kSumWarps - 1) / kSumWarps, most = 16ll * device_sm_count() / pairs;
  if (x > most) x = most;
  if (x < 1) x = 1;
  const dim3 grid((unsigned)x, (unsigned)c->kv_heads, (unsigned)p->batch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return c->head_dim == 64   ? kv_launch(fn, kv_summarise_kernel<64>, grid, 32 * kSumWarps, 0, 1, st, a)
         : c->head_dim == 96 ? kv_launch(fn, kv_summarise_kernel<96>, grid, 32 * kSumWarps, 0, 1, st, a)
                             : kv_launch(fn, kv_summarise_kernel<128>, grid, 32 * kSumWarps, 0, 1, st, a);
}

extern "C" size_t lw_kv_blocks_workspace_bytes(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens,
                                               int32_t table_width, int32_t blocks) {
  if (!c || !lw_kv_page_bytes(c->kv_heads, c->head_dim, c->page_tokens) || q_heads < 1 || q_heads % c->kv_heads ||
      q_tokens < 0 || q_tokens * c->kv_heads > 65535 || table_width < 0 || table_width > kMostWidth || blocks < 1 ||
      blocks > kMostWidth)
    return 0;
  return block_space(c, q_heads, q_tokens, blocks).bytes;
}

extern "C" lw_status lw_kv_attention_blocks(const lw_kv_cache* c, const lw_kv_attn* p, const lw_kv_blocks* k, void* ws,
                                            size_t ws_bytes, int32_t* d_status, void* stream) {
  const char* fn = "lw_kv_attention_blocks";
  clear_error();
  lw_status s = check_kv_attention(c, p);
  if (s != LW_OK) return s;
  if (!k) return fail(LW_ERR_INVALID_ARG, "%s: NULL blocks", fn);
  if (p->causal != 1 || p->window != 0) return fail(LW_ERR_UNSUPPORTED, "%s: causal attention without a window only", fn);
  if (!(p->scale > 0.f)) return fail(LW_ERR_UNSUPPORTED, "%s: scale %g is not positive", fn, (double)p->scale);
  if (k->blocks < 1 || k->blocks > kMostWidth || k->first < 0 || k->recent < 1 ||
      (int64_t)k->first + k->recent > k->blocks)
    return fail(LW_ERR_INVALID_ARG, "%s: blocks %d, first %d, recent %d", fn, k->blocks, k->first, k->recent);
  if (p->table_width > kMostWidth) return fail(LW_ERR_SHAPE, "%s: page table of %d pages (at most %d)", fn, p->table_width, kMostWidth);
  if (p->q_tokens * c->kv_heads > 65535)
    return fail(LW_ERR_SHAPE, "%s: %lld query tokens of %d key/value heads", fn, (long long)p->q_tokens, c->kv_heads);
  const int group = p->q_heads / c->kv_heads;
  if (group > kMostGroup) return fail(LW_ERR_SHAPE, "%s: %d query heads a key/value head (at most %d)", fn, group, kMostGroup);
  const lw_kv_cache v = by_head(c);
  if (v.n_pages > ((1ll << 32) - 1) / c->page_tokens || v.n_pages > (1ll << 31) - 1)
    return fail(LW_ERR_SHAPE, "%s: %lld pages of %d heads of %d tokens", fn, (long long)c->n_pages, c->kv_heads, c->page_tokens);
  if ((int64_t)k->blocks * c->page_tokens > kKvMost)
    return fail(LW_ERR_SHAPE, "%s: %d blocks of %d tokens", fn, k->blocks, c->page_tokens);
  if (p->q_tokens == 0) return LW_OK;
  if (!k->summary || (reinterpret_cast<uintptr_t>(k->summary) & 15u) || reinterpret_cast<uintptr_t>(k->chosen) % 4)
    return fail(LW_ERR_INVALID_ARG, "%s: summary missing, or an address is not aligned to its type", fn);
  const BlockSpace at = block_space(c, p->q_heads, p->q_tokens, k->blocks);
  if (!ws || ws_bytes < at.bytes || (reinterpret_cast<uintptr_t>(ws) & 15u))
    return fail(LW_ERR_INVALID_ARG, "%s: workspace missing, misaligned or %zu bytes of %zu", fn, ws_bytes, at.bytes);
  uint8_t* w = static_cast<uint8_t*>(ws);
  BlockArgs a{};
  a.p = *p;
  a.s = *k;
  a.pages = reinterpret_cast<int32_t*>(w + at.pages);
  a.lens = reinterpret_cast<int32_t*>(w + at.lens);
  a.n_pages = c->n_pages;
  a.page_tokens = c->page_tokens;
  a.heads = c->kv_heads;
  a.group = group;
  a.status = d_status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  s = c->head_dim == 64   ? launch_choose_t<64>(a, st)
      : c->head_dim == 96 ? launch_choose_t<96>(a, st)
                          : launch_choose_t<128>(a, st);
  if (s != LW_OK) return s;
  lw_kv_attn one = *p;
  one.q_start = nullptr;
  one.kv_len = a.lens;
  one.page_table = a.pages;
  one.table_stride = one.table_width = k->blocks;
  one.q_tokens = p->q_tokens * c->kv_heads;
  one.batch = (int32_t)one.q_tokens;
  one.q_heads = group;
  one.max_q = 1;
  return launch_kv_attention(&v, &one, c->kv_heads, ws, d_status, st);
}
