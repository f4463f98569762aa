// Host checks and launchers of the key/value cache calls.  Internal.
#pragma once

#include <cuda_runtime.h>

#include "lw_internal.h"

namespace lw {

int device_sm_count();
int resident_blocks(const void* kernel, int threads, size_t smem);

// The most rows (query tokens times heads) of an attention call, and keys of its
// page table: 32-bit numbers with room for the rows and keys that the last row
// tile (256 rows) and unit (256 keys) run past the end.
constexpr int64_t kKvMost = (1ll << 31) - 1024;

// Views of the cache and of rows of heads, checked by every call.
lw_status check_kv_cache(const lw_kv_cache* c);
inline bool kv_type_ok(int32_t t) { return t == LW_F32 || t == LW_F16 || t == LW_BF16; }
inline int kv_type_bytes(int32_t t) { return t == LW_F32 ? 4 : 2; }
// Whether every head row starts on a 16-byte boundary
inline bool kv_rows_aligned(const void* p, int64_t token_stride, int64_t head_stride, int32_t t) {
  const int64_t n = 16 / kv_type_bytes(t);
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && token_stride % n == 0 && head_stride % n == 0;
}

// Bytes of workspace of an attention call of q_tokens tokens in all.
size_t kv_attention_workspace(const lw_kv_cache* c, int32_t q_heads, int64_t q_tokens);
lw_status launch_kv_attention(const lw_kv_cache* c, const lw_kv_attn* a, void* ws, int32_t* status,
                              cudaStream_t st);

}  // namespace lw
