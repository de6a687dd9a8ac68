// Prefill over the block-scaled 8-bit cache (attn_prefill_paged_block_scaled).
// Chunks of few rows go to the decode kernel, which reads the codes themselves
// (prefill_has_few_rows). For the others the pages' values are written to the
// workspace as dense bf16 (code * 2^e has 4 significant bits, so that is exact) and
// the dense prefill kernel attends to them. The first step moves 3 bytes per cached
// element and kv head (and the second one 2 more), at HBM's rate; the second one is
// bound by the softmax and tensor chain. 1844 rows over 30617 keys, 32/8 heads of
// 128: 30 us and 790-830 us (1080-1140 TFLOP/s); 5 chunks of up to 300 rows over up
// to 3300 keys, 16/4 heads: 49 us in all; 8 first chunks of up to 512 rows, 32/8
// heads: 46 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace attn {

// Keys of the dense copy: the caller's bound on the lengths, or what a table row can hold.
static int dense_width(const attn_prefill_params& p) {
  const long long cap = (long long)p.max_blocks_per_seq * 16;
  return (int)(p.seqlen_k < cap ? p.seqlen_k : cap);
}

static size_t dense_bytes(const attn_prefill_params& p) {
  const size_t n = (size_t)p.batch * p.num_kv_heads * dense_width(p) * p.head_dim * 2;
  return (n + 255) / 256 * 256;
}

// The call over the dense copy at `k`, V behind K.
static attn_prefill_params dense_params(const attn_prefill_params& p, uint8_t* k) {
  const int width = dense_width(p);
  attn_prefill_params d = p;
  d.k_cache = d.v_cache = nullptr;
  d.block_table = nullptr;
  d.max_blocks_per_seq = d.num_blocks = d.block_size = 0;
  d.k = width > 0 ? k : nullptr;
  d.v = width > 0 ? k + dense_bytes(p) : nullptr;
  d.seqlen_k = width;
  d.k_row_stride = d.v_row_stride = p.head_dim;
  d.k_head_stride = d.v_head_stride = (int64_t)width * p.head_dim;
  d.k_batch_stride = d.v_batch_stride = (int64_t)p.num_kv_heads * width * p.head_dim;
  return d;
}

size_t prefill_block_scaled_workspace_bytes(const attn_prefill_params& p) {
  if (p.batch == 0 || p.seqlen_q == 0) return 0;
  if (prefill_has_few_rows(p)) return prefill_few_rows_workspace_bytes(p);
  return 2 * dense_bytes(p) + prefill_split_workspace_bytes(dense_params(p, nullptr));
}

attn_status_t launch_prefill_block_scaled(const attn_prefill_params& p, const uint8_t* k_scales,
                                          const uint8_t* v_scales, void* workspace, cudaStream_t stream) {
  if (prefill_has_few_rows(p)) return launch_prefill_few_rows(p, k_scales, v_scales, workspace, stream);
  const int width = dense_width(p);
  uint8_t* k = reinterpret_cast<uint8_t*>(workspace);
  uint8_t* v = k + dense_bytes(p);
  const attn_gather_params g = {p.k_cache, p.v_cache, k_scales, v_scales, p.block_table, p.seqlens_k, k, v,
                                p.error_flags, p.batch, p.num_kv_heads, p.head_dim, width, p.num_blocks,
                                p.block_size, p.max_blocks_per_seq, ATTN_DTYPE_FP8_E4M3};
  // The prefill kernel reads whole tiles of 128 keys: the rest of a sequence's
  // last tile is cleared, nothing behind it is touched.
  const attn_status_t st = launch_gather(g, 128, true, stream);
  if (st != ATTN_OK) return st;
  return launch_prefill_behind(dense_params(p, k), v + dense_bytes(p), stream);
}

}  // namespace attn
