// Rotary positions on dense or packed query / key rows (attn_rotary), for sm_100a.
//
// One pass: every row is read and written once, two 16-byte vectors per thread
// and head, so the kernel is bound by HBM; the 64-bit angle reduction and the
// sine and cosine are computed once per (token, pair) and head group.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "rotary.cuh"

namespace attn {
namespace rotary {

constexpr int THREADS = 256;

template <typename TI, typename TO, bool INTER>
__global__ void __launch_bounds__(THREADS, 3) rotary_kernel(const Rows r, const Turn t) {
  turn_rows<TI, TO, INTER>(r, t, (long long)blockIdx.x * THREADS + threadIdx.x);
}

template <typename TI, typename TO>
static attn_status_t launch(const Rows& r, const Turn& t, bool interleaved, cudaStream_t stream) {
  const long long threads = r.tokens * r.head_groups * r.units;
  const long long blocks = (threads + THREADS - 1) / THREADS;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  if (interleaved)
    rotary_kernel<TI, TO, true><<<(unsigned)blocks, THREADS, 0, stream>>>(r, t);
  else
    rotary_kernel<TI, TO, false><<<(unsigned)blocks, THREADS, 0, stream>>>(r, t);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace rotary

attn_status_t launch_rotary(const attn_rotary_params& p, cudaStream_t stream) {
  rotary::Rows r;
  memset(&r, 0, sizeof(r));
  r.q = p.q, r.k = p.k, r.q_out = p.q_out, r.k_out = p.k_out;
  r.positions = p.positions;
  r.tokens = (long long)p.batch * p.seqlen;
  r.seqlen = p.seqlen;
  r.hq = p.num_q_heads;
  r.heads = p.num_q_heads + (p.k ? p.num_k_heads : 0);
  if (r.tokens == 0 || r.heads == 0) return ATTN_OK;
  r.units = p.head_dim / 16;
  r.head_groups = rotary::head_groups_for(r.tokens, r.heads, r.units, device_sm_count());
  r.q_bs = p.q_batch_stride, r.q_hs = p.q_head_stride, r.q_rs = p.q_row_stride;
  r.k_bs = p.k_batch_stride, r.k_hs = p.k_head_stride, r.k_rs = p.k_row_stride;
  r.qo_bs = p.qo_batch_stride, r.qo_hs = p.qo_head_stride, r.qo_rs = p.qo_row_stride;
  r.ko_bs = p.ko_batch_stride, r.ko_hs = p.ko_head_stride, r.ko_rs = p.ko_row_stride;
  const rotary::Turn t = {p.inv_freq, p.rotary_dim, p.magnitude, p.inverse ? -1.f : 1.f};
  const bool inter = p.interleaved != 0;
  if (p.in_dtype == ATTN_DTYPE_BF16)
    return p.out_dtype == ATTN_DTYPE_BF16 ? rotary::launch<__nv_bfloat16, __nv_bfloat16>(r, t, inter, stream)
                                          : rotary::launch<__nv_bfloat16, float>(r, t, inter, stream);
  return p.out_dtype == ATTN_DTYPE_BF16 ? rotary::launch<float, __nv_bfloat16>(r, t, inter, stream)
                                        : rotary::launch<float, float>(r, t, inter, stream);
}

}  // namespace attn
