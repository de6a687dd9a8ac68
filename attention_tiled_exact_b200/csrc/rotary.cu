// Rotary positions on dense or packed query / key rows (attn_rotary), for sm_100a.
//
// One pass: every row is read and written once (turn_rows). It is bound by HBM
// for many rows: queries and keys of 4 x 40 heads x 2048 x 128 in bf16 take 28.6-29.6
// us (168 MB, 5.7-5.9 TB/s, of 6.4 TB/s of a plain elementwise kernel; the angles,
// with which every CTA begins, cost 0.5 us of it), 8504 packed rows of 32 heads 21-23
// us (6.1-6.6 TB/s). 64 rows take 2.5 us, a launch and three dependent loads.
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "rotary.cuh"

namespace attn {
namespace rotary {

template <typename TI, typename TO, bool INTER, int D, bool BY_HEADS>
__global__ void __launch_bounds__(THREADS, CTAS_PER_SM) rotary_kernel(const Rows r, const Turn t) {
  extern __shared__ __align__(16) uint8_t smem[];
  turn_rows<TI, TO, INTER, D, BY_HEADS>(r, t, blockIdx.x, blockIdx.y, smem);
}

template <typename TI, typename TO, bool INTER, int D, bool BY_HEADS>
static attn_status_t launch(const Rows& r, const Turn& t, cudaStream_t stream) {
  if (r.head_groups > 65535) return ATTN_ERR_INVALID_ARG;
  auto kern = rotary_kernel<TI, TO, INTER, D, BY_HEADS>;
  static DeviceOnce setup;
  const attn_status_t st = setup.run([&]() -> attn_status_t {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, ring_bytes<TI>()) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
  });
  if (st != ATTN_OK) return st;
  kern<<<dim3(r.tiles, r.head_groups), THREADS, ring_bytes<TI>(), stream>>>(r, t);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <typename TI, typename TO, bool INTER>
static attn_status_t launch(const Rows& r, const Turn& t, int head_dim, cudaStream_t stream) {
  if (head_dim == 128)
    return r.by_heads ? launch<TI, TO, INTER, 128, true>(r, t, stream) : launch<TI, TO, INTER, 128, false>(r, t, stream);
  return r.by_heads ? launch<TI, TO, INTER, 64, true>(r, t, stream) : launch<TI, TO, INTER, 64, false>(r, t, stream);
}

template <typename TI, typename TO>
static attn_status_t launch(const Rows& r, const Turn& t, int head_dim, bool inter, cudaStream_t stream) {
  return inter ? launch<TI, TO, true>(r, t, head_dim, stream) : launch<TI, TO, false>(r, t, head_dim, stream);
}

}  // namespace rotary

attn_status_t launch_rotary(const attn_rotary_params& p, cudaStream_t stream) {
  rotary::Rows r;
  memset(&r, 0, sizeof(r));
  r.q = p.q, r.k = p.k, r.q_out = p.q_out, r.k_out = p.k_out;
  r.positions = p.positions;
  if ((long long)p.batch * p.seqlen > INT32_MAX) return ATTN_ERR_INVALID_ARG;
  r.tokens = p.batch * p.seqlen;
  r.seqlen = p.seqlen;
  r.hq = p.num_q_heads;
  r.heads = p.num_q_heads + (p.k ? p.num_k_heads : 0);
  if (r.tokens == 0 || r.heads == 0) return ATTN_OK;
  r.q_bs = p.q_batch_stride, r.q_hs = p.q_head_stride, r.q_rs = p.q_row_stride;
  r.k_bs = p.k_batch_stride, r.k_hs = p.k_head_stride, r.k_rs = p.k_row_stride;
  // Rows next to one another: heads, if they are closer than tokens.
  rotary::plan_rows(r, p.head_dim, r.hq > 1 && r.q_hs < r.q_rs, device_sm_count());
  r.qo_bs = p.qo_batch_stride, r.qo_hs = p.qo_head_stride, r.qo_rs = p.qo_row_stride;
  r.ko_bs = p.ko_batch_stride, r.ko_hs = p.ko_head_stride, r.ko_rs = p.ko_row_stride;
  const rotary::Turn t = {p.inv_freq, p.rotary_dim, p.magnitude, p.inverse ? -1.f : 1.f};
  const bool inter = p.interleaved != 0;
  if (p.in_dtype == ATTN_DTYPE_BF16)
    return p.out_dtype == ATTN_DTYPE_BF16 ? rotary::launch<__nv_bfloat16, __nv_bfloat16>(r, t, p.head_dim, inter, stream)
                                          : rotary::launch<__nv_bfloat16, float>(r, t, p.head_dim, inter, stream);
  return p.out_dtype == ATTN_DTYPE_BF16 ? rotary::launch<float, __nv_bfloat16>(r, t, p.head_dim, inter, stream)
                                        : rotary::launch<float, float>(r, t, p.head_dim, inter, stream);
}

}  // namespace attn
