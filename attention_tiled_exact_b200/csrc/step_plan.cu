// The plan of a step over a paged cache (attn_plan_paged_step), for sm_100a:
// prefix sums of the new tokens and of the blocks they need, then one position
// and slot for each token and one table entry for each new block.
//
// One launch of one thread-block cluster. Every CTA scans the requests itself
// (a few integers per thread, from L2) instead of waiting for another's sums,
// keeps a chunk of the prefix sums in shared memory, and fills its share of
// the chunk's rows, each finding its request by binary search. The cluster's
// barrier stands between the last read of the lengths and the writes of the
// advanced state, which may be the same memory. The bytes are few (8 per token
// out): what bounds it is the launch and the chain load - scan - search - load.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace plan {

namespace cg = cooperative_groups;

constexpr int THREADS = 512;
constexpr int CHUNK = 2048;  // requests whose prefix sums are in shared memory at once
constexpr int PER = CHUNK / THREADS;
constexpr int BS = 16;

struct Args {
  const int32_t* seq_lens;
  const int32_t* new_lens;
  int32_t* table;
  const int32_t* free_blocks;
  const int32_t* num_used;
  int32_t* seq_out;
  int32_t* cu;
  int32_t* positions;
  int32_t* slots;
  int32_t* used_out;
  int32_t* flags;
  int batch, max_blocks, num_blocks, num_free, total_q;
};

// Sums of (tokens, blocks) in front of this thread's requests, over the block.
__device__ __forceinline__ void scan_pair(long long& tok, long long& blk, long long& tok_all, long long& blk_all,
                                          long long (*sums)[2]) {
  const int lane = lane_id(), warp = warp_id();
  long long t = tok, k = blk;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, t, d), b = __shfl_up_sync(0xffffffffu, k, d);
    if (lane >= d) t += a, k += b;
  }
  if (lane == 31) sums[warp][0] = t, sums[warp][1] = k;
  __syncthreads();
  long long t0 = 0, k0 = 0;
  tok_all = blk_all = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) t0 = tok_all, k0 = blk_all;
    tok_all += sums[w][0];
    blk_all += sums[w][1];
  }
  tok = t0 + t - tok;
  blk = k0 + k - blk;
  __syncthreads();
}

__global__ void __launch_bounds__(THREADS) plan_kernel(const Args a) {
  __shared__ int s_cu[CHUNK + 1];    // the chunk's first rows, clipped to total_q
  __shared__ int s_seq[CHUNK];       // cached tokens
  __shared__ int s_base[CHUNK];      // place of the request's first new block in the free list, clipped to num_free
  __shared__ long long s_sums[THREADS / 32][2];
  __shared__ unsigned long long s_taken;  // blocks taken for the tokens that have a row
  if (threadIdx.x == 0) s_taken = 0;  // the first scan's barriers stand before its first use
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int cap = a.max_blocks * BS;
  int faults = 0;
  int used = a.num_used ? a.num_used[0] : 0;
  if (used < 0 || used > a.num_free) {
    faults |= ATTN_FAULT_NO_BLOCK;
    used = used < 0 ? 0 : a.num_free;
  }
  long long tok_before = 0, blk_before = 0;  // of the chunks so far
  // A request's lengths, bounded to its table row.
  auto lengths = [&](int b, int& s, int& n) {
    s = a.seq_lens[b];
    n = a.new_lens[b];
    if (s < 0 || s > cap) {
      faults |= ATTN_FAULT_BAD_LENGTH;
      s = s < 0 ? 0 : cap;
    }
    if (n < 0 || n > cap - s) {
      faults |= ATTN_FAULT_BAD_LENGTH;
      n = n < 0 ? 0 : cap - s;
    }
  };
  for (int c0 = 0; c0 < a.batch; c0 += CHUNK) {
    const int count = min(CHUNK, a.batch - c0);
    int s[PER], n[PER];
    long long tok = 0, blk = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = threadIdx.x * PER + i;
      s[i] = n[i] = 0;
      if (j < count) lengths(c0 + j, s[i], n[i]);
      tok += n[i];
      blk += (s[i] + n[i] + BS - 1) / BS - (s[i] + BS - 1) / BS;
    }
    long long tok_all, blk_all;
    scan_pair(tok, blk, tok_all, blk_all, s_sums);
    tok += tok_before;
    blk += blk_before + used;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = threadIdx.x * PER + i;
      if (j < count) {
        s_cu[j] = (int)min(tok, (long long)a.total_q);
        s_seq[j] = s[i];
        s_base[j] = (int)min(blk, (long long)a.num_free);
        if (rank == 0) a.cu[c0 + j] = s_cu[j];
        if (rank == 0 && n[i] > 0 && tok < a.total_q) {
          const int rows = (int)min((long long)n[i], a.total_q - tok);
          const int need = (s[i] + rows + BS - 1) / BS - (s[i] + BS - 1) / BS;
          if (need) atomicAdd(&s_taken, (unsigned long long)need);
        }
      }
      tok += n[i];
      blk += (s[i] + n[i] + BS - 1) / BS - (s[i] + BS - 1) / BS;
    }
    tok_before += tok_all;
    blk_before += blk_all;
    if (threadIdx.x == 0) s_cu[count] = (int)min(tok_before, (long long)a.total_q);
    __syncthreads();
    const int end = s_cu[count];
    for (int t = s_cu[0] + rank * THREADS + threadIdx.x; t < end; t += ranks * THREADS) {
      int lo = 0, hi = count;  // the last request whose first row is <= t: it has row t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t) lo = mid; else hi = mid;
      }
      const int pos = s_seq[lo] + (t - s_cu[lo]);
      const int col = pos / BS, had = (s_seq[lo] + BS - 1) / BS;
      int32_t* entry = a.table + (long long)(c0 + lo) * a.max_blocks + col;
      const int at = s_base[lo] + (col - had);  // both terms below 2^30
      int id = -1;
      if (col >= had && at >= a.num_free) {
        faults |= ATTN_FAULT_NO_BLOCK;
      } else {
        id = col < had ? *entry : a.free_blocks[at];
        if (id < 0 || id >= a.num_blocks) {
          faults |= ATTN_FAULT_BAD_BLOCK;
          id = -1;
        }
      }
      if (col >= had && pos % BS == 0) *entry = id;
      a.positions[t] = pos;
      a.slots[t] = id < 0 ? -1 : id * BS + pos % BS;
    }
    __syncthreads();  // the chunk's sums are overwritten next
  }
  for (long long t = min(tok_before, (long long)a.total_q) + rank * THREADS + threadIdx.x; t < a.total_q;
       t += ranks * THREADS) {
    a.positions[t] = -1;
    a.slots[t] = -1;
  }
  if (tok_before > a.total_q) faults |= ATTN_FAULT_BAD_LENGTH;
  cluster.sync();  // every CTA has read the lengths and num_used
  if (rank == 0) {
    const int end = (int)min(tok_before, (long long)a.total_q);
    for (int b = threadIdx.x; b < a.batch; b += THREADS) {
      int s, n;
      lengths(b, s, n);
      a.seq_out[b] = s + ((b + 1 < a.batch ? a.cu[b + 1] : end) - a.cu[b]);  // a.cu: this CTA's own writes
    }
    if (threadIdx.x == 0) {
      a.cu[a.batch] = end;
      a.used_out[0] = (int)min((long long)(used + s_taken), (long long)a.num_free);
    }
  }
  if (faults && a.flags) atomicOr(a.flags, faults);
}

}  // namespace plan

attn_status_t launch_plan(const attn_plan_params& p, cudaStream_t stream) {
  const plan::Args a = {p.seq_lens, p.new_lens, p.block_table, p.free_blocks, p.num_used, p.seq_lens_out,
                        p.cu_seqlens_q, p.positions, p.slot_map, p.num_used_out, p.error_flags, p.batch,
                        p.max_blocks_per_seq, p.num_blocks, p.num_free, p.total_q};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.total_q > 4 * plan::THREADS ? 8 : 1;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(attr[0].val.clusterDim.x);
  cfg.blockDim = dim3(plan::THREADS);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, plan::plan_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

}  // namespace attn
