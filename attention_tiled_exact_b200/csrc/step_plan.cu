// The plan of a step over a paged cache (attn_plan_paged_step), for sm_100a:
// prefix sums of the new tokens and of the blocks they need, then one position
// and slot for each token and one table entry for each new block.
//
// Every CTA scans the requests itself (a few integers per thread, from L2)
// instead of waiting for another's sums, keeps a chunk of the prefix sums in
// shared memory, and fills its share of the chunk's rows four at a time: one
// binary search for the first row's request, then a walk (one at a time in a
// small step: 64 rows of 64 requests are 1.2 us faster than four at a time). A step of
// up to SMALL rows is one CTA, a larger one takes as many CTAs as its rows fill.
// The first CTA also advances the state; if the new state lies over the old one,
// which the others may still be reading, a dependent launch of one CTA does.
// The bytes are few (8 per token out): what bounds it is the launch and the
// chain load - scan - search - load. One token for each of 64 sequences: 4.2 us;
// 208,000 rows of 300 requests: 5.4 us (53 us by one cluster of 8 CTAs, a row at a
// time), over the old state 6.8 us.
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace plan {

constexpr int THREADS = 512;
constexpr int CHUNK = 2048;  // requests whose prefix sums are in shared memory at once
constexpr int PER = CHUNK / THREADS;
constexpr int BS = 16;
constexpr int SMALL = 4 * THREADS;  // rows that one CTA fills in one round

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
  int vec;  // positions and slots are 16-byte aligned
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

// Bounds a request's cached tokens s and the new ones it asks for to its table row;
// n: the new ones that it gets. Its rows in the step are all that it asks for,
// because the caller's rows lie by that, and a request over its limit must not
// move those behind it.
__device__ __forceinline__ void bound(const Args& a, int& s, int& asked, int& n, int& faults) {
  const int cap = a.max_blocks * BS, s0 = s, asked0 = asked;
  s = min(max(s, 0), cap);
  asked = max(asked, 0);
  n = min(asked, cap - s);
  if (s != s0 || n != asked0) faults |= ATTN_FAULT_BAD_LENGTH;
}

__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + BS - 1) / BS; }

// Blocks in use before the step, bounded to the free list.
__device__ __forceinline__ int used_before(const Args& a, int& faults) {
  const int used = a.num_used[0];
  if (used >= 0 && used <= a.num_free) return used;
  faults |= ATTN_FAULT_NO_BLOCK;
  return used < 0 ? 0 : a.num_free;
}

// By one CTA, when a.cu is complete and nobody reads the old state any more:
// the lengths and the blocks in use, for the rows that the step has.
__device__ __forceinline__ void advance_state(const Args& a, int used, long long (*sums)[2]) {
  long long none = 0, taken = 0;
  int ignored = 0;  // the fill has flagged them
  for (int b = threadIdx.x; b < a.batch; b += THREADS) {
    int s = a.seq_lens[b], asked = a.new_lens[b], n;
    bound(a, s, asked, n, ignored);
    const int end = s + min(n, a.cu[b + 1] - a.cu[b]);
    taken += blocks_of(end) - blocks_of(s);
    a.seq_out[b] = end;
  }
  long long all, none_all;
  scan_pair(none, taken, none_all, all, sums);
  if (threadIdx.x == 0) a.used_out[0] = (int)min(used + all, (long long)a.num_free);
}

// ADVANCE: the first CTA advances the state. More than one may run with it only if
// the new state is apart from the old one.
template <bool ADVANCE>
__global__ void __launch_bounds__(THREADS) plan_kernel(const Args a) {
  __shared__ int s_cu[CHUNK + 1];    // the chunk's first rows, clipped to total_q
  __shared__ int s_seq[CHUNK];       // cached tokens
  __shared__ int s_base[CHUNK];      // place of the request's first new block in the free list, clipped to num_free
  __shared__ long long s_sums[THREADS / 32][2];
  const int rank = (int)blockIdx.x, ranks = (int)gridDim.x;
  if constexpr (!ADVANCE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int faults = 0;
  const int used = used_before(a, faults);
  // A thread's rows: in a small step one, because rows of different requests
  // follow one another, each with its load of a table or free-list entry.
  const int rows = ADVANCE && a.total_q <= THREADS ? 1 : 4;
  const int cap = a.max_blocks * BS;
  bool advanced = false, dropped = false;    // dropped: some request asks for more than its table row holds
  long long tok_before = 0, blk_before = 0;  // rows and blocks of the chunks so far
  int last = 0;  // the end of the rows that this thread's requests have a token for
  for (int c0 = 0; c0 < a.batch; c0 += CHUNK) {
    const int count = min(CHUNK, a.batch - c0);
    int s[PER], n[PER], asked[PER];
    long long tok = 0, blk = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int j = threadIdx.x * PER + i;
      s[i] = j < count ? a.seq_lens[c0 + j] : 0;
      asked[i] = j < count ? a.new_lens[c0 + j] : 0;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      bound(a, s[i], asked[i], n[i], faults);
      tok += asked[i];
      blk += blocks_of(s[i] + n[i]) - blocks_of(s[i]);
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
        if (n[i] > 0 && tok < a.total_q) last = (int)min(tok + n[i], (long long)a.total_q);
      }
      tok += asked[i];
      blk += blocks_of(s[i] + n[i]) - blocks_of(s[i]);
    }
    tok_before += tok_all;
    blk_before += blk_all;
    if (ADVANCE && rank == 0 && a.batch <= CHUNK && tok_before <= a.total_q) {  // every row of every request has its place
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int j = threadIdx.x * PER + i;
        if (j < count) a.seq_out[j] = s[i] + n[i];
      }
      if (threadIdx.x == 0) a.used_out[0] = (int)min(used + blk_before, (long long)a.num_free);
      advanced = true;
    }
    if (threadIdx.x == 0) s_cu[count] = (int)min(tok_before, (long long)a.total_q);
    __syncthreads();
    const int begin = s_cu[0], end = s_cu[count];
    // Rows 4 i .. 4 i + 3 (or row i), as far as they are the chunk's.
    for (int i = begin / rows + rank * THREADS + threadIdx.x; (long long)rows * i < end; i += ranks * THREADS) {
      const int t0 = max(rows * i, begin), t1 = (int)min((long long)rows * i + rows, (long long)end);
      int lo = 0, hi = count;  // the last request whose first row is <= t0: it has row t0
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_cu[mid] <= t0) lo = mid; else hi = mid;
      }
      int pos[4], slot[4];
      int id = -1, known = -1;  // the block of column `known` of request lo
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = rows * i + j;
        if (t < t0 || t >= t1) continue;
        while (t >= s_cu[lo + 1]) ++lo, known = -1;  // past requests without rows too
        const int nth = t - s_cu[lo];
        if (nth >= cap - s_seq[lo]) {  // a row without a token
          pos[j] = slot[j] = -1;
          continue;
        }
        const int p = s_seq[lo] + nth;
        const int col = p / BS, had = blocks_of(s_seq[lo]);
        if (col != known) {
          known = col;
          int32_t* entry = a.table + (long long)(c0 + lo) * a.max_blocks + col;
          const int at = s_base[lo] + (col - had);  // both terms below 2^30
          id = -1;
          if (col >= had && at >= a.num_free) {
            faults |= ATTN_FAULT_NO_BLOCK;
          } else {
            id = col < had ? *entry : a.free_blocks[at];
            if (id < 0 || id >= a.num_blocks) {
              faults |= ATTN_FAULT_BAD_BLOCK;
              id = -1;
            }
          }
          if (col >= had && p % BS == 0) *entry = id;
        }
        pos[j] = p;
        slot[j] = id < 0 ? -1 : id * BS + p % BS;
      }
      if (a.vec && t1 - t0 == 4) {
        *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<int4*>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int t = rows * i + j;
          if (t >= t0 && t < t1) a.positions[t] = pos[j], a.slots[t] = slot[j];
        }
      }
    }
    bool cut = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) cut |= n[i] < asked[i];
    dropped |= __syncthreads_or(cut) != 0;  // and the chunk's sums are overwritten next
  }
  for (long long t = min(tok_before, (long long)a.total_q) + rank * THREADS + threadIdx.x; t < a.total_q;
       t += ranks * THREADS) {
    a.positions[t] = -1;
    a.slots[t] = -1;
  }
  if (tok_before > a.total_q) faults |= ATTN_FAULT_BAD_LENGTH;
  if (faults && a.flags) atomicOr(a.flags, faults);
  if (rank != 0) return;
  int end = (int)min(tok_before, (long long)a.total_q);
  if (dropped) {
    // The step ends behind its last token: rows without one belong to a request
    // only where a later request's tokens follow.
#pragma unroll
    for (int d = 16; d; d >>= 1) last = max(last, __shfl_xor_sync(0xffffffffu, last, d));
    if (lane_id() == 0) s_sums[warp_id()][0] = last;
    __syncthreads();
    for (int w = 0; w < THREADS / 32; ++w) last = max(last, (int)s_sums[w][0]);
    end = last;
    for (int b = threadIdx.x; b < a.batch; b += THREADS)
      if (a.cu[b] > end) a.cu[b] = end;
  }
  if (threadIdx.x == 0) a.cu[a.batch] = end;
  if (ADVANCE && !advanced) {
    __syncthreads();
    advance_state(a, used, s_sums);
  }
}

__global__ void __launch_bounds__(THREADS) advance_kernel(const Args a) {
  __shared__ long long s_sums[THREADS / 32][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int ignored = 0;
  advance_state(a, used_before(a, ignored), s_sums);
}

}  // namespace plan

attn_status_t launch_plan(const attn_plan_params& p, cudaStream_t stream) {
  const bool vec = ((reinterpret_cast<uintptr_t>(p.positions) | reinterpret_cast<uintptr_t>(p.slot_map)) & 15u) == 0;
  const plan::Args a = {p.seq_lens, p.new_lens, p.block_table, p.free_blocks, p.num_used, p.seq_lens_out,
                        p.cu_seqlens_q, p.positions, p.slot_map, p.num_used_out, p.error_flags, p.batch,
                        p.max_blocks_per_seq, p.num_blocks, p.num_free, p.total_q, vec ? 1 : 0};
  const int want = p.total_q <= plan::SMALL ? 1 : (p.total_q + plan::SMALL - 1) / plan::SMALL, sms = device_sm_count();
  const int ctas = want < sms ? want : sms;
  const bool apart = (p.seq_lens_out + p.batch <= p.seq_lens || p.seq_lens + p.batch <= p.seq_lens_out) &&
                     p.num_used_out != p.num_used;
  if (ctas == 1 || apart) {
    plan::plan_kernel<true><<<ctas, plan::THREADS, 0, stream>>>(a);
    return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
  }
  plan::plan_kernel<false><<<ctas, plan::THREADS, 0, stream>>>(a);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(plan::THREADS);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaGetLastError() != cudaSuccess || cudaLaunchKernelEx(&cfg, plan::advance_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

}  // namespace attn
