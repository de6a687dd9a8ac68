// Writing the paged cache (attn_append_paged) and reading it back
// (attn_gather_paged), for sm_100a.
//
// Append, one launch with two kinds of blocks. The first blocks turn the query
// rows (turn_rows). In the others a warp owns one kv head of K or of V and a
// window of rows: it finds the runs of consecutive slots that start in the
// window, and handles a run (at most 16 tokens, one cache block) as a whole.
// A lane holds one 16-element unit of 16 * units / 32 of the block's tokens in
// registers: kept tokens (in front of the run) are read back as values, new
// ones are read and turned; one warp reduction gives the block's largest
// magnitude and with it the scale, and the codes go out. So a block's scale
// and codes come from one warp, without atomics, whatever the grid's order.
//   value -> code: e = smallest integer with amax <= 448 * 2^e,
//   code = e4m3(x * 2^-e), the only rounding of a key or value; it is made
//   from the fp32 turned key, not from a bf16 copy of it.
//
// Both kernels are bound by HBM (each element in and out once) for many
// tokens and by the launch and two dependent loads (slot, then row or block)
// for one token per sequence.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "block_scaled.cuh"
#include "internal.h"
#include "rotary.cuh"

namespace attn {
namespace cache {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int BS = 16;
constexpr unsigned FULL = 0xffffffffu;

struct Append {
  rotary::Rows rows;  // the queries (rows.heads == 0: none)
  rotary::Turn turn;  // rotary_dim 0: nothing is turned
  int q_blocks;       // blocks of the grid that turn queries
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  long long k_rs, k_hs, v_rs, v_hs;
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint8_t* k_scales;
  uint8_t* v_scales;
  const int32_t* slots;
  const int32_t* positions;
  int32_t* flags;
  int total, hkv, num_slots;
  int window;  // rows whose runs one warp handles: 1 or 16
};

// One run of `n` tokens from row `t` on, to offsets off0 .. off0 + n - 1 of a
// block whose codes (or bf16 elements) of this head start at `page`.
template <int D, bool FP8, bool INTER>
__device__ __forceinline__ void write_run(const Append& a, const __nv_bfloat16* x, long long rs, bool turn_rows,
                                          int t, int n, int off0, uint8_t* page, uint8_t* scale) {
  constexpr int UNITS = D / 16, GROUPS = 32 / UNITS, PER = BS / GROUPS;
  const int lane = lane_id();
  const int u = lane % UNITS, grp = lane / UNITS;
  const int rotary_dim = turn_rows ? a.turn.rotary_dim : 0;
  const bool turned = u * 16 < rotary_dim;
  const int2 off = rotary::unit_offsets<INTER>(u, rotary_dim);
  const float old_scale = FP8 && off0 > 0 ? bscale::scale_of(*scale) : 0.f;
  const int old_byte = FP8 && off0 > 0 ? *scale : -1;
  float val[PER][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int o = grp + GROUPS * i;  // this lane's token of the block
    if (o >= off0 && o < off0 + n) {
      const long long row = t + (o - off0);
      const __nv_bfloat16* src = x + row * rs;
      rotary::load8(src + off.x, &val[i][0]);
      rotary::load8(src + off.y, &val[i][8]);
      if (turned) {
        float c[8], s[8];
        rotary::unit_turn(a.turn, __ldg(a.positions + row), u, c, s);
        rotary::turn16<INTER>(val[i], c, s);
      }
    } else if (FP8 && o < off0) {
      bscale::load_codes8(page + o * D + off.x, &val[i][0]);
      bscale::load_codes8(page + o * D + off.y, &val[i][8]);
#pragma unroll
      for (int j = 0; j < 16; ++j) val[i][j] *= old_scale;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) val[i][j] = 0.f;
    }
    if constexpr (FP8) {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (!(fabsf(val[i][j]) < INFINITY)) val[i][j] = NAN;  // stored as NaN, and outside the maximum
        amax = fmaxf(amax, fabsf(val[i][j]));
      }
    }
  }
  if constexpr (FP8) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, d));
    const int e = bscale::exponent_for(amax);
    const float mul = bscale::pow2i(-e);
    const bool recode = e + bscale::BIAS != old_byte;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int o = grp + GROUPS * i;
      if (o < off0 + n && (o >= off0 || recode)) {
        bscale::store_codes8(page + o * D + off.x, &val[i][0], mul);
        bscale::store_codes8(page + o * D + off.y, &val[i][8], mul);
      }
    }
    if (lane == 0) *scale = (uint8_t)(e + bscale::BIAS);
  } else {
    __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(page);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int o = grp + GROUPS * i;
      if (o >= off0 && o < off0 + n) {
        rotary::store8(dst + o * D + off.x, &val[i][0]);
        rotary::store8(dst + o * D + off.y, &val[i][8]);
      }
    }
  }
}

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(THREADS) append_kernel(const Append a) {
  if ((int)blockIdx.x < a.q_blocks) {
    rotary::turn_rows<__nv_bfloat16, __nv_bfloat16, INTER>(a.rows, a.turn,
                                                           (long long)blockIdx.x * THREADS + threadIdx.x);
    return;
  }
  const int lane = lane_id();
  const long long item = (long long)(blockIdx.x - a.q_blocks) * WARPS + warp_id();
  const bool is_v = item & 1;
  const int h = (int)((item >> 1) % a.hkv);
  const long long first = (item >> 1) / a.hkv * a.window;  // the window's first row
  if (first >= a.total) return;
  // Lane i holds the slot of row first - 1 + i: the window's rows, the one in
  // front of it and the 15 that a run may reach into behind it.
  const long long row = first - 1 + lane;
  const int slot = row >= 0 && row < a.total ? __ldg(a.slots + row) : -1;
  const int before = __shfl_up_sync(FULL, slot, 1);
  const bool good = slot >= 0 && slot < a.num_slots;
  const bool mine = lane >= 1 && lane <= a.window && row < a.total;
  if (mine && slot >= a.num_slots && a.flags) atomicOr(a.flags, ATTN_FAULT_BAD_BLOCK);
  const bool follows = lane >= 1 && good && (slot & (BS - 1)) != 0 && before == slot - 1;
  const unsigned runs = __ballot_sync(FULL, mine && good && !follows), rest = __ballot_sync(FULL, follows);
  const __nv_bfloat16* x = is_v ? a.v + h * a.v_hs : a.k + h * a.k_hs;
  const long long rs = is_v ? a.v_rs : a.k_rs;
  uint8_t* pool = is_v ? a.v_cache : a.k_cache;
  uint8_t* scales = is_v ? a.v_scales : a.k_scales;
  for (unsigned left = runs; left; left &= left - 1) {
    const int i = __ffs(left) - 1;
    const int n = i == 31 ? 1 : 1 + __ffs(~(rest >> (i + 1))) - 1;  // rows that follow row i, and it
    const int at = __shfl_sync(FULL, slot, i);
    const long long blk = (long long)(at / BS) * a.hkv + h;
    write_run<D, FP8, INTER>(a, x, rs, !is_v, (int)(first - 1 + i), n, at % BS, pool + blk * (BS * D * (FP8 ? 1 : 2)),
                             FP8 ? scales + blk : nullptr);
  }
}

struct Gather {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* table;
  const int32_t* seq_lens;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int32_t* flags;
  int hkv, width, num_blocks, max_blocks, blocks;  // blocks: of 16 rows that `width` takes
  int zero_to;  // rows behind a sequence are cleared up to the next multiple of this (0: up to width)
  int flag_width;  // a sequence over width is a fault
};

// One warp per (sequence, block, kv head): 16 rows of K and of V. A lane
// holds 8-element vectors of both pages, all on their way before the first is
// stored, so that a warp's store covers 512 bytes in a row.
template <int D, bool FP8>
__global__ void __launch_bounds__(THREADS) gather_kernel(const Gather g, long long items) {
  // A dependent launch may set itself up; it waits for the whole of this one.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const long long item = (long long)blockIdx.x * WARPS + warp_id();
  if (item >= items) return;
  const int lane = lane_id();
  const int h = (int)(item % g.hkv);
  const int blk = (int)(item / g.hkv % g.blocks);
  const long long b = item / g.hkv / g.blocks;
  const int row0 = blk * BS;
  int len = __ldg(g.seq_lens + b);
  int id = blk < g.max_blocks ? __ldg(g.table + b * g.max_blocks + blk) : -1;
  if (lane == 0 && h == 0 && blk == 0 && g.flags &&
      (len < 0 || len > (long long)g.max_blocks * BS || (g.flag_width && len > g.width)))
    atomicOr(g.flags, ATTN_FAULT_BAD_LENGTH);
  len = min(min(max(len, 0), g.max_blocks * BS), g.width);
  const int end = g.zero_to ? min(g.width, (len + g.zero_to - 1) / g.zero_to * g.zero_to) : g.width;
  if (row0 >= end) return;
  if (row0 < len && (id < 0 || id >= g.num_blocks)) {
    if (lane == 0 && g.flags) atomicOr(g.flags, ATTN_FAULT_BAD_BLOCK);
    id = -1;
  }
  const int live = row0 < len && id >= 0 ? min(BS, len - row0) : 0, rows = min(BS, end - row0);
  using Raw = typename std::conditional<FP8, uint2, uint4>::type;
  constexpr int VECS = D / 8, STEPS = BS * VECS / 32;
  const long long at = (long long)id * g.hkv + h;
  Raw raw[2][STEPS];
  float scale[2];
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const Raw* page = reinterpret_cast<const Raw*>(which ? g.v_cache : g.k_cache) + at * (BS * VECS);
    scale[which] = FP8 && live > 0 ? bscale::scale_of(__ldg((which ? g.v_scales : g.k_scales) + at)) : 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      raw[which][i] = Raw{};
      if ((i * 32 + lane) / VECS < live) raw[which][i] = __ldg(page + i * 32 + lane);
    }
  }
  const long long out = ((b * g.hkv + h) * g.width + row0) * D;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    uint4* dst = reinterpret_cast<uint4*>((which ? g.v_out : g.k_out) + out);
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const int v = i * 32 + lane;
      if (v / VECS >= rows) continue;
      if constexpr (FP8) {
        const uint2 r = raw[which][i];
        const float mul = v / VECS < live ? scale[which] : 0.f;
        const float2 x0 = bscale::codes_to_float2(r.x & 0xffffu), x1 = bscale::codes_to_float2(r.x >> 16);
        const float2 x2 = bscale::codes_to_float2(r.y & 0xffffu), x3 = bscale::codes_to_float2(r.y >> 16);
        dst[v] = make_uint4(pack_bf16x2(x0.x * mul, x0.y * mul), pack_bf16x2(x1.x * mul, x1.y * mul),
                            pack_bf16x2(x2.x * mul, x2.y * mul), pack_bf16x2(x3.x * mul, x3.y * mul));
      } else {
        dst[v] = raw[which][i];
      }
    }
  }
}

}  // namespace cache

template <int D, bool FP8>
static attn_status_t launch_append_d(const cache::Append& a, bool inter, unsigned blocks, cudaStream_t stream) {
  if (inter)
    cache::append_kernel<D, FP8, true><<<blocks, cache::THREADS, 0, stream>>>(a);
  else
    cache::append_kernel<D, FP8, false><<<blocks, cache::THREADS, 0, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

attn_status_t launch_append(const attn_append_params& p, cudaStream_t stream) {
  if (p.total == 0) return ATTN_OK;
  cache::Append a;
  memset(&a, 0, sizeof(a));
  a.turn = {p.inv_freq, p.rotary_dim, p.magnitude, 1.f};
  a.k = reinterpret_cast<const __nv_bfloat16*>(p.k);
  a.v = reinterpret_cast<const __nv_bfloat16*>(p.v);
  a.k_rs = p.k_row_stride, a.k_hs = p.k_head_stride, a.v_rs = p.v_row_stride, a.v_hs = p.v_head_stride;
  a.k_cache = reinterpret_cast<uint8_t*>(p.k_cache);
  a.v_cache = reinterpret_cast<uint8_t*>(p.v_cache);
  a.k_scales = p.k_scales;
  a.v_scales = p.v_scales;
  a.slots = p.slot_map;
  a.positions = p.positions;
  a.flags = p.error_flags;
  a.total = p.total;
  a.hkv = p.num_kv_heads;
  a.num_slots = p.num_blocks * cache::BS;
  const int sms = device_sm_count();
  const bool turn_q = p.q && p.num_q_heads > 0;
  // Queries that stay as and where they are need no pass.
  if (turn_q && !(p.rotary_dim == 0 && p.q == p.q_out && p.q_row_stride == p.qo_row_stride &&
                  p.q_head_stride == p.qo_head_stride)) {
    rotary::Rows& r = a.rows;
    r.q = p.q, r.q_out = p.q_out;
    r.positions = p.positions;
    r.slots = p.slot_map;
    r.tokens = p.total, r.seqlen = p.total;
    r.hq = r.heads = p.num_q_heads;
    r.units = p.head_dim / 16;
    r.head_groups = rotary::head_groups_for(r.tokens, r.heads, r.units, sms);
    r.q_hs = p.q_head_stride, r.q_rs = p.q_row_stride;
    r.qo_hs = p.qo_head_stride, r.qo_rs = p.qo_row_stride;
    const long long threads = r.tokens * r.head_groups * r.units;
    const long long q_blocks = (threads + cache::THREADS - 1) / cache::THREADS;
    if (q_blocks > 0x3fffffffLL) return ATTN_ERR_INVALID_ARG;
    a.q_blocks = (int)q_blocks;
  }
  // A warp per row while that does not fill the machine (a decode step has one
  // run per row), a warp per 16 rows beyond (a chunk has one run per 16).
  a.window = 2LL * p.num_kv_heads * p.total <= 32LL * sms ? 1 : 16;
  const long long items = 2LL * p.num_kv_heads * ((p.total + a.window - 1) / a.window);
  const long long blocks = a.q_blocks + (items + cache::WARPS - 1) / cache::WARPS;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const bool fp8 = p.kv_dtype == ATTN_DTYPE_FP8_E4M3, inter = p.interleaved != 0;
  if (p.head_dim == 128)
    return fp8 ? launch_append_d<128, true>(a, inter, (unsigned)blocks, stream)
               : launch_append_d<128, false>(a, inter, (unsigned)blocks, stream);
  return fp8 ? launch_append_d<64, true>(a, inter, (unsigned)blocks, stream)
             : launch_append_d<64, false>(a, inter, (unsigned)blocks, stream);
}

attn_status_t launch_gather(const attn_gather_params& p, int zero_to, bool flag_width, cudaStream_t stream) {
  const int blocks = (p.width + cache::BS - 1) / cache::BS;
  const long long items = (long long)p.batch * blocks * p.num_kv_heads;
  if (items == 0) return ATTN_OK;
  const long long grid = (items + cache::WARPS - 1) / cache::WARPS;
  if (grid > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  const cache::Gather g = {reinterpret_cast<const uint8_t*>(p.k_cache), reinterpret_cast<const uint8_t*>(p.v_cache),
                           p.k_scales, p.v_scales, p.block_table, p.seq_lens,
                           reinterpret_cast<__nv_bfloat16*>(p.k_out), reinterpret_cast<__nv_bfloat16*>(p.v_out),
                           p.error_flags, p.num_kv_heads, p.width, p.num_blocks, p.max_blocks_per_seq, blocks,
                           zero_to, flag_width ? 1 : 0};
  const bool fp8 = p.kv_dtype == ATTN_DTYPE_FP8_E4M3;
  if (p.head_dim == 128) {
    if (fp8)
      cache::gather_kernel<128, true><<<(unsigned)grid, cache::THREADS, 0, stream>>>(g, items);
    else
      cache::gather_kernel<128, false><<<(unsigned)grid, cache::THREADS, 0, stream>>>(g, items);
  } else {
    if (fp8)
      cache::gather_kernel<64, true><<<(unsigned)grid, cache::THREADS, 0, stream>>>(g, items);
    else
      cache::gather_kernel<64, false><<<(unsigned)grid, cache::THREADS, 0, stream>>>(g, items);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
