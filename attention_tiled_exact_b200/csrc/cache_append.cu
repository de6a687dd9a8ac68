// Writing the paged cache (attn_append_paged) and reading it back
// (attn_gather_paged), for sm_100a.
//
// Append, one launch with two kinds of CTAs. The last ones turn the query rows
// (turn_rows); behind the others, whose chain of loads is longer, they fill the
// time that those wait (2048 rows of 32/8 heads 8.8 us, in front of them 11 us).
// The others own a window of rows and some of the K and V heads: they find the
// runs of consecutive slots that start in the window, compute the angles of the
// runs' rows once for all K heads, and two warps handle a run (at most 16 tokens,
// one cache block) of one head of K or V as a whole. A lane holds one 16-element
// unit of 16 * units / 64 of the block's tokens in registers: kept tokens (in
// front of the run) are read back as values, new ones are read and turned; one
// reduction gives the block's largest magnitude and with it the scale, and the
// codes go out. So a block's scale and codes come from one pair of warps,
// without atomics, whatever the grid's order.
//   value -> code: e = smallest integer with amax <= 448 * 2^e,
//   code = e4m3(x * 2^-e), the only rounding of a key or value; it is made
//   from the fp32 turned key, not from a bf16 copy of it.
//
// Both kernels read and write each element once. 8504 rows of 32/8 heads of 128:
// append 36 us (192 MB; the queries alone 23 us at 6.0 TB/s, the keys and values
// alone 20 us, where a run's load, reduction and store follow one another),
// gather 14.5 us (93 MB, 6.4 TB/s); with bf16 pages 36 us (209 MB) and 21 us (119 MB,
// 5.7 TB/s). A decode step of 32 rows takes 3.7 us and 3.5 us (bf16 3.0 and 3.7):
// the launch and two dependent loads (slot, then row or block).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "block_scaled.cuh"
#include "internal.h"
#include "rotary.cuh"

namespace attn {
namespace cache {

constexpr int THREADS = rotary::THREADS;
constexpr int WARPS = THREADS / 32;
constexpr int BS = 16;
constexpr unsigned FULL = 0xffffffffu;

struct Append {
  rotary::Rows rows;  // the queries (rows.heads == 0: none)
  rotary::Turn turn;  // rotary_dim 0: nothing is turned
  int kv_blocks;      // blocks of the grid in front of those that turn queries
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
  int window;      // rows whose runs one CTA handles, at most 16
  int items_per;   // items of a CTA: the K heads, then the V heads
  int chunks;      // CTAs that share a window's items
};

constexpr int PAIRS = WARPS / 2;       // pairs of warps, each with its own run
constexpr int SPAN = 31;               // rows that the runs of a window may reach over

constexpr int KV_STAGES = 2;           // runs whose rows are on their way
constexpr int KV_SLOTS = 4;            // 16-byte vectors of a thread and run: 32 elements

struct __align__(16) AppendSmem {
  uint4 ring[KV_STAGES][KV_SLOTS][THREADS];  // each thread's own
  float2 turn[SPAN][rotary::MAX_PAIRS];  // magnitude * (cos, sin) of the window's rows
  float amax[2][PAIRS][2];
};

// A lane's part of a run: unit u of the tokens grp + GROUPS * i of the block.
template <int D>
struct Lanes {
  static constexpr int UNITS = D / 16, GROUPS = 64 / UNITS, PER = BS / GROUPS;
  int u, grp;
  __device__ __forceinline__ Lanes() : u(lane_id() % UNITS), grp(lane_id() / UNITS + (warp_id() & 1) * (GROUPS / 2)) {}
};

// Starts the copies of the lane's part of a run (as in write_run) to its slots of
// a stage: of new tokens the rows, of kept ones (8-bit pages) the codes.
template <int D, bool FP8>
__device__ __forceinline__ void fetch_run(const __nv_bfloat16* x, long long rs, int rotary_dim, int t, int n, int off0,
                                          const uint8_t* page, uint4 (*stage)[THREADS]) {
  using L = Lanes<D>;
  const L l;
  const int2 off = rotary::unit_offsets<D>(l.u, rotary_dim);
#pragma unroll
  for (int i = 0; i < L::PER; ++i) {
    const int o = l.grp + L::GROUPS * i;
    const uint32_t to = smem_addr(&stage[2 * i][threadIdx.x]);
    if (o >= off0 && o < off0 + n) {
      const __nv_bfloat16* src = x + (long long)(t + o - off0) * rs;
#pragma unroll
      for (int v = 0; v < 2; ++v)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + v * (THREADS * 16)),
                     "l"(src + (v ? off.y : off.x))
                     : "memory");
    } else if (FP8 && o < off0) {
#pragma unroll
      for (int v = 0; v < 2; ++v)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to + v * (THREADS * 16)),
                     "l"(page + o * D + (v ? off.y : off.x))
                     : "memory");
    }
  }
}

// One run of `n` tokens from row `t` on, to offsets off0 .. off0 + n - 1 of a
// block whose codes (or bf16 elements) of this head start at `page`, by a pair
// of warps. turn: the angles of the first row, or NULL. old_byte: the block's
// scale so far, or -1 when nothing in front of the run is kept. amax_at: alternates
// from run to run.
template <int D, bool FP8, bool INTER>
__device__ __forceinline__ void write_run(const uint4 (*stage)[THREADS],
                                          const float2 (*turn)[rotary::MAX_PAIRS], int rotary_dim, int n, int off0,
                                          uint8_t* page, uint8_t* scale, int old_byte, float (*amax_at)[2]) {
  using L = Lanes<D>;
  constexpr int GROUPS = L::GROUPS, PER = L::PER;
  const L l;
  const int lane = lane_id(), pair = warp_id() / 2, half = warp_id() & 1, u = l.u, grp = l.grp;
  const bool turned = turn && u * 16 < rotary_dim;
  const int2 off = rotary::unit_offsets<D>(u, turn ? rotary_dim : 0);
  const float old_scale = old_byte >= 0 ? bscale::scale_of(old_byte) : 0.f;
  float val[PER][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int o = grp + GROUPS * i;  // this lane's token of the block
    if (o >= off0 && o < off0 + n) {
      rotary::load8(reinterpret_cast<const __nv_bfloat16*>(&stage[2 * i][threadIdx.x]), &val[i][0]);
      rotary::load8(reinterpret_cast<const __nv_bfloat16*>(&stage[2 * i + 1][threadIdx.x]), &val[i][8]);
    } else if (FP8 && o < off0) {
      bscale::load_codes8(reinterpret_cast<const uint8_t*>(&stage[2 * i][threadIdx.x]), &val[i][0]);
      bscale::load_codes8(reinterpret_cast<const uint8_t*>(&stage[2 * i + 1][threadIdx.x]), &val[i][8]);
#pragma unroll
      for (int j = 0; j < 16; ++j) val[i][j] *= old_scale;
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) val[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int o = grp + GROUPS * i;
    if (turned && o >= off0 && o < off0 + n) {
      float c[8], s[8];
      rotary::unit_turn<INTER>(turn[o - off0], u, rotary_dim, c, s);
      rotary::UnitTurn ut;
      ut.set(c, s);
      rotary::turn16<INTER>(val[i], ut);
    }
    if constexpr (FP8) {
#pragma unroll
      for (int j = 0; j < 16; ++j) amax = fmaxf(amax, fabsf(val[i][j]));  // passes over a NaN
    }
  }
  if (FP8 && amax == INFINITY) {  // an infinity is stored as NaN, and is outside the maximum
    amax = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (fabsf(val[i][j]) == INFINITY) val[i][j] = NAN;
        amax = fmaxf(amax, fabsf(val[i][j]));
      }
  }
  if constexpr (FP8) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(FULL, amax, d));
    if (lane == 0) amax_at[pair][half] = amax;
    named_bar_sync(1 + pair, 64);  // both warps have read the old scale, too
    amax = fmaxf(amax_at[pair][0], amax_at[pair][1]);
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
    if (lane == 0 && half == 0) *scale = (uint8_t)(e + bscale::BIAS);
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
__global__ void __launch_bounds__(THREADS, 4) append_kernel(const Append a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int item = blockIdx.x;
  if (item >= a.kv_blocks) {
    const int q_item = item - a.kv_blocks, group = q_item / a.rows.tiles;
    rotary::turn_rows<__nv_bfloat16, __nv_bfloat16, INTER, D, true>(a.rows, a.turn, q_item - group * a.rows.tiles, group,
                                                                    smem);
    return;
  }
  AppendSmem& sm = *reinterpret_cast<AppendSmem*>(smem);
  const int lane = lane_id();
  const int chunk = item % a.chunks;
  const long long first = (long long)(item / a.chunks) * a.window;  // the window's first row
  // Lane i holds the slot of row first - 1 + i: the window's rows, the one in
  // front of it and the 15 that a run may reach into behind it.
  const long long row = first - 1 + lane;
  const int slot = row >= 0 && row < a.total ? __ldg(a.slots + row) : -1;
  const int before = __shfl_up_sync(FULL, slot, 1);
  const bool good = slot >= 0 && slot < a.num_slots;
  const bool mine = lane >= 1 && lane <= a.window && row < a.total;
  if (mine && slot >= a.num_slots && a.flags && chunk == 0 && threadIdx.x < 32)
    atomicOr(a.flags, ATTN_FAULT_BAD_BLOCK);
  const bool follows = lane >= 1 && good && (slot & (BS - 1)) != 0 && before == slot - 1;
  const unsigned runs = __ballot_sync(FULL, mine && good && !follows), rest = __ballot_sync(FULL, follows);
  if (runs == 0) return;
  // The pair's runs: item by item (K or V of a head), and in each the window's runs.
  const int it0 = chunk * a.items_per, items = min(2 * a.hkv - it0, a.items_per);
  const int rotary_dim = a.turn.rotary_dim;
  struct Cursor {
    int it;
    unsigned left;
  };
  auto advance = [&](Cursor& c) {
    c.left &= c.left - 1;
    if (c.left == 0) c.it += PAIRS, c.left = runs;
  };
  // First lane of the cursor's run and its length.
  auto run_of = [&](const Cursor& c, int& i, int& n) {
    i = __ffs(c.left) - 1;
    n = i == 31 ? 1 : 1 + __ffs(~(rest >> (i + 1))) - 1;  // rows that follow row i, and it
  };
  // Starts the run's copies; its block's scale byte if tokens of the block are kept, or -1.
  auto fetch = [&](const Cursor& c, int stage) {
    int byte = -1;
    if (c.it < items) {
      int i, n;
      run_of(c, i, n);
      const int at = __shfl_sync(FULL, slot, i), off0 = at % BS, which = it0 + c.it;
      const bool is_v = which >= a.hkv;
      const int h = is_v ? which - a.hkv : which;
      const long long blk = (long long)(at / BS) * a.hkv + h;
      fetch_run<D, FP8>(is_v ? a.v + h * a.v_hs : a.k + h * a.k_hs, is_v ? a.v_rs : a.k_rs, is_v ? 0 : rotary_dim,
                        (int)(first - 1 + i), n, off0, (is_v ? a.v_cache : a.k_cache) + blk * (BS * D * (FP8 ? 1 : 2)),
                        sm.ring[stage]);
      if (FP8 && off0 > 0) byte = (is_v ? a.v_scales : a.k_scales)[blk];
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    return byte;
  };
  Cursor now = {warp_id() / 2, runs}, next = now;
  int stage = 0, byte_now = fetch(next, 0);
  const int pairs = it0 < a.hkv ? rotary_dim / 2 : 0;
  if (pairs > 0) {
    // The rows of the runs: from a run's first row to the last that follows it.
    unsigned rows = runs;
    for (int i = 0; i < BS - 1; ++i) rows |= (rows << 1) & rest;
    const int p = threadIdx.x % rotary::MAX_PAIRS;
    if (p < pairs)
      for (int r = threadIdx.x / rotary::MAX_PAIRS; r < SPAN; r += THREADS / rotary::MAX_PAIRS)
        if (rows >> (r + 1) & 1) sm.turn[r][p] = rotary::pair_turn(a.turn, __ldg(a.positions + first + r), p);
    __syncthreads();
  }
  while (now.it < items) {
    advance(next);
    const int byte_next = fetch(next, stage ^ 1);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    int i, n;
    run_of(now, i, n);
    const bool is_v = it0 + now.it >= a.hkv;
    const int h = it0 + now.it - (is_v ? a.hkv : 0), at = __shfl_sync(FULL, slot, i);
    const long long blk = (long long)(at / BS) * a.hkv + h;
    write_run<D, FP8, INTER>(sm.ring[stage], !is_v && pairs > 0 ? sm.turn + (i - 1) : nullptr, rotary_dim, n, at % BS,
                             (is_v ? a.v_cache : a.k_cache) + blk * (BS * D * (FP8 ? 1 : 2)),
                             FP8 ? (is_v ? a.v_scales : a.k_scales) + blk : nullptr, byte_now, sm.amax[stage]);
    now = next, byte_now = byte_next;
    stage ^= 1;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
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

template <int D, bool FP8, bool INTER>
static attn_status_t launch_append_kernel(const cache::Append& a, unsigned blocks, cudaStream_t stream) {
  constexpr int SMEM = (int)sizeof(cache::AppendSmem);
  static_assert(rotary::ring_bytes<__nv_bfloat16>() <= SMEM, "the query CTAs' ring");
  auto kern = cache::append_kernel<D, FP8, INTER>;
  static DeviceOnce setup;
  const attn_status_t st = setup.run([&]() -> attn_status_t {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
  });
  if (st != ATTN_OK) return st;
  kern<<<blocks, cache::THREADS, SMEM, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, bool FP8>
static attn_status_t launch_append_d(const cache::Append& a, bool inter, unsigned blocks, cudaStream_t stream) {
  return inter ? launch_append_kernel<D, FP8, true>(a, blocks, stream)
               : launch_append_kernel<D, FP8, false>(a, blocks, stream);
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
  long long q_blocks = 0;
  // Queries that stay as and where they are need no pass.
  if (turn_q && !(p.rotary_dim == 0 && p.q == p.q_out && p.q_row_stride == p.qo_row_stride &&
                  p.q_head_stride == p.qo_head_stride)) {
    rotary::Rows& r = a.rows;
    r.q = p.q, r.q_out = p.q_out;
    r.positions = p.positions;
    r.slots = p.slot_map;
    r.tokens = p.total, r.seqlen = p.total;
    r.hq = r.heads = p.num_q_heads;
    r.q_hs = p.q_head_stride, r.q_rs = p.q_row_stride;
    r.qo_hs = p.qo_head_stride, r.qo_rs = p.qo_row_stride;
    rotary::plan_rows(r, p.head_dim, true, sms);
    q_blocks = (long long)r.tiles * r.head_groups;
    if (q_blocks > 0x3fffffffLL) return ATTN_ERR_INVALID_ARG;
  }
  // Rows per CTA: as few as keep the grid within two rounds, 16 at most. A decode
  // step has a run per row, and a CTA's runs follow one another; a chunk has one
  // run per 16 rows, and CTAs without one end at once. (512 rows of 8 heads, a
  // sequence each: 2 rows 15 us, 16 rows 30 us; a chunk of about 2000 rows: 8 rows
  // 7 us, 1 row 11 us.) A window's K heads and then its V heads are shared out, in
  // multiples of four (a run for each pair of warps), as long as the grid stays
  // within two rounds: more CTAs compute more angles (8504 rows of 32/8 heads: 4
  // heads of K or V each 39 us, 8 heads 36 us; 11567 rows of 64: 4 heads 32 us, all
  // 16 28 us), fewer leave SMs empty (1071 rows of 32/8 heads of 128: 4 heads 7.6 us,
  // 8 heads 9.9 us).
  const int most = (2 * p.num_kv_heads + cache::PAIRS - 1) / cache::PAIRS;
  a.window = 1;
  while (a.window < cache::BS && ((long long)p.total + a.window - 1) / a.window * most > 8LL * sms) a.window *= 2;
  const long long windows = ((long long)p.total + a.window - 1) / a.window;
  const long long chunks = std::max(1LL, 8LL * sms / windows);
  const int heads = 2 * p.num_kv_heads;
  const long long items = (heads + chunks - 1) / chunks;
  a.items_per = (int)std::min<long long>(heads, (items + cache::PAIRS - 1) / cache::PAIRS * cache::PAIRS);
  a.chunks = (heads + a.items_per - 1) / a.items_per;
  const long long blocks = q_blocks + windows * a.chunks;
  if (blocks > 0x7fffffffLL) return ATTN_ERR_INVALID_ARG;
  a.kv_blocks = (int)(blocks - q_blocks);
  const bool fp8 = p.kv_dtype == ATTN_DTYPE_FP8_E4M3, inter = p.interleaved != 0;
  if (p.head_dim == 128)
    return fp8 ? launch_append_d<128, true>(a, inter, (unsigned)blocks, stream)
               : launch_append_d<128, false>(a, inter, (unsigned)blocks, stream);
  return fp8 ? launch_append_d<64, true>(a, inter, (unsigned)blocks, stream)
             : launch_append_d<64, false>(a, inter, (unsigned)blocks, stream);
}

attn_status_t launch_gather(const attn_gather_params& p, int zero_to, bool flag_width, cudaStream_t stream) {
  // With flag_width even a width of 0 is launched: it flags the lengths, and the
  // dependent launch behind it must not hang on whatever ran before.
  const int blocks = std::max((p.width + cache::BS - 1) / cache::BS, flag_width ? 1 : 0);
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
