// Attention of few query rows over the block-scaled 8-bit cache, for sm_100a:
// single tokens (attn_decode_paged_block_scaled) and short chunks
// (attn_prefill_paged_block_scaled where its tensor-core tiles would stand empty).
//
//   x_j = scale * (q . code_kj) 2^(ek_j),  O = sum_j 2^(ev_j) e^(x_j) code_vj / sum_j e^(x_j)
// with one exponent ek, ev for each 16-token block. A key's exponent multiplies
// its scores in fp32. A value's exponent goes into its weight, so the product
// with V runs on the codes themselves; because the weights enter that product
// in fp16, it keeps its own running maximum r of x_j + ev_j (in powers of two)
// beside the softmax's running maximum m of x_j: the weight 2^(x_j + ev_j - r)
// neither overflows nor vanishes while it matters, however far the exponents of
// a sequence's blocks lie apart (they reach over 2^230). Both maxima are kept stale
// until they grow by 2^8.
//
// A tile is up to 8 * HALVES query rows of one sequence and kv head (row i: token
// i / group, head i % group); a block is read from HBM once for the tile. The
// keys that a tile sees are dealt out evenly to the CTAs of a row of the grid,
// by the sequence's own length, so that every CTA of a sequence ends with the
// others. CLUSTER of them are a thread-block cluster and merge their results
// through distributed shared memory. Where that is the whole row of the grid,
// nothing goes through global memory and no second launch is needed (it cost
// 3 us of the 11 us of one sequence of 4097 tokens); a longer row, for few long
// sequences, leaves one partial result per cluster to a dependent launch.
//
// The 4 warps of a CTA walk every 4th block of a piece: K and V codes come
// through a per-warp ring of cp.async stages, are widened exactly to fp16
// (cvt.rn.f16x2.e4m3x2) and go to mma.sync m16n8k16 with fp32 sums. Both
// products are computed transposed, S' = K q' and O' = V' P', with the tokens or
// the elements as the 16 rows and the query rows as the 8 columns: half the
// products of the other order, which would pad 8 query rows to 16. P' changes
// its lane layout between the two with movmatrix.
// The ring's 16-byte chunks are swizzled so that the K reads (a row per 4 lanes)
// and the V reads (a column slice per 8 lanes) are free of bank conflicts.
// The running maxima move only when some lane's score exceeds them by 2^8: one
// vote per block stands in for the shuffles of a maximum over its tokens.
// Queries enter in fp16 too: each row is first scaled by a power of two that
// brings its largest element into [2^14, 2^15), and the scores are scaled back,
// so that no bf16 query overflows (elements 2^29 below the row's largest one
// round to fp16's step there, 2^-39 of the largest).
//
// Bound by HBM for full batches (64 sequences of 1K to 32K tokens, 32/8 heads of
// 128: 325-353 us, 6.2-6.7 TB/s; the other order of the products, with a maximum
// per block, took 384 us) and by its chain of length, table, pages, products and
// merge for few: one sequence of 4097 tokens 9.2 us, 8 of 4096 16-17 us (66 MB). The
// CTAs of a cluster read one another's results: sending them to the CTA that
// merges them, ahead of one barrier instead of two, took 0.7 us longer.
#include <cooperative_groups.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>

#include "block_scaled.cuh"
#include "bounds_check.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace bsdecode {

namespace cg = cooperative_groups;

constexpr int BS = 16;
constexpr int COMBINE_WARPS = 4;
constexpr int STAGES = 3;
constexpr int CLUSTER = 8;      // CTAs that merge through shared memory, at most
// Cache blocks: the least that a CTA is started for (2 per warp), the least per
// CTA of a row of several clusters, and the pieces of a grid of many rounds.
constexpr int MIN_BLOCKS = 8, LONG_BLOCKS = 32, EVEN_BLOCKS = 256;
constexpr int WIDE_CTAS = 1;  // CTAs per SM up to which they have 8 warps
constexpr float RESCALE_THRESHOLD = 8.0f;  // log2 units
constexpr float LN2 = 0.69314718055994530942f;
constexpr float LOG2E = 1.4426950408889634f;
constexpr unsigned FULL = 0xffffffffu;

struct Args {
  const __nv_bfloat16* q;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* cu_q;      // packed queries: sequence b has rows cu_q[b] .. cu_q[b + 1] - 1 of total_q
  const int32_t* q_lens;    // padded queries: rows of each sequence (NULL: max_q)
  void* o;
  float* lse;
  long long q_bs, q_hs, q_rs, o_bs, o_hs, o_rs, lse_bs, lse_hs;  // the LSE's row stride is 1
  float* part_o;     // [cluster][tile of the grid][row][D], normalised, in units of 2^shift
  float2* part_lse;  // [cluster][tile of the grid][row]: LSE (natural log) and shift
  int o_f32, causal;
  int batch, max_q, total_q, hkv, group, max_blocks, num_blocks, max_len;
  int tiles;        // row tiles per sequence and kv head (a bound)
  float scale_log2;
  int32_t* error_flags;
  int planted;
};

// CTAs of 4 warps per SM that the kernels are built for; half as many of 8.
template <int D, int HALVES>
constexpr int ctas_per_sm() {
  return HALVES == 2 ? 3 : D == 128 ? 4 : 5;
}
template <int D, int WARPS>
struct Ring {
  uint8_t kv[WARPS][STAGES][2][BS * D];
};
template <int D, int ROWS, int WARPS>
struct Merge {  // over the ring, when it is empty
  float m[WARPS][ROWS], r[WARPS][ROWS], l[WARPS][ROWS];
  float o[WARPS][ROWS][D];
  // The CTA's result: O in units of 2^r, for the other CTAs of its cluster to read.
  float cta_m[ROWS], cta_r[ROWS], cta_l[ROWS];
  float cta_o[ROWS][D];
};
template <int D, int ROWS, int WARPS>
constexpr int smem_bytes() {
  constexpr int ring = (int)sizeof(Ring<D, WARPS>), merge = (int)sizeof(Merge<D, ROWS, WARPS>);
  return ring > merge ? ring : merge;
}

// Byte offset of 16-byte chunk c of token `row` in a ring slot.
template <int D>
__device__ __forceinline__ int swz(int row, int c) {
  if constexpr (D == 128) return row * 128 + ((c ^ (row & 7)) << 4);
  const int line = row >> 1;
  return line * 128 + (((((row & 1) << 2) | c) ^ ((line & 3) << 1)) << 4);
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The 8 x 8 matrix of 16-bit elements whose row lane / 4 holds the lane's two, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Four codes as two fp16 pairs (elements 0, 1 and 2, 3).
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t r;
  memcpy(&r, &h, 4);
  return r;
}

// Tile blockIdx.z % tiles of sequence blockIdx.z / tiles, for every kv head.
struct Group {
  int b, row0, rows;  // rows of the tile (0: the sequence has no such tile)
  int seq, first;     // the sequence's batch coordinate and first row in the q, O and LSE tensors
  int len, n_q;       // cached tokens, query tokens
  int blocks;         // key blocks that the tile's last row sees
  int per_cta, used;  // of them for a CTA of the row of the grid, and CTAs that have some
};

template <int ROWS, int WARPS>
__device__ __forceinline__ Group group_of(const Args& a, int gi, int ctas) {
  Group g;
  g.b = a.tiles == 1 ? gi : gi / a.tiles;
  g.row0 = (gi - g.b * a.tiles) * ROWS;
  g.len = min(max(__ldg(a.seq_lens + g.b), 0), a.max_len);
  if (a.cu_q) {
    const int s0 = min(max(__ldg(a.cu_q + g.b), 0), a.total_q);
    g.n_q = min(max(__ldg(a.cu_q + g.b + 1), s0), a.total_q) - s0;
    g.seq = 0, g.first = s0;
  } else {
    g.seq = g.b, g.first = 0;
    g.n_q = a.q_lens ? max(__ldg(a.q_lens + g.b), 0) : a.max_q;
  }
  g.n_q = min(g.n_q, a.max_q);
  g.rows = max(0, min(ROWS, g.n_q * a.group - g.row0));
  int end = g.len;
  if (a.causal) end = min(end, g.len - g.n_q + (g.row0 + g.rows - 1) / a.group + 1);
  g.blocks = (max(end, 0) + BS - 1) / BS;
  // At least MIN_BLOCKS each, and as many for every warp.
  g.per_cta = max(MIN_BLOCKS, ((g.blocks + ctas - 1) / ctas + WARPS - 1) / WARPS * WARPS);
  g.used = max(1, (g.blocks + g.per_cta - 1) / g.per_cta);
  return g;
}

// Elements d .. d + 3 of the output of row i of a tile, and with element 0 its LSE.
__device__ __forceinline__ void store_row4(const Args& a, const Group& g, int kvh, int i, int d, float4 o, float lse) {
  const int token = g.first + (g.row0 + i) / a.group, head = kvh * a.group + (g.row0 + i) % a.group;
  const long long at = g.seq * a.o_bs + head * a.o_hs + token * a.o_rs + d;
  if (a.o_f32)
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.o) + at) = o;
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<__nv_bfloat16*>(a.o) + at) =
        make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
  if (d == 0 && a.lse) a.lse[g.seq * a.lse_bs + head * a.lse_hs + token] = lse;
}

__device__ __forceinline__ void add_scaled(float4& acc, float w, const float4& x) {
  acc.x = fmaf(w, x.x, acc.x), acc.y = fmaf(w, x.y, acc.y), acc.z = fmaf(w, x.z, acc.z), acc.w = fmaf(w, x.w, acc.w);
}

// Divides O (in units of 2^R) by a row's sum (in units of 2^M): O is then in units
// of 2^shift. Returns the row's LSE.
__device__ __forceinline__ float divide_row(float M, float R, float sum, float4& acc, float& shift) {
  const float Ms = M == -INFINITY ? 0.f : M, Rs = R == -INFINITY ? 0.f : R;
  const bool empty = sum == 0.f;  // a NaN is not an empty row
  const float inv = empty ? 0.f : 1.f / sum;
  acc.x = empty ? 0.f : acc.x * inv;
  acc.y = empty ? 0.f : acc.y * inv;
  acc.z = empty ? 0.f : acc.z * inv;
  acc.w = empty ? 0.f : acc.w * inv;
  shift = empty ? 0.f : Rs - Ms;
  return empty ? -INFINITY : (Ms + log2f(sum)) * LN2;
}

// A row's sum and O as output and LSE.
__device__ __forceinline__ float finish_row(float M, float R, float sum, float4& acc) {
  float shift;
  const float lse = divide_row(M, R, sum, acc, shift);
  const float back = exp2f(0.5f * shift);  // applied twice: 2^shift may leave fp32 where O does not
  acc.x = acc.x * back * back;
  acc.y = acc.y * back * back;
  acc.z = acc.z * back * back;
  acc.w = acc.w * back * back;
  return lse;
}

// CTAs of a cluster: the row of the grid up to CLUSTER.
__device__ __forceinline__ int cluster_size() { return min((int)gridDim.x, CLUSTER); }

template <int D, int HALVES, bool CLUSTERED, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, ctas_per_sm<D, HALVES>() * 4 / WARPS) few_rows_kernel(const Args a) {
  constexpr int ROWS = 8 * HALVES, THREADS = 32 * WARPS;
  constexpr int KSTEPS = D / 16, MT = D / 16;
  constexpr int COPIES = BS * D / (16 * 32);  // 16-byte copies per lane and block
  extern __shared__ __align__(128) uint8_t smem[];
  Ring<D, WARPS>& ring = *reinterpret_cast<Ring<D, WARPS>*>(smem);
  const int warp = warp_id(), lane = lane_id();
  const int gq = lane >> 2, tq = lane & 3;
  const int split = blockIdx.x, kvh = blockIdx.y;
  const Group grp = group_of<ROWS, WARPS>(a, blockIdx.z, gridDim.x);
  const int b = grp.b;
  if (split == 0 && kvh == 0 && threadIdx.x == 0 && a.error_flags &&
      (unsigned)__ldg(a.seq_lens + b) > (unsigned)a.max_len)
    atomicOr(a.error_flags, ATTN_FAULT_BAD_LENGTH);
  // Without rows, or the whole cluster without keys (the first one writes the rows of none).
  if (grp.rows == 0 || (CLUSTERED ? split / cluster_size() * cluster_size() : split) >= grp.used) return;
  const int blk_begin = min(grp.blocks, split * grp.per_cta), blk_end = min(grp.blocks, blk_begin + grp.per_cta);
  const int n_mine = max(0, (blk_end - blk_begin - warp + WARPS - 1) / WARPS);
  const int32_t* table = a.block_table + (long long)b * a.max_blocks;
  // Row i of the tile: its token and head, and the keys that it sees.
  auto token_of = [&](int i) { return (grp.row0 + i) / a.group; };
  auto head_of = [&](int i) { return kvh * a.group + (grp.row0 + i) % a.group; };

  // Lane i holds the table entry of this warp's block 32 k + i: one batch of 32
  // is in use for issuing copies, the next one is on its way.
  auto entry_of = [&](int batch) {
    const int n = batch * 32 + lane;
    const int blk = blk_begin + warp + n * WARPS;
    if (n >= n_mine || !ATTN_IN_BOUNDS(blk >= 0 && blk < a.max_blocks, ATTN_SITE_DECODE_TABLE, a.error_flags,
                                       a.planted))
      return -1;
    const int id = __ldg(table + blk);
    if (id >= 0 && id < a.num_blocks) return id;
    if (a.error_flags) atomicOr(a.error_flags, ATTN_FAULT_BAD_BLOCK);
    return -1;
  };
  // Its scale bytes: k | v << 8, or -1 without a block.
  auto scales_of = [&](int id) {
    if (id < 0) return -1;
    const long long at = (long long)id * a.hkv + kvh;
    return (int)__ldg(a.k_scales + at) | (int)__ldg(a.v_scales + at) << 8;
  };
  int id_issue = entry_of(0), id_next = n_mine > 32 ? entry_of(1) : -1;
  int sc_issue = scales_of(id_issue), sc_use = sc_issue;

  const uint32_t ring_at = smem_addr(&ring.kv[warp][0][0][0]);
  auto issue = [&](int n) {
    if (n < n_mine) {
      if (n > 0 && (n & 31) == 0) {
        id_issue = id_next;
        id_next = entry_of((n >> 5) + 1);
        sc_issue = scales_of(id_issue);
      }
      const int id = __shfl_sync(FULL, id_issue, n & 31);
      if (id >= 0) {
        const long long off = ((long long)id * a.hkv + kvh) * (BS * D);
        const uint32_t dst = ring_at + (n % STAGES) * (2 * BS * D);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const int c = i * 32 + lane;
          const uint32_t to = dst + swz<D>(c / (D / 16), c % (D / 16));
          cp_async16(to, a.k_cache + off + c * 16);
          cp_async16(to + BS * D, a.v_cache + off + c * 16);
        }
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) issue(s);

  // B fragments of q: row gq (and gq + 8), elements (D / 4) tq + 4 step + 0..3,
  // the order in which the lane reads its K row slices.
  uint32_t qb[HALVES][KSTEPS][2];
  float mul[HALVES][2];  // score of the scaled query of rows 2 tq, 2 tq + 1 (+ 8 h) -> log2 units
  int limit[HALVES][2];  // keys that these rows see
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    const int g = gq + 8 * h;
    const __nv_bfloat16* src =
        a.q + grp.seq * a.q_bs + (grp.first + token_of(g)) * a.q_rs + head_of(g) * a.q_hs + (D / 4) * tq;
    uint32_t w[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (g < grp.rows) r = __ldg(reinterpret_cast<const uint4*>(src) + i);
      w[4 * i] = r.x, w[4 * i + 1] = r.y, w[4 * i + 2] = r.z, w[4 * i + 3] = r.w;
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
      top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
    top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
    top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
    // 2^e scales the row; bounded so that 2^e and 2^-e are normal fp32 numbers.
    const int e = min(max(14 - ((int)(__float_as_uint(top) >> 23) - 127), -113), 113);
    const float up = top > 0.f ? bscale::pow2i(e) : 1.f;
    const float back = a.scale_log2 * (top > 0.f ? bscale::pow2i(-e) : 1.f);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mul[h][j] = __shfl_sync(FULL, back, 4 * (2 * tq + j));
      limit[h][j] = a.causal ? min(grp.len, grp.len - grp.n_q + token_of(2 * tq + j + 8 * h) + 1) : grp.len;
    }
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t x = w[2 * ks + j];
        qb[h][ks][j] = pack_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
      }
  }

  // O of element (D / 8) gq + 2 mt + i / 2, row 2 tq + i % 2 (+ 8 h) in ot[h][mt][i], in units of 2^r.
  float ot[HALVES][MT][4];
  float m[HALVES][2], r[HALVES][2], l[HALVES][2];  // l: this lane's tokens only, until the end
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) ot[h][mt][i] = 0.f;
#pragma unroll
    for (int j = 0; j < 2; ++j) m[h][j] = r[h][j] = -INFINITY, l[h][j] = 0.f;
  }

  for (int n = 0; n < n_mine; ++n) {
    issue(n + STAGES - 1);
    cp_async_wait<STAGES - 1>();
    __syncwarp();
    // The issuing side is at most STAGES - 1 blocks ahead: it enters a new batch
    // of 32 before this side does.
    if ((n & 31) == 0) sc_use = sc_issue;
    const int sc = __shfl_sync(FULL, sc_use, n & 31);
    const int tok0 = (blk_begin + warp + n * WARPS) * BS;
    const int n_valid = sc < 0 ? 0 : min(BS, grp.len - tok0);
    if (n_valid > 0) {
      const uint8_t* kblk = ring.kv[warp][n % STAGES][0];
      const uint8_t* vblk = ring.kv[warp][n % STAGES][1];
      // ---- S' = K q': tokens gq (x[h][0], x[h][1]: rows 2 tq, 2 tq + 1) and gq + 8 (x[h][2], x[h][3])
      float x[HALVES][4];
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[h][i] = 0.f;
      {
        uint32_t kw[2][D / 16];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int i = 0; i < D / 64; ++i) {
            const uint4 w = *reinterpret_cast<const uint4*>(kblk + swz<D>(8 * nt + gq, (D / 64) * tq + i));
            kw[nt][4 * i] = w.x, kw[nt][4 * i + 1] = w.y, kw[nt][4 * i + 2] = w.z, kw[nt][4 * i + 3] = w.w;
          }
#pragma unroll
        for (int ks = 0; ks < KSTEPS; ++ks) {
          uint32_t ka[4];
          widen4(kw[0][ks], ka[0], ka[2]);
          widen4(kw[1][ks], ka[1], ka[3]);
#pragma unroll
          for (int h = 0; h < HALVES; ++h) mma_f16(x[h], ka, qb[h][ks][0], qb[h][ks][1]);
        }
      }
      // ---- the two running maxima and the weights
      const float k_mul = bscale::scale_of(sc & 0xff);
      const int vb = sc >> 8;
      const float ev = vb == 255 ? NAN : (float)(vb - bscale::BIAS);
      bool over = false;
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f = mul[h][j] * k_mul;
          x[h][j] = tok0 + gq < limit[h][j] ? x[h][j] * f : -INFINITY;
          x[h][2 + j] = tok0 + gq + 8 < limit[h][j] ? x[h][2 + j] * f : -INFINITY;
          const float top = fmaxf(x[h][j], x[h][2 + j]);
          over |= top - m[h][j] > RESCALE_THRESHOLD || top + ev - r[h][j] > RESCALE_THRESHOLD;
        }
      if (__any_sync(FULL, over)) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float top = fmaxf(x[h][j], x[h][2 + j]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(FULL, top, d));
            const float m_new = fmaxf(m[h][j], top), r_new = fmaxf(r[h][j], top + ev);
            if (m_new > m[h][j]) {
              l[h][j] *= ex2_approx(m[h][j] - m_new);
              m[h][j] = m_new;
            }
            if (r_new > r[h][j]) {
              const float alpha = ex2_approx(r[h][j] - r_new);
              r[h][j] = r_new;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt) ot[h][mt][j] *= alpha, ot[h][mt][2 + j] *= alpha;
            }
          }
      }
      uint32_t pb[HALVES][2];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          // The softmax's weight for the sum, and the weight of the codes for O: an
          // exponential of its own, because 2^(ev + m - r), its ratio to the other one,
          // may be anything from 2^-250 to 2^250 (as fast as a product of the two: 8
          // sequences of 4096 tokens 16.3 us).
          const float ms = m[h][j] == -INFINITY ? 0.f : m[h][j];
          const float up = r[h][j] == -INFINITY ? ev : ev - r[h][j];
          l[h][j] += ex2_approx(x[h][j] - ms) + ex2_approx(x[h][2 + j] - ms);
          p[j] = ex2_approx(x[h][j] + up);
          p[2 + j] = ex2_approx(x[h][2 + j] + up);
        }
        // fp16 weights: half a step is 2^-11 of the weight, below the rounding of a bf16 result.
        pb[h][0] = transpose8x8(pack_f16x2(p[0], p[1]));
        pb[h][1] = transpose8x8(pack_f16x2(p[2], p[3]));
      }
      // ---- O' += V' P' on the codes: tokens 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9, elements (D / 8) gq + ..
      uint32_t vr[4][D / 32];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int tk = 2 * tq + (i & 1) + 8 * (i >> 1);
        if constexpr (D == 128) {
          const uint4 w = *reinterpret_cast<const uint4*>(vblk + swz<D>(tk, gq));
          vr[i][0] = w.x, vr[i][1] = w.y, vr[i][2] = w.z, vr[i][3] = w.w;
        } else {
          const uint2 w = *reinterpret_cast<const uint2*>(vblk + swz<D>(tk, gq >> 1) + 8 * (gq & 1));
          vr[i][0] = w.x, vr[i][1] = w.y;
        }
      }
      if (n_valid < BS) {  // a weight of 0 must not meet what lies behind the last token
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (2 * tq + (i & 1) + 8 * (i >> 1) >= n_valid)
#pragma unroll
            for (int w = 0; w < D / 32; ++w) vr[i][w] = 0u;
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;  // bytes 2, 3 or 0, 1 of both tokens, interleaved
          uint32_t va[4];
          widen4(__byte_perm(vr[0][w], vr[1][w], sel), va[0], va[1]);
          widen4(__byte_perm(vr[2][w], vr[3][w], sel), va[2], va[3]);
#pragma unroll
          for (int h = 0; h < HALVES; ++h) mma_f16(ot[h][2 * w + half], va, pb[h][0], pb[h][1]);
        }
    }
    __syncwarp();  // the slot is refilled by the next issue
  }
  cp_async_wait<0>();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- merge the warps
  __syncthreads();  // the ring becomes the merge buffer
  Merge<D, ROWS, WARPS>& mg = *reinterpret_cast<Merge<D, ROWS, WARPS>*>(smem);
#pragma unroll
  for (int h = 0; h < HALVES; ++h)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) l[h][j] += __shfl_xor_sync(FULL, l[h][j], d);
      const int g = 8 * h + 2 * tq + j;
      if (gq == 0) mg.m[warp][g] = m[h][j], mg.r[warp][g] = r[h][j], mg.l[warp][g] = l[h][j];
      float2* dst = reinterpret_cast<float2*>(&mg.o[warp][g][(D / 8) * gq]);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) dst[mt] = make_float2(ot[h][mt][j], ot[h][mt][2 + j]);
    }
  __syncthreads();
  for (int i = threadIdx.x; i < grp.rows * (D / 4); i += THREADS) {
    const int row = i / (D / 4), d = i % (D / 4) * 4;
    float M = -INFINITY, R = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, mg.m[w][row]), R = fmaxf(R, mg.r[w][row]);
    const float Ms = M == -INFINITY ? 0.f : M, Rs = R == -INFINITY ? 0.f : R;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      sum = fmaf(ex2_approx(mg.m[w][row] - Ms), mg.l[w][row], sum);
      add_scaled(acc, ex2_approx(mg.r[w][row] - Rs), *reinterpret_cast<const float4*>(&mg.o[w][row][d]));
    }
    if constexpr (CLUSTERED) {
      *reinterpret_cast<float4*>(&mg.cta_o[row][d]) = acc;
      if (d == 0) mg.cta_m[row] = M, mg.cta_r[row] = R, mg.cta_l[row] = sum;
    } else {
      const float lse = finish_row(M, R, sum, acc);
      store_row4(a, grp, kvh, row, d, acc, lse);
    }
  }
  if constexpr (CLUSTERED) {
    // ---- merge the cluster: each CTA a part of the rows' elements
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), first = split - rank;
    const int size = cluster_size(), n = min(size, grp.used - first);  // CTAs of the cluster with keys, or the first one
    const bool part = grp.used > CLUSTER;
    cluster.sync();
    for (int i = threadIdx.x * size + rank; i < grp.rows * (D / 4); i += size * THREADS) {
      const int row = i / (D / 4), d = i % (D / 4) * 4;
      float m[CLUSTER], r[CLUSTER], l[CLUSTER];
      float4 o[CLUSTER];
      float M = -INFINITY, R = -INFINITY;
#pragma unroll
      for (int c = 0; c < CLUSTER; ++c) {
        m[c] = r[c] = -INFINITY;
        l[c] = 0.f;
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < n) {
          const Merge<D, ROWS, WARPS>& of = *cluster.map_shared_rank(&mg, c);
          m[c] = of.cta_m[row], r[c] = of.cta_r[row], l[c] = of.cta_l[row];
          o[c] = *reinterpret_cast<const float4*>(&of.cta_o[row][d]);
        }
        M = fmaxf(M, m[c]), R = fmaxf(R, r[c]);
      }
      const float Ms = M == -INFINITY ? 0.f : M, Rs = R == -INFINITY ? 0.f : R;
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int c = 0; c < CLUSTER; ++c) {
        sum = fmaf(ex2_approx(m[c] - Ms), l[c], sum);
        add_scaled(acc, ex2_approx(r[c] - Rs), o[c]);
      }
      if (!part) {
        const float lse = finish_row(M, R, sum, acc);
        store_row4(a, grp, kvh, row, d, acc, lse);
      } else {
        float shift;
        const float lse = divide_row(M, R, sum, acc, shift);
        const long long at = (((long long)(split / CLUSTER) * gridDim.z + blockIdx.z) * a.hkv + kvh) * ROWS + row;
        if (ATTN_IN_BOUNDS(split / CLUSTER < (int)gridDim.x / CLUSTER && row < ROWS, ATTN_SITE_DECODE_PARTIAL,
                           a.error_flags, a.planted)) {
          *reinterpret_cast<float4*>(a.part_o + at * D + d) = acc;
          if (d == 0) a.part_lse[at] = make_float2(lse, shift);
        }
      }
    }
    cluster.sync();  // the others have read this CTA's shared memory
  }
}

// Merges the clusters' partial results of one row (blockIdx.x) of one tile and kv
// head: O = sum_s e^(lse_s - lse) 2^(shift_s) O_s, dealt out to 4 warps. The weights
// e^(lse_s) and e^(lse_s) 2^(shift_s) have their own maxima, as in the splits.
// A dependent launch: it is set up while the last splits run.
template <int D, int ROWS, int SPLIT_WARPS>
__global__ void __launch_bounds__(32 * COMBINE_WARPS) combine_kernel(const Args a, int ctas) {
  constexpr int PER = D / 32;
  __shared__ float s_m[COMBINE_WARPS], s_r[COMBINE_WARPS], s_sum[COMBINE_WARPS];
  __shared__ __align__(16) float s_acc[COMBINE_WARPS][D];
  const int row = blockIdx.x, kvh = blockIdx.y, warp = warp_id(), lane = lane_id();
  const Group grp = group_of<ROWS, SPLIT_WARPS>(a, blockIdx.z, ctas);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= grp.rows || grp.used <= CLUSTER) return;
  const int n = (grp.used + CLUSTER - 1) / CLUSTER;
  const long long first = ((long long)blockIdx.z * a.hkv + kvh) * ROWS + row, step = (long long)gridDim.z * a.hkv * ROWS;
  float M = -INFINITY, R = -INFINITY;
  for (int i = threadIdx.x; i < n; i += 32 * COMBINE_WARPS) {
    const float2 y = __ldcg(a.part_lse + first + i * step);
    M = fmaxf(M, y.x), R = fmaxf(R, fmaf(y.x, LOG2E, y.y));
  }
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, d)), R = fmaxf(R, __shfl_xor_sync(FULL, R, d));
  if (lane == 0) s_m[warp] = M, s_r[warp] = R;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < COMBINE_WARPS; ++w) M = fmaxf(M, s_m[w]), R = fmaxf(R, s_r[w]);
  const float Ms = M == -INFINITY ? 0.f : M, Rs = R == -INFINITY ? 0.f : R;
  float sum = 0.f, acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int i = warp; i < n; i += COMBINE_WARPS) {
    if (!ATTN_IN_BOUNDS(i < ctas / CLUSTER, ATTN_SITE_COMBINE, a.error_flags, a.planted)) break;
    const float2 y = __ldcg(a.part_lse + first + i * step);
    const float w = ex2_approx(fmaf(y.x, LOG2E, y.y) - Rs);
    const float* src = a.part_o + (first + i * step) * D + lane * PER;
    float x[PER];
    if constexpr (PER == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      x[0] = v.x, x[1] = v.y;
    }
    sum += ex2_approx((y.x - Ms) * LOG2E);
#pragma unroll
    for (int k = 0; k < PER; ++k) acc[k] = fmaf(w, x[k], acc[k]);
  }
#pragma unroll
  for (int k = 0; k < PER; ++k) s_acc[warp][lane * PER + k] = acc[k];
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  const int d = threadIdx.x * 4;
  if (d >= D) return;
  sum = 0.f;
  float4 out = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < COMBINE_WARPS; ++w) {
    sum += s_sum[w];
    add_scaled(out, 1.f, *reinterpret_cast<const float4*>(&s_acc[w][d]));
  }
  // The sum is relative to a power of e: in powers of two for finish_row.
  const float lse = finish_row(Ms * LOG2E, Rs, sum, out);
  store_row4(a, grp, kvh, row, d, out, lse);
}

// CTAs in a row of the grid. Enough that the grid fills the machine once, and
// not a second time in part (8 sequences of 4096 tokens, 64 tiles: 8 CTAs each
// 17 us, 4 CTAs 18 us, 16 CTAs 25 us; 32 of 2048, 256 tiles: 2 CTAs 28 us, 1 CTA
// 30 us, 4 CTAs 32 us). A grid that is larger anyway is cut into
// pieces of EVEN_BLOCKS, so that a long sequence at its end does not run alone
// (64 sequences of 1K to 32K tokens, 512 tiles: 8 CTAs 325 us, 4 CTAs 333 us,
// 1 CTA 470 us, 16 CTAs 364 us). A row of more than one cluster costs a merge through
// memory and is taken for LONG_BLOCKS per CTA (one sequence of 32768 tokens
// and one kv head: 64 CTAs 11 us, 8 CTAs 45 us).
static int ctas_per_tile(const Args& a, int num_splits, int slots) {
  const long long blocks = (a.max_len + BS - 1) / BS, tiles = (long long)a.batch * a.tiles * a.hkv;
  long long n = num_splits;
  if (n == 0) {
    n = slots / tiles;
    if (n <= CLUSTER) n = std::max(n, std::min<long long>(CLUSTER, blocks / EVEN_BLOCKS));
    n = std::min(n, std::max(blocks / LONG_BLOCKS, std::min<long long>(CLUSTER, blocks / MIN_BLOCKS)));
  } else {
    n = std::min(n, std::max(1ll, blocks / MIN_BLOCKS));
  }
  if (n > CLUSTER) return (int)(n / CLUSTER * CLUSTER);
  return n >= 8 ? 8 : n >= 4 ? 4 : n >= 2 ? 2 : 1;
}

template <int D, int HALVES, bool CLUSTERED, int WARPS>
static attn_status_t launch_grid(const Args& a, int ctas, cudaStream_t stream) {
  constexpr int ROWS = 8 * HALVES, SMEM = smem_bytes<D, ROWS, WARPS>();
  auto kern = few_rows_kernel<D, HALVES, CLUSTERED, WARPS>;
  static DeviceOnce setup;
  const attn_status_t st = setup.run([&]() -> attn_status_t {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
  });
  if (st != ATTN_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas < CLUSTER ? ctas : CLUSTER;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(ctas, a.hkv, a.batch * a.tiles);
  cfg.blockDim = dim3(32 * WARPS);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = CLUSTERED ? 1 : 0;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e == cudaSuccess && ctas > CLUSTER) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    const long long rows = (long long)a.max_q * a.group;
    cfg.gridDim = dim3(rows < ROWS ? (int)rows : ROWS, a.hkv, a.batch * a.tiles);
    cfg.blockDim = dim3(32 * COMBINE_WARPS);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, combine_kernel<D, ROWS, WARPS>, a, ctas);
  }
  if (e == cudaSuccess) return ATTN_OK;
  cudaGetLastError();
  return ATTN_ERR_CUDA;
}

// With `bytes` only the workspace's size: O, then LSE and shift of the partial results.
template <int D, int HALVES>
static attn_status_t launch(Args a, int num_splits, void* workspace, size_t* bytes, cudaStream_t stream) {
  constexpr int ROWS = 8 * HALVES;
  a.tiles = (int)(((long long)a.max_q * a.group + ROWS - 1) / ROWS);
  const int sms = device_sm_count(), ctas = ctas_per_tile(a, num_splits, sms * ctas_per_sm<D, HALVES>());
  const size_t n = ctas > CLUSTER ? (size_t)(ctas / CLUSTER) * a.batch * a.tiles * a.hkv * ROWS : 0;
  const size_t lse_at = n * D * sizeof(float);
  if (bytes) {
    *bytes = (lse_at + n * sizeof(float2) + 255) / 256 * 256;
    return ATTN_OK;
  }
  a.part_o = reinterpret_cast<float*>(workspace);
  a.part_lse = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(workspace) + lse_at);
  if (ctas == 1) return launch_grid<D, HALVES, false, 4>(a, ctas, stream);
  // A warp's blocks follow one another, 0.6 us each, so a grid that leaves SMs
  // empty deals a CTA's blocks to 8 warps: one sequence of 4097 tokens, 32/8 heads,
  // 9.1 us (4 warps 10.3), of 32768 tokens, 8/1 heads, 11.3 us (12.5). A
  // grid of several CTAs per SM has the warps already, and with 8 it takes two
  // rounds (8 sequences of 4096 tokens, 3.5 CTAs per SM: 4 warps 17 us, 8 22 us).
  const bool wide = (long long)ctas * a.batch * a.tiles * a.hkv <= WIDE_CTAS * (long long)sms;
  return wide ? launch_grid<D, HALVES, true, 8>(a, ctas, stream) : launch_grid<D, HALVES, true, 4>(a, ctas, stream);
}

// Launches, or with `bytes` only gives the workspace's size.
static attn_status_t dispatch(const Args& a, int head_dim, int num_splits, void* workspace, size_t* bytes, cudaStream_t stream) {
  const bool wide = (long long)a.max_q * a.group > 8;
  if (head_dim == 128)
    return wide ? launch<128, 2>(a, num_splits, workspace, bytes, stream) : launch<128, 1>(a, num_splits, workspace, bytes, stream);
  return wide ? launch<64, 2>(a, num_splits, workspace, bytes, stream) : launch<64, 1>(a, num_splits, workspace, bytes, stream);
}

static Args decode_args(const attn_decode_params& p, const uint8_t* k_scales, const uint8_t* v_scales) {
  Args a;
  memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(p.q);
  a.k_cache = reinterpret_cast<const uint8_t*>(p.k_cache);
  a.v_cache = reinterpret_cast<const uint8_t*>(p.v_cache);
  a.k_scales = k_scales, a.v_scales = v_scales;
  a.block_table = p.block_table;
  a.seq_lens = p.seq_lens;
  a.o = p.o, a.lse = p.lse;
  a.o_f32 = p.o_dtype == ATTN_DTYPE_F32;
  a.q_bs = a.o_bs = (long long)p.num_q_heads * p.head_dim;
  a.q_hs = a.o_hs = p.head_dim;
  a.lse_bs = p.num_q_heads, a.lse_hs = 1;
  a.batch = p.batch, a.max_q = 1;
  a.hkv = p.num_kv_heads, a.group = p.num_q_heads / p.num_kv_heads;
  a.max_blocks = p.max_blocks_per_seq, a.num_blocks = p.num_blocks;
  const int cap = p.max_blocks_per_seq * BS;
  a.max_len = p.max_seq_len > 0 && p.max_seq_len < cap ? p.max_seq_len : cap;
  a.scale_log2 = p.scale * LOG2E;
  a.error_flags = p.error_flags;
  a.planted = planted_bounds_site();
  return a;
}

// A chunk's tiles; max_q rows at most per sequence.
static Args chunk_args(const attn_prefill_params& p, const uint8_t* k_scales, const uint8_t* v_scales) {
  Args a;
  memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(p.q);
  a.k_cache = reinterpret_cast<const uint8_t*>(p.k_cache);
  a.v_cache = reinterpret_cast<const uint8_t*>(p.v_cache);
  a.k_scales = k_scales, a.v_scales = v_scales;
  a.block_table = p.block_table;
  a.seq_lens = p.seqlens_k;
  a.cu_q = p.cu_seqlens_q, a.q_lens = p.seqlens_q;
  a.o = p.o, a.lse = p.lse;
  a.o_f32 = p.o_dtype == ATTN_DTYPE_F32;
  a.q_bs = p.q_batch_stride, a.q_hs = p.q_head_stride, a.q_rs = p.q_row_stride;
  a.o_bs = p.o_batch_stride, a.o_hs = p.o_head_stride, a.o_rs = p.o_row_stride;
  a.lse_hs = p.cu_seqlens_q ? p.total_q : p.seqlen_q, a.lse_bs = (long long)p.num_q_heads * p.seqlen_q;
  a.causal = p.causal ? 1 : 0;
  a.batch = p.batch, a.max_q = p.seqlen_q, a.total_q = p.cu_seqlens_q ? p.total_q : 0;
  a.hkv = p.num_kv_heads, a.group = p.num_q_heads / p.num_kv_heads;
  a.max_blocks = p.max_blocks_per_seq, a.num_blocks = p.num_blocks;
  const int cap = p.max_blocks_per_seq * BS;
  a.max_len = p.seqlen_k < cap ? p.seqlen_k : cap;
  a.scale_log2 = p.scale * LOG2E;
  a.error_flags = p.error_flags;
  a.planted = planted_bounds_site();
  return a;
}

}  // namespace bsdecode

bool prefill_has_few_rows(const attn_prefill_params& p) {
  using namespace bsdecode;
  const long long tiles = ((long long)p.seqlen_q * (p.num_q_heads / p.num_kv_heads) + 15) / 16;
  if (p.batch * tiles > 65535 || p.num_kv_heads > 65535) return false;
  // Estimates of both sides in ns, from the bounds of the lengths: which is the
  // smaller is all that they are for, a call itself may take less than half or
  // more than twice of one (few sequences fill no machine, ragged ones are shorter
  // than their bound). Measured (chunk, context, query / kv heads, head_dim; this
  // side against the other, in us): 1, 6000, 8/1, 128: 9.5 against 27; 3 x 22, 3000,
  // 16/4, 128: 15.5 against 23; 4 x 16, 6000, 32/8, 128: 46 against 50; 4 x 100, 500,
  // 32/8, 128: 26.5 against 27; 1 x 64, 30000, 32/8, 128: 146 against 82; 6 x 64, 3000,
  // 32/8, 64: 56 against 35; 5 x 300, 3000, 16/4, 128: 138 against 49. Of 30 shapes it
  // chooses the slower side of two, 4 x 100, 400, 8/2, 128 (18 against 14) and the
  // fourth above.
  const int cap = p.max_blocks_per_seq * BS, len = p.seqlen_k < cap ? p.seqlen_k : cap;
  const double blocks = (len + BS - 1) / BS, wide = p.head_dim / 128.0;
  const double few = 4000 + p.batch * tiles * (double)p.num_kv_heads * blocks * (p.head_dim == 128 ? 1.1 : 0.45);
  const double dense = (len > 512 ? 20000 : 9000) + p.batch * (double)p.num_kv_heads * len * wide * 0.154 +
                       (double)prefill_split_items(p) * ((len + 127) / 128) * 15 * wide;
  return few < dense;
}

size_t prefill_few_rows_workspace_bytes(const attn_prefill_params& p) {
  size_t bytes = 0;
  bsdecode::dispatch(bsdecode::chunk_args(p, nullptr, nullptr), p.head_dim, 0, nullptr, &bytes, nullptr);
  return bytes;
}

attn_status_t launch_prefill_few_rows(const attn_prefill_params& p, const uint8_t* k_scales, const uint8_t* v_scales,
                                      void* workspace, cudaStream_t stream) {
  return bsdecode::dispatch(bsdecode::chunk_args(p, k_scales, v_scales), p.head_dim, 0, workspace, nullptr, stream);
}

size_t decode_block_scaled_workspace_bytes(const attn_decode_params& p) {
  size_t bytes = 0;
  if (p.batch > 0) bsdecode::dispatch(bsdecode::decode_args(p, nullptr, nullptr), p.head_dim, p.num_splits, nullptr, &bytes, nullptr);
  return bytes;
}

attn_status_t launch_decode_block_scaled(const attn_decode_params& p, const uint8_t* k_scales, const uint8_t* v_scales,
                                         void* workspace, cudaStream_t stream) {
  return bsdecode::dispatch(bsdecode::decode_args(p, k_scales, v_scales), p.head_dim, p.num_splits, workspace, nullptr, stream);
}

}  // namespace attn
