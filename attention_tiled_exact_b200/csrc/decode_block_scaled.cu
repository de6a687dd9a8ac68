// Single-token attention over the block-scaled 8-bit cache
// (attn_decode_paged_block_scaled), for sm_100a.
//
//   x_j = scale * (q . code_kj) 2^(ek_j),  O = sum_j 2^(ev_j) e^(x_j) code_vj / sum_j e^(x_j)
// with one exponent ek, ev for each 16-token block. A key's exponent multiplies
// its scores in fp32. A value's exponent goes into its weight, so the product
// with V runs on the codes themselves; because the weights enter that product
// in fp16, it keeps its own running maximum r of x_j + ev_j (in powers of two)
// beside the softmax's running maximum m of x_j: the weight 2^(x_j + ev_j - r)
// neither overflows nor vanishes while it matters, however far the exponents of
// a sequence's blocks lie apart. Both maxima are kept stale until they grow by
// 2^8.
//
// One CTA of 4 warps handles one split of one (sequence, kv head), so a block is
// read from HBM once for the group. Each warp walks every 4th block: K and V
// codes come through a per-warp ring of cp.async stages, are widened exactly to
// fp16 (cvt.rn.f16x2.e4m3x2) and go to mma.sync m16n8k16 with fp32 sums. Both
// products are computed transposed, S' = K q' and O' = V' P', with the tokens or
// the elements as the 16 rows and the group's heads as the 8 columns: half the
// products of the other order, which would pad a group of 8 to 16 rows. P'
// changes its lane layout between the two with movmatrix.
// The ring's 16-byte chunks are swizzled so that the K reads (a row per 4 lanes)
// and the V reads (a column slice per 8 lanes) are free of bank conflicts.
// The running maxima move only when some lane's score exceeds them by 2^8: one
// vote per block stands in for the shuffles of a maximum over its tokens.
// Queries enter in fp16 too: each row is first scaled by a power of two that
// brings its largest element into [2^14, 2^15), and the scores are scaled back,
// so that no bf16 query overflows (elements 2^29 below the row's largest one
// round to fp16's step there, 2^-39 of the largest).
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "block_scaled.cuh"
#include "bounds_check.cuh"
#include "internal.h"
#include "sm100_ptx.cuh"

namespace attn {
namespace bsdecode {

constexpr int BS = 16;
constexpr int WARPS = 4;
constexpr int THREADS = WARPS * 32;
constexpr int STAGES = 3;
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
  void* o;
  float* lse;
  int o_f32;
  float* part_o;    // [split][row][D], normalised
  float* part_lse;  // [split][row], natural log
  int batch, hq, hkv, group, max_blocks, num_blocks, split_tokens;
  float scale_log2;
  int32_t* error_flags;
  int planted;
};

template <int D>
struct Ring {
  uint8_t kv[WARPS][STAGES][2][BS * D];
};
template <int D, int ROWS>
struct Merge {
  float m[WARPS][ROWS], r[WARPS][ROWS], l[WARPS][ROWS];
  float o[WARPS][ROWS][D];
};
template <int D, int ROWS>
constexpr int smem_bytes() {
  return (int)(sizeof(Ring<D>) > sizeof(Merge<D, ROWS>) ? sizeof(Ring<D>) : sizeof(Merge<D, ROWS>));
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

// The cached tokens that sequence b's call sees: its length, bounded to its
// table and to the plan's splits (flagged where it was longer or negative).
__device__ __forceinline__ int bounded_len(const Args& a, int b, int max_splits, bool flag) {
  int len = __ldg(a.seq_lens + b);
  const int cap = (int)min((long long)a.max_blocks * BS, (long long)max_splits * a.split_tokens);
  if (len < 0 || len > cap) {
    if (flag && a.error_flags) atomicOr(a.error_flags, ATTN_FAULT_BAD_LENGTH);
    len = len < 0 ? 0 : cap;
  }
  return len;
}

template <typename T>
__device__ __forceinline__ T* o_row(const Args& a, int b, int head, int d) {
  return reinterpret_cast<T*>(a.o) + ((long long)b * a.hq + head) * d;
}

// HALVES: groups of 8 columns that hold query heads (group <= 8 * HALVES).
template <int D, int HALVES>
__global__ void __launch_bounds__(THREADS, HALVES == 1 ? 4 : 3) split_kernel(const Args a) {
  constexpr int ROWS = 8 * HALVES;
  constexpr int KSTEPS = D / 16, MT = D / 16;
  constexpr int COPIES = BS * D / (16 * 32);  // 16-byte copies per lane and block
  extern __shared__ __align__(128) uint8_t smem[];
  Ring<D>& ring = *reinterpret_cast<Ring<D>*>(smem);
  const int split = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z, max_splits = gridDim.x;
  const int warp = warp_id(), lane = lane_id();
  const int gq = lane >> 2, tq = lane & 3;

  const int T = a.split_tokens;
  const int L = bounded_len(a, b, max_splits, split == 0 && kvh == 0 && threadIdx.x == 0);
  const int n_splits = max(1, (L + T - 1) / T);
  if (split >= n_splits) return;
  const int t_begin = split * T, t_end = min(L, t_begin + T);
  const int blk_begin = t_begin / BS, blk_end = (t_end + BS - 1) / BS;
  const int n_mine = max(0, (blk_end - blk_begin - warp + WARPS - 1) / WARPS);
  const int32_t* table = a.block_table + (long long)b * a.max_blocks;

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

  // B fragments of q: head gq (and gq + 8), elements (D / 4) tq + 4 step + 0..3,
  // the order in which the lane reads its K row slices.
  uint32_t qb[HALVES][KSTEPS][2];
  float mul[HALVES][2];  // score of the scaled query of heads 2 tq, 2 tq + 1 (+ 8 h) -> log2 units
#pragma unroll
  for (int h = 0; h < HALVES; ++h) {
    const int g = gq + 8 * h;
    const __nv_bfloat16* src = a.q + ((long long)b * a.hq + kvh * a.group + g) * D + (D / 4) * tq;
    uint32_t w[D / 8];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      uint4 r = make_uint4(0u, 0u, 0u, 0u);
      if (g < a.group) r = __ldg(reinterpret_cast<const uint4*>(src) + i);
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
    for (int j = 0; j < 2; ++j) mul[h][j] = __shfl_sync(FULL, back, 4 * (2 * tq + j));
#pragma unroll
    for (int ks = 0; ks < KSTEPS; ++ks)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t x = w[2 * ks + j];
        qb[h][ks][j] = pack_f16x2(__uint_as_float(x << 16) * up, __uint_as_float(x & 0xffff0000u) * up);
      }
  }

  // O of element (D / 8) gq + 2 mt + i / 2, head 2 tq + i % 2 (+ 8 h) in ot[h][mt][i], in units of 2^r.
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
    const int n_valid = sc < 0 ? 0 : min(BS, t_end - (blk_begin + warp + n * WARPS) * BS);
    if (n_valid > 0) {
      const uint8_t* kblk = ring.kv[warp][n % STAGES][0];
      const uint8_t* vblk = ring.kv[warp][n % STAGES][1];
      // ---- S' = K q': tokens gq (x[h][0], x[h][1]: heads 2 tq, 2 tq + 1) and gq + 8 (x[h][2], x[h][3])
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
          x[h][j] = gq < n_valid ? x[h][j] * f : -INFINITY;
          x[h][2 + j] = gq + 8 < n_valid ? x[h][2 + j] * f : -INFINITY;
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
          const float ms = m[h][j] == -INFINITY ? 0.f : m[h][j];
          // 2^(ev + m - r): the softmax's weight to O's. Bounded, so that a weight of 0 stays 0.
          float f = r[h][j] == -INFINITY ? ev : ev + ms - r[h][j];
          f = ex2_approx(f > 126.f ? 126.f : f);
          p[j] = ex2_approx(x[h][j] - ms);
          p[2 + j] = ex2_approx(x[h][2 + j] - ms);
          l[h][j] += p[j] + p[2 + j];
          p[j] *= f;
          p[2 + j] *= f;
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
  Merge<D, ROWS>& mg = *reinterpret_cast<Merge<D, ROWS>*>(smem);
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
  const long long rows = (long long)a.batch * a.hq;
  for (int i = threadIdx.x; i < a.group * D; i += THREADS) {
    const int g = i / D, d = i % D;
    float M = -INFINITY, R = -INFINITY;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, mg.m[w][g]), R = fmaxf(R, mg.r[w][g]);
    const float Ms = M == -INFINITY ? 0.f : M, Rs = R == -INFINITY ? 0.f : R;
    float sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      sum = fmaf(ex2_approx(mg.m[w][g] - Ms), mg.l[w][g], sum);
      acc = fmaf(ex2_approx(mg.r[w][g] - Rs), mg.o[w][g][d], acc);
    }
    const bool empty = sum == 0.f;  // a NaN is not an empty row
    const float back = exp2f(0.5f * (Rs - Ms));  // applied twice: 2^(R - M) may leave fp32 where O does not
    const float out = empty ? 0.f : acc / sum * back * back;
    const float lse = empty ? -INFINITY : (Ms + log2f(sum)) * LN2;
    const int head = kvh * a.group + g;
    const long long row = (long long)b * a.hq + head;
    if (n_splits == 1) {
      if (a.o_f32)
        o_row<float>(a, b, head, D)[d] = out;
      else
        o_row<__nv_bfloat16>(a, b, head, D)[d] = __float2bfloat16_rn(out);
      if (d == 0 && a.lse) a.lse[row] = lse;
    } else if (ATTN_IN_BOUNDS(split >= 0 && split < max_splits && row >= 0 && row < rows, ATTN_SITE_DECODE_PARTIAL,
                              a.error_flags, a.planted)) {
      a.part_o[((long long)split * rows + row) * D + d] = out;
      if (d == 0) a.part_lse[(long long)split * rows + row] = lse;
    }
  }
}

// One block per row of more than one split: O = sum_s e^(lse_s - lse) O_s, the
// splits dealt out to 4 warps. A dependent launch: it is set up while the last
// splits run.
template <int D>
__global__ void __launch_bounds__(THREADS) combine_kernel(const Args a, int max_splits) {
  constexpr int PER = D / 32;
  __shared__ float s_m[WARPS], s_sum[WARPS], s_acc[WARPS][D];
  const int row = blockIdx.x, b = row / a.hq, warp = warp_id(), lane = lane_id();
  const int T = a.split_tokens, L = bounded_len(a, b, max_splits, false);
  const int n = (L + T - 1) / T;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (n <= 1) return;
  const long long rows = (long long)a.batch * a.hq;
  const float* lse = a.part_lse + row;
  float M = -INFINITY;
  for (int s = threadIdx.x; s < n; s += THREADS) M = fmaxf(M, __ldcg(lse + s * rows));
#pragma unroll
  for (int d = 16; d; d >>= 1) M = fmaxf(M, __shfl_xor_sync(FULL, M, d));
  if (lane == 0) s_m[warp] = M;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_m[w]);
  const float Ms = M == -INFINITY ? 0.f : M;
  float sum = 0.f, acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll 4
  for (int s = warp; s < n; s += WARPS) {
    const float w = ex2_approx((__ldcg(lse + s * rows) - Ms) * LOG2E);
    const float* src = a.part_o + (s * rows + row) * D + lane * PER;
    float x[PER];
    if constexpr (PER == 4) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      const float2 v = __ldcg(reinterpret_cast<const float2*>(src));
      x[0] = v.x, x[1] = v.y;
    }
    sum += w;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = fmaf(w, x[i], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_acc[warp][lane * PER + i] = acc[i];
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) sum += s_sum[w];
  const bool empty = sum == 0.f;
  if (threadIdx.x < D) {
    float out = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) out += s_acc[w][threadIdx.x];
    out = empty ? 0.f : out / sum;
    if (a.o_f32)
      reinterpret_cast<float*>(a.o)[(long long)row * D + threadIdx.x] = out;
    else
      reinterpret_cast<__nv_bfloat16*>(a.o)[(long long)row * D + threadIdx.x] = __float2bfloat16_rn(out);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[row] = empty ? -INFINITY : Ms + log2f(sum) * LN2;
}

template <int D, int HALVES>
static attn_status_t launch(const Args& a, int max_splits, cudaStream_t stream) {
  constexpr int SMEM = smem_bytes<D, 8 * HALVES>();
  auto kern = split_kernel<D, HALVES>;
  static DeviceOnce setup;
  const attn_status_t st = setup.run([&]() -> attn_status_t {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) != cudaSuccess) {
      cudaGetLastError();
      return ATTN_ERR_CUDA;
    }
    return ATTN_OK;
  });
  if (st != ATTN_OK) return st;
  kern<<<dim3(max_splits, a.hkv, a.batch), THREADS, SMEM, stream>>>(a);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (max_splits <= 1) return ATTN_OK;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.batch * a.hq);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, combine_kernel<D>, a, max_splits) != cudaSuccess) {
    cudaGetLastError();
    return ATTN_ERR_CUDA;
  }
  return ATTN_OK;
}

}  // namespace bsdecode

DecodePlan plan_decode_block_scaled(const attn_decode_params& p) {
  using namespace bsdecode;
  DecodePlan plan;
  const int cap = p.max_blocks_per_seq * BS;
  const int max_len = p.max_seq_len > 0 && p.max_seq_len < cap ? p.max_seq_len : cap;
  constexpr int UNIT = BS * WARPS;
  int T;
  if (p.num_splits > 0) {
    T = (max_len + p.num_splits - 1) / p.num_splits;
  } else {
    const long long pairs = (long long)p.batch * p.num_kv_heads;
    long long per_seq = pairs > 0 ? (32LL * device_sm_count() + pairs - 1) / pairs : 1;
    T = (int)((max_len + per_seq - 1) / per_seq);
    if (T < 512) T = 512;
  }
  T = (T + UNIT - 1) / UNIT * UNIT;
  plan.split_tokens = T;
  plan.max_splits = (max_len + T - 1) / T;
  const size_t rows = (size_t)p.batch * p.num_q_heads;
  const size_t po = (plan.max_splits * rows * p.head_dim * sizeof(float) + 255) / 256 * 256;
  const size_t pl = (plan.max_splits * rows * sizeof(float) + 255) / 256 * 256;
  plan.workspace_bytes = plan.max_splits > 1 ? po + pl : 0;
  return plan;
}

attn_status_t launch_decode_block_scaled(const attn_decode_params& p, const uint8_t* k_scales, const uint8_t* v_scales,
                                         const DecodePlan& plan, void* workspace, cudaStream_t stream) {
  using namespace bsdecode;
  Args a;
  memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(p.q);
  a.k_cache = reinterpret_cast<const uint8_t*>(p.k_cache);
  a.v_cache = reinterpret_cast<const uint8_t*>(p.v_cache);
  a.k_scales = k_scales;
  a.v_scales = v_scales;
  a.block_table = p.block_table;
  a.seq_lens = p.seq_lens;
  a.o = p.o;
  a.lse = p.lse;
  a.o_f32 = p.o_dtype == ATTN_DTYPE_F32;
  const size_t rows = (size_t)p.batch * p.num_q_heads;
  if (plan.max_splits > 1) {
    a.part_o = reinterpret_cast<float*>(workspace);
    a.part_lse = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(workspace) +
                                          (plan.max_splits * rows * p.head_dim * sizeof(float) + 255) / 256 * 256);
  }
  a.batch = p.batch;
  a.hq = p.num_q_heads;
  a.hkv = p.num_kv_heads;
  a.group = p.num_q_heads / p.num_kv_heads;
  a.max_blocks = p.max_blocks_per_seq;
  a.num_blocks = p.num_blocks;
  a.split_tokens = plan.split_tokens;
  a.scale_log2 = p.scale * LOG2E;
  a.error_flags = p.error_flags;
  a.planted = planted_bounds_site();
  const bool wide = a.group > 8;
  if (p.head_dim == 128)
    return wide ? launch<128, 2>(a, plan.max_splits, stream) : launch<128, 1>(a, plan.max_splits, stream);
  return wide ? launch<64, 2>(a, plan.max_splits, stream) : launch<64, 1>(a, plan.max_splits, stream);
}

}  // namespace attn
