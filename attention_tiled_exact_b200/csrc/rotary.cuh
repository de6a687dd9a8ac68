// Rotary positions: the turn of 16 row elements by one thread, shared by the
// rotary kernel and the cache append.
//
// A row of head_dim elements is cut into head_dim / 16 units of two 8-element
// vectors. A unit below rotary_dim / 16 owns elements 8 u .. 8 u + 7 and
// rotary_dim / 2 + 8 u .. + 7 of the turned part: 8 pairs, whichever way they lie
// (half layout: pairs 8 u .., an element from each vector; interleaved: 4 pairs
// in each vector). The other units own the rest in the same way, so that
// neighbouring lanes always move neighbouring 16 bytes.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "sm100_ptx.cuh"

namespace attn {
namespace rotary {

struct Turn {
  const double* inv_freq;
  int rotary_dim;
  float magnitude;
  float sign;  // -1: the inverse turn
};

// Element offsets of a unit's two 8-element vectors.
template <int D>
__device__ __forceinline__ int2 unit_offsets(int u, int rotary_dim) {
  const bool in_turned = u * 16 < rotary_dim;
  const int v = in_turned ? u : u - rotary_dim / 16;
  const int first = in_turned ? 0 : rotary_dim, half = (in_turned ? rotary_dim : D - rotary_dim) / 2;
  return make_int2(first + 8 * v, first + half + 8 * v);
}

// The i-th of a turned unit's 8 pairs.
template <bool INTER>
__device__ __forceinline__ int unit_pair(int u, int i, int rotary_dim) {
  if (!INTER) return 8 * u + i;
  return 4 * u + i + (i < 4 ? 0 : rotary_dim / 4 - 4);
}

// magnitude * (cos, sin) of position * inv_freq[pair]. The angle is reduced to
// half turns in fp64 (an fp32 product is off by half a step of the angle, 0.03
// rad at position 10^6), the product as a sum of two numbers: rounded to one it is
// off by 2^-20.6 rad at 2^31 radians, with the second one by less than 2^-50 at
// any position. The remainder, in [-1, 1], goes to fp32 as a sum hi + lo
// whose second part enters to first order, cos(a + d) = cos a - d sin a: rounded
// to hi alone it would be off by up to 2^-23.3 rad, more than all that follows,
// and an 8-bit key is made from the result.
__device__ __forceinline__ float2 pair_turn(const Turn& t, int position, int pair) {
  constexpr double INV_PI = 0.31830988618379067154, INV_PI_LO = -1.9678676675182486e-17;  // their sum is 1 / pi
  constexpr float PI = 3.14159265358979f;
  const double freq = __ldg(t.inv_freq + pair), at = (double)position;
  const double f = freq * INV_PI, f_lo = fma(freq, INV_PI, -f) + freq * INV_PI_LO;
  double h = at * f;
  const double h_lo = fma(at, f, -h) + at * f_lo;
  h -= 2.0 * rint(0.5 * h);  // exact
  h += h_lo;
  const float hi = (float)h, d = PI * (float)(h - (double)hi);
  float si, co;
  sincospif(hi, &si, &co);
  return make_float2(fmaf(-d, si, co) * t.magnitude, fmaf(d, co, si) * t.magnitude * t.sign);
}

constexpr int MAX_PAIRS = 64;

// The angles of unit u out of a row of them.
template <bool INTER>
__device__ __forceinline__ void unit_turn(const float2* row, int u, int rotary_dim, float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 y = *reinterpret_cast<const float4*>(row + unit_pair<INTER>(u, 2 * j, rotary_dim));
    c[2 * j] = y.x, s[2 * j] = y.y, c[2 * j + 1] = y.z, s[2 * j + 1] = y.w;
  }
}

// magnitude * (cos, sin, -sin) of a unit's 8 pairs, two pairs per register pair
// (the packed fp32 instructions take two at a time).
struct UnitTurn {
  float2 c[4], s[4], ns[4];
  __device__ __forceinline__ void set(const float (&co)[8], const float (&si)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = make_float2(co[2 * i], co[2 * i + 1]);
      s[i] = make_float2(si[2 * i], si[2 * i + 1]);
      ns[i] = make_float2(-si[2 * i], -si[2 * i + 1]);
    }
  }
};

template <bool INTER>
__device__ __forceinline__ void turn16(float (&x)[16], const UnitTurn& t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = INTER ? 4 * i : 2 * i, b = INTER ? 4 * i + 1 : 2 * i + 8, d = INTER ? 2 : 1;
    const float2 x1 = make_float2(x[a], x[a + d]), x2 = make_float2(x[b], x[b + d]);
    const float2 y1 = __ffma2_rn(x2, t.ns[i], __fmul2_rn(x1, t.c[i]));
    const float2 y2 = __ffma2_rn(x1, t.s[i], __fmul2_rn(x2, t.c[i]));
    x[a] = y1.x, x[a + d] = y1.y, x[b] = y2.x, x[b + d] = y2.y;
  }
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float* x) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                            pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
}

// Rows of up to two tensors (q's heads, then k's) that share positions.
struct Rows {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  const int32_t* positions;  // NULL: the row's index in its sequence
  const int32_t* slots;      // not NULL: rows with a negative slot are left alone, not those with a negative position
  int tokens;                // batch * seqlen
  int seqlen, hq, heads;     // heads = hq + the heads of k
  int head_groups;           // CTAs that share a tile's heads
  int tiles;                 // token tiles of the CTAs
  int by_heads;              // which of a warp's rows lie next to one another (below)
  long long q_bs, q_hs, q_rs, k_bs, k_hs, k_rs;
  long long qo_bs, qo_hs, qo_rs, ko_bs, ko_hs, ko_rs;
};

constexpr int THREADS = 256;
constexpr int CTAS_PER_SM = 4;
constexpr int STAGES = 4;  // rows of a thread that are on their way, and the one in use
template <typename T>
constexpr int ring_bytes() {
  return STAGES * THREADS * 16 * (int)sizeof(T);
}

// A thread's own slots in shared memory: vector v of stage s of thread t at
// (s * vectors + v) * THREADS + t, so that a warp's accesses are 512 bytes in a row.
template <typename T>
struct Ring {
  static constexpr int VECS = 16 * (int)sizeof(T) / 16;  // 16-byte vectors of 16 elements
  uint4* mine;
  __device__ __forceinline__ explicit Ring(uint8_t* smem) : mine(reinterpret_cast<uint4*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ void fetch(int stage, const T* lo, const T* hi) {
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const T* src = v < VECS / 2 ? lo + v * (16 / (int)sizeof(T)) : hi + (v - VECS / 2) * (16 / (int)sizeof(T));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(mine + (stage * VECS + v) * THREADS)),
                   "l"(src)
                   : "memory");
    }
  }
  __device__ __forceinline__ void get(int stage, float* x) const {
#pragma unroll
    for (int v = 0; v < VECS; ++v) {
      const uint4 r = mine[(stage * VECS + v) * THREADS];
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[8 * v + 2 * i] = __uint_as_float(w[i] << 16);
          x[8 * v + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[4 * v + i] = __uint_as_float(w[i]);
      }
    }
  }
};

// A tile of tokens, and of their heads every head_groups-th set from `group`. A
// warp's lanes hold the units of a row (16-byte vectors, whole 128-byte lines
// for head_dim 128), and of the rows that lie next to it in memory: the next
// tokens' in [.., head, token, element], or (BY_HEADS) the next heads' in [token,
// head, element], a set of them per step, which share their angles. The rows
// come through a ring of cp.async stages in shared memory that belongs to the
// thread alone; the first ones are fetched before the position is known. What
// this costs is instructions as much as bytes: no division by a variable, the
// loop unrolled over the ring, pointers that advance by addition, packed products.
template <int D, bool BY_HEADS>
struct Warp {
  static constexpr int UNITS = D / 16, ROWS = 32 / UNITS;
  static constexpr int HEADS = BY_HEADS ? ROWS : 1, TOKENS = ROWS / HEADS;
  static constexpr int TILE = THREADS / 32 * TOKENS;
};

template <typename TI, typename TO, bool INTER, int D, bool BY_HEADS>
__device__ __forceinline__ void turn_rows(const Rows& r, const Turn& t, int tile, int group_index, uint8_t* smem) {
  using W = Warp<D, BY_HEADS>;
  const int lane = lane_id(), u = lane % W::UNITS, row = lane / W::UNITS, hsub = BY_HEADS ? row : 0;
  const long long token_at = (long long)tile * W::TILE + warp_id() * W::TOKENS + (BY_HEADS ? 0 : row);
  const bool live = token_at < r.tokens;
  const int token = live ? (int)token_at : 0;
  const int group = group_index * W::HEADS + hsub, step = r.head_groups * W::HEADS;
  const int b = token / r.seqlen, pos_in_seq = token - b * r.seqlen;
  const bool turned = u * 16 < t.rotary_dim;
  const int2 off = unit_offsets<D>(u, t.rotary_dim);
  const int second = off.y - off.x;  // from the unit's first vector to its second
  const TI* q = reinterpret_cast<const TI*>(r.q) + b * r.q_bs + pos_in_seq * r.q_rs + off.x;
  const TI* k = reinterpret_cast<const TI*>(r.k) + b * r.k_bs + pos_in_seq * r.k_rs + off.x;
  Ring<TI> ring(smem);
  // The next row to fetch: its head, counted on through q and k, and its address.
  int fetch_h = live ? group : r.heads;
  const TI* fetch_at = group < r.hq ? q + group * r.q_hs : k + (group - r.hq) * r.k_hs;
  long long fetch_step = step * (group < r.hq ? r.q_hs : r.k_hs);
  auto fetch = [&](int stage) {
    if (fetch_h < r.heads) {
      ring.fetch(stage, fetch_at, fetch_at + second);
      const bool was_q = fetch_h < r.hq;
      fetch_h += step;
      fetch_at += fetch_step;
      if (was_q && fetch_h >= r.hq) {
        fetch_at = k + (fetch_h - r.hq) * r.k_hs;
        fetch_step = step * r.k_hs;
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) fetch(i);
  const int position = !live ? -1 : r.positions ? __ldg(r.positions + token) : pos_in_seq;
  const bool skipped = !live || (r.slots ? __ldg(r.slots + token) < 0 : position < 0);
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
  if constexpr (BY_HEADS) {  // the lanes of a unit compute PER of its angles each
    constexpr int PER = 8 / W::HEADS;
    float2 mine[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i)
      mine[i] = turned && !skipped ? pair_turn(t, position, unit_pair<INTER>(u, hsub * PER + i, t.rotary_dim)) : make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = __shfl_sync(0xffffffffu, mine[i % PER].x, i / PER * W::UNITS + u);
      s[i] = __shfl_sync(0xffffffffu, mine[i % PER].y, i / PER * W::UNITS + u);
    }
  } else if (turned && !skipped) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 y = pair_turn(t, position, unit_pair<INTER>(u, i, t.rotary_dim));
      c[i] = y.x, s[i] = y.y;
    }
  }
  UnitTurn turn;
  turn.set(c, s);
  TO* ko = reinterpret_cast<TO*>(r.k_out) + b * r.ko_bs + pos_in_seq * r.ko_rs + off.x;
  TO* to = group < r.hq ? reinterpret_cast<TO*>(r.q_out) + b * r.qo_bs + pos_in_seq * r.qo_rs + group * r.qo_hs + off.x
                        : ko + (group - r.hq) * r.ko_hs;
  long long to_step = step * (group < r.hq ? r.qo_hs : r.ko_hs);
  int h = skipped ? r.heads : group;
  while (h < r.heads) {
#pragma unroll
    for (int stage = 0; stage < STAGES; ++stage) {
      if (h >= r.heads) break;
      fetch((stage + STAGES - 1) % STAGES);
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      float x[16];
      ring.get(stage, x);
      if (turned) turn16<INTER>(x, turn);
      store8(to, x);
      store8(to + second, x + 8);
      const bool was_q = h < r.hq;
      h += step;
      to += to_step;
      if (was_q && h >= r.hq) {
        to = ko + (h - r.hq) * r.ko_hs;
        to_step = step * r.ko_hs;
      }
    }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Token tiles, and the head groups for which the CTAs end soonest. The SM with
// the most CTAs decides: per CTA its steps and what it begins with (1.5 steps), and
// a tenth of a step per step for the chain of one CTA's loads, which few CTAs
// hide. Over 100 shapes of 64 to 16384 rows, 8 to 64 query heads and both layouts
// this is 0.8 % behind the best number on average. Queries and keys of 8192 tokens
// and 40 heads of 128, by tokens: 4 groups 27.9 us, 1 group 29.2 us, 2 groups (one
// round) 29.2 us, 40 groups 69 us; of 16384 tokens and 72 heads: 2 groups 95 us,
// 1 group 110 us.
inline void plan_rows(Rows& r, int head_dim, bool by_heads, int sm_count) {
  const int rows = 32 / (head_dim / 16), warp_heads = by_heads ? rows : 1;
  r.by_heads = by_heads ? 1 : 0;
  const int tile_tokens = THREADS / 32 * (rows / warp_heads);
  r.tiles = (int)(((long long)r.tokens + tile_tokens - 1) / tile_tokens);
  const int sets = (r.heads + warp_heads - 1) / warp_heads;
  long long best = 0;
  for (int g = 1; g <= sets; ++g) {
    const long long steps = (sets + g - 1) / g, ctas = (r.tiles * (long long)g + sm_count - 1) / sm_count;
    const long long cost = ctas * (10 * steps + 15) + steps;
    if (g == 1 || cost < best) best = cost, r.head_groups = g;
  }
}

}  // namespace rotary
}  // namespace attn
