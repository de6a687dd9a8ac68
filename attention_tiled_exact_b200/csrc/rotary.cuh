// Rotary positions: the turn of 16 row elements by one thread, shared by the
// rotary kernel and the cache append.
//
// A row of head_dim elements is cut into head_dim / 16 units. A unit below
// rotary_dim / 16 turns the pairs 8 u .. 8 u + 7, whichever way the pairs lie
// (half layout: elements 8 u .. and rotary_dim / 2 + 8 u ..; interleaved: 16 u
// .. 16 u + 15); the units above copy 16 elements. Either way a thread moves two
// 8-element vectors per row and reuses its 8 angles for every head of a token.
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
template <bool INTER>
__device__ __forceinline__ int2 unit_offsets(int u, int rotary_dim) {
  if (!INTER && u * 16 < rotary_dim) return make_int2(8 * u, rotary_dim / 2 + 8 * u);
  return make_int2(16 * u, 16 * u + 8);
}

// magnitude * (cos, sin) of position * inv_freq for the pairs of unit u. The
// angle is reduced to half turns in fp64 (an fp32 product is off by half a
// step of the angle, 0.03 rad at position 10^6) and only the remainder, in
// [-1, 1], goes to fp32.
__device__ __forceinline__ void unit_turn(const Turn& t, int position, int u, float (&c)[8], float (&s)[8]) {
  constexpr double INV_PI = 0.31830988618379067154;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    double h = (double)position * (__ldg(t.inv_freq + 8 * u + i) * INV_PI);
    h -= 2.0 * rint(0.5 * h);
    float si, co;
    sincospif((float)h, &si, &co);
    c[i] = co * t.magnitude;
    s[i] = si * t.magnitude * t.sign;
  }
}

template <bool INTER>
__device__ __forceinline__ void turn16(float (&x)[16], const float (&c)[8], const float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : i + 8;
    const float x1 = x[a], x2 = x[b];
    x[a] = x1 * c[i] - x2 * s[i];
    x[b] = x2 * c[i] + x1 * s[i];
  }
}

// Eight row elements as they lie in memory, and as fp32.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* x) {
  Raw8<T> r;
  r.load(p);
  r.get(x);
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
  long long tokens;          // batch * seqlen
  int seqlen, hq, heads;     // heads = hq + the heads of k
  int units;                 // head_dim / 16
  int head_groups;           // threads that share a token's heads
  long long q_bs, q_hs, q_rs, k_bs, k_hs, k_rs;
  long long qo_bs, qo_hs, qo_rs, ko_bs, ko_hs, ko_rs;
};

// Thread `index` of tokens * head_groups * units: unit index % units of one
// token, for every head_groups-th head. Neighbouring lanes hold a row's units
// (16-byte vectors, whole 128-byte lines for head_dim 128), then the next
// token's. The rows of several heads are on their way while the angles are
// computed, and the next ones while these are turned; they stay packed until
// they are used, which keeps the kernel at 64 registers and 32 warps per SM.
template <typename TI, typename TO, bool INTER>
__device__ __forceinline__ void turn_rows(const Rows& r, const Turn& t, long long index) {
  const int u = (int)(index % r.units);
  const long long row = index / r.units;
  const long long token = row % r.tokens;
  const int group = (int)(row / r.tokens);
  if (group >= r.head_groups) return;
  const long long b = token / r.seqlen, pos_in_seq = token - b * r.seqlen;
  const int position = r.positions ? __ldg(r.positions + token) : (int)pos_in_seq;
  if (r.slots ? __ldg(r.slots + token) < 0 : position < 0) return;
  const bool turned = u * 16 < t.rotary_dim;
  const int2 off = unit_offsets<INTER>(u, t.rotary_dim);
  const TI* q = reinterpret_cast<const TI*>(r.q) + b * r.q_bs + pos_in_seq * r.q_rs;
  const TI* k = reinterpret_cast<const TI*>(r.k) + b * r.k_bs + pos_in_seq * r.k_rs;
  TO* qo = reinterpret_cast<TO*>(r.q_out) + b * r.qo_bs + pos_in_seq * r.qo_rs;
  TO* ko = reinterpret_cast<TO*>(r.k_out) + b * r.ko_bs + pos_in_seq * r.ko_rs;
  constexpr int BATCH = sizeof(TI) == 2 ? 2 : 1;
  Raw8<TI> raw[2][BATCH][2];
  auto fetch = [&](int h0, Raw8<TI> (&to)[BATCH][2]) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = h0 + i * r.head_groups;
      if (h < r.heads) {
        const TI* src = h < r.hq ? q + h * r.q_hs : k + (h - r.hq) * r.k_hs;
        to[i][0].load(src + off.x);
        to[i][1].load(src + off.y);
      }
    }
  };
  fetch(group, raw[0]);
  float c[8], s[8];
  if (turned) unit_turn(t, position, u, c, s);
  auto finish = [&](int h0, const Raw8<TI> (&from)[BATCH][2]) {
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int h = h0 + i * r.head_groups;
      if (h < r.heads) {
        float x[16];
        from[i][0].get(x);
        from[i][1].get(x + 8);
        if (turned) turn16<INTER>(x, c, s);
        TO* dst = h < r.hq ? qo + h * r.qo_hs : ko + (h - r.hq) * r.ko_hs;
        store8(dst + off.x, x);
        store8(dst + off.y, x + 8);
      }
    }
  };
  const int step = BATCH * r.head_groups;
  for (int h0 = group; h0 < r.heads; h0 += 2 * step) {
    fetch(h0 + step, raw[1]);
    finish(h0, raw[0]);
    fetch(h0 + 2 * step, raw[0]);
    finish(h0 + step, raw[1]);
  }
}

// Threads that share a token's heads: one thread per head while the tokens
// alone do not fill the machine, and fewer as they do, so that the angles of a
// token are computed once for several heads.
inline int head_groups_for(long long tokens, int heads, int units, int sm_count) {
  const long long want = 2048LL * sm_count;  // threads: two rounds of 1024 per SM
  long long g = tokens > 0 ? (want + tokens * units - 1) / (tokens * units) : 1;
  const long long least = (heads + 15) / 16;  // at most 16 heads a thread
  if (g < least) g = least;
  return (int)(g > heads ? heads : g);
}

}  // namespace rotary
}  // namespace attn
