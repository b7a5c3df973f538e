// attn_group.h -- what the one-token attention steps do with 32 keys and values that a wave holds in
// registers (attn_decode.hip, attn_paged.hip).
//
// No operand is moved between lanes on the way: in group coordinates key
// 8u + 4t + r (u = 0..3 quarter of the wave, t = 0, 1, r = 0..3) is row 4u + r
// of score tile t, so that a lane of quarter u holds the scores of keys 8u ..
// 8u+7 of its column, which is the order of the second product's B operand; the
// value rows 8u .. 8u+7 of lane c hold elements EV c .. EV c + EV - 1 of the
// head, and the product's row c stands for element EV c + j in the j-th of EV
// products.
//
// q (times scale and log2 e) and, for bf16 caches, the probabilities enter as
// sums of two bf16 values, so their rounding does not show in o; the matrix
// cores are idle enough for twice the products.  An infinity in the cache takes part in the
// first of the two products alone (times a second part of 0 or of the other sign it would be
// a NaN): a wave whose sums come out as NaN, as they do then, goes over its keys once more and takes
// infinities and NaN out of the second products.
#pragma once

#include "attn.h"
#include "pages.h"

namespace dynconv {

namespace {

// o from the joined sums (t = 0: every score was -infinity, no key has a weight)
__device__ __forceinline__ float quotient(float s, float t) { return t == 0.f ? 0.f : s / t; }

template <typename T> struct Pair { uint4 hi, lo; };  // a B operand as hi + lo (fp32: hi alone)

// bf16 rounding of 8 values and of what it left
__device__ __forceinline__ Pair<bf16> split8(const float (&f)[8]) {
  bf16x8 h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = (bf16)f[i];
    l[i] = (bf16)(f[i] - (float)h[i]);
  }
  return {__builtin_bit_cast(uint4, h), __builtin_bit_cast(uint4, l)};
}
// the same of values that may be infinite: their first part alone
__device__ __forceinline__ Pair<bf16> split8_any(const float (&f)[8]) {
  bf16x8 h, l;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h[i] = (bf16)f[i];
    const float rest = f[i] - (float)h[i];
    l[i] = (bf16)(__builtin_fabsf(rest) < INFINITY ? rest : 0.f);
  }
  return {__builtin_bit_cast(uint4, h), __builtin_bit_cast(uint4, l)};
}

template <typename T, int DH>
struct Group {
  static constexpr int E = 16 / (int)sizeof(T), NS = DH / (4 * E), EV = DH / 16;
  static constexpr int VW = EV * (int)sizeof(T) / 4;  // dwords of a value piece: 2, 4 or 8
  uint4 k[2][NS];
  uint32_t v[8][VW];
};

// Running softmax of a wave: its 16 columns' maximum, partial sum and values.
template <typename T, int DH>
struct State {
  using G = Group<T, DH>;
  float m, l;
  f32x4 acc[G::EV];

  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int j = 0; j < G::EV; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[j][r] = 0.f;
  }
  // Whether some lane's sum or value is a NaN (uniform).
  __device__ __forceinline__ bool spoilt() const {
    bool bad = l != l;
#pragma unroll
    for (int j = 0; j < G::EV; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) bad |= acc[j][r] != acc[j][r];
    return __ballot(bad) != 0;
  }

  // GUARD: infinities and NaN of the cache enter the first products alone.
  // q[i]: step i of the columns' operand; seen(i): whether they see key i of the group.
  template <bool GUARD, typename Q, typename SEEN>
  __device__ __forceinline__ void add(const G &x, const Q &q, SEEN seen, int lane) {
    const int u = lane >> 4;
    f32x4 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][r] = 0.f;
#pragma unroll
      for (int i = 0; i < G::NS; ++i) {
        const Pair<T> c = q[i];
        if constexpr (sizeof(T) == 2) {
          s[t] = mfma16(as_bf16x8(x.k[t][i]), as_bf16x8(c.hi), s[t]);
          s[t] = mfma16(as_bf16x8(GUARD ? part_of<T, Part::KEEP>(x.k[t][i]) : x.k[t][i]), as_bf16x8(c.lo), s[t]);
        } else {
          const uint4 &a = x.k[t][i], &b = c.hi;
          s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.x), __uint_as_float(b.x), s[t], 0, 0, 0);
          s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.y), __uint_as_float(b.y), s[t], 0, 0, 0);
          s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.z), __uint_as_float(b.z), s[t], 0, 0, 0);
          s[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.w), __uint_as_float(b.w), s[t], 0, 0, 0);
        }
      }
    }
    float mx = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if (!seen(8 * u + 4 * t + r)) s[t][r] = -INFINITY;
        mx = fmaxf(mx, s[t][r]);
      }
    mx = half_max(mx);
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    if (__ballot(mx > m) != 0) {
      const float up = fmaxf(m, mx);
      const float f = up == m ? 1.f : __builtin_amdgcn_exp2f(m - up);
      m = up;
      l *= f;
#pragma unroll
      for (int j = 0; j < G::EV; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[j][r] *= f;
    }
    const float m0 = m == -INFINITY ? 0.f : m;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(s[i >> 2][i & 3] - m0);
      l += p[i];
    }
    if constexpr (sizeof(T) == 2) {
      const Pair<bf16> pb = split8(p);
#pragma unroll
      for (int j = 0; j < G::EV; ++j) {
        // element j of the 8 value rows: halves of dwords j/2 taken together
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = __builtin_amdgcn_perm(x.v[2 * i + 1][j / 2], x.v[2 * i][j / 2], (j & 1) ? 0x07060302u : 0x05040100u);
        const uint4 a = make_uint4(w[0], w[1], w[2], w[3]);
        acc[j] = mfma16(as_bf16x8(a), as_bf16x8(pb.hi), acc[j]);
        acc[j] = mfma16(as_bf16x8(GUARD ? part_of<T, Part::KEEP>(a) : a), as_bf16x8(pb.lo), acc[j]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < G::EV; ++j)
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.v[i][j]), p[i], acc[j], 0, 0, 0);
    }
  }
};

}  // namespace

}  // namespace dynconv
