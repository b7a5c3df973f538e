// attn_decode.hip -- attention of one new token per sequence over its cache.
//
// Bound by the cache: every key and value row is read once.  A block takes one
// sequence, one key/value head with up to 16 of its query heads as the columns
// of 16 x 16 matrix-core tiles, and a stretch of the cache; its 8 waves take
// groups of 32 keys in turn, straight from memory to registers, each with its own running
// maximum and sum, joined through LDS at the end.  Stretches of one sequence
// are joined by a second kernel.
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
#include <algorithm>
#include <type_traits>

#include "attn_decode.h"
#include "kernels.h"
#include "rope.h"

namespace dynconv {

namespace {

constexpr int kWaves = 8;
constexpr int kGroup = 32;                 // keys a wave takes at a time
constexpr int kSorted = 256;               // sequences that are worth being put in order of length
constexpr int kFloor = kWaves * kGroup;    // keys that are worth a block of their own

// Groups of 32 cached keys that each of n_split blocks takes, and the blocks that get any.
__device__ __forceinline__ int groups_per_split(int n, int n_split) {
  return max((((n + kGroup - 1) / kGroup) + n_split - 1) / n_split, kWaves);
}
__device__ __forceinline__ int active_splits(int n, int n_split) {
  const int ng = (n + kGroup - 1) / kGroup, per = groups_per_split(n, n_split);
  return max(1, (ng + per - 1) / per);
}

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

  // keys row0 .. row0+31 of the cache, those below n
  __device__ __forceinline__ void fetch(const char *kc, const char *vc, int64_t krow, int64_t vrow, int row0, int n,
                                        int hd, int lane) {
    const __amdgpu_buffer_rsrc_t rk = make_rsrc(kc + (int64_t)row0 * krow, kOutside);
    const __amdgpu_buffer_rsrc_t rv = make_rsrc(vc + (int64_t)row0 * vrow, kOutside);
    const int m = lane & 15, u = lane >> 4;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int row = 8 * (m >> 2) + 4 * t + (m & 3);
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const int chunk = 4 * s + u;
        const bool in = row0 + row < n && chunk * E < hd;
        k[t][s] = buf_load16(rk, in ? (uint32_t)row * (uint32_t)krow + chunk * 16u : kOutside);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = 8 * u + i;
      const uint32_t off = (uint32_t)row * (uint32_t)vrow + (uint32_t)(m * EV * (int)sizeof(T));
      const bool there = row0 + row < n;
      if constexpr (VW == 2) {
        const uint2 x = buf_load8(rv, there && m * EV < hd ? off : kOutside);
        v[i][0] = x.x;
        v[i][1] = x.y;
      } else {
#pragma unroll
        for (int w = 0; w < VW / 4; ++w) {
          const uint4 x = buf_load16(rv, there && m * EV + w * E < hd ? off + 16u * w : kOutside);
          v[i][4 * w] = x.x;
          v[i][4 * w + 1] = x.y;
          v[i][4 * w + 2] = x.z;
          v[i][4 * w + 3] = x.w;
        }
      }
    }
  }
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
  template <bool GUARD>
  __device__ __forceinline__ void add(const G &x, const Pair<T> (&q)[G::NS], int first, int n, int lane) {
    const int u = lane >> 4;
    f32x4 s[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) s[t][r] = 0.f;
#pragma unroll
      for (int i = 0; i < G::NS; ++i) {
        if constexpr (sizeof(T) == 2) {
          s[t] = mfma16(as_bf16x8(x.k[t][i]), as_bf16x8(q[i].hi), s[t]);
          s[t] = mfma16(as_bf16x8(GUARD ? part_of<T, Part::KEEP>(x.k[t][i]) : x.k[t][i]), as_bf16x8(q[i].lo), s[t]);
        } else {
          const uint4 &a = x.k[t][i], &b = q[i].hi;
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
        if (first + 8 * u + 4 * t + r >= n) s[t][r] = -INFINITY;
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

template <typename T, int DH>
__global__ __launch_bounds__(kWaves * 64, 1) void attn_decode_kernel(DecodeArgs a) {
  using GP = Group<T, DH>;
  constexpr int THREADS = kWaves * 64, LD = DH + 4;  // (rows shifted by 16 bytes against bank conflicts)
  __shared__ __align__(16) float qs[17][LD];  // 16 query heads times scale log2 e, then the new key
  __shared__ __align__(16) float sums[kWaves][16][LD];
  __shared__ float tops[kWaves][16], tots[kWaves][16];
  __shared__ int chosen;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int split = blockIdx.x;
  // Blocks start in the order of their index: the longest sequences first, so that the last
  // blocks to start are short ones (64 sequences of 0 to 8191 keys: 127 -> 117 us).
  int b = blockIdx.z;
  if (a.B > 1 && a.B <= kSorted) {
    int *len = (int *)&sums[0][0][0];
    for (int i = tid; i < a.B; i += THREADS) len[i] = a.lengths[i];
    __syncthreads();
    for (int i = tid; i < a.B; i += THREADS) {
      const int n = len[i];
      int before = 0;
      for (int j = 0; j < a.B; ++j) before += len[j] > n || (len[j] == n && j < i);
      if (before == (int)blockIdx.z) chosen = i;
    }
    __syncthreads();
    b = uniform(chosen);
  }
  const int per = a.H / a.G, blocks = (per + 15) / 16;
  const int g = blockIdx.y / blocks, cb = blockIdx.y % blocks;
  const int e0 = g * per + cb * 16, cols = min(16, per - cb * 16);
  const int n = uniform(a.lengths[b]);
  const bool idle = n < 0 || n >= a.capacity;
  if (idle) {
    if (split == 0)
      for (int i = tid; i < cols * a.hd; i += THREADS)
        *(T *)(a.o.p + b * a.o.batch + (e0 + i / a.hd) * a.o.head + (i % a.hd) * sizeof(T)) = from_f32<T>(0.f);
    return;
  }
  if (split >= active_splits(n, a.n_split)) return;
  const int gps = groups_per_split(n, a.n_split);
  const int first = split * gps * kGroup, stop = (int)min((int64_t)n, (int64_t)first + (int64_t)gps * kGroup);

  char *kc = a.kc.p + b * a.kc.batch + g * a.kc.head, *vc = a.vc.p + b * a.vc.batch + g * a.vc.head;
  GP x;
  const int row0 = first + wave * kGroup;
  if (row0 < stop) x.fetch(kc, vc, a.kc.row, a.vc.row, row0, stop, a.hd, lane);

  // q and the new key, turned, in LDS; the new key and value into the cache
  for (int i = tid; i < 17 * LD; i += THREADS) (&qs[0][0])[i] = 0.f;
  __syncthreads();
  const float c = a.scale * kLog2e;
  const int half = a.hd / 2;
  for (int i = tid; i < (cols + 1) * half; i += THREADS) {
    const int hh = i / half, p = i % half;
    const bool key = hh == cols;
    const T *src = key ? (const T *)(a.k.p + b * a.k.batch + g * a.k.head)
                       : (const T *)(a.q.p + b * a.q.batch + (e0 + hh) * a.q.head);
    int i0, i1;
    float cs = 1.f, sn = 0.f;
    if (p < a.rot / 2) {
      i0 = a.interleaved ? 2 * p : p;
      i1 = a.interleaved ? 2 * p + 1 : p + a.rot / 2;
      turn(n, a.freqs[p], cs, sn);
      cs *= a.factor;
      sn *= a.factor;
    } else {
      i0 = 2 * p;  // (rot is even: the rest starts at 2 (rot/2))
      i1 = 2 * p + 1;
    }
    const float u = to_f32(src[i0]), w = to_f32(src[i1]);
    float r0 = u, r1 = w;
    if (p < a.rot / 2) turn_pair(u, w, cs, sn, r0, r1);
    if (key) {
      const T k0 = from_f32<T>(r0), k1 = from_f32<T>(r1);
      qs[16][i0] = to_f32(k0);
      qs[16][i1] = to_f32(k1);
      if (split == 0 && cb == 0) {
        T *kr = (T *)(kc + (int64_t)n * a.kc.row), *vr = (T *)(vc + (int64_t)n * a.vc.row);
        const T *vs = (const T *)(a.v.p + b * a.v.batch + g * a.v.head);
        kr[i0] = k0;
        kr[i1] = k1;
        vr[2 * p] = vs[2 * p];
        vr[2 * p + 1] = vs[2 * p + 1];
      }
    } else {
      qs[hh][i0] = r0 * c;
      qs[hh][i1] = r1 * c;
    }
  }
  __syncthreads();
  const int m16 = lane & 15, u4 = lane >> 4;
  Pair<T> q[GP::NS];
#pragma unroll
  for (int s = 0; s < GP::NS; ++s) {
    const float *f = &qs[m16][(4 * s + u4) * GP::E];
    if constexpr (sizeof(T) == 2) {
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = f[i];
      q[s] = split8_any(w);
    } else {
      q[s].hi = *reinterpret_cast<const uint4 *>(f);
    }
  }

  State<T, DH> st;
  // the next group is on the way while this one is used, where the registers hold both (fp32 rows
  // of 512 bytes: 128 registers a group; eight waves' loads keep the memory busy there)
  constexpr bool AHEAD = sizeof(T) * DH <= 256;
  // The wave's keys, x holding its first group if it has any.
  auto pass = [&](auto guard) {
    constexpr bool GUARD = decltype(guard)::value;
    st.clear();
    for (int row = row0; row < stop; row += kWaves * kGroup) {
      const int next = row + kWaves * kGroup;
      if constexpr (AHEAD && !GUARD) {
        GP y;
        if (next < stop) y.fetch(kc, vc, a.kc.row, a.vc.row, next, stop, a.hd, lane);
        st.template add<GUARD>(x, q, row, stop, lane);
        if (next < stop) x = y;
      } else {
        st.template add<GUARD>(x, q, row, stop, lane);
        if (next < stop) x.fetch(kc, vc, a.kc.row, a.vc.row, next, stop, a.hd, lane);
      }
    }
    if (split == 0 && wave == kWaves - 1) {  // the new token: a group of one key (its wave has the fewest others)
      GP y;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int s = 0; s < GP::NS; ++s) {
          y.k[t][s] = make_uint4(0, 0, 0, 0);
          if (t == 0 && m16 == 0) {
            const float *f = &qs[16][(4 * s + u4) * GP::E];
            if constexpr (sizeof(T) == 2) {
              float w[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) w[i] = f[i];
              y.k[t][s] = split8(w).hi;
            } else {
              y.k[t][s] = *reinterpret_cast<const uint4 *>(f);
            }
          }
        }
      const char *vs = a.v.p + b * a.v.batch + g * a.v.head;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int w = 0; w < GP::VW; ++w) {
          const int at = m16 * GP::EV * (int)sizeof(T) + 4 * w;
          y.v[i][w] = i == 0 && u4 == 0 && at < a.hd * (int)sizeof(T) ? *(const uint32_t *)(vs + at) : 0u;
        }
      st.template add<GUARD>(y, q, 0, 1, lane);
    }
  };
  pass(std::false_type());
  if constexpr (sizeof(T) == 2) {
    if (__builtin_expect(st.spoilt(), 0)) {
      if (row0 < stop) x.fetch(kc, vc, a.kc.row, a.vc.row, row0, stop, a.hd, lane);
      pass(std::true_type());
    }
  }

  // join the waves
  float l = half_sum(st.l);
  l += __shfl_xor(l, 16);
  if (u4 == 0) {
    tops[wave][m16] = st.m;
    tots[wave][m16] = l;
  }
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < GP::EV; j += 4)
      *reinterpret_cast<float4 *>(&sums[wave][m16][GP::EV * (4 * u4 + r) + j]) =
          make_float4(st.acc[j][r], st.acc[j + 1][r], st.acc[j + 2][r], st.acc[j + 3][r]);
  __syncthreads();
  for (int i = tid; i < cols * a.hd; i += THREADS) {
    const int col = i / a.hd, d = i % a.hd;
    float top = tops[0][col];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) top = fmaxf(top, tops[w][col]);
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = tops[w][col];
      const float f = mw == -INFINITY ? (tots[w][col] == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(mw - top);
      s = __builtin_fmaf(f, sums[w][col][d], s);
      t = __builtin_fmaf(f, tots[w][col], t);
    }
    if (a.n_split == 1) {
      *(T *)(a.o.p + b * a.o.batch + (e0 + col) * a.o.head + d * sizeof(T)) = from_f32<T>(quotient(s, t));
    } else {
      const int64_t at = ((int64_t)b * a.H + e0 + col) * a.n_split + split;
      a.part[at * a.hd + d] = s;
      if (d == 0) {
        float *ml = a.part + (int64_t)a.B * a.H * a.n_split * a.hd + at * 2;
        ml[0] = top;
        ml[1] = t;
      }
    }
  }
}

// o from the stretches of a sequence: a block for a query head.
template <typename T>
__global__ __launch_bounds__(128) void attn_decode_join_kernel(DecodeArgs a) {
  const int e = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  const int n = a.lengths[b];
  if (n < 0 || n >= a.capacity || d >= a.hd) return;  // (idle: its zeros are written)
  const int k = active_splits(n, a.n_split);
  const int64_t at = ((int64_t)b * a.H + e) * a.n_split;
  const float *ml = a.part + (int64_t)a.B * a.H * a.n_split * a.hd + at * 2;
  float top = -INFINITY;
  for (int i = 0; i < k; ++i) top = fmaxf(top, ml[2 * i]);
  float s = 0.f, t = 0.f;
  for (int i = 0; i < k; ++i) {
    const float f = ml[2 * i] == -INFINITY ? (ml[2 * i + 1] == 0.f ? 0.f : 1.f) : __builtin_amdgcn_exp2f(ml[2 * i] - top);
    s = __builtin_fmaf(f, a.part[(at + i) * a.hd + d], s);
    t = __builtin_fmaf(f, ml[2 * i + 1], t);
  }
  *(T *)(a.o.p + b * a.o.batch + e * a.o.head + d * sizeof(T)) = from_f32<T>(quotient(s, t));
}

template <typename T>
int launch(const DecodeArgs &a, hipStream_t st) {
  const int per = a.H / a.G;
  const dim3 grid(a.n_split, a.G * ((per + 15) / 16), a.B);
  if (a.hd <= 64) attn_decode_kernel<T, 64><<<grid, dim3(kWaves * 64), 0, st>>>(a);
  else attn_decode_kernel<T, 128><<<grid, dim3(kWaves * 64), 0, st>>>(a);
  if (a.n_split > 1) attn_decode_join_kernel<T><<<dim3(a.H, a.B), dim3(128), 0, st>>>(a);
  return DYNCONV_OK;
}

}  // namespace

// Three blocks for a CU (64 sequences of 0 to 8191 keys, 4 key/value heads: 117 us, 4.8 TB/s of
// the cache; with 2 or 4: 119 and 128 us, each block costs some 3 us around its keys), but no
// block with less than one group for each of its waves, and no join for caches that a
// single block reads in a few steps.
int decode_splits(int64_t B, int H, int G, int64_t capacity) {
  const int64_t blocks = std::max<int64_t>(1, B * G * ((H / G + 15) / 16));
  if (capacity <= 4 * kFloor) return 1;
  const int64_t want = (768 + blocks - 1) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, (capacity + kFloor - 1) / kFloor, 64}));
}

int attn_decode(const DecodeArgs &a, int dtype, hipStream_t st) {
  return dtype == DYNCONV_BF16 ? launch<bf16>(a, st) : launch<float>(a, st);
}

}  // namespace dynconv
