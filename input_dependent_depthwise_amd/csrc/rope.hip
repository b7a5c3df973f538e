// rope.hip -- rotary positions on the heads of a row.
//
// Bound by memory: each element is read and written once.  A block takes a few
// tokens whole: its threads form the cosines and sines of each (token, pair) once, in LDS,
// while their first vectors are on the way, and then walk over the heads, neighbouring lanes on
// neighbouring vectors of the row (16384 tokens of 20 heads of 128, bf16, half of each turned: 34 to 38 us
// with the card, 4.5 to 4.9 TB/s where a large copy has 5.2; fp32, whole heads: 63 us, 5.3 TB/s of which the
// 256 MB cache serves a part; bf16 with a thread for a pair and token that walks over the heads: 41 us).  No table is
// read from memory, and the fp64 reduction of an angle is paid once for all heads.
#include <algorithm>

#include "attn.h"
#include "kernels.h"
#include "rope.h"

namespace dynconv {

namespace {

// Position of token t of batch row b: given, or its index in its document (of
// the last offset at or before it) or row.
__device__ __forceinline__ int position_of(const RopeArgs &a, int b, int t) {
  if (a.pos) return a.pos[(int64_t)b * a.T + t];
  if (!a.cu) return t;
  int lo = 0, hi = a.n_seqs + 1;  // the first j with cu[j] > t, or n_seqs + 1
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (a.cu[mid] > t) hi = mid;
    else lo = mid + 1;
  }
  return lo > 0 ? t - a.cu[lo - 1] : t;
}

template <int BYTES> struct Raw;
template <> struct Raw<16> { typedef uint4 type; };
template <> struct Raw<8> { typedef uint2 type; };
template <> struct Raw<4> { typedef uint32_t type; };

template <typename T, int E>
__device__ __forceinline__ void get(const char *p, float (&f)[E]) {
  typedef typename Raw<E * sizeof(T)>::type R;
  const R r = *reinterpret_cast<const R *>(p);
  T v[E];
  __builtin_memcpy(v, &r, sizeof(r));
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = to_f32(v[i]);
}
template <typename T, int E>
__device__ __forceinline__ void put(char *p, const float (&f)[E]) {
  typedef typename Raw<E * sizeof(T)>::type R;
  T v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = from_f32<T>(f[i]);
  R r;
  __builtin_memcpy(&r, v, sizeof(r));
  *reinterpret_cast<R *>(p) = r;
}

// Unit u < rot / 2E of a head: pairs uE .. uE+E-1, in the vectors at elements
// uE and rot/2 + uE (halves) or 2uE and 2uE + E (interleaved); the units after
// those copy the rest of the head, two vectors each.
constexpr int kPairs = 1024;  // cosines and sines a block holds

template <typename T, int E>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int units, int tokens) {
  __shared__ float2 cs[kPairs];
  const int tid = threadIdx.x, pairs = a.rot / 2, turned = a.rot / (2 * E);
  const int64_t token0 = (int64_t)blockIdx.x * tokens, all = (int64_t)a.B * a.T;
  const int nt = (int)min((int64_t)tokens, all - token0), per = a.H * units, n = nt * per;
  for (int i0 = 0; i0 < n; i0 += 256) {
    const int i = i0 + tid;
    float p[E], q[E];
    char *y = nullptr;
    int tok = 0, u = 0, second = 0;  // second: bytes from the first vector to the other, 0: none
    if (i < n) {
      tok = i / per;
      const int e = (i - tok * per) / units;
      u = i - tok * per - e * units;
      const int64_t token = token0 + tok;
      const int b = (int)(token / a.T), t = (int)(token - (int64_t)b * a.T);
      int first;
      if (u < turned) {
        first = a.interleaved ? 2 * u * E : u * E;
        second = (a.interleaved ? E : pairs) * (int)sizeof(T);
      } else {
        first = a.rot + (u - turned) * 2 * E;
        second = first + E < a.hd ? E * (int)sizeof(T) : 0;
      }
      y = a.y + b * a.yb + t * a.yr + e * a.yh + first * (int)sizeof(T);
      const char *x = a.x + b * a.xb + t * a.xr + e * a.xh + first * (int)sizeof(T);
      get<T, E>(x, p);
      get<T, E>(x + second, q);
    }
    if (i0 == 0) {
      for (int j = tid; j < nt * pairs; j += 256) {
        const int64_t token = token0 + j / pairs;
        const int b = (int)(token / a.T), t = (int)(token - (int64_t)b * a.T);
        float c, s;
        turn(position_of(a, b, t), a.freqs[j % pairs], c, s);
        cs[j] = make_float2(c * a.factor, s * (a.factor * a.sign));
      }
      __syncthreads();
    }
    if (i >= n) continue;
    if (u < turned) {
      const float2 *w = cs + tok * pairs + u * E;
      float f[E], g[E];
      if (a.interleaved) {
#pragma unroll
        for (int m = 0; m < E / 2; ++m) {
          turn_pair(p[2 * m], p[2 * m + 1], w[m].x, w[m].y, f[2 * m], f[2 * m + 1]);
          turn_pair(q[2 * m], q[2 * m + 1], w[E / 2 + m].x, w[E / 2 + m].y, g[2 * m], g[2 * m + 1]);
        }
      } else {
#pragma unroll
        for (int m = 0; m < E; ++m) turn_pair(p[m], q[m], w[m].x, w[m].y, f[m], g[m]);
      }
      put<T, E>(y, f);
      put<T, E>(y + second, g);
    } else {
      put<T, E>(y, p);
      if (second) put<T, E>(y + second, q);
    }
  }
}

// Any rot_dim, head_dim, strides: a thread per pair (or per single element of the rest).
template <typename T>
__global__ __launch_bounds__(256) void rope_single_kernel(RopeArgs a, int units, int heads) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(i % units);
  const int64_t token = i / units;
  if (token >= (int64_t)a.B * a.T) return;
  const int b = (int)(token / a.T), t = (int)(token % a.T);
  const int e0 = blockIdx.y * heads, e1 = min(e0 + heads, a.H);
  const char *x = a.x + b * a.xb + t * a.xr + e0 * a.xh;
  char *y = a.y + b * a.yb + t * a.yr + e0 * a.yh;
  if (u >= a.rot / 2) {
    const int at = a.rot / 2 + u;
    for (int e = e0; e < e1; ++e, x += a.xh, y += a.yh) ((T *)y)[at] = ((const T *)x)[at];
    return;
  }
  const int i0 = a.interleaved ? 2 * u : u, i1 = a.interleaved ? 2 * u + 1 : u + a.rot / 2;
  float cs, sn;
  turn(position_of(a, b, t), a.freqs[u], cs, sn);
  cs *= a.factor;
  sn *= a.factor * a.sign;
  for (int e = e0; e < e1; ++e, x += a.xh, y += a.yh) {
    const float p = to_f32(((const T *)x)[i0]), q = to_f32(((const T *)x)[i1]);
    float f, g;
    turn_pair(p, q, cs, sn, f, g);
    ((T *)y)[i0] = from_f32<T>(f);
    ((T *)y)[i1] = from_f32<T>(g);
  }
}

// Heads of one thread: all of them, or fewer while there are not enough threads to fill the chip.
int heads_per_thread(int64_t threads, int H) {
  int n = H;
  while (n > 1 && threads * ((H + n - 1) / n) < (int64_t)256 * 1024) n = (n + 1) / 2;
  return n;
}

constexpr int64_t kMaxBlocks = (1 << 24) - 1;  // of 256 threads, below 2^32 threads in all

template <typename T, int E>
int launch(const RopeArgs &a, hipStream_t st) {
  const int units = a.rot / (2 * E) + (a.in_place ? 0 : ((a.hd - a.rot) / E + 1) / 2);
  // tokens of a block: two units for a thread, no more than leave a block for every CU or fit
  // the block's pairs (four units, or two loaded before either is turned: 34.3 -> 36.3 us
  // for 16384 tokens of 20 heads of 128, half of each turned)
  const int64_t all = (int64_t)a.B * a.T;
  const int64_t tokens = std::max<int64_t>(1, std::min<int64_t>({(512 + a.H * units - 1) / (a.H * units), all / 256,
                                                                 kPairs / (a.rot / 2)}));
  const int64_t blocks = (all + tokens - 1) / tokens;
  if (blocks > kMaxBlocks) return DYNCONV_E_LIMIT;
  rope_kernel<T, E><<<dim3((unsigned)blocks), dim3(256), 0, st>>>(a, units, (int)tokens);
  return DYNCONV_OK;
}

template <typename T>
int launch_single(const RopeArgs &a, hipStream_t st) {
  const int units = a.rot / 2 + (a.in_place ? 0 : a.hd - a.rot);
  const int64_t n = (int64_t)a.B * a.T * units;
  const int heads = heads_per_thread(n, a.H);
  if ((n + 255) / 256 > kMaxBlocks) return DYNCONV_E_LIMIT;
  rope_single_kernel<T><<<dim3((unsigned)((n + 255) / 256), (a.H + heads - 1) / heads), dim3(256), 0, st>>>(a, units, heads);
  return DYNCONV_OK;
}

}  // namespace

int rope(const RopeArgs &a, int dtype, int vec_bytes, hipStream_t st) {
  if (a.rot > 2 * kPairs) vec_bytes = 0;
  if (dtype == DYNCONV_BF16) {
    if (vec_bytes == 16) return launch<bf16, 8>(a, st);
    return vec_bytes == 8 ? launch<bf16, 4>(a, st) : launch_single<bf16>(a, st);
  }
  if (vec_bytes == 16) return launch<float, 4>(a, st);
  return vec_bytes == 8 ? launch<float, 2>(a, st) : launch_single<float>(a, st);
}

}  // namespace dynconv
