// rope.hip -- rotary positions on the heads of a row.
//
// Bound by memory: each element is read and written once.  A thread holds E
// pairs of one token (two vectors of E elements), forms their E angles once
// and walks over heads with them, so that the fp64 reduction of an angle is paid
// once for many heads and no table of cosines is read.
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

// Unit u < rot / 2E of a token: pairs uE .. uE+E-1, in the vectors at elements
// uE and rot/2 + uE (halves) or 2uE and 2uE + E (interleaved); the units after
// those copy the rest of the head, two vectors each.
template <typename T, int E>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs a, int units, int heads) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int u = (int)(i % units);
  const int64_t token = i / units;
  if (token >= (int64_t)a.B * a.T) return;
  const int b = (int)(token / a.T), t = (int)(token % a.T);
  const int turned = a.rot / (2 * E);
  const int e0 = blockIdx.y * heads, e1 = min(e0 + heads, a.H);
  const char *x = a.x + b * a.xb + t * a.xr + e0 * a.xh;
  char *y = a.y + b * a.yb + t * a.yr + e0 * a.yh;
  if (u >= turned) {
    const int at = a.rot + (u - turned) * 2 * E;
    const bool two = at + E < a.hd;
    for (int e = e0; e < e1; ++e, x += a.xh, y += a.yh) {
      float p[E], q[E];
      get<T, E>(x + at * sizeof(T), p);
      if (two) get<T, E>(x + (at + E) * sizeof(T), q);
      put<T, E>(y + at * sizeof(T), p);
      if (two) put<T, E>(y + (at + E) * sizeof(T), q);
    }
    return;
  }
  const int at0 = (a.interleaved ? 2 * u * E : u * E) * (int)sizeof(T);
  const int at1 = (a.interleaved ? 2 * u * E + E : a.rot / 2 + u * E) * (int)sizeof(T);
  const int pos = position_of(a, b, t);
  float cs[E], sn[E];
#pragma unroll
  for (int k = 0; k < E; ++k) {
    turn(pos, a.freqs[u * E + k], cs[k], sn[k]);
    cs[k] *= a.factor;
    sn[k] *= a.factor * a.sign;
  }
#pragma unroll 4
  for (int e = e0; e < e1; ++e, x += a.xh, y += a.yh) {
    float p[E], q[E], f[E], g[E];
    get<T, E>(x + at0, p);
    get<T, E>(x + at1, q);
    if (a.interleaved) {
#pragma unroll
      for (int k = 0; k < E / 2; ++k) {
        turn_pair(p[2 * k], p[2 * k + 1], cs[k], sn[k], f[2 * k], f[2 * k + 1]);
        turn_pair(q[2 * k], q[2 * k + 1], cs[E / 2 + k], sn[E / 2 + k], g[2 * k], g[2 * k + 1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < E; ++k) turn_pair(p[k], q[k], cs[k], sn[k], f[k], g[k]);
    }
    put<T, E>(y + at0, f);
    put<T, E>(y + at1, g);
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

template <typename T, int E>
void launch(const RopeArgs &a, hipStream_t st) {
  const int units = a.rot / (2 * E) + (a.in_place ? 0 : ((a.hd - a.rot) / E + 1) / 2);
  const int64_t n = (int64_t)a.B * a.T * units;
  const int heads = heads_per_thread(n, a.H);
  rope_kernel<T, E><<<dim3((unsigned)((n + 255) / 256), (a.H + heads - 1) / heads), dim3(256), 0, st>>>(a, units, heads);
}

template <typename T>
void launch_single(const RopeArgs &a, hipStream_t st) {
  const int units = a.rot / 2 + (a.in_place ? 0 : a.hd - a.rot);
  const int64_t n = (int64_t)a.B * a.T * units;
  const int heads = heads_per_thread(n, a.H);
  rope_single_kernel<T><<<dim3((unsigned)((n + 255) / 256), (a.H + heads - 1) / heads), dim3(256), 0, st>>>(a, units, heads);
}

}  // namespace

int rope(const RopeArgs &a, int dtype, int vec_bytes, hipStream_t st) {
  if (dtype == DYNCONV_BF16) {
    if (vec_bytes == 16) launch<bf16, 8>(a, st);
    else if (vec_bytes == 8) launch<bf16, 4>(a, st);
    else launch_single<bf16>(a, st);
  } else {
    if (vec_bytes == 16) launch<float, 4>(a, st);
    else if (vec_bytes == 8) launch<float, 2>(a, st);
    else launch_single<float>(a, st);
  }
  return DYNCONV_OK;
}

}  // namespace dynconv
