// rope.h -- the turn of a rotary pair (rope.hip, attn_decode.hip).
#pragma once

#include "common.h"

namespace dynconv {

constexpr double kInvTwoPi = 0.15915494309189533577;

// cos and sin of the angle position * freq (radians).  The angle is taken to
// turns and reduced in fp64 (to a quarter turn, then [-pi/4, pi/4]); sine and cosine
// there are their Taylor polynomials of degree 11 and 12, whose remainders are
// below 2^-33.
__device__ __forceinline__ void turn(int position, double freq, float &cs, float &sn) {
  const double t = (double)position * (freq * kInvTwoPi);
  const double q = __builtin_rint(4.0 * t);  // quarter turns
  const float a = (float)((4.0 * t - q) * 1.57079632679489661923);
  const int k = (int)(q - 4.0 * __builtin_floor(0.25 * q));  // q mod 4
  const float x = a * a;
  float s = -2.5052108e-8f, c = 2.0876757e-9f;
  s = __builtin_fmaf(s, x, 2.7557319e-6f);
  s = __builtin_fmaf(s, x, -1.9841270e-4f);
  s = __builtin_fmaf(s, x, 8.3333333e-3f);
  s = __builtin_fmaf(s, x, -1.6666667e-1f);
  s = __builtin_fmaf(s * x, a, a);
  c = __builtin_fmaf(c, x, -2.7557319e-7f);
  c = __builtin_fmaf(c, x, 2.4801587e-5f);
  c = __builtin_fmaf(c, x, -1.3888889e-3f);
  c = __builtin_fmaf(c, x, 4.1666667e-2f);
  c = __builtin_fmaf(c, x, -0.5f);
  c = __builtin_fmaf(c, x, 1.0f);
  const float cq = (k & 1) ? s : c, sq = (k & 1) ? c : s;
  cs = (k == 1 || k == 2) ? -cq : cq;
  sn = (k >= 2) ? -sq : sq;
}

// The turned pair, the same bits wherever a pair is turned.
__device__ __forceinline__ void turn_pair(float a, float b, float cs, float sn, float &x, float &y) {
  x = __builtin_fmaf(-b, sn, a * cs);
  y = __builtin_fmaf(a, sn, b * cs);
}

struct RopeArgs {
  const char *x;
  char *y;
  int64_t xb, xr, xh, yb, yr, yh;  // batch, row and head strides in bytes
  int B, T, H, hd, rot;
  bool interleaved, in_place;
  float factor, sign;  // sign: -1 turns back
  const double *freqs;
  const int32_t *pos;  // [B, T] or NULL
  const int32_t *cu;
  int n_seqs;
};
// vec: elements that a 16- or 8-byte access of both views may take (0: single elements)
int rope(const RopeArgs &a, int dtype, int vec_bytes, hipStream_t st);

}  // namespace dynconv
