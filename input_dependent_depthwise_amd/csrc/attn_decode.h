// attn_decode.h -- arguments of the one-token attention step (attn_decode.hip).
#pragma once

#include "attn.h"

namespace dynconv {

struct DecodeArgs {
  AttnView q, k, v, o, kc, vc;
  int B, H, G, hd, capacity;
  int n_split;         // blocks along the cache for one sequence and key/value head
  int rot;             // 0: no rotation
  bool interleaved;
  float scale, factor;
  const double *freqs;
  const int32_t *lengths;
  float *part;         // n_split > 1: sums [B, H, n_split, hd], then maximum and sum [B, H, n_split, 2]
};
int decode_splits(int64_t B, int H, int G, int64_t capacity);
int attn_decode(const DecodeArgs &a, int dtype, hipStream_t st);

}  // namespace dynconv
