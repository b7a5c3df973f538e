// attn_bwd_bf16.hip -- the attention backward for bf16 tensors, and its dispatch.
#include <algorithm>
#include <cmath>

#include "attn_bwd.h"

namespace dynconv {

// At most two blocks for a CU (of unequal work: early keys have more queries; packed documents
// make it more unequal, then four); within that, the fewest microseconds by a tile's time against
// the time to write and join a split's fp32 sums.  bf16, whole backward, with 1, 2, 4 and 8
// splits: 16 + 4 heads of 128, 4096 tokens (128 blocks) 724, 445, 332, 362 us; 12 heads of 64,
// 1024 tokens (96 blocks, 16 tiles) 46, 44, 42, 47; 4 rows of 512 tokens (192, 8 tiles) 38, 48,
// 54, 69.
int attn_bwd_splits(const AttnArgs &a, int dtype) {
  const double blocks = (double)((a.T + 127) / 128) * a.G * a.B, tiles = (double)((a.T + 63) / 64) * (a.H / a.G);
  const double tile_us = (dtype == DYNCONV_BF16 ? 1.0 : 8.0) * (a.hd <= 64 ? 1.4 : a.hd <= 96 ? 2.1 : 2.8);
  const double split_us = 16.0 * a.B * a.T * a.G * a.hd / 4.5e6, join_us = 4.0;
  int best = 1;
  if (a.window) {
    // Through a window the blocks are alike, a window and their own keys' queries each: what counts is the rounds of the chip
    // (two blocks on a CU where their registers leave room).
    const double reach = (double)((std::min<int64_t>(a.T, (int64_t)a.window + 127) + 63) / 64) * (a.H / a.G);
    const double at_once = dtype == DYNCONV_BF16 && a.hd <= 64 ? 512 : 256;
    double least = 0;
    for (int n = 1; n <= 8 && n <= reach && n * blocks < (1 << 24); ++n) {
      const double us = std::ceil(blocks * n / at_once) * std::ceil(reach / n) * tile_us + (n > 1 ? n * split_us + join_us : 0.0);
      if (n == 1 || us < least) {
        least = us;
        best = n;
      }
    }
    return best;
  }
  double least = tiles * tile_us;
  for (int n = 2; n <= 8 && n <= tiles && (n - 1) * blocks < (a.cu ? 1024 : 512); ++n) {
    const double us = tiles / n * tile_us + n * split_us + join_us;
    if (us < least) {
      least = us;
      best = n;
    }
  }
  return best;
}

int attn_bwd(const AttnArgs &a, int dtype, hipStream_t st) {
  return dtype == DYNCONV_BF16 ? dispatch_bf16<false>(a, st) : attn_bwd_fp32(a, st);
}

}  // namespace dynconv
