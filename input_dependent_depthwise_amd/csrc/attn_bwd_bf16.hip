// attn_bwd_bf16.hip -- the attention backward for bf16 tensors, and its dispatch.
#include <algorithm>

#include "attn_bwd.h"

namespace dynconv {

// Two blocks for a CU (of unequal work: early keys have more queries; packed documents make it
// more unequal, then four), each with enough query tiles of 64 to be worth the fp32 sums that a
// split costs to write and join.  bf16, whole backward, with 1, 2, 4 and 8 splits: 16 + 4 heads of
// 128, 4096 tokens (128 blocks) 724, 445, 332, 362 us; 12 heads of 64, 1024 tokens (96 blocks, at
// most 16 tiles each) 46, 44, 42, 47; 4 rows of 512 tokens (192, at most 8) 38, 48, 54, 69.  A tile
// takes several times as long in fp32.
int attn_bwd_splits(int64_t B, int64_t T, int H, int G, int dtype, bool packed) {
  const int64_t blocks = (T + 127) / 128 * G * B, tiles = (T + 63) / 64 * (H / G);
  const int64_t want = ((packed ? 1024 : 512) + blocks - 1) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, tiles / (dtype == DYNCONV_BF16 ? 8 : 1), 8}));
}

int attn_bwd(const AttnArgs &a, int dtype, hipStream_t st) {
  if (dtype != DYNCONV_BF16) return attn_bwd_fp32(a, st);
  return a.hd <= 64 ? launch<bf16, 64, 64>(a, st) : launch<bf16, 128, 64>(a, st);
}

}  // namespace dynconv
