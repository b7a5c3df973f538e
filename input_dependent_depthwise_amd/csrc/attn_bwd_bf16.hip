// attn_bwd_bf16.hip -- the attention backward for bf16 tensors, and its dispatch.
#include <algorithm>

#include "attn_bwd.h"

namespace dynconv {

int attn_bwd_splits(int64_t B, int64_t T, int H, int G) {
  const int64_t blocks = (T + 127) / 128 * G * B, steps = (T + 63) / 64 * (H / G);
  const int64_t want = (1024 + blocks - 1) / blocks;
  return (int)std::max<int64_t>(1, std::min<int64_t>({want, steps, 16}));
}

int attn_bwd(const AttnArgs &a, int dtype, hipStream_t st) {
  if (dtype != DYNCONV_BF16) return attn_bwd_fp32(a, st);
  return a.hd <= 64 ? launch<bf16, 64, 64>(a, st) : launch<bf16, 128, 64>(a, st);
}

}  // namespace dynconv
