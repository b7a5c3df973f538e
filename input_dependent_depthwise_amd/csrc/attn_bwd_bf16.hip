// attn_bwd_bf16.hip -- the attention backward for bf16 tensors, and its dispatch.
#include "attn_bwd.h"

namespace dynconv {

int attn_bwd_splits(int64_t B, int64_t T, int H, int G) {
  (void)B;
  (void)T;
  (void)H;
  (void)G;
  return 1;
}

int attn_bwd(const AttnArgs &a, int dtype, hipStream_t st) {
  if (dtype != DYNCONV_BF16) return attn_bwd_fp32(a, st);
  return a.hd <= 64 ? launch<bf16, 64, 64>(a, st) : launch<bf16, 128, 64>(a, st);
}

}  // namespace dynconv
