// attn_bwd_fp32.hip -- the attention backward for fp32 tensors.
#include "attn_bwd.h"

namespace dynconv {

int attn_bwd_fp32(const AttnArgs &a, hipStream_t st) {
  if (a.hd <= 32) return launch<float, 32, 64>(a, st);
  return a.hd <= 64 ? launch<float, 64, 32>(a, st) : launch<float, 128, 32>(a, st);
}

}  // namespace dynconv
