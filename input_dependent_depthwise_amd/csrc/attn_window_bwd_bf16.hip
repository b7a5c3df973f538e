// attn_window_bwd_bf16.hip -- the backward of attention through a window for bf16 tensors, and its dispatch.
#include "attn_bwd.h"

namespace dynconv {

int attn_window_bwd(const AttnArgs &a, int dtype, hipStream_t st) {
  return dtype == DYNCONV_BF16 ? dispatch_bf16<true>(a, st) : attn_window_bwd_fp32(a, st);
}

}  // namespace dynconv
