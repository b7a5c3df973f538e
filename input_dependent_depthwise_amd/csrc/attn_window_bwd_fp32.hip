// attn_window_bwd_fp32.hip -- the backward of attention through a window for fp32 tensors.
#include "attn_bwd.h"

namespace dynconv {

int attn_window_bwd_fp32(const AttnArgs &a, hipStream_t st) { return dispatch_fp32<true>(a, st); }

}  // namespace dynconv
