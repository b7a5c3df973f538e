// attn_bwd_fp32.hip -- the attention backward for fp32 tensors.
#include "attn_bwd.h"

namespace dynconv {

int attn_bwd_fp32(const AttnArgs &a, hipStream_t st) { return dispatch_fp32<false>(a, st); }

}  // namespace dynconv
