// attn_window_fwd.hip -- causal attention through a sliding window, forward.
#include "attn_fwd.h"

namespace dynconv {

int attn_window_fwd(const AttnArgs &a, int dtype, hipStream_t st) { return dispatch<true>(a, dtype, st); }

}  // namespace dynconv
