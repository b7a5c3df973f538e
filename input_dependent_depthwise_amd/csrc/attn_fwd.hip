// attn_fwd.hip -- causal attention over whole sequences, forward.
#include "attn_fwd.h"

namespace dynconv {

int attn_fwd(const AttnArgs &a, int dtype, hipStream_t st) { return dispatch<false>(a, dtype, st); }

}  // namespace dynconv
