// layer_heads_bf16.hip -- the forward scan over heads for bfloat16 I/O.
#include "layer_heads_fwd.h"

namespace ssm {

hipError_t heads_fwd_bf16(const HeadsArgs &a, hipStream_t s) { return heads_fwd_io<BF16>(a, s); }

}  // namespace ssm
