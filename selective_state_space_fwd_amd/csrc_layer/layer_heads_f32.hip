// layer_heads_f32.hip -- the forward scan over heads for float32 I/O.
#include "layer_heads_fwd.h"

namespace ssm {

hipError_t heads_fwd_f32(const HeadsArgs &a, hipStream_t s) { return heads_fwd_io<F32>(a, s); }

}  // namespace ssm
