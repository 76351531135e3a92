// kernels_attn_any.hip -- linear attention, bf16: the walk's instances for rows of any
// alignment and length.
#include "attn_walk.hpp"

namespace ssd {

hipError_t launch_attn_any(const AttnArgs& A, bool full, hipStream_t st) { return launch<false>(A, full, st); }

}  // namespace ssd
