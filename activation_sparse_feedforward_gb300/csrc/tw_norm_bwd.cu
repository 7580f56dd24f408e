// Layer norm's backward: see tw_norm.cu.
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_norm_bwd(const NormBwdArgs& a, cudaStream_t s) { return norm_bwd_any<false>(a, s); }

}  // namespace tw
