// Backward of root-mean-square norm (tw_rms_norm_bwd), with the gradient that comes along the
// residual stream and the sum over rows of the weight's gradient.
//
//   xh = x rstd;  g = dy w;  dx = rstd (g - xh sum(g xh) / d) + dres;  dw = sum_t dy xh
//
// The form of layer norm's backward (tw_norm.cu) without the mean's terms. Bound by HBM.
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_rms_bwd(const NormBwdArgs& a, cudaStream_t s) { return norm_bwd_any<true>(a, s); }

}  // namespace tw
