// Backward of root-mean-square norm (tw_rms_norm_bwd), with the gradient that comes along the
// residual stream and the sum over rows of the weight's gradient.
//
//   xh = x rstd;  g = dy w;  dx = rstd (g - xh sum(g xh) / d) + dres;  dw = sum_t dy xh
//
// The form of layer norm's backward (tw_norm.cu) without the mean's terms. Bound by HBM: one
// GB300, 16384 x 2048 bf16 with the residual's gradient and fp32 weights 45.3 us for 268 MB
// (0.87 of the copy rate, 6777 GB/s). Rows off 16 bytes that lie alike in all matrices: bf16 0.27
// (515 columns) to 0.58 (4001), fp32 0.65 to 0.81; others 0.2 to 0.45. 1048576
// rows of 64 columns, several to a warp, 74 us without the residual's gradient (0.80; a warp
// each 457).
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_rms_bwd(const NormBwdArgs& a, cudaStream_t s) { return norm_bwd_any<true>(a, s); }

}  // namespace tw
