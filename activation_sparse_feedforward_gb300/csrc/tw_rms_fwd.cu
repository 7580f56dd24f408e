// Root-mean-square norm over the rows of [T, d], after an optional residual add
// (tw_rms_norm_fwd).
//
//   s = x + r rounded to the type;  rstd = (sum s^2 / d + eps)^-1/2;  y = s rstd w
//
// The form of layer norm's forward (tw_norm.cu) with one sum, so one barrier, a row. Bound
// by HBM: one GB300, 16384 x 2048 bf16 with residual, its sum and fp32 weights 44.8 us for
// 268 MB (0.88 of the copy rate, 6777 GB/s). Rows off 16 bytes that lie
// alike in all matrices (a dense x, y, r of any width) run at 0.45 (515 columns bf16, where half
// of a team's lanes have nothing) to 0.9 of that rate, others at 0.35 to 0.5, bound by the
// instructions that put their vectors together. Rows of up to 256 columns go several to a warp:
// 1048576 of 64 bf16 46 us (0.86; with a warp each 147).
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_rms_fwd(const NormFwdArgs& a, cudaStream_t s) { return norm_fwd<RMS_NORM>(a, s); }

}  // namespace tw
