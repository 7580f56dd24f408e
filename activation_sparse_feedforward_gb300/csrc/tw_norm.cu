// Layer norm over the rows of [T, d], forward (with the residual add before it) and
// backward (with the gradient that comes along the residual stream, and the sums over
// rows of the weight's and bias's gradients).
//
//   s = x + r rounded to the type;  mu = sum s / d;  rstd = (sum (s - mu)^2 / d + eps)^-1/2
//   xh = (s - mu) rstd;  y = xh w + b
//   g = dy w;  c1 = sum g / d;  c2 = sum g xh / d;  dx = rstd (g - c1 - xh c2) + dres
//   dw = sum_t dy xh;  db = sum_t dy
//
// A row is read once and stays in the registers of its team of warps, so the variance
// is the two-sweep one (no cancellation of large means) at no extra traffic. All
// statistics and sums are fp32; y, dx and s are rounded once.
//
// Both directions are bound by HBM: CTAs stay for many rows, a team keeps the rows it
// will take next on their way through its own places of a ring in shared memory (each
// thread copies and reads back its own 16 bytes, so the ring needs no barrier), and
// weights and column sums stay in registers. Rows off 16 bytes go through the ring as the
// aligned vectors that they lie in, and are put together from two of them (those instructions,
// and in the forward's 80 registers spills of 8 to 144 bytes a thread, bound them: 32672 x 1027
// fp16 forward 55 us, 0.36 of the copy rate). Rows too wide for a ring are loaded straight
// into registers, of which 1024 threads have too few (spills of 8 to 392 bytes a thread in
// the forward, 536 to 656 in the backward).
//
// Measured on one GB300 against the copy rate (6681 GB/s), bf16 with fp32 weights: forward
// 16384 x 2048 with residual and saved statistics 45.4 us (0.89); backward 16384 x 2048
// with the residual's gradient and both sums 46.8 us (0.86), fp32 8191 x 8192 without the
// residual's 130 us (0.92). One read of each input: no second sweep from HBM.
//
// The kernels are in tw_norm_rows.cuh, the backward's launches in tw_norm_bwd.cu.
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_norm_fwd(const NormFwdArgs& a, cudaStream_t s) { return norm_fwd<LAYER_NORM>(a, s); }

}  // namespace tw
