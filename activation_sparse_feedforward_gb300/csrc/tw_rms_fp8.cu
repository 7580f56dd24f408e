// Root-mean-square norm with an output in 8 bits (tw_rms_norm_fwd_fp8): e4m3 with an fp32
// scale a row, or one for each 128 columns.
//
//   y = s rstd w in fp32;  scale = max(max |y| / 448, 2^-126);  q = e4m3(y / scale)
//
// The row's maximum is that of |s w|, times rstd: it needs no rstd, so it shares the barrier
// of the row's sum. A group's is taken by shuffles among the 16 or 32 lanes that hold its
// 128 columns. y itself never leaves the registers. Bound by HBM: bytes in, half or a
// quarter of them out.
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_rms_fp8(const NormFwdArgs& a, int group, cudaStream_t s) {
  return group == 0 ? norm_fwd<RMS_FP8_ROW>(a, s) : norm_fwd<RMS_FP8_GROUP>(a, s);
}

}  // namespace tw
