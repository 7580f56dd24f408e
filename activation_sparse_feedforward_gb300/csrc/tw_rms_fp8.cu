// Root-mean-square norm with an output in 8 bits (tw_rms_norm_fwd_fp8): e4m3 with an fp32
// scale a row, or one for each 128 columns.
//
//   y = s rstd w in fp32;  scale = max(max |y| / 448, 2^-126);  q = e4m3(y / scale)
//
// The row's maximum is that of |s w|, times rstd: it needs no rstd, so it shares the barrier
// of the row's sum. A group's is taken by shuffles among the 16 or 32 lanes that hold its
// 128 columns. y itself never leaves the registers. (|s w| rounds in fp32 before rstd: a row
// where it passes 3.4e38 has scale inf, though y may be finite.) Bound by HBM: bytes in, half
// or a quarter of them out. One GB300, 8191 x 8192 bf16, a scale for each 128 columns: 37.0 us
// for 203 MB (0.81 of the copy rate, 6777 GB/s); with 800 threads an SM in place of 1024, and a
// division in place of the reciprocal, 47. Eight rows of 2048 take 6.7 us, the call's own time.
#include "tw_norm_rows.cuh"

namespace tw {

cudaError_t launch_rms_fp8(const NormFwdArgs& a, int group, cudaStream_t s) {
  return group == 0 ? norm_fwd<RMS_FP8_ROW>(a, s) : norm_fwd<RMS_FP8_GROUP>(a, s);
}

}  // namespace tw
