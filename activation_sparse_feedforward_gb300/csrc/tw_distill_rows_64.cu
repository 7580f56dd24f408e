// The distillation with one CTA of 64 threads a row (a translation unit of its own, so
// that the sizes compile in parallel).
#include "tw_distill_rows.cuh"

namespace tw {

cudaError_t launch_distill_rows_64(const DistillArgs& a, cudaStream_t s) { return distill_rows_any<64>(a, s); }

}  // namespace tw
