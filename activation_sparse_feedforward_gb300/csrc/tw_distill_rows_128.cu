// The distillation with one CTA of 128 threads a row (a translation unit of its own, so
// that the sizes compile in parallel).
#include "tw_distill_rows.cuh"

namespace tw {

cudaError_t launch_distill_rows_128(const DistillArgs& a, cudaStream_t s) { return distill_rows_any<128>(a, s); }

}  // namespace tw
