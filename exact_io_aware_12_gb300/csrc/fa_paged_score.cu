// Attention of a decode step over a paged key/value cache whose scores are capped by a tanh, or
// biased by distance (fa_paged_kernel.cuh).
#include "fa_paged_kernel.cuh"

namespace fa {

cudaError_t launch_fwd_paged_score(const PagedArgs& a, cudaStream_t stream) { return launch_paged<true>(a, stream); }

}  // namespace fa
