// Attention of a decode step over a paged key/value cache: the kernels of
// fa_paged_kernel.cuh for scores as they come, and the sizes that a call's plan gives.
#include "fa_paged_kernel.cuh"

namespace fa {

size_t paged_workspace(const PagedCache& c, int H, int Nq, int window, int sinks, bool fp8) {
    return paged_plan(c, H, Nq, window, sinks, fp8).bytes;
}

long long paged_max_tiles(int B, int H, int H_kv, int Nq, int max_pages, int shift) {
    const long long groups = (static_cast<long long>(H / H_kv) * Nq + 63) / 64;
    return groups * H_kv * B * ((static_cast<long long>(max_pages) << shift) / kPagedTile + kSegmentTiles);
}

cudaError_t launch_fwd_paged(const PagedArgs& a, cudaStream_t stream) { return launch_paged<false>(a, stream); }

}  // namespace fa
