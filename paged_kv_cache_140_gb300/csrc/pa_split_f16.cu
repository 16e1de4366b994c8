// The split decode kernel for f16 caches.
#include "pa_split_kernel.cuh"

namespace pa {

cudaError_t launch_split_f16(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                             cudaStream_t stream) {
    return launch_split_ct<kCacheF16>(p, head_dim, cols, m, grid, smem, stream);
}

}  // namespace pa
