// The split decode kernel for e4m3 caches.
#include "pa_split_kernel.cuh"

namespace pa {

cudaError_t launch_split_e4m3(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                             cudaStream_t stream) {
    return launch_split_ct<kCacheE4M3>(p, head_dim, cols, m, grid, smem, stream);
}

}  // namespace pa
