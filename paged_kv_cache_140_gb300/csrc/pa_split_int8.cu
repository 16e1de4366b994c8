// The split decode kernel for int8 caches.
#include "pa_split_kernel.cuh"

namespace pa {

cudaError_t launch_split_int8(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                             cudaStream_t stream) {
    return launch_split_ct<kCacheInt8>(p, head_dim, cols, m, grid, smem, stream);
}

}  // namespace pa
