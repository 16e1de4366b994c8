// The split decode kernel for bf16 caches.
#include "pa_split_kernel.cuh"

namespace pa {

cudaError_t launch_split_bf16(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                             cudaStream_t stream) {
    return launch_split_ct<kCacheBF16>(p, head_dim, cols, m, grid, smem, stream);
}

}  // namespace pa
