// Host-side interface between the C ABI (pa_api.cu) and the tensor-core kernel
// for prefixes shared by many sequences (pa_shared_prefix.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa_split.h"

namespace pa {

constexpr int kSharedTile = 128;   // query rows per tile, tokens per K/V tile

size_t shared_prefix_smem(int head_dim);

// Units are (group, range of unit_tokens, KV head, query tile or pair of query
// tiles): `tiles` of them cover max_group_size sequences, `units_per_list` ranges
// the longest prefix, and the grid has one CTA for each; or, for a list `padded` with
// empty groups, about as many CTAs as there are units, which take those that there are
// in turn.  Range r writes the partial r of its rows, or with `pairs` 2 r and 2 r + 1.
// unit_tokens is a multiple of kSharedTile; block_size a power of two, 8 to 128.
cudaError_t launch_shared_prefix(const SplitParams &p, int head_dim, bool bf16, bool pairs, int grid, bool padded, int tiles,
                                 int unit_tokens, int units_per_list, const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, cudaStream_t stream);

}  // namespace pa
