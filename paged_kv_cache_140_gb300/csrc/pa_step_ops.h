// Host-side interface between the C ABI (pa_api.cu) and the kernels of a serving
// step around its attention: block tables (pa_tables.cu), and norm, rotation and
// cache write (pa_rope.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "pa_divisor.cuh"

namespace pa {

// Sequences of one call: the kernel keeps 20 bytes for each in shared memory.
constexpr int kTablesMaxSeqs = 8192;

struct TablesParams {
    int32_t *block_tables;       // [num_seqs, max_blocks]
    int max_blocks;
    const int32_t *lens;
    const int32_t *changes;
    int32_t *out_lens;           // may be lens
    int num_seqs;
    int32_t *free_blocks;        // [free_capacity]: a stack, the next block to take last
    int64_t free_capacity;
    const int32_t *free_count;
    int32_t *out_free_count;     // may be free_count
    int64_t num_blocks;
    Divisor block;               // the block size
    int32_t *cu_seqlens;         // [num_seqs + 1]
    int64_t *slots;              // [num_tokens]
    int64_t *positions;          // [num_tokens]
    int64_t num_tokens;
    int *err_flag;
};

cudaError_t launch_update_tables(const TablesParams &p, cudaStream_t stream);

// What the rotated keys and the values become in the cache.
constexpr int kRopeHalf = 0;     // rows of the inputs' type
constexpr int kRopeE4M3 = 1;     // e4m3 codes, one scale per tensor
constexpr int kRopeRows = 2;     // e4m3 codes, a scale per row
constexpr int kRopeInt8 = 3;     // int8 codes, a scale per row
constexpr int kRopeInt4 = 4;     // 4-bit codes, a scale and zero per 64 elements

struct RopeParams {
    const uint16_t *src[3];      // query, key, value
    int64_t stride[3];           // elements between tokens
    uint16_t *out_q;             // [num_tokens, hq, D]
    void *cache[2];              // K, V
    void *scales[2];
    float scale[2];              // kRopeE4M3
    const int64_t *slots;
    const int64_t *positions;
    const double *inv_freq;      // [rot / 2]
    const uint16_t *weight[2];   // norms of queries and keys, or null
    float eps, factor;
    int64_t num_tokens;
    int hq, hkv, rot;
    int interleaved;
    int64_t num_slots;
    int bs;
    int *err_flag;
};

cudaError_t launch_rope_and_cache(const RopeParams &p, int head_dim, bool bf16, int kind, int sms, cudaStream_t stream);

}  // namespace pa
