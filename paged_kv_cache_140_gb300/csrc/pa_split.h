// Host-side interface between the C ABI (pa_api.cu) and the split decode
// kernels (pa_split_kernel.cuh, one instantiating file per cache type), their
// merge (pa_split_merge.cu), the shared-prefix kernel (pa_shared_prefix.cu) and
// the quantised cache's write and read-back (pa_quant_ops.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

// Cache element types of the split kernels.  The 8-bit ones carry one float
// scale per token and KV head.
constexpr int kCacheF16 = 0, kCacheBF16 = 1, kCacheE4M3 = 2, kCacheInt8 = 3;

// Entries (sequences, or chunks of groups) of one launch: the kernel keeps 12
// bytes for each in shared memory; longer lists take several launches.
constexpr int kSplitEntries = 2048;
// CTAs of a launch at most (a row of the workspace for each).
constexpr int kSplitMaxCtas = 256;
constexpr int kRowFinal = -1, kRowCut = 1;

// What a launch's entries are.
constexpr int kSplitDecode = 0;   // sequences, whole contexts; results final where one partition holds them
constexpr int kSplitSuffix = 1;   // sequences past their shared blocks; partial results only
constexpr int kSplitPrefix = 2;   // (group, chunk of its sequences) over the group's shared blocks; partial only
constexpr int kSplitWhole = 3;    // as kSplitDecode, the shared blocks read through the group's first sequence

struct SplitParams {
    void *out;
    int out_dtype;               // pa_dtype value
    const uint16_t *q;           // [num_seqs, Hq, D]
    int q_bf16;
    const int32_t *block_tables; // [num_seqs, max_blocks_per_seq]
    const int32_t *context_lens; // [num_seqs]
    int max_blocks_per_seq;
    int max_context_len;
    int num_seqs;
    int num_heads;
    int num_kv_heads;
    int log2_group;              // query heads per KV head
    int block_size;
    int64_t num_blocks;
    float scale_log2;            // softmax scale * log2(e)
    int partition_size;          // tokens per partition, a multiple of 16, at most 32 blocks
    int max_parts;               // partial results per (sequence, KV head) in the workspace
    int part_off;                // where this launch's start among them
    // Workspace rows: one per (sequence, KV head, part, head of the group), then
    // those of cut items, per (launch, CTA, head of its box, query row).
    float *ws_ml;                // [rows, 4]: reference, sum, and as ints 0, kRowFinal (the output is written) or
                                 // kRowCut with the row, after cut_row, of what the next CTA did of the item
    float *ws_acc;               // [rows, D]: weighted sum
    int cut;                     // CTAs take equal shares of the slots, items may be cut
    int cut_cols;                // query rows per head in a cut item's rows
    int64_t cut_row;             // where the cut items' rows of this launch start
    int64_t prefix_cut_row;      // join: where those of the prefix launches start
    uint32_t cut_rows, prefix_cut_rows;   // join: how many there are of each
    const float *k_scales;       // 8-bit caches: [num_blocks, bs, Hkv]
    const float *v_scales;
    int *err_flag;
    int mode;
    const int32_t *shared_lens;  // suffix, prefix, whole: [num_seqs] tokens a sequence shares with its group
    const int32_t *cu_groups;    // prefix, whole: [num_groups + 1]
    int num_groups;
    int chunks, chunk_seqs;      // prefix: a group's sequences are taken chunk_seqs at a time
    int max_group_size;
    int max_shared_len;
    int e0, entries;             // this launch's entries
    int log2_heads;              // KV heads per box: 1, 2, 4 or 8
    int stages;                  // ring depth
    int late_wait;               // the previous kernel is the call's own prefix kernel, whose results this
                                 // one does not read: wait for it only at the end
};

// The state a launch needs in shared memory beyond its ring, and a ring slot.
struct SplitSmem {
    size_t fixed, slot;
};
SplitSmem split_smem(int head_dim, int cols, int cache, int log2_heads, int entries);

// KV heads per box: the largest power of two up to 8 that divides Hkv.
inline int split_log2_heads(int num_kv_heads) {
    int l = 0;
    while (l < 3 && num_kv_heads % (2 << l) == 0) ++l;
    return l;
}

// 16-token stages of one ring slot (a slot feeds every consumer warp once).
int split_slot_stages(int cache, int log2_heads);

// The caches viewed as (dim, token, head), boxes {min(128 bytes, row), min(16,
// bs), heads}; 8-bit caches with 4 or 8 heads per box: the scales as (head,
// token), boxes {heads, min(16, bs)}.
struct SplitMaps {
    CUtensorMap k, v, ks, vs;
};

// `cols`: query rows per KV head and entry (1, 2, 4 or 8).
cudaError_t launch_split_f16(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                             cudaStream_t stream);
cudaError_t launch_split_bf16(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                              cudaStream_t stream);
cudaError_t launch_split_e4m3(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                              cudaStream_t stream);
cudaError_t launch_split_int8(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                              cudaStream_t stream);

// Joins partial results into output rows.  Sequence s has per_part partials for
// each prefix_part tokens of its shared blocks at index 0.. and one for each
// partition_size of the rest at p.part_off.. (p.mode kSplitDecode: no shared
// blocks, and sequences of one partition are final already).  holes: every second
// partial of a prefix may be empty.
cudaError_t launch_split_merge(const SplitParams &p, int head_dim, int prefix_part, int per_part, bool holes, int sms,
                               cudaStream_t stream);

// Quantising write and read-back (cache: kCacheE4M3 or kCacheInt8).
cudaError_t launch_quant_write(const void *key, const void *value, int64_t key_stride, int64_t value_stride,
                               void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                               const int64_t *slot_mapping, int64_t num_tokens, int64_t num_slots, int num_kv_heads,
                               int head_dim, bool bf16, int cache, int sms, int *err_flag, cudaStream_t stream);

cudaError_t launch_quant_gather(void *out_k, void *out_v, int out_dtype, const void *k_cache, const void *v_cache,
                                int cache, const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                int max_blocks_per_seq, const int32_t *cu_seqlens, const int32_t *seq_starts,
                                int num_seqs, int64_t num_tokens, int num_kv_heads, int head_dim, int block_size,
                                int64_t num_blocks, int *err_flag, cudaStream_t stream);

}  // namespace pa
