// The exported C ABI (declared in include/pa.h): argument validation,
// partition and workspace planning, TMA descriptor encoding and launches.
// The library allocates no memory and keeps no state between calls beyond
// cached device attributes (per device ordinal) and the driver entry point.
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <stdlib.h>

#include <algorithm>
#include <atomic>
#include <initializer_list>
#include <mutex>
#include <numeric>

#include "pa.h"
#include "pa_cache_ops.h"
#include "pa_internal.h"
#include "pa_prefill.h"
#include "pa_shared_prefix.h"
#include "pa_split.h"
#include "pa_split_plan.h"
#include "pa_step_ops.h"

#define PA_EXPORT extern "C" __attribute__((visibility("default")))

namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool half_dtype(pa_dtype d) { return d == PA_F16 || d == PA_BF16; }
bool cache_dtype_ok(pa_dtype d) { return half_dtype(d) || d == PA_FP8_E4M3; }
int elem_bytes(pa_dtype d) { return d == PA_FP8_E4M3 ? 1 : 2; }
bool scale_ok(float s) { return s > 0.f && s < 3.0e38f; }
bool supported_head_dim(int d) { return d == 64 || d == 128; }
bool supported_block_size(int bs) { return bs == 8 || (bs >= 16 && bs <= 256 && bs % 16 == 0); }
bool supported_group(int g) { return g == 1 || g == 2 || g == 4 || g == 8; }

int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

struct DeviceInfo {
    int sms = 0;
    int smem_optin = 0;
};

// Attributes of the current device, read once per device ordinal (they are
// properties of the hardware and do not change while the process runs).
constexpr int kMaxDevices = 64;

bool device_info(DeviceInfo &info) {
    static DeviceInfo cache[kMaxDevices];
    static std::atomic<bool> valid[kMaxDevices];
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    if (dev >= 0 && dev < kMaxDevices && valid[dev].load(std::memory_order_acquire)) {
        info = cache[dev];
        return true;
    }
    DeviceInfo d;
    if (cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return false;
    if (cudaDeviceGetAttribute(&d.smem_optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
        cudaSuccess)
        return false;
    if (dev >= 0 && dev < kMaxDevices) {
        std::lock_guard<std::mutex> lock(mu);
        cache[dev] = d;
        valid[dev].store(true, std::memory_order_release);
    }
    info = d;
    return true;
}

// Tuning overrides read once from the environment (documented in pa.h):
// PA_DECODE_COOP=0 keeps every shape on the per-warp decode kernel;
// PA_DECODE_COOP_STAGES, PA_DECODE_STAGES and PA_DECODE_WARPS set ring depths
// and warps per CTA; PA_DECODE_INTERLEAVE=0 gives each per-warp pipeline a
// contiguous run of items.  Results stay within the documented tolerance under
// any setting; only speed changes.
struct Tuning {
    int stages = 0;  // 0: default
    int warps = 0;
    int interleave = 1;
    int coop = 1;            // 0: never use the CTA-cooperative decode kernel
    int coop_stages = 0;     // 0: default
};

int env_int(const char *name, int lo, int hi) {
    const char *v = getenv(name);
    if (v == nullptr) return 0;
    const int x = atoi(v);
    return (x >= lo && x <= hi) ? x : 0;
}

const Tuning &tuning() {
    static const Tuning t = [] {
        Tuning r;
        r.stages = env_int("PA_DECODE_STAGES", 2, 8);
        r.warps = env_int("PA_DECODE_WARPS", 1, 16);
        const char *il = getenv("PA_DECODE_INTERLEAVE");
        r.interleave = (il != nullptr && il[0] == '0') ? 0 : 1;
        const char *co = getenv("PA_DECODE_COOP");
        r.coop = (co != nullptr && co[0] == '0') ? 0 : 1;
        r.coop_stages = env_int("PA_DECODE_COOP_STAGES", 2, 8);
        return r;
    }();
    return t;
}

// Partition length in tokens for pa_decode; 0 when the request is invalid.
int resolve_partition(int max_context_len, int block_size, int requested) {
    const int cap = 32 * block_size;
    if (requested != 0) {
        if (requested < 16 || requested % 16 != 0 || requested > cap) return 0;
        // A partition's block ids sit in the 32 lanes of a warp.  Partitions start at most
        // block_size - gcd inside a block; a long one that reaches into a 33rd from there
        // is cut to whole blocks.
        if (requested > cap - block_size + std::gcd(requested, block_size) && max_context_len > requested)
            return requested - requested % block_size;
        return requested;
    }
    int P;
    if (max_context_len <= 256)
        P = static_cast<int>(std::max<int64_t>(16, round_up(max_context_len, 16)));
    else if (max_context_len <= 8192)
        P = 256;
    else
        P = 512;
    return std::min(P, cap);
}

struct WorkspacePlan {
    int partition = 0;
    int max_partitions = 1;
    size_t ml_off = 0, acc_off = 0, bytes = 0;
};

bool plan_workspace(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                    int max_context_len, int partition_size, WorkspacePlan &w) {
    if (num_seqs < 0 || num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads != 0)
        return false;
    if (!supported_group(num_heads / num_kv_heads) || !supported_head_dim(head_dim) ||
        !supported_block_size(block_size) || max_context_len < 0)
        return false;
    w.partition = resolve_partition(max_context_len, block_size, partition_size);
    if (w.partition == 0) return false;
    w.max_partitions = std::max(1, (max_context_len + w.partition - 1) / w.partition);
    if (w.max_partitions <= 1) {
        w.bytes = 0;
        return true;
    }
    const int G = num_heads / num_kv_heads;
    const int64_t slots = static_cast<int64_t>(num_seqs) * num_kv_heads * w.max_partitions;
    w.ml_off = 0;
    w.acc_off = round_up(slots * G * 2 * 4, 256);
    w.bytes = w.acc_off + static_cast<size_t>(slots) * G * head_dim * 4;
    return true;
}

// Tensor map over a cache [NB * bs, Hkv, D] with 128-byte boxes of one KV
// head's row and min(bs, 16) rows, 128-byte swizzle.
bool encode_cache_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int block_size,
                      int num_kv_heads, int head_dim, int es) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim),
                                static_cast<cuuint64_t>(num_kv_heads),
                                static_cast<cuuint64_t>(num_blocks) * block_size};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(head_dim) * es,
                                   static_cast<cuuint64_t>(num_kv_heads) * head_dim * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), 1u,
                               static_cast<cuuint32_t>(std::min(block_size, 16))};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
              const_cast<void *>(cache), dims, strides,
              box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over a cache [NB * bs, Hkv, D] of `es`-byte elements with its
// dimensions taken in the order (dim, token, head): a box {128 / es, 16, 8}
// is one 128-byte column block of 16 token rows for 8 consecutive KV heads,
// landing as 8 per-head tiles of 16 rows x 128 bytes, 128-byte swizzle (the
// cooperative decode kernel).
bool encode_cache_map_heads8(CUtensorMap *map, const void *cache, int64_t num_blocks, int block_size,
                             int num_kv_heads, int head_dim, int es) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim),
                                static_cast<cuuint64_t>(num_blocks) * block_size,
                                static_cast<cuuint64_t>(num_kv_heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(num_kv_heads) * head_dim * es,
                                   static_cast<cuuint64_t>(head_dim) * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), 16u, 8u};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
              const_cast<void *>(cache), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The address a kernel on the current device may use for `p`: device or
// managed memory as is, page-locked host memory through its mapped device
// pointer.  False for anything else (e.g. pageable host memory), which the
// caller rejects before any launch.
bool device_address(const void *p, const void **out) {
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    if (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) {
        *out = p;
        return true;
    }
    if (a.type == cudaMemoryTypeHost && a.devicePointer != nullptr) {
        *out = a.devicePointer;
        return true;
    }
    return false;
}

}  // namespace

PA_EXPORT const char *pa_status_string(pa_status s) {
    switch (s) {
        case PA_OK: return "ok";
        case PA_ERR_INVALID_ARG: return "invalid argument";
        case PA_ERR_UNSUPPORTED: return "unsupported shape or dtype";
        case PA_ERR_CUDA: return "CUDA error";
        case PA_ERR_WORKSPACE: return "decode workspace missing or too small";
        case PA_ERR_DEVICE_BOUNDS: return "device-side index out of bounds (see err_flag bits)";
    }
    return "unknown status";
}

PA_EXPORT int pa_version(void) { return 200; }

PA_EXPORT pa_status pa_reshape_and_cache(const void *key, const void *value, void *k_cache,
                                         void *v_cache, const int64_t *slot_mapping,
                                         int64_t num_tokens, int64_t num_blocks, int block_size,
                                         int num_kv_heads, int head_dim, pa_dtype dtype,
                                         pa_dtype cache_dtype, float k_scale, float v_scale,
                                         int *err_flag, void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || !half_dtype(dtype) || !cache_dtype_ok(cache_dtype))
        return PA_ERR_INVALID_ARG;
    const bool fp8 = cache_dtype == PA_FP8_E4M3;
    if (!fp8 && cache_dtype != dtype) return PA_ERR_UNSUPPORTED;
    if (fp8 && (!scale_ok(k_scale) || !scale_ok(v_scale))) return PA_ERR_INVALID_ARG;
    const int64_t row_elems = static_cast<int64_t>(num_kv_heads) * head_dim;
    if ((row_elems * 2) % 16 != 0 || row_elems % 8 != 0) return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    cudaError_t e;
    if (fp8)
        e = pa::launch_reshape_and_cache_fp8(key, value, k_cache, v_cache, slot_mapping, num_tokens,
                                             num_blocks * block_size, row_elems, dtype == PA_BF16,
                                             k_scale, v_scale, err_flag,
                                             static_cast<cudaStream_t>(stream));
    else
        e = pa::launch_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, num_tokens,
                                         num_blocks * block_size, row_elems * 2, err_flag,
                                         static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_EXPORT pa_status pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *block_mapping,
                                   int64_t num_pairs, int64_t num_blocks, int block_size,
                                   int num_kv_heads, int head_dim, pa_dtype dtype, int *err_flag,
                                   void *stream) {
    if (num_pairs < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || !cache_dtype_ok(dtype))
        return PA_ERR_INVALID_ARG;
    const int64_t block_bytes =
        static_cast<int64_t>(block_size) * num_kv_heads * head_dim * elem_bytes(dtype);
    if (block_bytes % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PA_OK;
    if (!k_cache || !v_cache || !block_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    cudaError_t e = pa::launch_copy_blocks(k_cache, v_cache, k_cache, v_cache, block_mapping, num_pairs,
                                           num_blocks, num_blocks, block_bytes, err_flag,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_EXPORT pa_status pa_copy_blocks_layers(void *kv_cache, int num_layers, const int64_t *block_mapping,
                                          int64_t num_pairs, int64_t num_blocks, int block_size,
                                          int num_kv_heads, int head_dim, pa_dtype dtype, int *err_flag,
                                          void *stream) {
    if (num_layers < 0 || num_pairs < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || !cache_dtype_ok(dtype))
        return PA_ERR_INVALID_ARG;
    if (num_layers > 65535) return PA_ERR_UNSUPPORTED;
    const int64_t block_bytes =
        static_cast<int64_t>(block_size) * num_kv_heads * head_dim * elem_bytes(dtype);
    if (block_bytes % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0 || num_layers == 0) return PA_OK;
    if (!kv_cache || !block_mapping || !aligned16(kv_cache)) return PA_ERR_INVALID_ARG;
    // [layers, 2, num_blocks, ...]: layer l's K at l * 2 * NB blocks, its V right after.
    uint8_t *base = static_cast<uint8_t *>(kv_cache);
    const int64_t cache_bytes = num_blocks * block_bytes;
    cudaError_t e = pa::launch_copy_blocks(base, base + cache_bytes, base, base + cache_bytes, block_mapping,
                                           num_pairs, num_blocks, num_blocks, block_bytes, err_flag,
                                           static_cast<cudaStream_t>(stream), num_layers, 2 * cache_bytes);
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_EXPORT pa_status pa_swap_blocks(const void *src_k, const void *src_v, void *dst_k, void *dst_v,
                                   const int64_t *block_mapping, int64_t num_pairs,
                                   int64_t src_num_blocks, int64_t dst_num_blocks, int block_size,
                                   int num_kv_heads, int head_dim, pa_dtype dtype, int *err_flag,
                                   void *stream) {
    if (num_pairs < 0 || src_num_blocks <= 0 || dst_num_blocks <= 0 || block_size <= 0 ||
        num_kv_heads <= 0 || head_dim <= 0 || !cache_dtype_ok(dtype))
        return PA_ERR_INVALID_ARG;
    const int64_t block_bytes =
        static_cast<int64_t>(block_size) * num_kv_heads * head_dim * elem_bytes(dtype);
    if (block_bytes % 16 != 0) return PA_ERR_UNSUPPORTED;
    if (num_pairs == 0) return PA_OK;
    if (!src_k || !src_v || !dst_k || !dst_v || !block_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(src_k) || !aligned16(src_v) || !aligned16(dst_k) || !aligned16(dst_v))
        return PA_ERR_INVALID_ARG;
    const void *sk, *sv, *dk, *dv, *bm;
    if (!device_address(src_k, &sk) || !device_address(src_v, &sv) || !device_address(dst_k, &dk) ||
        !device_address(dst_v, &dv) || !device_address(block_mapping, &bm))
        return PA_ERR_INVALID_ARG;
    cudaError_t e = pa::launch_copy_blocks(sk, sv, const_cast<void *>(dk), const_cast<void *>(dv),
                                           static_cast<const int64_t *>(bm), num_pairs, src_num_blocks,
                                           dst_num_blocks, block_bytes, err_flag,
                                           static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_EXPORT size_t pa_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads,
                                          int head_dim, int block_size, int max_context_len,
                                          int partition_size) {
    WorkspacePlan w;
    if (!plan_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                        partition_size, w))
        return static_cast<size_t>(-1);
    return w.bytes;
}

PA_EXPORT int pa_decode_partition_size(int num_seqs, int num_heads, int num_kv_heads,
                                       int head_dim, int block_size, int max_context_len,
                                       int partition_size) {
    WorkspacePlan w;
    if (!plan_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                        partition_size, w))
        return 0;
    return w.partition;
}

PA_EXPORT pa_status pa_decode_workspace_init(void *workspace, size_t workspace_bytes,
                                             void *stream) {
    if (workspace_bytes == 0) return PA_OK;
    if (workspace == nullptr) return PA_ERR_INVALID_ARG;
    return cudaMemsetAsync(workspace, 0, workspace_bytes, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

namespace {

// pa_decode and pa_decode_append share everything but the new rows.
pa_status decode_impl(void *out, pa_dtype out_dtype, const void *query, pa_dtype q_dtype,
                      const void *new_k, const void *new_v,
                      const void *k_cache, const void *v_cache, pa_dtype kv_dtype,
                      float k_scale, float v_scale,
                              const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *context_lens, int max_context_len, int num_seqs,
                              int num_heads, int num_kv_heads, int head_dim, int block_size,
                              int64_t num_blocks, float scale, int partition_size,
                              void *workspace, size_t workspace_bytes, int *err_flag,
                              void *stream) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0 || max_context_len < 0)
        return PA_ERR_INVALID_ARG;
    if (!half_dtype(q_dtype) || !cache_dtype_ok(kv_dtype) ||
        (out_dtype != PA_F16 && out_dtype != PA_BF16 && out_dtype != PA_F32))
        return PA_ERR_INVALID_ARG;
    const bool fp8 = kv_dtype == PA_FP8_E4M3;
    if (fp8 && (!scale_ok(k_scale) || !scale_ok(v_scale))) return PA_ERR_INVALID_ARG;
    if (!fp8 && kv_dtype != q_dtype) return PA_ERR_UNSUPPORTED;     // 16-bit caches: same type as q
    if (fp8 && head_dim != 128) return PA_ERR_UNSUPPORTED;
    if (num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (!supported_group(num_heads / num_kv_heads) || !supported_head_dim(head_dim) ||
        !supported_block_size(block_size))
        return PA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size)
        return PA_ERR_INVALID_ARG;
    if (num_blocks * block_size > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (!(scale == scale)) return PA_ERR_INVALID_ARG;
    WorkspacePlan w;
    if (!plan_workspace(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                        partition_size, w))
        return PA_ERR_INVALID_ARG;
    // Work is counted in 16-token stages in 32-bit arithmetic on the device.
    const int64_t max_units = static_cast<int64_t>(num_seqs) * num_kv_heads *
                              std::max<int64_t>(1, (max_context_len + 15) / 16);
    if (max_units >= (int64_t{1} << 31)) return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if ((new_k == nullptr) != (new_v == nullptr)) return PA_ERR_INVALID_ARG;
    if (new_k && (!aligned16(new_k) || !aligned16(new_v))) return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;
    if (w.bytes > 0 && (workspace == nullptr || workspace_bytes < w.bytes || !aligned16(workspace)))
        return PA_ERR_WORKSPACE;

    DeviceInfo dev;
    if (!device_info(dev)) return PA_ERR_CUDA;
    const int G = num_heads / num_kv_heads;
    // Ring depth and warps per CTA (PA_DECODE_STAGES / PA_DECODE_WARPS override
    // the defaults for tuning); fewer warps are used if shared memory is short.
    const Tuning &tune = tuning();
    const int stages = tune.stages > 0 ? tune.stages : pa::kDefaultStages;
    const int max_warps = head_dim == 128 ? 12 : 16;
    const int def_warps = head_dim == 128 ? (fp8 ? pa::kDefaultWarpsFp8 : pa::kDefaultWarps128) : 16;
    int warps = tune.warps > 0 ? std::min(tune.warps, max_warps) : def_warps;
    const int es = elem_bytes(kv_dtype);
    while (warps > 1 && pa::decode_smem_bytes(head_dim, G, es, warps, stages, num_seqs) >
                            static_cast<size_t>(dev.smem_optin))
        --warps;
    const size_t smem_used = pa::decode_smem_bytes(head_dim, G, es, warps, stages, num_seqs);
    if (smem_used > static_cast<size_t>(dev.smem_optin)) return PA_ERR_UNSUPPORTED;

    pa::DecodeParams p{};
    p.out = out;
    p.out_dtype = static_cast<int>(out_dtype);
    p.q = query;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f * (fp8 ? k_scale : 1.0f);
    p.v_scale = fp8 ? v_scale : 1.0f;
    p.partition_size = w.partition;
    p.max_partitions = w.max_partitions;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.ws_ml = w.bytes ? reinterpret_cast<float *>(ws + w.ml_off) : nullptr;
    p.ws_acc = w.bytes ? reinterpret_cast<float *>(ws + w.acc_off) : nullptr;
    p.err_flag = err_flag;
    p.stages = stages;
    p.new_k = new_k;
    p.new_v = new_v;
    p.k_cache_w = const_cast<void *>(k_cache);
    p.v_cache_w = const_cast<void *>(v_cache);
    p.k_scale_w = k_scale;
    p.v_scale_w = v_scale;
    p.interleave = tune.interleave;

    const int kv = fp8 ? (q_dtype == PA_F16 ? 2 : 3) : (kv_dtype == PA_BF16 ? 1 : 0);
    // Caches whose KV heads come in groups of 8 run the CTA-cooperative
    // kernel (8-head TMA boxes); everything else the per-warp kernel.  With
    // new rows to append, an append kernel writes them first (quantised for
    // an e4m3 cache) and the cooperative kernel, chained by programmatic
    // dependent launch, waits for it only before the stages that hold them.
    if (tune.coop && head_dim == 128 && num_kv_heads % 8 == 0 && block_size % 16 == 0) {
        // a slot holds one 16-token stage of a 16-bit cache or two of an e4m3
        // cache: 64 KB either way
        int cst = tune.coop_stages > 0 ? tune.coop_stages : 3;
        while (cst > 2 && pa::decode_coop_smem_bytes(G, es, cst, num_seqs) > static_cast<size_t>(dev.smem_optin))
            --cst;
        const size_t csmem = pa::decode_coop_smem_bytes(G, es, cst, num_seqs);
        CUtensorMap ck, cv;
        if (csmem > 0 && csmem <= static_cast<size_t>(dev.smem_optin) &&
            encode_cache_map_heads8(&ck, k_cache, num_blocks, block_size, num_kv_heads, head_dim, es) &&
            encode_cache_map_heads8(&cv, v_cache, num_blocks, block_size, num_kv_heads, head_dim, es)) {
            p.stages = cst;
            if (new_k != nullptr) {
                const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
                const cudaError_t ea =
                    fp8 ? pa::launch_append_rows_fp8(new_k, new_v, const_cast<void *>(k_cache),
                                                     const_cast<void *>(v_cache), block_tables, context_lens,
                                                     max_blocks_per_seq, max_context_len, block_size, num_blocks,
                                                     num_seqs, row, q_dtype == PA_BF16, k_scale, v_scale, err_flag,
                                                     static_cast<cudaStream_t>(stream))
                        : pa::launch_append_rows(new_k, new_v, const_cast<void *>(k_cache),
                                                 const_cast<void *>(v_cache), block_tables, context_lens,
                                                 max_blocks_per_seq, max_context_len, block_size, num_blocks,
                                                 num_seqs, row * 2, err_flag, static_cast<cudaStream_t>(stream));
                if (ea != cudaSuccess) return PA_ERR_CUDA;
                p.new_k = p.new_v = nullptr;
                p.defer_wait = 1;
            }
            const cudaError_t e = pa::launch_decode_coop(p, G, kv, ck, cv, dev.sms, csmem,
                                                         static_cast<cudaStream_t>(stream));
            return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
        }
    }
    CUtensorMap tk, tv;
    if (!encode_cache_map(&tk, k_cache, num_blocks, block_size, num_kv_heads, head_dim, es) ||
        !encode_cache_map(&tv, v_cache, num_blocks, block_size, num_kv_heads, head_dim, es))
        return PA_ERR_CUDA;
    cudaError_t e = pa::launch_decode(p, head_dim, G, kv, tk, tv, dev.sms, warps,
                                      smem_used, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

PA_EXPORT pa_status pa_decode(void *out, pa_dtype out_dtype, const void *query, pa_dtype q_dtype,
                              const void *k_cache, const void *v_cache, pa_dtype kv_dtype,
                              float k_scale, float v_scale, const int32_t *block_tables,
                              int max_blocks_per_seq, const int32_t *context_lens,
                              int max_context_len, int num_seqs, int num_heads, int num_kv_heads,
                              int head_dim, int block_size, int64_t num_blocks, float scale,
                              int partition_size, void *workspace, size_t workspace_bytes,
                              int *err_flag, void *stream) {
    return decode_impl(out, out_dtype, query, q_dtype, nullptr, nullptr, k_cache, v_cache, kv_dtype,
                       k_scale, v_scale, block_tables, max_blocks_per_seq, context_lens,
                       max_context_len, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, scale, partition_size, workspace, workspace_bytes, err_flag,
                       stream);
}

PA_EXPORT pa_status pa_decode_append(void *out, pa_dtype out_dtype, const void *query,
                                     pa_dtype q_dtype, const void *key, const void *value,
                                     void *k_cache, void *v_cache, pa_dtype kv_dtype, float k_scale,
                                     float v_scale, const int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *context_lens,
                                     int max_context_len, int num_seqs, int num_heads,
                                     int num_kv_heads, int head_dim, int block_size,
                                     int64_t num_blocks, float scale, int partition_size,
                                     void *workspace, size_t workspace_bytes, int *err_flag,
                                     void *stream) {
    if (num_seqs > 0 && (key == nullptr || value == nullptr)) return PA_ERR_INVALID_ARG;
    return decode_impl(out, out_dtype, query, q_dtype, key, value, k_cache, v_cache, kv_dtype,
                       k_scale, v_scale, block_tables, max_blocks_per_seq, context_lens,
                       max_context_len, num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                       num_blocks, scale, partition_size, workspace, workspace_bytes, err_flag,
                       stream);
}

namespace {

// Tensor map over a dense 3-D array [d2][d1][d0] of `es`-byte elements with
// a (128 / es, box1, box2) box (128 bytes wide) and 128-byte swizzle.
bool encode_map_128b(CUtensorMap *map, const void *ptr, int es, int64_t d0, int64_t d1, int64_t d2, int box1,
                     int box2) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d0), static_cast<cuuint64_t>(d1),
                                static_cast<cuuint64_t>(d2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d0) * es, static_cast<cuuint64_t>(d0 * d1) * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / es), static_cast<cuuint32_t>(box1),
                               static_cast<cuuint32_t>(box2)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, es == 4 ? CU_TENSOR_MAP_DATA_TYPE_UINT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
              const_cast<void *>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

PA_EXPORT pa_status pa_prefill(void *out, pa_dtype out_dtype, const void *query,
                               const void *k_cache, const void *v_cache, pa_dtype kv_dtype,
                               const int32_t *block_tables, int max_blocks_per_seq,
                               const int32_t *context_lens, const int32_t *cu_seqlens_q,
                               int num_seqs, int64_t num_tokens, int max_q_len, int num_heads,
                               int num_kv_heads, int head_dim, int block_size, int64_t num_blocks,
                               float scale, int *err_flag, void *stream) {
    if (num_seqs < 0 || num_tokens < 0 || max_q_len < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
        head_dim <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq <= 0)
        return PA_ERR_INVALID_ARG;
    if (!half_dtype(kv_dtype) || (out_dtype != PA_F16 && out_dtype != PA_BF16 && out_dtype != PA_F32))
        return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    const int G = num_heads / num_kv_heads;
    if (G > pa::kPrefillTile || (G & (G - 1)) != 0) return PA_ERR_UNSUPPORTED;
    if (!supported_head_dim(head_dim)) return PA_ERR_UNSUPPORTED;
    if (block_size < 8 || block_size > pa::kPrefillTile || (block_size & (block_size - 1)) != 0)
        return PA_ERR_UNSUPPORTED;
    if (num_blocks * block_size > INT32_MAX || num_tokens > INT32_MAX) return PA_ERR_UNSUPPORTED;
    if (!(scale > 0.f) || scale > 3.0e38f) return PA_ERR_INVALID_ARG;
    int lg = 0;
    while ((1 << lg) < G) ++lg;
    const int tokens_per_tile = pa::kPrefillTile / G;
    const int64_t tiles = (static_cast<int64_t>(max_q_len) + tokens_per_tile - 1) / tokens_per_tile;
    const int64_t grid = static_cast<int64_t>(num_seqs) * num_kv_heads * ((tiles + 1) / 2);
    if (grid >= (int64_t{1} << 31)) return PA_ERR_UNSUPPORTED;
    if (grid == 0 || num_tokens == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens || !cu_seqlens_q)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache))
        return PA_ERR_INVALID_ARG;

    DeviceInfo dev;
    if (!device_info(dev)) return PA_ERR_CUDA;
    const size_t smem = pa::prefill_smem_bytes(head_dim);
    // + the kernel's static shared memory (barriers, the sequence order), under 8 KB
    if (smem + 8192 > static_cast<size_t>(dev.smem_optin)) return PA_ERR_UNSUPPORTED;

    CUtensorMap tq, tk, tv, to;
    const int out_es = out_dtype == PA_F32 ? 4 : 2;
    if (!encode_map_128b(&tq, query, 2, head_dim, num_heads, num_tokens, G, tokens_per_tile) ||
        !encode_map_128b(&tk, k_cache, 2, head_dim, num_kv_heads, num_blocks * block_size, 1, block_size) ||
        !encode_map_128b(&tv, v_cache, 2, head_dim, num_kv_heads, num_blocks * block_size, 1, block_size) ||
        !encode_map_128b(&to, out, out_es, head_dim, num_heads, num_tokens, G, tokens_per_tile))
        return PA_ERR_CUDA;

    pa::PrefillParams p{};
    p.q = query;
    p.out = out;
    p.out_dtype = static_cast<int>(out_dtype);
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.cu_seqlens_q = cu_seqlens_q;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    p.log2_group = lg;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.max_q_len = max_q_len;
    p.tiles_per_seq = static_cast<int>(tiles);
    p.pairs_per_seq = static_cast<int>((tiles + 1) / 2);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.err_flag = err_flag;
    cudaError_t e = pa::launch_prefill(p, head_dim, kv_dtype == PA_BF16, tq, tk, tv, to, smem,
                                       static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// ------------------------- quantised cache, and decode with shared prefixes

namespace {

bool quant_dtype(pa_dtype d) { return d == PA_FP8_E4M3 || d == PA_INT8; }
bool out_dtype_ok(pa_dtype d) { return d == PA_F16 || d == PA_BF16 || d == PA_F32; }
int split_cache(pa_dtype d) {
    return d == PA_F16 ? pa::kCacheF16 : d == PA_BF16 ? pa::kCacheBF16 : d == PA_FP8_E4M3 ? pa::kCacheE4M3 : pa::kCacheInt8;
}

using pa::kSmsTarget;
using pa::kSplitEntries;
using pa::split_partition;

// A group with more query rows per KV head than this has its prefix computed on
// the tensor-core kernel, whose 128-row tiles read each K/V row once for up to
// 256 query rows; up to it the split kernel does, which reads them once for every
// 8 rows.  Whole calls, 16 prompts of 2,000 tokens: 8 rows 51 us split against 57,
// 12 rows 72 against 61, 24 rows 93 against 69 (one prompt of 4,000 to 8,000 tokens:
// 33 against 27, 30 against 24, 34 against 24; 64 of 1,000 with 4 rows 256 against 282).
constexpr int kSharedSplitRows = 8;

// Tokens per unit of the tensor-core prefix kernel, for `lists` lists (groups x
// tiles x KV heads) of up to `tokens`: the cut with the least estimated time, whole
// waves of CTAs times the tiles of one unit plus a CTA's own start and end.  Pairs
// of query tiles take one CTA per SM, about 2 us per K/V tile and five times that to
// start and end; single ones two, each a little slower, which hide one another's
// ends.  The prefixes of several groups are taken to be of any length up to the
// longest alike, with a tenth more units than that gives: a second wave costs more
// than longer units (24 groups of 0 to 4,096 tokens: 130 us, with shorter units 135
// to 148).
int shared_unit(int64_t lists, int tokens, bool paired, bool several) {
    const int tiles = std::max(1, (tokens + pa::kSharedTile - 1) / pa::kSharedTile);
    const int64_t ctas = paired ? kSmsTarget : 2 * kSmsTarget;
    const double tile = paired ? 1.0 : 1.1, ends = paired ? 5.0 : 3.0;
    int best = tiles;
    double best_cost = 1e30;
    for (int per = tiles; per >= 1; per = std::min(per - 1, per * 15 / 16)) {
        const int64_t units =
            several ? static_cast<int64_t>(1.1 * lists * (0.5 * tiles / per + 0.5)) : lists * ((tiles + per - 1) / per);
        const double cost = static_cast<double>((units + ctas - 1) / ctas) * (per * tile + ends);
        if (cost < best_cost) {
            best_cost = cost;
            best = per;
        }
    }
    return best * pa::kSharedTile;
}

// A batch whose shared prefixes, read again for every sequence, cost at most this
// many more bytes of K/V is decoded in one pass that does read them again: it
// takes one launch in place of three, and the second reads come from L2.
constexpr int64_t kSharedWholeBytes = 8 << 20;

struct SplitPlan {
    int log2_heads = 0, G = 1;
    bool padded = false;         // the list of groups is taken to be padded with empty ones
    int64_t groups = 0;          // groups that the prefixes are planned for
    int partition = 0;           // decode and suffix entries
    int parts = 1;               // their partials per row
    bool whole = false;          // shared prefixes are not worth a pass of their own
    bool prefix_tc = false;      // shared prefixes: on the tensor-core kernel (else the split kernel)
    int prefix_cols = 0;         // split kernel: query rows per entry
    bool prefix_paired = false;  // tensor-core kernel: query tiles in pairs (more than one per group)
    int prefix_tiles = 0;        // query tiles (pairs) per group
    int prefix_part = 0;         // tokens per prefix_per partials
    int prefix_per = 1, prefix_parts = 0;
    int max_parts = 1;
    int max_shares = 0;
    int64_t cut_row = 0, prefix_cut_row = 0, rows = 0;
    size_t acc_off = 0, bytes = 0;
};

bool split_shape_ok(int num_heads, int num_kv_heads, int head_dim, int block_size) {
    return num_heads % num_kv_heads == 0 && supported_group(num_heads / num_kv_heads) && supported_head_dim(head_dim) &&
           supported_block_size(block_size);
}

// The cut of a call and the workspace for its partial results.  `shared`: the
// shared blocks of up to max_shared_len tokens are computed per group.
bool plan_split(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size, int max_context_len,
                int partition_size, int cache, bool shared, int num_groups, int max_group_size, int max_shared_len,
                SplitPlan &w) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_context_len < 0)
        return false;
    if (!split_shape_ok(num_heads, num_kv_heads, head_dim, block_size)) return false;
    w.G = num_heads / num_kv_heads;
    w.log2_heads = pa::split_log2_heads(num_kv_heads);
    const int64_t ngroups = num_kv_heads >> w.log2_heads;
    const int slot_tokens = 16 * pa::split_slot_stages(cache, w.log2_heads);
    if (shared) {
        if (num_groups < 0 || max_group_size < 0 || max_shared_len < 0 || max_shared_len > max_context_len) return false;
        max_group_size = std::min(max_group_size, num_seqs);
        const int shared_tokens = max_shared_len / block_size * block_size;
        // A list of at least as many groups as sequences shares nothing or is padded with
        // empty ones (as the fixed list of a captured step is): it is planned for the
        // fewest groups that hold all sequences.  A shorter one is taken at its word.
        w.padded = num_groups >= num_seqs && max_group_size > 1;
        w.groups = w.padded ? (static_cast<int64_t>(num_seqs) + max_group_size - 1) / max_group_size : num_groups;
        w.whole = static_cast<double>(std::max<int64_t>(0, num_seqs - w.groups)) * shared_tokens * num_kv_heads * head_dim *
                      4 <= kSharedWholeBytes;
    }
    // Private parts are about as long as the bounds differ (only the cut goes by
    // that; a part may be longer).
    const int64_t part_len = shared && !w.whole ? std::max(256, max_context_len - max_shared_len) : max_context_len;
    w.partition = split_partition(num_seqs * ngroups, ngroups, part_len, block_size, slot_tokens, partition_size);
    if (w.partition == 0) return false;
    w.parts = std::max(1, static_cast<int>((static_cast<int64_t>(max_context_len) + w.partition - 1) / w.partition));
    w.max_parts = w.parts;
    int64_t prefix_entries = 0;
    if (shared && !w.whole) {
        const int shared_tokens = max_shared_len / block_size * block_size;
        const int64_t rows = static_cast<int64_t>(max_group_size) * w.G;
        w.prefix_tc = rows > kSharedSplitRows && block_size <= pa::kSharedTile && (block_size & (block_size - 1)) == 0;
        if (w.prefix_tc) {
            w.prefix_paired = rows > pa::kSharedTile;
            w.prefix_per = w.prefix_paired ? 2 : 1;
            const int per = w.prefix_per * pa::kSharedTile;
            w.prefix_tiles = static_cast<int>((rows + per - 1) / per);
            w.prefix_part = shared_unit(w.groups * w.prefix_tiles * num_kv_heads, shared_tokens, w.prefix_paired, w.groups > 1);
        }
        w.prefix_cols = w.G;
        while (w.prefix_cols < 8 && w.prefix_cols < static_cast<int64_t>(max_group_size) * w.G) w.prefix_cols *= 2;
        const int chunk_seqs = w.prefix_cols / w.G;
        const int64_t chunks = (static_cast<int64_t>(max_group_size) + chunk_seqs - 1) / chunk_seqs;
        if (!w.prefix_tc) {
            prefix_entries = num_groups * chunks;
            w.prefix_part = split_partition(w.groups * chunks * ngroups, ngroups, max_shared_len, block_size, slot_tokens, 0);
        }
        w.prefix_parts = (shared_tokens + w.prefix_part - 1) / w.prefix_part * w.prefix_per;
        w.max_parts += w.prefix_parts;
    }
    if ((!shared || w.whole) && w.max_parts <= 1) return true;
    // Rows of (reference, sum, weighted sum): one per partial, and for cut items
    // one per launch, CTA and head of its box.
    w.max_shares = cache == pa::kCacheInt4 ? 2 * pa::kSplitMaxCtas : pa::kSplitMaxCtas;
    const int64_t per_launch = static_cast<int64_t>(w.max_shares) << w.log2_heads;
    w.cut_row = static_cast<int64_t>(num_seqs) * num_heads * w.max_parts;
    w.prefix_cut_row = w.cut_row + (num_seqs + kSplitEntries - 1) / kSplitEntries * per_launch * w.G;
    w.rows = w.prefix_cut_row +
             (prefix_entries + kSplitEntries - 1) / kSplitEntries * per_launch * w.prefix_cols;
    w.acc_off = static_cast<size_t>(round_up(w.rows * 4 * 4, 256));
    w.bytes = w.acc_off + static_cast<size_t>(w.rows) * head_dim * 4;
    return true;
}

// Tensor map over a cache [NB * bs, Hkv, D] taken as (dim, token, head): boxes
// of min(128 bytes, row) x min(16, bs) tokens x `heads` heads, swizzled by the
// box row's width.
bool encode_split_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int block_size, int num_kv_heads,
                      int head_dim, int es, int heads) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const int row = std::min(128, head_dim * es);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(num_blocks) * block_size,
                                static_cast<cuuint64_t>(num_kv_heads)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(num_kv_heads) * head_dim * es,
                                   static_cast<cuuint64_t>(head_dim) * es};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(row / es), static_cast<cuuint32_t>(std::min(block_size, 16)),
                               static_cast<cuuint32_t>(heads)};
    const cuuint32_t estr[3] = {1u, 1u, 1u};
    return fn(map, es == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
              const_cast<void *>(cache), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              row == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
              : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                          : CU_TENSOR_MAP_SWIZZLE_32B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over scales [NB * bs, Hkv] (32-bit), boxes of `heads` heads x
// min(16, bs) tokens.
bool encode_scale_map(CUtensorMap *map, const float *scales, int64_t num_blocks, int block_size, int num_kv_heads,
                      int heads) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(num_kv_heads), static_cast<cuuint64_t>(num_blocks) * block_size};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(num_kv_heads) * 4};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(std::min(block_size, 16))};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float *>(scales), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Tensor map over the scale words [NB, Hkv, bs, groups] of a 4-bit cache taken as
// (token and group, block and head), boxes of min(16, bs) tokens x `heads` heads.
bool encode_word_map(CUtensorMap *map, const void *words, int64_t num_blocks, int block_size, int num_kv_heads,
                     int groups, int heads) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(block_size) * groups,
                                static_cast<cuuint64_t>(num_blocks) * num_kv_heads};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(block_size) * groups * 4};
    const cuuint32_t box[2] = {static_cast<cuuint32_t>(std::min(block_size, 16) * groups), static_cast<cuuint32_t>(heads)};
    const cuuint32_t estr[2] = {1u, 1u};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void *>(words), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One pass of the split kernel over `entries` entries (p.mode says which).
pa_status run_split(pa::SplitParams p, int cache, int head_dim, int cols, int entries, int max_len,
                    const pa::SplitMaps &maps, const DeviceInfo &dev, cudaStream_t stream) {
    const int64_t per_entry = static_cast<int64_t>(p.num_kv_heads >> p.log2_heads) *
                              std::max<int64_t>(1, (static_cast<int64_t>(max_len) + p.partition_size - 1) / p.partition_size);
    for (int64_t e = 0; e < entries; e += kSplitEntries) {
        p.e0 = static_cast<int>(e);
        p.entries = static_cast<int>(std::min<int64_t>(kSplitEntries, entries - e));
        const pa::SplitSmem need = pa::split_smem(head_dim, cols, cache, p.log2_heads, p.entries);
        const size_t room = static_cast<size_t>(dev.smem_optin);
        if (need.fixed + 2 * need.slot > room) return PA_ERR_UNSUPPORTED;
        p.stages = static_cast<int>(std::min<size_t>(8, (room - need.fixed) / need.slot));
        const size_t smem = need.fixed + p.stages * need.slot;
        const int grid = static_cast<int>(std::min<int64_t>(std::min(dev.sms, pa::kSplitMaxCtas), p.entries * per_entry));
        p.part_div = pa::divisor(p.partition_size);
        p.block_div = pa::divisor(p.block_size);
        p.share_div = pa::divisor(grid * pa::split_teams(cols, cache));
        auto launch = cache == pa::kCacheF16    ? pa::launch_split_f16
                      : cache == pa::kCacheBF16 ? pa::launch_split_bf16
                      : cache == pa::kCacheE4M3 ? pa::launch_split_e4m3
                      : cache == pa::kCacheInt8 ? pa::launch_split_int8
                                                : pa::launch_split_int4;
        if (launch(p, head_dim, cols, maps, grid, smem, stream) != cudaSuccess) return PA_ERR_CUDA;
    }
    return PA_OK;
}

// Checks shared by pa_quant_decode and pa_decode_shared; PA_OK lets them go on.
pa_status check_split(pa_dtype out_dtype, pa_dtype q_dtype, int max_blocks_per_seq, int max_context_len, int num_seqs,
                      int num_heads, int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale) {
    if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
        max_blocks_per_seq <= 0 || max_context_len < 0)
        return PA_ERR_INVALID_ARG;
    if (!half_dtype(q_dtype) || !out_dtype_ok(out_dtype)) return PA_ERR_INVALID_ARG;
    if (num_heads % num_kv_heads != 0) return PA_ERR_INVALID_ARG;
    if (!split_shape_ok(num_heads, num_kv_heads, head_dim, block_size)) return PA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(max_context_len) > static_cast<int64_t>(max_blocks_per_seq) * block_size)
        return PA_ERR_INVALID_ARG;
    if (num_blocks > INT32_MAX / block_size || num_seqs >= (1 << 27) || max_context_len > (1 << 30))
        return PA_ERR_UNSUPPORTED;
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return PA_ERR_INVALID_ARG;
    // Work is counted in 16-token stages in 32-bit arithmetic on the device,
    // and one join warp per output row.
    const int64_t stages = static_cast<int64_t>(num_kv_heads) * (max_context_len / 16 + 1);
    if (stages * std::min(num_seqs, kSplitEntries) >= (int64_t{1} << 31) ||
        static_cast<int64_t>(num_seqs) * num_heads >= (int64_t{1} << 31))
        return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

pa::SplitParams split_params(void *out, pa_dtype out_dtype, const void *query, pa_dtype q_dtype,
                             const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                             int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int block_size,
                             int64_t num_blocks, float scale, const SplitPlan &w, void *workspace, int *err_flag) {
    pa::SplitParams p{};
    p.out = out;
    p.out_dtype = static_cast<int>(out_dtype);
    p.q = static_cast<const uint16_t *>(query);
    p.q_bf16 = q_dtype == PA_BF16;
    p.block_tables = block_tables;
    p.context_lens = context_lens;
    p.max_blocks_per_seq = max_blocks_per_seq;
    p.max_context_len = max_context_len;
    p.num_seqs = num_seqs;
    p.num_heads = num_heads;
    p.num_kv_heads = num_kv_heads;
    while ((1 << p.log2_group) < w.G) ++p.log2_group;
    p.block_size = block_size;
    p.num_blocks = num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.partition_size = w.partition;
    p.max_parts = w.max_parts;
    if (w.bytes) {
        p.ws_ml = static_cast<float *>(workspace);
        p.ws_acc = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + w.acc_off);
        p.cut_row = w.cut_row;
        p.prefix_cut_row = w.prefix_cut_row;
        p.cut_rows = static_cast<uint32_t>(w.prefix_cut_row - w.cut_row);
        p.prefix_cut_rows = static_cast<uint32_t>(w.rows - w.prefix_cut_row);
        p.cut_cols = w.G;
        p.max_shares = w.max_shares;
        p.cut = 1;
    }
    p.err_flag = err_flag;
    p.log2_heads = w.log2_heads;
    return p;
}

}  // namespace

namespace {

// The quantised calls for any codes; `cache` is the codes' kCache value, scales float
// per row or, for 4-bit codes, words per group.
bool quant_slots_ok(int cache, int64_t num_blocks, int block_size, int num_kv_heads) {
    if (cache != pa::kCacheInt4) return true;
    return num_blocks <= INT32_MAX / block_size && num_blocks <= INT32_MAX / num_kv_heads;
}

pa_status quant_write(const void *key, const void *value, int64_t key_stride, int64_t value_stride, void *k_cache,
                      void *v_cache, void *k_scales, void *v_scales, const int64_t *slot_mapping, int64_t num_tokens,
                      int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, pa_dtype dtype, int cache,
                      int *err_flag, void *stream) {
    if (num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 || !half_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || num_kv_heads > (1 << 20) ||
        !quant_slots_ok(cache, num_blocks, block_size, num_kv_heads))
        return PA_ERR_UNSUPPORTED;
    const int64_t row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (key_stride < row || value_stride < row || key_stride % 8 != 0 || value_stride % 8 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!key || !value || !k_cache || !v_cache || !k_scales || !v_scales || !slot_mapping) return PA_ERR_INVALID_ARG;
    if (!aligned16(key) || !aligned16(value) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) ||
        !aligned16(v_scales))
        return PA_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return PA_ERR_CUDA;
    const cudaError_t e = pa::launch_quant_write(
        key, value, key_stride, value_stride, k_cache, v_cache, static_cast<float *>(k_scales),
        static_cast<float *>(v_scales), slot_mapping, num_tokens, num_blocks * block_size, block_size, num_kv_heads,
        head_dim, dtype == PA_BF16, cache, dev.sms, err_flag, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status quant_gather(void *out_k, void *out_v, pa_dtype out_dtype, const void *k_cache, const void *v_cache, int cache,
                       const void *k_scales, const void *v_scales, const int32_t *block_tables, int max_blocks_per_seq,
                       const int32_t *cu_seqlens, const int32_t *seq_starts, int num_seqs, int64_t num_tokens,
                       int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, int *err_flag, void *stream) {
    if (num_seqs < 0 || num_tokens < 0 || num_blocks <= 0 || block_size <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
        max_blocks_per_seq <= 0 || !out_dtype_ok(out_dtype))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || num_kv_heads > (1 << 20) || num_tokens > INT32_MAX ||
        !quant_slots_ok(cache, num_blocks, block_size, num_kv_heads))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!out_k || !out_v || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !cu_seqlens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out_k) || !aligned16(out_v) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) ||
        !aligned16(v_scales))
        return PA_ERR_INVALID_ARG;
    const cudaError_t e = pa::launch_quant_gather(
        out_k, out_v, static_cast<int>(out_dtype), k_cache, v_cache, cache, static_cast<const float *>(k_scales),
        static_cast<const float *>(v_scales), block_tables, max_blocks_per_seq, cu_seqlens, seq_starts, num_seqs,
        num_tokens, num_kv_heads, head_dim, block_size, num_blocks, err_flag, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

size_t quant_workspace(int cache, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                       int max_context_len, int partition_size) {
    SplitPlan w;
    if (!plan_split(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, partition_size, cache,
                    false, 0, 0, 0, w))
        return static_cast<size_t>(-1);
    return w.bytes;
}

pa_status quant_decode(void *out, pa_dtype out_dtype, const void *query, pa_dtype q_dtype, const void *k_cache,
                       const void *v_cache, int cache, const float *k_scales, const float *v_scales,
                       const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                       int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                       int64_t num_blocks, float scale, int partition_size, void *workspace, size_t workspace_bytes,
                       int *err_flag, void *stream) {
    const pa_status st = check_split(out_dtype, q_dtype, max_blocks_per_seq, max_context_len, num_seqs, num_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, scale);
    if (st != PA_OK) return st;
    if (!quant_slots_ok(cache, num_blocks, block_size, num_kv_heads)) return PA_ERR_UNSUPPORTED;
    // 4-bit caches: an item weighs one unit more than its slots
    if (cache == pa::kCacheInt4 && static_cast<int64_t>(num_kv_heads) * (max_context_len / 16 + 1) *
                                           std::min(num_seqs, kSplitEntries) >= (int64_t{1} << 30))     // (so that their sum stays below 2^31)
        return PA_ERR_UNSUPPORTED;
    SplitPlan w;
    if (!plan_split(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, partition_size, cache,
                    false, 0, 0, 0, w))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !k_scales || !v_scales || !block_tables || !context_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scales) ||
        !aligned16(v_scales))
        return PA_ERR_INVALID_ARG;
    if (w.bytes > 0 && (workspace == nullptr || workspace_bytes < w.bytes || !aligned16(workspace)))
        return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    if (!device_info(dev)) return PA_ERR_CUDA;
    const int box_heads = 1 << w.log2_heads;
    const bool four = cache == pa::kCacheInt4;
    // 4-bit rows: as many heads to a row of the boxes as make up 128 bytes
    const int side = four ? std::min(box_heads, 256 / head_dim) : 1;
    const int row = four ? side * head_dim / 2 : head_dim, groups = head_dim / 64;
    pa::SplitMaps maps{};
    if (!encode_split_map(&maps.k, k_cache, num_blocks, block_size, num_kv_heads / side, row, 1, box_heads / side) ||
        !encode_split_map(&maps.v, v_cache, num_blocks, block_size, num_kv_heads / side, row, 1, box_heads / side))
        return PA_ERR_CUDA;
    // where the kernel takes scales as boxes (pa_split_kernel.cuh)
    if (four && std::min(block_size, 16) * groups * 4 * box_heads >= 128 &&
        (!encode_word_map(&maps.ks, k_scales, num_blocks, block_size, num_kv_heads, groups, box_heads) ||
         !encode_word_map(&maps.vs, v_scales, num_blocks, block_size, num_kv_heads, groups, box_heads)))
        return PA_ERR_CUDA;
    if (!four && box_heads >= 4 &&
        (!encode_scale_map(&maps.ks, k_scales, num_blocks, block_size, num_kv_heads, box_heads) ||
         !encode_scale_map(&maps.vs, v_scales, num_blocks, block_size, num_kv_heads, box_heads)))
        return PA_ERR_CUDA;
    pa::SplitParams p = split_params(out, out_dtype, query, q_dtype, block_tables, max_blocks_per_seq, context_lens,
                                     max_context_len, num_seqs, num_heads, num_kv_heads, block_size, num_blocks, scale,
                                     w, workspace, err_flag);
    p.k_scales = k_scales;
    p.v_scales = v_scales;
    p.mode = pa::kSplitDecode;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    const pa_status r = run_split(p, cache, head_dim, w.G, num_seqs, max_context_len, maps, dev, s);
    if (r != PA_OK || w.max_parts <= 1) return r;
    return pa::launch_split_merge(p, head_dim, 1, 1, false, dev.sms, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace

PA_EXPORT pa_status pa_quant_reshape_and_cache(const void *key, const void *value, int64_t key_stride,
                                               int64_t value_stride, void *k_cache, void *v_cache, float *k_scales,
                                               float *v_scales, const int64_t *slot_mapping, int64_t num_tokens,
                                               int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                                               pa_dtype dtype, pa_dtype cache_dtype, int *err_flag, void *stream) {
    if (!quant_dtype(cache_dtype)) return PA_ERR_INVALID_ARG;
    return quant_write(key, value, key_stride, value_stride, k_cache, v_cache, k_scales, v_scales, slot_mapping,
                       num_tokens, num_blocks, block_size, num_kv_heads, head_dim, dtype, split_cache(cache_dtype),
                       err_flag, stream);
}

PA_EXPORT pa_status pa_quant_gather(void *out_k, void *out_v, pa_dtype out_dtype, const void *k_cache,
                                    const void *v_cache, pa_dtype cache_dtype, const float *k_scales,
                                    const float *v_scales, const int32_t *block_tables, int max_blocks_per_seq,
                                    const int32_t *cu_seqlens, const int32_t *seq_starts, int num_seqs,
                                    int64_t num_tokens, int num_kv_heads, int head_dim, int block_size,
                                    int64_t num_blocks, int *err_flag, void *stream) {
    if (!quant_dtype(cache_dtype)) return PA_ERR_INVALID_ARG;
    return quant_gather(out_k, out_v, out_dtype, k_cache, v_cache, split_cache(cache_dtype), k_scales, v_scales,
                        block_tables, max_blocks_per_seq, cu_seqlens, seq_starts, num_seqs, num_tokens, num_kv_heads,
                        head_dim, block_size, num_blocks, err_flag, stream);
}

PA_EXPORT size_t pa_quant_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                                int block_size, int max_context_len, int partition_size) {
    return quant_workspace(pa::kCacheInt8, num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                           partition_size);
}

PA_EXPORT pa_status pa_quant_decode(void *out, pa_dtype out_dtype, const void *query, pa_dtype q_dtype,
                                    const void *k_cache, const void *v_cache, pa_dtype cache_dtype,
                                    const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                    int max_blocks_per_seq, const int32_t *context_lens, int max_context_len,
                                    int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                    int64_t num_blocks, float scale, int partition_size, void *workspace,
                                    size_t workspace_bytes, int *err_flag, void *stream) {
    if (!quant_dtype(cache_dtype)) return PA_ERR_INVALID_ARG;
    return quant_decode(out, out_dtype, query, q_dtype, k_cache, v_cache, split_cache(cache_dtype), k_scales, v_scales,
                        block_tables, max_blocks_per_seq, context_lens, max_context_len, num_seqs, num_heads,
                        num_kv_heads, head_dim, block_size, num_blocks, scale, partition_size, workspace,
                        workspace_bytes, err_flag, stream);
}

PA_EXPORT pa_status pa_int4_reshape_and_cache(const void *key, const void *value, int64_t key_stride,
                                              int64_t value_stride, void *k_cache, void *v_cache, void *k_scales,
                                              void *v_scales, const int64_t *slot_mapping, int64_t num_tokens,
                                              int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                                              pa_dtype dtype, int *err_flag, void *stream) {
    return quant_write(key, value, key_stride, value_stride, k_cache, v_cache, k_scales, v_scales, slot_mapping,
                       num_tokens, num_blocks, block_size, num_kv_heads, head_dim, dtype, pa::kCacheInt4, err_flag,
                       stream);
}

PA_EXPORT pa_status pa_int4_gather(void *out_k, void *out_v, pa_dtype out_dtype, const void *k_cache,
                                   const void *v_cache, const void *k_scales, const void *v_scales,
                                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *cu_seqlens,
                                   const int32_t *seq_starts, int num_seqs, int64_t num_tokens, int num_kv_heads,
                                   int head_dim, int block_size, int64_t num_blocks, int *err_flag, void *stream) {
    return quant_gather(out_k, out_v, out_dtype, k_cache, v_cache, pa::kCacheInt4, k_scales, v_scales, block_tables,
                        max_blocks_per_seq, cu_seqlens, seq_starts, num_seqs, num_tokens, num_kv_heads, head_dim,
                        block_size, num_blocks, err_flag, stream);
}

PA_EXPORT size_t pa_int4_decode_workspace_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                               int block_size, int max_context_len, int partition_size) {
    return quant_workspace(pa::kCacheInt4, num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len,
                           partition_size);
}

PA_EXPORT pa_status pa_int4_decode(void *out, pa_dtype out_dtype, const void *query, pa_dtype q_dtype,
                                   const void *k_cache, const void *v_cache, const void *k_scales, const void *v_scales,
                                   const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                   int max_context_len, int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                   int block_size, int64_t num_blocks, float scale, int partition_size, void *workspace,
                                   size_t workspace_bytes, int *err_flag, void *stream) {
    return quant_decode(out, out_dtype, query, q_dtype, k_cache, v_cache, pa::kCacheInt4,
                        static_cast<const float *>(k_scales), static_cast<const float *>(v_scales), block_tables,
                        max_blocks_per_seq, context_lens, max_context_len, num_seqs, num_heads, num_kv_heads, head_dim,
                        block_size, num_blocks, scale, partition_size, workspace, workspace_bytes, err_flag, stream);
}

PA_EXPORT pa_status pa_update_tables(int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                     const int32_t *changes, int32_t *out_lens, int num_seqs, int32_t *free_blocks,
                                     int64_t free_capacity, const int32_t *free_count, int32_t *out_free_count,
                                     int64_t num_blocks, int block_size, int32_t *cu_seqlens, int64_t *slot_mapping,
                                     int64_t *positions, int64_t num_tokens, int *err_flag, void *stream) {
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || free_capacity < 0 || num_blocks <= 0 || block_size <= 0 || num_tokens < 0)
        return PA_ERR_INVALID_ARG;
    if (num_seqs > pa::kTablesMaxSeqs || static_cast<int64_t>(max_blocks_per_seq) * block_size > (1 << 30) ||
        num_tokens > (1 << 30) || free_capacity > (1 << 30) || num_blocks > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (!cu_seqlens || !free_count || !out_free_count) return PA_ERR_INVALID_ARG;
    if (num_seqs > 0 && (!block_tables || !context_lens || !changes || !out_lens)) return PA_ERR_INVALID_ARG;
    if ((num_tokens > 0 && (!slot_mapping || !positions)) || (free_capacity > 0 && !free_blocks)) return PA_ERR_INVALID_ARG;
    const pa::TablesParams p{block_tables, max_blocks_per_seq, context_lens,   changes,    out_lens,
                             num_seqs,     free_blocks,        free_capacity,  free_count, out_free_count,
                             num_blocks,   pa::divisor(block_size), cu_seqlens, slot_mapping, positions,
                             num_tokens,   err_flag};
    return pa::launch_update_tables(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

PA_EXPORT pa_status pa_rope_and_cache(void *out_q, const void *query, const void *key, const void *value, int64_t q_stride,
                                      int64_t key_stride, int64_t value_stride, void *k_cache, void *v_cache,
                                      pa_dtype cache_dtype, void *k_scales, void *v_scales, float k_scale, float v_scale,
                                      const int64_t *slot_mapping, const int64_t *positions, const double *inv_freq,
                                      int rot_dim, int interleaved, float factor, const void *q_weight,
                                      const void *k_weight, float eps, int64_t num_tokens, int num_heads,
                                      int num_kv_heads, int head_dim, pa_dtype dtype, int64_t num_blocks, int block_size,
                                      int *err_flag, void *stream) {
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_blocks <= 0 || block_size <= 0 ||
        !half_dtype(dtype))
        return PA_ERR_INVALID_ARG;
    if (!supported_head_dim(head_dim) || num_heads > (1 << 20) || num_kv_heads > (1 << 20) || num_tokens > INT32_MAX)
        return PA_ERR_UNSUPPORTED;
    if (rot_dim <= 0 || rot_dim > head_dim || rot_dim % 8 != 0) return PA_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !(factor == factor)) return PA_ERR_INVALID_ARG;
    // what the cache holds
    int kind;
    const bool scales = k_scales != nullptr && v_scales != nullptr;
    if (cache_dtype == dtype) {
        kind = pa::kRopeHalf;
    } else if (cache_dtype == PA_FP8_E4M3 && !k_scales && !v_scales) {
        if (!scale_ok(k_scale) || !scale_ok(v_scale)) return PA_ERR_INVALID_ARG;
        kind = pa::kRopeE4M3;
    } else if (quant_dtype(cache_dtype) || cache_dtype == PA_INT4) {
        if (num_tokens > 0 && !scales) return PA_ERR_INVALID_ARG;
        kind = cache_dtype == PA_INT4 ? pa::kRopeInt4 : cache_dtype == PA_INT8 ? pa::kRopeInt8 : pa::kRopeRows;
        if (kind == pa::kRopeInt4 && !quant_slots_ok(pa::kCacheInt4, num_blocks, block_size, num_kv_heads))
            return PA_ERR_UNSUPPORTED;
    } else {
        return half_dtype(cache_dtype) ? PA_ERR_UNSUPPORTED : PA_ERR_INVALID_ARG;
    }
    const int64_t q_row = static_cast<int64_t>(num_heads) * head_dim, kv_row = static_cast<int64_t>(num_kv_heads) * head_dim;
    if (q_stride < q_row || key_stride < kv_row || value_stride < kv_row || q_stride % 8 != 0 || key_stride % 8 != 0 ||
        value_stride % 8 != 0)
        return PA_ERR_INVALID_ARG;
    if (num_tokens == 0) return PA_OK;
    if (!out_q || !query || !key || !value || !k_cache || !v_cache || !slot_mapping || !positions || !inv_freq)
        return PA_ERR_INVALID_ARG;
    for (const void *x : {static_cast<const void *>(out_q), query, key, value, static_cast<const void *>(k_cache),
                          static_cast<const void *>(v_cache), q_weight, k_weight, static_cast<const void *>(k_scales),
                          static_cast<const void *>(v_scales)})
        if (!aligned16(x)) return PA_ERR_INVALID_ARG;
    if (out_q == query && q_stride != q_row) return PA_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!device_info(dev)) return PA_ERR_CUDA;
    pa::RopeParams p{};
    p.src[0] = static_cast<const uint16_t *>(query);
    p.src[1] = static_cast<const uint16_t *>(key);
    p.src[2] = static_cast<const uint16_t *>(value);
    p.stride[0] = q_stride;
    p.stride[1] = key_stride;
    p.stride[2] = value_stride;
    p.out_q = static_cast<uint16_t *>(out_q);
    p.cache[0] = k_cache;
    p.cache[1] = v_cache;
    p.scales[0] = k_scales;
    p.scales[1] = v_scales;
    p.scale[0] = k_scale;
    p.scale[1] = v_scale;
    p.slots = slot_mapping;
    p.positions = positions;
    p.inv_freq = inv_freq;
    p.weight[0] = static_cast<const uint16_t *>(q_weight);
    p.weight[1] = static_cast<const uint16_t *>(k_weight);
    p.eps = eps;
    p.factor = factor;
    p.num_tokens = num_tokens;
    p.hq = num_heads;
    p.hkv = num_kv_heads;
    p.rot = rot_dim;
    p.interleaved = interleaved != 0;
    p.num_slots = num_blocks * block_size;
    p.bs = block_size;
    p.err_flag = err_flag;
    return pa::launch_rope_and_cache(p, head_dim, dtype == PA_BF16, kind, dev.sms, static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

PA_EXPORT size_t pa_decode_shared_workspace_size(int num_seqs, int num_groups, int max_group_size, int num_heads,
                                                 int num_kv_heads, int head_dim, int block_size, int max_context_len,
                                                 int max_shared_len, int partition_size) {
    SplitPlan w;
    if (!plan_split(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, partition_size,
                    pa::kCacheF16, true, num_groups, max_group_size, max_shared_len, w))
        return static_cast<size_t>(-1);
    return w.bytes;
}

PA_EXPORT pa_status pa_decode_shared(void *out, pa_dtype out_dtype, const void *query, const void *k_cache,
                                     const void *v_cache, pa_dtype kv_dtype, const int32_t *block_tables,
                                     int max_blocks_per_seq, const int32_t *context_lens, int max_context_len,
                                     const int32_t *cu_groups, int num_groups, int max_group_size,
                                     const int32_t *shared_lens, int max_shared_len, int num_seqs, int num_heads,
                                     int num_kv_heads, int head_dim, int block_size, int64_t num_blocks, float scale,
                                     int partition_size, void *workspace, size_t workspace_bytes, int *err_flag,
                                     void *stream) {
    if (num_groups < 0 || max_group_size < 0 || max_shared_len < 0 || max_shared_len > max_context_len || !(scale >= 0.f))
        return PA_ERR_INVALID_ARG;
    const pa_status st = check_split(out_dtype, kv_dtype, max_blocks_per_seq, max_context_len, num_seqs, num_heads,
                                     num_kv_heads, head_dim, block_size, num_blocks, scale);
    if (st != PA_OK) return st;
    if (static_cast<int64_t>(num_groups) * max_group_size < num_seqs) return PA_ERR_INVALID_ARG;
    const int cache = split_cache(kv_dtype);
    SplitPlan w;
    if (!plan_split(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_context_len, partition_size, cache,
                    true, num_groups, max_group_size, max_shared_len, w))
        return PA_ERR_INVALID_ARG;
    if (num_seqs == 0) return PA_OK;
    if (!out || !query || !k_cache || !v_cache || !block_tables || !context_lens || !cu_groups || !shared_lens)
        return PA_ERR_INVALID_ARG;
    if (!aligned16(out) || !aligned16(query) || !aligned16(k_cache) || !aligned16(v_cache)) return PA_ERR_INVALID_ARG;
    if (w.bytes > 0 && (workspace == nullptr || workspace_bytes < w.bytes || !aligned16(workspace)))
        return PA_ERR_WORKSPACE;
    DeviceInfo dev;
    if (!device_info(dev)) return PA_ERR_CUDA;
    pa::SplitMaps maps{};
    if (!encode_split_map(&maps.k, k_cache, num_blocks, block_size, num_kv_heads, head_dim, 2, 1 << w.log2_heads) ||
        !encode_split_map(&maps.v, v_cache, num_blocks, block_size, num_kv_heads, head_dim, 2, 1 << w.log2_heads))
        return PA_ERR_CUDA;
    pa::SplitParams p = split_params(out, out_dtype, query, kv_dtype, block_tables, max_blocks_per_seq, context_lens,
                                     max_context_len, num_seqs, num_heads, num_kv_heads, block_size, num_blocks, scale,
                                     w, workspace, err_flag);
    p.shared_lens = shared_lens;
    p.cu_groups = cu_groups;
    p.num_groups = num_groups;
    p.max_group_size = max_group_size;
    p.max_shared_len = max_shared_len;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (w.whole) {
        p.mode = pa::kSplitWhole;
        const pa_status r = run_split(p, cache, head_dim, w.G, num_seqs, max_context_len, maps, dev, s);
        if (r != PA_OK || w.max_parts <= 1) return r;
        return pa::launch_split_merge(p, head_dim, 1, 1, false, dev.sms, s) == cudaSuccess ? PA_OK : PA_ERR_CUDA;
    }
    if (w.prefix_parts > 0 && w.prefix_tc) {
        if (pa::shared_prefix_smem(head_dim) + 1024 > static_cast<size_t>(dev.smem_optin)) return PA_ERR_UNSUPPORTED;
        const int ranges = w.prefix_parts / w.prefix_per, tile_seqs = pa::kSharedTile / w.G;
        int64_t grid = w.groups * ranges * num_kv_heads * w.prefix_tiles;
        // at least a whole wave where there may be more units than planned for
        if (w.padded) grid = std::max(grid, kSmsTarget * (w.prefix_paired ? 1 : 2));
        if (grid >= (int64_t{1} << 31)) return PA_ERR_UNSUPPORTED;
        CUtensorMap tq, sk, sv;
        if (!encode_map_128b(&tq, query, 2, head_dim, num_heads, num_seqs, w.G, tile_seqs) ||
            !encode_map_128b(&sk, k_cache, 2, head_dim, num_kv_heads, num_blocks * block_size, 1, block_size) ||
            !encode_map_128b(&sv, v_cache, 2, head_dim, num_kv_heads, num_blocks * block_size, 1, block_size))
            return PA_ERR_CUDA;
        if (pa::launch_shared_prefix(p, head_dim, kv_dtype == PA_BF16, w.prefix_paired, static_cast<int>(grid), w.padded,
                                     w.prefix_tiles, w.prefix_part, ranges, tq, sk, sv, s) != cudaSuccess)
            return PA_ERR_CUDA;
    } else if (w.prefix_parts > 0) {
        pa::SplitParams pre = p;
        pre.mode = pa::kSplitPrefix;
        pre.cut_row = w.prefix_cut_row;
        pre.cut_cols = w.prefix_cols;
        pre.partition_size = w.prefix_part;
        pre.chunk_seqs = w.prefix_cols / w.G;
        pre.chunks = (std::min(max_group_size, num_seqs) + pre.chunk_seqs - 1) / pre.chunk_seqs;
        if (static_cast<int64_t>(num_groups) * pre.chunks >= (int64_t{1} << 31)) return PA_ERR_UNSUPPORTED;
        const pa_status r = run_split(pre, cache, head_dim, w.prefix_cols, num_groups * pre.chunks, max_shared_len,
                                      maps, dev, s);
        if (r != PA_OK) return r;
    }
    p.mode = pa::kSplitSuffix;
    p.part_off = w.prefix_parts;
    p.late_wait = w.prefix_parts > 0;
    const pa_status r = run_split(p, cache, head_dim, w.G, num_seqs, max_context_len, maps, dev, s);
    if (r != PA_OK) return r;
    return pa::launch_split_merge(p, head_dim, std::max(1, w.prefix_part), w.prefix_per,
                                  w.prefix_tc && w.prefix_paired, dev.sms, s) == cudaSuccess
               ? PA_OK
               : PA_ERR_CUDA;
}

PA_EXPORT pa_status pa_check_err_flag(int *err_flag, int clear, int *flag_out, void *stream) {
    if (err_flag == nullptr) return PA_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int host = 0;
    if (cudaMemcpyAsync(&host, err_flag, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return PA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return PA_ERR_CUDA;
    if (clear && cudaMemsetAsync(err_flag, 0, sizeof(int), s) != cudaSuccess) return PA_ERR_CUDA;
    if (flag_out) *flag_out = host;
    return host == 0 ? PA_OK : PA_ERR_DEVICE_BOUNDS;
}
