// The quantised cache's write and read-back: 8-bit codes (e4m3 or int8) with
// one 32-bit scale per token and KV head.
//
// For a row x of D elements (one token, one KV head), in 32-bit arithmetic,
//     a = max(max |x_i|, 2^-60),  scale = a / qmax,  code_i = rn(x_i (qmax / a)),
// qmax = 448 (e4m3) or 127 (int8), rn to nearest with ties to even; the row
// stands for code_i * scale.  The floor on a keeps qmax / a finite and gives a
// row of zeros the codes 0.  A row that holds an infinity or NaN gets the
// scale NaN and codes 0, so that it reads back, and attends, as NaN.
//
// Both are data movement: per row, write reads 2 D bytes and writes D + 4,
// read-back reads D + 4 and writes 2 D (16-bit output).  A thread takes 16
// elements of a row (32 bytes of 16-bit values, 16 of codes), so that a row is
// D / 16 neighbouring lanes, whose maximum takes two or three shuffles and no
// shared memory; each thread has several rows in flight.
#include "pa_decode_common.cuh"
#include "pa_device.cuh"
#include "pa_split.h"

namespace pa {

namespace {

using decode_common::kFull;
using decode_common::launch_pdl;

constexpr float kAmaxFloor = 8.673617379884035e-19f;   // 2^-60
constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t vmax_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Four values -> four int8 codes.  v + 1.5 * 2^23 holds round(v) (nearest,
// ties to even) in its low bits for |v| < 2^22.
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
    constexpr float k = 12582912.f;
    const uint32_t ia = __float_as_uint(__fadd_rn(a, k)), ib = __float_as_uint(__fadd_rn(b, k));
    const uint32_t ic = __float_as_uint(__fadd_rn(c, k)), id = __float_as_uint(__fadd_rn(d, k));
    return __byte_perm(__byte_perm(ia, ib, 0x0040u), __byte_perm(ic, id, 0x0040u), 0x5410u);
}

// One 32-byte store (dst on a 32-byte boundary).
__device__ __forceinline__ void store32(void *dst, const uint32_t (&h)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(h[0]), "r"(h[1]), "r"(h[2]),
                 "r"(h[3]), "r"(h[4]), "r"(h[5]), "r"(h[6]), "r"(h[7])
                 : "memory");
}

struct QuantWrite {
    const uint16_t *src[2];      // key, value
    int64_t stride[2];           // elements between tokens
    uint8_t *codes[2];
    float *scales[2];
    const int64_t *slots;
    uint32_t rows;               // tokens * Hkv, per tensor
    uint32_t hkv;
    int64_t num_slots;
    int *err_flag;
};

// One row part (16 elements) per thread and step; U steps of a thread are
// loaded before the first is reduced.
template <int D, bool BF16, int CT, int U>
__global__ void __launch_bounds__(kThreads) quant_write_kernel(const __grid_constant__ QuantWrite p) {
    constexpr int LPR = D / 16;              // lanes per row
    constexpr int RPB = kThreads / LPR;      // rows per block and step
    constexpr float kMax = CT == kCacheE4M3 ? 448.f : 127.f;
    pdl_wait();
    pdl_launch_dependents();
    const int part = threadIdx.x % LPR;
    const uint32_t r0 = blockIdx.x * (RPB * U) + threadIdx.x / LPR;
    const int kv = blockIdx.y;
    uint4 a[U], b[U];
    int64_t slot[U];
    uint32_t head[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t r = r0 + u * RPB;
        slot[u] = -1;
        a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
        if (r >= p.rows) continue;
        const uint32_t tok = r / p.hkv;
        head[u] = r - tok * p.hkv;
        slot[u] = __ldg(p.slots + tok);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.src[kv] + static_cast<int64_t>(tok) * p.stride[kv] +
                                                           static_cast<int64_t>(head[u]) * D + part * 16);
        a[u] = __ldg(src);
        b[u] = __ldg(src + 1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t w[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
        uint32_t m2 = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m2 = vmax_u16x2(m2, w[i] & 0x7fff7fffu);
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) m2 = vmax_u16x2(m2, __shfl_xor_sync(kFull, m2, o));
        const uint32_t m = max(m2 & 0xffffu, m2 >> 16);   // the largest magnitude's bits
        const bool finite = m < (BF16 ? 0x7f80u : 0x7c00u);
        const float amax = fmaxf(finite ? Half2x<BF16>::to_float2(m).x : 0.f, kAmaxFloor);
        const float inv = __fdiv_rn(kMax, amax);
        uint32_t code[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = Half2x<BF16>::to_float2(w[2 * i]), y = Half2x<BF16>::to_float2(w[2 * i + 1]);
            const float v0 = __fmul_rn(x.x, inv), v1 = __fmul_rn(x.y, inv);
            const float v2 = __fmul_rn(y.x, inv), v3 = __fmul_rn(y.y, inv);
            if constexpr (CT == kCacheE4M3)
                code[i] = f32x2_to_e4m3x2(v0, v1) | (f32x2_to_e4m3x2(v2, v3) << 16);
            else
                code[i] = int8x4(v0, v1, v2, v3);
            if (!finite) code[i] = 0u;
        }
        if (slot[u] < 0) continue;
        if (slot[u] >= p.num_slots) {
            report(p.err_flag, 0x1 /* PA_FLAG_BAD_SLOT */);
            continue;
        }
        const int64_t row = slot[u] * p.hkv + head[u];
        *reinterpret_cast<uint4 *>(p.codes[kv] + row * D + part * 16) = make_uint4(code[0], code[1], code[2], code[3]);
        if (part == 0) p.scales[kv][row] = finite ? __fdiv_rn(amax, kMax) : __uint_as_float(0x7fc00000u);
    }
}

// ------------------------------------------------------------- read-back

constexpr int kGatherTokens = 8;      // dense rows per block
constexpr int kSmemSeqs = 1024;       // sequences whose bounds a block keeps in shared memory

struct QuantGather {
    void *out[2];
    const uint8_t *codes[2];
    const float *scales[2];
    const int32_t *tables;
    const int32_t *cu;
    const int32_t *starts;       // may be null
    int max_blocks;
    int num_seqs;
    int64_t num_tokens;
    int hkv;
    int bs;
    int64_t num_blocks;
    int wide_out;                // both outputs start on a 32-byte boundary
    int *err_flag;
};

// OUT: 0 f16, 1 bf16, 2 f32.
template <int D, int CT, int OUT>
__global__ void __launch_bounds__(kThreads) quant_gather_kernel(const __grid_constant__ QuantGather p) {
    constexpr int LPR = D / 16;
    __shared__ int64_t src_slot[kGatherTokens];   // >= 0: cache slot; -1: no such slot (zeros); -2: not a row
    __shared__ int32_t cu_s[kSmemSeqs + 1];
    pdl_wait();
    pdl_launch_dependents();
    const int B = p.num_seqs;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kGatherTokens;
    const bool in_smem = B <= kSmemSeqs;
    const bool tell = blockIdx.x == 0;
    for (int i = threadIdx.x; i <= B; i += blockDim.x) {
        if (!in_smem && !tell) break;
        const int32_t c = __ldg(p.cu + i);
        if (in_smem) cu_s[i] = c;
        // one block looks the bounds over: from 0, never falling, at most num_tokens
        if (tell && ((i == 0 && c != 0) || (i > 0 && c < __ldg(p.cu + i - 1)) || c < 0 ||
                     static_cast<int64_t>(c) > p.num_tokens))
            report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
    }
    __syncthreads();
    if (threadIdx.x < kGatherTokens) {
        const int64_t t = t0 + threadIdx.x;
        auto cu = [&](int i) -> int64_t { return in_smem ? cu_s[i] : __ldg(p.cu + i); };
        int64_t slot = -2;
        if (t < p.num_tokens && t < cu(B)) {
            int a = 0, b = B;                     // the last sequence that starts at or before t
            while (b - a > 1) {
                const int m = (a + b) >> 1;
                if (cu(m) <= t) a = m; else b = m;
            }
            if (cu(a) <= t && t < cu(a + 1)) {
                const int64_t pos = t - cu(a) + (p.starts != nullptr ? __ldg(p.starts + a) : 0);
                slot = -1;
                if (pos >= 0 && pos < static_cast<int64_t>(p.max_blocks) * p.bs) {
                    const int32_t id = __ldg(p.tables + static_cast<int64_t>(a) * p.max_blocks + pos / p.bs);
                    if (id >= 0 && static_cast<int64_t>(id) < p.num_blocks)
                        slot = static_cast<int64_t>(id) * p.bs + pos % p.bs;
                    else
                        report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
                } else {
                    report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
                }
            }
        }
        src_slot[threadIdx.x] = slot;
    }
    __syncthreads();
    // row parts of this block: (token, tensor, head, part), U in flight per thread
    const int per_tensor = p.hkv * LPR, per_tok = 2 * per_tensor;
    const int n = kGatherTokens * per_tok;
    constexpr int U = 4;
    for (int i0 = threadIdx.x; i0 < n; i0 += U * kThreads) {
        uint4 w[U];
        float sc[U];
        int64_t dst[U];
        int kv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kThreads;
            dst[u] = -1;
            if (i >= n) continue;
            const int tok = i / per_tok;
            const int64_t slot = src_slot[tok];
            if (slot == -2) continue;
            const int rem = i - tok * per_tok;
            kv[u] = rem >= per_tensor;
            const int off = rem - kv[u] * per_tensor;       // head * LPR + part
            dst[u] = (t0 + tok) * per_tensor + off;
            w[u] = make_uint4(0u, 0u, 0u, 0u);
            sc[u] = 0.f;
            if (slot >= 0) {
                w[u] = __ldcs(reinterpret_cast<const uint4 *>(p.codes[kv[u]]) + slot * per_tensor + off);
                sc[u] = __ldg(p.scales[kv[u]] + slot * p.hkv + off / LPR);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (dst[u] < 0) continue;
            const uint32_t c4[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
            float v[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (CT == kCacheE4M3) {
                    uint32_t lo, hi;
                    e4m3x4_to_f16x2x2(c4[k], lo, hi);
                    const float2 a = Half2x<false>::to_float2(lo), b = Half2x<false>::to_float2(hi);
                    v[4 * k] = a.x; v[4 * k + 1] = a.y; v[4 * k + 2] = b.x; v[4 * k + 3] = b.y;
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[4 * k + j] = static_cast<float>(static_cast<int8_t>(c4[k] >> (8 * j)));
                }
            }
            if constexpr (OUT == 2) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out[kv[u]]) + dst[u] * 16);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    __stcs(o + k, make_float4(v[4 * k] * sc[u], v[4 * k + 1] * sc[u], v[4 * k + 2] * sc[u],
                                              v[4 * k + 3] * sc[u]));
            } else {
                uint32_t h[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) h[k] = pack2<OUT == 1>(v[2 * k] * sc[u], v[2 * k + 1] * sc[u]);
                uint16_t *o = static_cast<uint16_t *>(p.out[kv[u]]) + dst[u] * 16;
                if (p.wide_out) {
                    store32(o, h);
                } else {
                    reinterpret_cast<uint4 *>(o)[0] = make_uint4(h[0], h[1], h[2], h[3]);
                    reinterpret_cast<uint4 *>(o)[1] = make_uint4(h[4], h[5], h[6], h[7]);
                }
            }
        }
    }
}

template <int D, bool BF16, int CT>
cudaError_t write_t(const QuantWrite &p, int sms, cudaStream_t stream) {
    constexpr int RPB = kThreads / (D / 16);
    // Four rows per thread once that still gives every SM 8 blocks.
    const uint32_t blocks4 = (p.rows + RPB * 4 - 1) / (RPB * 4);
    if (blocks4 * 2 >= static_cast<uint32_t>(8 * sms))
        return launch_pdl(quant_write_kernel<D, BF16, CT, 4>, dim3(blocks4, 2), dim3(kThreads), 0, stream, p);
    return launch_pdl(quant_write_kernel<D, BF16, CT, 1>, dim3((p.rows + RPB - 1) / RPB, 2), dim3(kThreads), 0, stream,
                      p);
}

template <int D>
cudaError_t write_d(const QuantWrite &p, bool bf16, int cache, int sms, cudaStream_t stream) {
    if (cache == kCacheE4M3)
        return bf16 ? write_t<D, true, kCacheE4M3>(p, sms, stream) : write_t<D, false, kCacheE4M3>(p, sms, stream);
    return bf16 ? write_t<D, true, kCacheInt8>(p, sms, stream) : write_t<D, false, kCacheInt8>(p, sms, stream);
}

template <int D, int CT>
cudaError_t gather_t(const QuantGather &p, int out_dtype, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((p.num_tokens + kGatherTokens - 1) / kGatherTokens));
    if (out_dtype == 0) return launch_pdl(quant_gather_kernel<D, CT, 0>, grid, dim3(kThreads), 0, stream, p);
    if (out_dtype == 1) return launch_pdl(quant_gather_kernel<D, CT, 1>, grid, dim3(kThreads), 0, stream, p);
    return launch_pdl(quant_gather_kernel<D, CT, 2>, grid, dim3(kThreads), 0, stream, p);
}

}  // namespace

cudaError_t launch_quant_write(const void *key, const void *value, int64_t key_stride, int64_t value_stride,
                               void *k_cache, void *v_cache, float *k_scales, float *v_scales,
                               const int64_t *slot_mapping, int64_t num_tokens, int64_t num_slots, int num_kv_heads,
                               int head_dim, bool bf16, int cache, int sms, int *err_flag, cudaStream_t stream) {
    // tokens per launch such that row indices stay below 2^30
    const int64_t most = (int64_t{1} << 30) / num_kv_heads;
    for (int64_t t = 0; t < num_tokens; t += most) {
        const int64_t n = num_tokens - t < most ? num_tokens - t : most;
        QuantWrite p;
        p.src[0] = static_cast<const uint16_t *>(key) + t * key_stride;
        p.src[1] = static_cast<const uint16_t *>(value) + t * value_stride;
        p.stride[0] = key_stride;
        p.stride[1] = value_stride;
        p.codes[0] = static_cast<uint8_t *>(k_cache);
        p.codes[1] = static_cast<uint8_t *>(v_cache);
        p.scales[0] = k_scales;
        p.scales[1] = v_scales;
        p.slots = slot_mapping + t;
        p.rows = static_cast<uint32_t>(n * num_kv_heads);
        p.hkv = static_cast<uint32_t>(num_kv_heads);
        p.num_slots = num_slots;
        p.err_flag = err_flag;
        const cudaError_t e =
            head_dim == 128 ? write_d<128>(p, bf16, cache, sms, stream) : write_d<64>(p, bf16, cache, sms, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t launch_quant_gather(void *out_k, void *out_v, int out_dtype, const void *k_cache, const void *v_cache,
                                int cache, const float *k_scales, const float *v_scales, const int32_t *block_tables,
                                int max_blocks_per_seq, const int32_t *cu_seqlens, const int32_t *seq_starts,
                                int num_seqs, int64_t num_tokens, int num_kv_heads, int head_dim, int block_size,
                                int64_t num_blocks, int *err_flag, cudaStream_t stream) {
    QuantGather p;
    p.out[0] = out_k;
    p.out[1] = out_v;
    p.codes[0] = static_cast<const uint8_t *>(k_cache);
    p.codes[1] = static_cast<const uint8_t *>(v_cache);
    p.scales[0] = k_scales;
    p.scales[1] = v_scales;
    p.tables = block_tables;
    p.cu = cu_seqlens;
    p.starts = seq_starts;
    p.max_blocks = max_blocks_per_seq;
    p.num_seqs = num_seqs;
    p.num_tokens = num_tokens;
    p.hkv = num_kv_heads;
    p.bs = block_size;
    p.num_blocks = num_blocks;
    p.wide_out = ((reinterpret_cast<uintptr_t>(out_k) | reinterpret_cast<uintptr_t>(out_v)) & 31u) == 0;
    p.err_flag = err_flag;
    if (head_dim == 128)
        return cache == kCacheE4M3 ? gather_t<128, kCacheE4M3>(p, out_dtype, stream)
                                   : gather_t<128, kCacheInt8>(p, out_dtype, stream);
    return cache == kCacheE4M3 ? gather_t<64, kCacheE4M3>(p, out_dtype, stream)
                               : gather_t<64, kCacheInt8>(p, out_dtype, stream);
}

}  // namespace pa
