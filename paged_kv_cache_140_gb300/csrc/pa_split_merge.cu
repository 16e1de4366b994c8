// Joins the partial softmax states of the split decode kernels
// (pa_split_kernel.cuh) and of the shared-prefix kernel (pa_shared_prefix.cu):
//     M = max m_j,   out = sum_j 2^(m_j - M) acc_j / sum_j 2^(m_j - M) l_j,
// partials in index order, in 32 bits, rounded once to the output type.
//
// Bound by reading the partials, most of which the previous kernel left in L2.
// A row (sequence, query head) is joined by 1 to 8 warps, as many as fill the
// GPU; each holds D / 32 columns per lane and has 8 partials in flight.
#include "pa_split_kernel.cuh"

namespace pa {

namespace {

template <int D>
__global__ void __launch_bounds__(256)
    split_merge_kernel(const __grid_constant__ SplitParams p, int prefix_part, int per_part, int wt) {
    constexpr int DPL = D / 32;
    __shared__ float red_o[8][D];
    __shared__ float red_l[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int G = 1 << p.log2_group;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * (8 / wt) + warp / wt;
    const int sub = warp % wt;
    pdl_wait();
    bool active = task < static_cast<int64_t>(p.num_seqs) * p.num_heads;
    int npre = 0, np = 0, s = 0, hq = 0;
    if (active) {
        s = static_cast<int>(task / p.num_heads);
        hq = static_cast<int>(task % p.num_heads);
        const int ctx = context_of(p, s, false);
        int shared = 0;
        if (p.mode != kSplitDecode) {
            shared = shared_blocks(p, s, ctx, false) * p.block_size;
            npre = (shared + prefix_part - 1) / prefix_part * per_part;
        }
        np = npre + (ctx - shared + p.partition_size - 1) / p.partition_size;
        active = np > 1 || p.mode != kSplitDecode;
    }
    const int d0 = lane * DPL;
    float l = 0.f, o[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) o[i] = 0.f;
    if (active) {
        // partial j: workspace row slot(j) * G + head of the group
        const int64_t base = (static_cast<int64_t>(s) * p.num_kv_heads + (hq >> p.log2_group)) * p.max_parts;
        auto row = [&](int j) -> int64_t {
            return ((base + (j < npre ? j : p.part_off + j - npre)) << p.log2_group) + (hq & (G - 1));
        };
        float mx = -INFINITY;
        for (int j = lane; j < np; j += 32) mx = fmaxf(mx, __ldcg(p.ws_ml + 2 * row(j)));
        const float M = warp_max(mx);
        const int per = (np + wt - 1) / wt;
        const int jb = min(np, sub * per), je = min(np, jb + per);
        for (int j0 = jb; j0 < je; j0 += 32) {
            float w = 0.f;
            if (j0 + lane < je) {
                const float2 ml = __ldcg(reinterpret_cast<const float2 *>(p.ws_ml + 2 * row(j0 + lane)));
                // An empty partial (nothing was added; its row need not exist) is passed
                // over; any other without a finite reference counts fully, its sum being
                // no number.
                if (ml.x == -INFINITY) {
                    w = ml.y == 0.f ? -1.f : 1.f;
                } else {
                    w = fast_exp2(ml.x - M);
                }
                l = fmaf(ml.y, w, l);
            }
            const int cnt = min(32, je - j0);
            for (int u0 = 0; u0 < cnt; u0 += 8) {
                float v[8][DPL], wj[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    wj[u] = __shfl_sync(kFull, w, (u0 + u) & 31);
#pragma unroll
                    for (int i = 0; i < DPL; ++i) v[u][i] = 0.f;
                    if (u0 + u < cnt && wj[u] >= 0.f) {
                        const float *a = p.ws_acc + row(j0 + u0 + u) * D + d0;
                        if constexpr (DPL == 4) {
                            const float4 x = __ldcg(reinterpret_cast<const float4 *>(a));
                            v[u][0] = x.x; v[u][1] = x.y; v[u][2] = x.z; v[u][3] = x.w;
                        } else {
                            const float2 x = __ldcg(reinterpret_cast<const float2 *>(a));
                            v[u][0] = x.x; v[u][1] = x.y;
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int i = 0; i < DPL; ++i) o[i] = fmaf(v[u][i], wj[u], o[i]);
            }
        }
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) l += __shfl_xor_sync(kFull, l, x);
    }
    if (wt > 1) {
#pragma unroll
        for (int i = 0; i < DPL; ++i) red_o[warp][d0 + i] = o[i];
        if (lane == 0) red_l[warp] = l;
        __syncthreads();
        if (sub != 0) return;
        for (int k = 1; k < wt; ++k) {
#pragma unroll
            for (int i = 0; i < DPL; ++i) o[i] += red_o[warp + k][d0 + i];
            l += red_l[warp + k];
        }
    }
    if (!active) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < DPL; ++i) o[i] *= inv;
    store_row<D>(p.out, p.out_dtype, (static_cast<int64_t>(s) * p.num_heads + hq) * D + d0, o);
}

template <int D, int CT>
SplitSmem smem_for(int cols, int log2_heads, int entries) {
    using L = SplitLayout<D, 1, CT>;
    const int H = 1 << log2_heads;
    SplitSmem s;
    s.fixed = 1024 + static_cast<size_t>(kQueryRing) * cols * D * 2 * H +
              static_cast<size_t>(L::kWarps - H) * cols * L::kStateBytes + L::kWarps * 8 * sizeof(float2) +
              (2 * kQueryRing + 16) * 8 + 32 * 4 + static_cast<size_t>(entries) * 12 + 16;
    s.slot = L::kSlotBytes + sizeof(SlotMeta) + 16;
    return s;
}

}  // namespace

SplitSmem split_smem(int head_dim, int cols, int cache, int log2_heads, int entries) {
    if (cache >= kCacheE4M3)
        return head_dim == 128 ? smem_for<128, kCacheInt8>(cols, log2_heads, entries)
                               : smem_for<64, kCacheInt8>(cols, log2_heads, entries);
    return head_dim == 128 ? smem_for<128, kCacheF16>(cols, log2_heads, entries)
                           : smem_for<64, kCacheF16>(cols, log2_heads, entries);
}

int split_slot_stages(int cache, int log2_heads) {
    return (cache >= kCacheE4M3 ? SplitLayout<128, 8, kCacheInt8>::kTiles : SplitLayout<128, 8, kCacheF16>::kTiles) >>
           log2_heads;
}

cudaError_t launch_split_merge(const SplitParams &p, int head_dim, int prefix_part, int per_part, int sms,
                               cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_heads;
    // one warp per row, more while the rows leave warps idle and there is something to share out
    int wt = 1;
    while (wt < 8 && rows * wt * 2 <= static_cast<int64_t>(sms) * 16 && p.max_parts >= 8 * wt) wt *= 2;
    const int64_t blocks = (rows + 8 / wt - 1) / (8 / wt);
    auto kern = head_dim == 128 ? split_merge_kernel<128> : split_merge_kernel<64>;
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p, prefix_part, per_part, wt);
}

}  // namespace pa
