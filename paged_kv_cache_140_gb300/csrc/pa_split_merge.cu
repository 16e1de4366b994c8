// Joins the partial softmax states of the split decode kernels
// (pa_split_kernel.cuh) and of the shared-prefix kernel (pa_shared_prefix.cu):
//     M = max m_j,   out = sum_j 2^(m_j - M) acc_j / sum_j 2^(m_j - M) l_j,
// partials in index order, in 32 bits, rounded once to the output type.
//
// Bound by latency and by reading the partials, most of which the previous kernel
// left in L2.  A row (sequence, query head) is joined by 1 to 8 warps, as many as
// fill the GPU; a warp requests the states and rows of 4 partials at once, so that
// up to 4 partials cost one trip to memory after the lengths, and carries a
// running (M, l, acc) over further ones.
#include "pa_split_kernel.cuh"

namespace pa {

namespace {

constexpr int kBatch = 4;     // partials a warp loads at a time

template <int D>
__global__ void __launch_bounds__(256)
    split_merge_kernel(const __grid_constant__ SplitParams p, int prefix_part, int per_part, int wt) {
    constexpr int DPL = D / 32;
    __shared__ float red_o[8][D];
    __shared__ float2 red_ml[8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * (8 / wt) + warp / wt;
    const int sub = warp % wt;
    const bool row_ok = task < static_cast<int64_t>(p.num_seqs) * p.num_heads;
    const int s = row_ok ? static_cast<int>(task / p.num_heads) : 0;
    const int hq = row_ok ? static_cast<int>(task % p.num_heads) : 0;
    const int G = 1 << p.log2_group, d0 = lane * DPL;
    pdl_wait();
    int npre = 0, np = 0;
    if (row_ok) {
        const int ctx = context_of(p, s, false);
        int shared = 0;
        if (!final_mode(p.mode)) {
            shared = shared_blocks(p, s, ctx, false) * p.block_size;
            npre = (shared + prefix_part - 1) / prefix_part * per_part;
        }
        np = npre + (ctx - shared + p.partition_size - 1) / p.partition_size;
    }
    // A list of one partition has written its output unless it was cut; no other
    // row is final.  (No private part and no prefix: a zero row.)
    bool active = row_ok && (np > 0 || !final_mode(p.mode));
    float M = -INFINITY, l = 0.f, o[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) o[i] = 0.f;
    auto add = [&](float2 ml, const float (&v)[DPL]) {
        if (ml.x == -INFINITY && ml.y == 0.f) return;      // empty: its row may be anything
        const float mb = fmaxf(M, ml.x);
        const float al = M == -INFINITY ? 1.f : fast_exp2(M - mb);
        // (a state without a finite reference whose sum is no number counts fully)
        const float w = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - mb);
        M = mb;
        l = fmaf(ml.y, w, l * al);
#pragma unroll
        for (int i = 0; i < DPL; ++i) o[i] = fmaf(v[i], w, o[i] * al);
    };
    auto load_row = [&](int64_t r, float (&v)[DPL]) {
        const float *a = p.ws_acc + r * D + d0;
        if constexpr (DPL == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(a));
            v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
        } else {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(a));
            v[0] = x.x; v[1] = x.y;
        }
    };
    if (active) {
        const float4 *states = reinterpret_cast<const float4 *>(p.ws_ml);
        // partial j: workspace row slot(j) * G + head of the group
        const int64_t base = (static_cast<int64_t>(s) * p.num_kv_heads + (hq >> p.log2_group)) * p.max_parts;
        for (int j0 = sub * kBatch; active && j0 < np; j0 += wt * kBatch) {
            // states and rows are requested together
            float4 st[kBatch];
            float v[kBatch][DPL];
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                st[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
                for (int i = 0; i < DPL; ++i) v[u][i] = 0.f;
                const int j = j0 + u;
                if (j < np) {
                    const int64_t r = ((base + (j < npre ? j : p.part_off + j - npre)) << p.log2_group) + (hq & (G - 1));
                    st[u] = __ldcg(states + r);
                    load_row(r, v[u]);
                }
            }
#pragma unroll
            for (int u = 0; u < kBatch; ++u) {
                const int kind = __float_as_int(st[u].z);
                if (kind == kRowFinal) active = false;
                add(make_float2(st[u].x, st[u].y), v[u]);
                if (kind == kRowCut) {   // few: what a second CTA did of the item
                    const int64_t r = (j0 + u < npre ? p.prefix_cut_row : p.cut_row) + __float_as_int(st[u].w);
                    const float4 x = __ldcg(states + r);
                    float w[DPL];
                    load_row(r, w);
                    add(make_float2(x.x, x.y), w);
                }
            }
        }
        if (final_mode(p.mode) && np == 0) active = false;
    }
    if (wt > 1) {
#pragma unroll
        for (int i = 0; i < DPL; ++i) red_o[warp][d0 + i] = o[i];
        if (lane == 0) red_ml[warp] = make_float2(M, l);
        __syncthreads();
        if (sub != 0) return;
        float mb = M;
        for (int k = 1; k < wt; ++k) mb = fmaxf(mb, red_ml[warp + k].x);
        const float al = M == -INFINITY ? 1.f : fast_exp2(M - mb);
        l *= al;
#pragma unroll
        for (int i = 0; i < DPL; ++i) o[i] *= al;
        for (int k = 1; k < wt; ++k) {
            const float2 ml = red_ml[warp + k];
            const float w = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - mb);
            l = fmaf(ml.y, w, l);
#pragma unroll
            for (int i = 0; i < DPL; ++i) o[i] = fmaf(red_o[warp + k][d0 + i], w, o[i]);
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
    while (wt < 8 && rows * wt * 2 <= static_cast<int64_t>(sms) * 32 && p.max_parts > kBatch * wt) wt *= 2;
    const int64_t blocks = (rows + 8 / wt - 1) / (8 / wt);
    auto kern = head_dim == 128 ? split_merge_kernel<128> : split_merge_kernel<64>;
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p, prefix_part, per_part, wt);
}

}  // namespace pa
