// Joins the partial softmax states of the split decode kernels
// (pa_split_kernel.cuh) and of the shared-prefix kernel (pa_shared_prefix.cu):
//     M = max m_j,   out = sum_j 2^(m_j - M) acc_j / sum_j 2^(m_j - M) l_j,
// partials in index order, in 32 bits, rounded once to the output type.
//
// Bound by latency and by reading the partials, most of which the previous kernel
// left in L2.  A row (sequence, query head) is joined by 1 to 8 warps, as many as
// fill the GPU, each carrying a running (M, l, acc).  States and rows of 4 partials
// are requested together, so that up to 4 cost one trip to memory after the lengths.
// Where every second partial may be empty (pairs of query tiles, `holes`) a warp
// takes 32 states first and then the rows that hold something: 100 us against 102
// for one prompt before 256 sequences, but 143 against 142 where none is empty.
#include "pa_split_kernel.cuh"

namespace pa {

namespace {

constexpr int kBatch = 4;     // partials a warp loads at a time, states and rows
constexpr int kRows = 8;      // rows at a time where states were loaded before

template <int D, bool kHoles>
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
        auto row_of = [&](int j) -> int64_t {
            return ((base + (j < npre ? j : p.part_off + j - npre)) << p.log2_group) + (hq & (G - 1));
        };
        // what a second CTA did of a cut item: few
        auto add_cut = [&](float4 st, int j) {
            // (a row that no kernel wrote, after a reported error, may hold any index)
            const uint32_t at = __float_as_uint(st.w);
            if (__float_as_int(st.z) != kRowCut || at >= (j < npre ? p.prefix_cut_rows : p.cut_rows)) return;
            const int64_t r = (j < npre ? p.prefix_cut_row : p.cut_row) + at;
            const float4 x = __ldcg(states + r);
            float w[DPL];
            load_row(r, w);
            add(make_float2(x.x, x.y), w);
        };
        if constexpr (!kHoles) {
            for (int j0 = sub * kBatch; active && j0 < np; j0 += wt * kBatch) {
                // states and rows are requested together
                float4 st[kBatch];
                float v[kBatch][DPL];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    st[u] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < DPL; ++i) v[u][i] = 0.f;
                    if (j0 + u < np) {
                        st[u] = __ldcg(states + row_of(j0 + u));
                        load_row(row_of(j0 + u), v[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    if (__float_as_int(st[u].z) == kRowFinal) active = false;
                    add(make_float2(st[u].x, st[u].y), v[u]);
                    add_cut(st[u], j0 + u);
                }
            }
        } else {
            // the states of up to 32 first, one per lane, then the rows that hold something
            const int per = (np + wt - 1) / wt, end = min(np, (sub + 1) * per);
            for (int c0 = sub * per; c0 < end; c0 += 32) {
                float4 st = make_float4(-INFINITY, 0.f, 0.f, 0.f);
                if (c0 + lane < end) st = __ldcg(states + row_of(c0 + lane));
                // (an empty state that was cut still names the row of what follows it)
                uint32_t left = __ballot_sync(kFull, !(st.x == -INFINITY && st.y == 0.f) || __float_as_int(st.z) == kRowCut);
                while (left != 0) {
                    int at[kRows];
                    float v[kRows][DPL];
#pragma unroll
                    for (int u = 0; u < kRows; ++u) {
                        at[u] = left != 0 ? __ffs(left) - 1 : -1;
                        left &= left - 1;
                        if (at[u] >= 0) load_row(row_of(c0 + at[u]), v[u]);
                    }
#pragma unroll
                    for (int u = 0; u < kRows; ++u) {
                        if (at[u] < 0) break;
                        const float4 one = make_float4(__shfl_sync(kFull, st.x, at[u]), __shfl_sync(kFull, st.y, at[u]),
                                                       __shfl_sync(kFull, st.z, at[u]), __shfl_sync(kFull, st.w, at[u]));
                        add(make_float2(one.x, one.y), v[u]);
                        add_cut(one, c0 + at[u]);
                    }
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
    using L = SplitLayout<D, 1, CT>;         // (a state's size is by its rows; teams are told here)
    const int H = 1 << log2_heads, teams = split_teams(cols, CT);
    const int states = L::k4 && H < L::kWarps ? L::kWarps : L::kWarps - H;
    SplitSmem s;
    s.fixed = 1024 +
              teams * (static_cast<size_t>(kQueryRing) * cols * D * 2 * H + static_cast<size_t>(states) * cols * L::kStateBytes +
                       L::kWarps * 8 * sizeof(float2) + (2 * kQueryRing + 16) * 8) +
              32 * 4 + static_cast<size_t>(entries) * 12 + 16;
    s.slot = teams * (L::kSlotBytes + sizeof(SlotMeta) + 16);
    return s;
}

}  // namespace

SplitSmem split_smem(int head_dim, int cols, int cache, int log2_heads, int entries) {
    if (cache == kCacheInt4)
        return head_dim == 128 ? smem_for<128, kCacheInt4>(cols, log2_heads, entries)
                               : smem_for<64, kCacheInt4>(cols, log2_heads, entries);
    if (cache >= kCacheE4M3)
        return head_dim == 128 ? smem_for<128, kCacheInt8>(cols, log2_heads, entries)
                               : smem_for<64, kCacheInt8>(cols, log2_heads, entries);
    return head_dim == 128 ? smem_for<128, kCacheF16>(cols, log2_heads, entries)
                           : smem_for<64, kCacheF16>(cols, log2_heads, entries);
}

int split_teams(int cols, int cache) {
    if (cache != kCacheInt4) return 1;
    return cols == 8 ? SplitLayout<128, 8, kCacheInt4>::kTeams : SplitLayout<128, 1, kCacheInt4>::kTeams;
}

int split_slot_stages(int cache, int log2_heads) {
    return (cache == kCacheInt4   ? SplitLayout<128, 8, kCacheInt4>::kTiles
            : cache >= kCacheE4M3 ? SplitLayout<128, 8, kCacheInt8>::kTiles
                                  : SplitLayout<128, 8, kCacheF16>::kTiles) >>
           log2_heads;
}

cudaError_t launch_split_merge(const SplitParams &p, int head_dim, int prefix_part, int per_part, bool holes, int sms,
                               cudaStream_t stream) {
    const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_heads;
    // one warp per row, more while the rows leave warps idle and there is something to share out
    int wt = 1;
    while (wt < 8 && rows * wt * 2 <= static_cast<int64_t>(sms) * 32 && p.max_parts > kBatch * wt) wt *= 2;
    const int64_t blocks = (rows + 8 / wt - 1) / (8 / wt);
    auto kern = head_dim == 128 ? (holes ? split_merge_kernel<128, true> : split_merge_kernel<128, false>)
                                : (holes ? split_merge_kernel<64, true> : split_merge_kernel<64, false>);
    return launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, stream, p, prefix_part, per_part, wt);
}

}  // namespace pa
