// A step's bookkeeping on the GPU: block tables, lengths, slot map and positions
// from how many tokens each sequence gains or loses.
//
// With n_s the length of sequence s, c_s its change, n'_s = max(0, n_s + c_s) and
// b(n) = ceil(n / block_size): a sequence gives back its blocks b(n'_s) .. b(n_s) - 1
// or takes b(n'_s) - b(n_s) new ones.  The free blocks are a stack.  Numbering the
// R blocks that are given back by sequence and place, number j goes to cell
// count + R - 1 - j; numbering the N that are taken the same way, number k comes
// from cell count + R - 1 - k.  So what a step took, a step that undoes it puts back
// where it lay, and no order depends on timing.  Three prefix sums over the
// sequences (tokens, blocks taken, blocks given back) say everything else.
//
// Bound by latency: a handful of dependent trips to memory and the sums.  One
// cluster of CTAs, so that a barrier among them separates reading lengths and
// counts from writing them (outputs may be the inputs), and putting blocks onto
// the stack from taking them off it.  Every CTA computes all sums in shared memory
// (cheaper than handing them round); blocks are then taken by the warps alike, 32
// neighbours at a time, which find their sequences together.  The tokens' slots and
// positions follow from what this wrote: by the same CTA where there is one and few
// tokens, else by a second kernel on all SMs.
//
// Measured (GB300, in a graph): 4 sequences 2.8 us, 256 that gain 6,561 tokens 7.0, 4,096 that
// gain 54,240 14.7.  With the tokens on the cluster's 8 SMs too the last took 20 to 22.
#include "pa_decode_common.cuh"
#include "pa_device.cuh"
#include "pa_step_ops.h"

namespace pa {

namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kTableThreads = 1024;
constexpr int kFlagNoBlocks = 0x20;      // PA_FLAG_NO_BLOCKS

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
// Everything written before is seen by all of the cluster after.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The last i < n with at[i] <= k, for the k = k0 + lane of a warp (at[0] = 0, borders never
// fall): of k0 by 32 probes at a time, from there by the next 32 borders, one to a lane.
__device__ __forceinline__ int find(const int32_t *at, int n, int k0, int lane) {
    const int end = n, k = k0 + lane;
    int i = 0;
    while (n > 1) {
        const int step = (n + 31) >> 5;
        const bool le = lane * step < n && at[i + lane * step] <= k0;
        const int c = __popc(__ballot_sync(kFull, le)) - 1;
        i += c * step;
        n = min(step, n - c * step);
    }
    int r = i;
    for (int w = i + 1;; w += 32) {
        const int border = w + lane < end ? at[w + lane] : 0x7fffffff;
        int c = 0;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const int x = __shfl_sync(kFull, border, c + o - 1);
            if (x <= k) c += o;
        }
        const int last = __shfl_sync(kFull, border, 31);
        if (c == 31 && last <= k) c = 32;
        r += c;          // (0 where the border behind k was met before)
        if (!__any_sync(kFull, c == 32)) return r;
    }
}

// Slots and positions of the 32 tokens from t0 on, one to a lane, out of updated tables;
// `len_of(s)`: a sequence's new length.
template <typename Len>
__device__ __forceinline__ void token_slots(const TablesParams &p, const int32_t *cu, int tokens, int t0, int lane, Len len_of) {
    const int t = t0 + lane;
    int64_t slot = -1, pos = 0;
    if (t0 < tokens) {
        const int s = find(cu, p.num_seqs, t0, lane);
        if (t < tokens) {
            const int behind = (s + 1 < p.num_seqs ? cu[s + 1] : tokens) - t;      // tokens from t to the sequence's end
            const uint32_t at = static_cast<uint32_t>(len_of(s) - behind), blk = divided(at, p.block);
            const int32_t id = p.block_tables[static_cast<int64_t>(s) * p.max_blocks + blk];
            pos = at;
            if (id >= 0 && id < p.num_blocks)
                slot = static_cast<int64_t>(id) * p.block.by + (at - blk * p.block.by);
            else
                report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
        }
    }
    if (t < p.num_tokens) {
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

// kTokens: the new tokens' slots and positions too (one CTA).
template <bool kTokens>
__global__ void __launch_bounds__(kTableThreads) update_tables_kernel(const __grid_constant__ TablesParams p) {
    extern __shared__ int32_t smem[];
    __shared__ uint32_t warp_tot[3][32], sum_s[3], size_s[2];
    __shared__ int bad_s;
    const int B = p.num_seqs;
    // per sequence: its blocks before and after, and the sums before it
    int32_t *had_s = smem, *has_s = had_s + B, *cu = has_s + B, *need = cu + B, *back = need + B;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const uint32_t bs = p.block.by;
    const int32_t most = static_cast<int32_t>(p.max_blocks * bs);      // at most 2^30
    if (threadIdx.x == 0) bad_s = 0;
    if (threadIdx.x < 2) size_s[threadIdx.x] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int64_t count = *p.free_count;
    // ---- lengths and the three sums: each thread takes neighbouring sequences, all loads first.
    // No term passes 2^30; the sums are taken modulo 2^32, and once more without the terms' 14
    // lowest bits, which cannot overflow and tells of a sum that passes 2^31. ----
    constexpr int kPer = (kTablesMaxSeqs + kTableThreads - 1) / kTableThreads;
    const int per = (B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int i0 = static_cast<int>(threadIdx.x) * per;
    int32_t n32[kPer], c32[kPer];
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        n32[k] = c32[k] = 0;
        if (k < per && i0 + k < B) {
            n32[k] = p.lens[i0 + k];
            c32[k] = p.changes[i0 + k];
        }
    }
    uint32_t v[3] = {0, 0, 0}, incl[3], total[3];
    uint32_t size[2] = {0, 0};                 // of tokens gained and blocks given back (those taken are fewer than tokens)
    int bad = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        if (k >= per) break;
        const int32_t n = n32[k], c = c32[k];
        uint32_t had = 0, has = 0, gained = 0;
        if (n < 0 || n > most || c > most - n) {
            bad = 1;
        } else {
            had = divided(static_cast<uint32_t>(n) + bs - 1, p.block);
            has = divided(static_cast<uint32_t>(max(n + c, 0)) + bs - 1, p.block);
            gained = static_cast<uint32_t>(max(c, 0));
        }
        if (i0 + k < B) {
            had_s[i0 + k] = static_cast<int32_t>(had);
            has_s[i0 + k] = static_cast<int32_t>(has);
            cu[i0 + k] = static_cast<int32_t>(v[0]);          // (from this thread's first sequence on)
            need[i0 + k] = static_cast<int32_t>(v[1]);
            back[i0 + k] = static_cast<int32_t>(v[2]);
        }
        const uint32_t up = has > had ? has - had : 0u, down = had > has ? had - has : 0u;
        v[0] += gained;
        v[1] += up;
        v[2] += down;
        size[0] += gained >> 14;
        size[1] += down >> 14;
    }
    const bool busy = warp * 32 * per < B;     // (shuffles of warps without a sequence would only hold the others up)
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        incl[k] = v[k];
        if (busy)
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t x = __shfl_up_sync(kFull, incl[k], o);
                if (lane >= o) incl[k] += x;
            }
        if (lane == 31) warp_tot[k][warp] = incl[k];
    }
    if (busy) {
        size[0] = __reduce_add_sync(kFull, size[0]);
        size[1] = __reduce_add_sync(kFull, size[1]);
        if (lane < 2 && size[lane]) atomicAdd(&size_s[lane], size[lane]);
    }
    if (bad) bad_s = 1;
    __syncthreads();
    if (warp < 3) {                            // the warps' totals summed, a warp for each of the three
        const uint32_t w = lane < nw ? warp_tot[warp][lane] : 0u;
        uint32_t x = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kFull, x, o);
            if (lane >= o) x += y;
        }
        if (lane < nw) warp_tot[warp][lane] = x - w;
        if (lane == 31) sum_s[warp] = x;
    }
    __syncthreads();
    uint32_t base[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        base[k] = warp_tot[k][warp] + incl[k] - v[k];
        total[k] = sum_s[k];
    }
#pragma unroll
    for (int k = 0; k < kPer; ++k)
        if (k < per && i0 + k < B) {
            cu[i0 + k] += static_cast<int32_t>(base[0]);
            need[i0 + k] += static_cast<int32_t>(base[1]);
            back[i0 + k] += static_cast<int32_t>(base[2]);
        }
    // 2^17 terms' worth of 2^14, less what each of the terms may have lost
    const bool huge = max(size_s[0], size_s[1]) >= (1u << 17) - kTablesMaxSeqs;
    __syncthreads();
    const int64_t T = total[0], N = total[1], R = total[2], top = count + R;
    const bool bad_len = bad_s || huge || T > p.num_tokens;
    const bool bad_free = count < 0 || count > p.free_capacity || (!huge && (top > p.free_capacity || N > top));
    const bool refused = bad_len || bad_free;
    if (refused && rank == 0 && threadIdx.x == 0)
        report(p.err_flag, (bad_len ? 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */ : 0) | (bad_free ? kFlagNoBlocks : 0));
    if (ctas > 1) cluster_sync();       // all of it is read
    const int me = static_cast<int>(rank * blockDim.x + threadIdx.x), all = static_cast<int>(ctas * blockDim.x);
    const int me0 = me - lane;          // the first of my warp's
    // ---- blocks given back ----
    if (!refused && R > 0) {
        for (int64_t j0 = me0; j0 < R; j0 += all) {
            const int s = find(back, B, static_cast<int>(j0), lane);
            const int64_t j = j0 + lane;
            if (j < R) {
                const int32_t id = p.block_tables[static_cast<int64_t>(s) * p.max_blocks + has_s[s] + (j - back[s])];
                if (id < 0 || id >= p.num_blocks) report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
                p.free_blocks[top - 1 - j] = id;
            }
        }
        if (ctas > 1) cluster_sync(); else __syncthreads();
    }
    // ---- lengths, bounds, and blocks taken ----
    for (int i = me; i < B; i += all) {
        // (the old length and the change once more, each by the thread that writes the new one)
        const int32_t n = p.lens[i], c = p.changes[i];
        p.out_lens[i] = refused ? n : n + max(c, -n);
        p.cu_seqlens[i] = refused ? 0 : cu[i];
    }
    if (me == 0) {
        p.cu_seqlens[B] = refused ? 0 : static_cast<int32_t>(T);
        *p.out_free_count = static_cast<int32_t>(refused ? count : top - N);
    }
    if (!refused)
        for (int64_t k0 = me0; k0 < N; k0 += all) {
            const int s = find(need, B, static_cast<int>(k0), lane);
            const int64_t k = k0 + lane;
            if (k < N) {
                const int32_t id = p.free_blocks[top - 1 - k];
                if (id < 0 || id >= p.num_blocks) report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
                p.block_tables[static_cast<int64_t>(s) * p.max_blocks + had_s[s] + (k - need[s])] = id;
            }
        }
    if constexpr (kTokens) {
        __syncthreads();                // tables and lengths are written
        const int tokens = refused ? 0 : static_cast<int>(T);
        for (int t0 = me0; t0 < p.num_tokens; t0 += all)
            token_slots(p, cu, tokens, t0, lane, [&](int s) { return p.out_lens[s]; });
    }
}

// Slots and positions after update_tables_kernel<false>, 32 tokens to a warp.
__global__ void __launch_bounds__(256) token_slots_kernel(const __grid_constant__ TablesParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) - lane;
    if (t0 >= p.num_tokens) return;
    // (without sequences there is no bound to read but cu_seqlens[0], which is 0)
    token_slots(p, p.cu_seqlens, p.cu_seqlens[p.num_seqs], static_cast<int>(t0), lane, [&](int s) { return p.out_lens[s]; });
}

}  // namespace

cudaError_t launch_update_tables(const TablesParams &p, cudaStream_t stream) {
    const size_t smem = static_cast<size_t>(p.num_seqs) * 5 * sizeof(int32_t);
    // In a graph, us.  The tokens by the same CTA up to 2,048 of them, two rounds of its threads: 5.6
    // with 100 sequences and 989 tokens (by a kernel behind it 6.6), 11.8 with 1,000 and 1,689 (11.8); 128
    // and 2,702 7.3 (7.0), 256 and 7,725 11.3 (7.6).
    // One CTA up to as many sequences as it has threads: 1,024 of a token each 8.2 (a cluster of 8: 9.5),
    // 512 with 8,279 tokens 8.6 (9.0), though 1,000 with 15,680 11.0 (10.1); above it 8: 1,500 with
    // 2,428 tokens 11.4 (one CTA 14.2), 4,096 with 53,583 14.8 (31.1), though 2,048 of a token each 10.4 (9.9).
    // Fewer threads, whose barriers are shorter, for steps of up to 128 sequences and 256 tokens: 4
    // of a token each 2.9 (1,024 threads: 3.7), 128 4.2 (4.9), though 100 with 190 tokens and as many blocks
    // to move take 5.8 (5.4); with more tokens, 100 and 989, they take 9.5 (5.6).
    const bool fused = p.num_seqs <= kTableThreads && p.num_tokens <= 2 * kTableThreads;
    const unsigned ctas = p.num_seqs <= kTableThreads ? 1 : 8;
    const unsigned threads = fused && p.num_seqs <= 128 && p.num_tokens <= 256 ? 128 : kTableThreads;
    auto kernel = fused ? update_tables_kernel<true> : update_tables_kernel<false>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(kTablesMaxSeqs * 5 * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    if (e != cudaSuccess || fused || p.num_tokens == 0) return e;
    return decode_common::launch_pdl(token_slots_kernel, dim3(static_cast<unsigned>((p.num_tokens + 255) / 256)), dim3(256),
                                     0, stream, p);
}

}  // namespace pa
