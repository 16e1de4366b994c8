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
// (cheaper than handing them round); items, blocks and tokens alike, are then taken
// by all threads alike and find their sequence by bisection.
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

__device__ __forceinline__ int64_t shfl_up64(int64_t v, int o) { return __shfl_up_sync(kFull, v, o); }

// The last i < n with at[i] <= k (at[0] = 0).
__device__ __forceinline__ int find(const int32_t *at, int n, int k) {
    int a = 0, b = n;
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (at[m] <= k) a = m; else b = m;
    }
    return a;
}

__global__ void __launch_bounds__(kTableThreads) update_tables_kernel(const __grid_constant__ TablesParams p) {
    extern __shared__ int32_t smem[];
    __shared__ int64_t warp_tot[3][32];
    __shared__ int bad_s;
    const int B = p.num_seqs;
    int32_t *old_s = smem, *new_s = old_s + B, *cu = new_s + B, *need = cu + B + 1, *back = need + B + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const uint32_t rank = cluster_rank(), ctas = cluster_size();
    const int64_t bs = p.block_size, most = static_cast<int64_t>(p.max_blocks) * bs;
    const uint32_t ubs = static_cast<uint32_t>(bs);
    if (threadIdx.x == 0) bad_s = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    const int64_t count = *p.free_count;
    // ---- lengths and the three sums (64 bits until they are known to be in range) ----
    int64_t total[3] = {0, 0, 0};
    int bad = 0;
    for (int b0 = 0; b0 < B; b0 += blockDim.x) {
        const int i = b0 + threadIdx.x;
        int64_t v[3] = {0, 0, 0};
        int64_t n = 0, m = 0;
        if (i < B) {
            n = p.lens[i];
            const int64_t c = p.changes[i];
            if (n < 0 || n > most || n + c > most) {
                bad = 1;
                n = m = 0;
            } else {
                m = n + c > 0 ? n + c : 0;
                const int64_t had = (n + bs - 1) / bs, has = (m + bs - 1) / bs;
                v[0] = c > 0 ? c : 0;
                v[1] = has > had ? has - had : 0;
                v[2] = had > has ? had - has : 0;
            }
        }
        int64_t incl[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            incl[k] = v[k];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = shfl_up64(incl[k], o);
                if (lane >= o) incl[k] += x;
            }
            if (lane == 31) warp_tot[k][warp] = incl[k];
        }
        __syncthreads();
        int64_t before[3];
#pragma unroll
        for (int k = 0; k < 3; ++k) {          // every warp sums the warps' totals
            const int64_t w = lane < nw ? warp_tot[k][lane] : 0;
            int64_t x = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = shfl_up64(x, o);
                if (lane >= o) x += y;
            }
            before[k] = total[k] + __shfl_sync(kFull, x - w, warp);
            total[k] += __shfl_sync(kFull, x, 31);
        }
        if (i < B) {
            old_s[i] = static_cast<int32_t>(n);
            new_s[i] = static_cast<int32_t>(m);
            // (sums beyond 32 bits make the whole call refused below)
            cu[i] = static_cast<int32_t>(before[0] + incl[0] - v[0]);
            need[i] = static_cast<int32_t>(before[1] + incl[1] - v[1]);
            back[i] = static_cast<int32_t>(before[2] + incl[2] - v[2]);
        }
        __syncthreads();
    }
    if (bad) bad_s = 1;
    if (threadIdx.x == 0) {
        cu[B] = static_cast<int32_t>(total[0]);
        need[B] = static_cast<int32_t>(total[1]);
        back[B] = static_cast<int32_t>(total[2]);
    }
    __syncthreads();
    const int64_t T = total[0], N = total[1], R = total[2], top = count + R;
    const bool bad_len = bad_s || T > p.num_tokens;
    const bool bad_free = count < 0 || count > p.free_capacity || top > p.free_capacity || N > top;
    const bool refused = bad_len || bad_free;
    if (refused && rank == 0 && threadIdx.x == 0)
        report(p.err_flag, (bad_len ? 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */ : 0) | (bad_free ? kFlagNoBlocks : 0));
    if (ctas > 1) cluster_sync();       // all of it is read
    const int me = static_cast<int>(rank * blockDim.x + threadIdx.x), all = static_cast<int>(ctas * blockDim.x);
    // ---- blocks given back ----
    if (!refused && R > 0) {
        for (int j = me; j < R; j += all) {
            const int s = find(back, B, j);
            const int has = static_cast<int>((static_cast<uint32_t>(new_s[s]) + ubs - 1) / ubs);
            const int32_t id = p.block_tables[static_cast<int64_t>(s) * p.max_blocks + has + j - back[s]];
            if (id < 0 || id >= p.num_blocks) report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
            p.free_blocks[top - 1 - j] = id;
        }
        if (ctas > 1) cluster_sync(); else __syncthreads();
    }
    // ---- lengths, bounds, and blocks taken ----
    for (int i = me; i < B; i += all) {
        if (refused) {
            // (read again, as they are; each by the thread that writes it)
            p.out_lens[i] = p.lens[i];
            p.cu_seqlens[i] = 0;
        } else {
            p.out_lens[i] = new_s[i];
            p.cu_seqlens[i] = cu[i];
        }
    }
    if (me == 0) {
        p.cu_seqlens[B] = refused ? 0 : static_cast<int32_t>(T);
        *p.out_free_count = static_cast<int32_t>(refused ? count : top - N);
    }
    if (!refused)
        for (int k = me; k < N; k += all) {
            const int s = find(need, B, k);
            const int had = static_cast<int>((static_cast<uint32_t>(old_s[s]) + ubs - 1) / ubs);
            const int32_t id = p.free_blocks[top - 1 - k];
            if (id < 0 || id >= p.num_blocks) report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
            p.block_tables[static_cast<int64_t>(s) * p.max_blocks + had + k - need[s]] = id;
        }
    // ---- new tokens ----
    for (int64_t t = me; t < p.num_tokens; t += all) {
        int64_t slot = -1, pos = 0;
        if (!refused && t < T) {
            const int s = find(cu, B, static_cast<int>(t));
            pos = old_s[s] + (t - cu[s]);
            const uint32_t blk = static_cast<uint32_t>(pos) / ubs;
            const uint32_t had = (static_cast<uint32_t>(old_s[s]) + ubs - 1) / ubs;
            // a new block's id from where its table entry comes from, which another thread may write later
            const int32_t id = blk < had ? p.block_tables[static_cast<int64_t>(s) * p.max_blocks + blk]
                                         : p.free_blocks[top - 1 - (need[s] + static_cast<int64_t>(blk - had))];
            if (id >= 0 && id < p.num_blocks)
                slot = static_cast<int64_t>(id) * bs + (static_cast<uint32_t>(pos) - blk * ubs);
            else
                report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
        }
        p.slots[t] = slot;
        p.positions[t] = pos;
    }
}

}  // namespace

cudaError_t launch_update_tables(const TablesParams &p, cudaStream_t stream) {
    const size_t smem = (static_cast<size_t>(p.num_seqs) * 5 + 3) * sizeof(int32_t);
    const cudaError_t e = cudaFuncSetAttribute(update_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>((kTablesMaxSeqs * 5 + 3) * sizeof(int32_t)));
    if (e != cudaSuccess) return e;
    const int64_t items = p.num_seqs > p.num_tokens ? p.num_seqs : p.num_tokens;
    // one CTA up to 2,048 items; beyond, 8 share them
    const unsigned ctas = items <= 2 * kTableThreads ? 1 : 8;
    const unsigned threads = items <= 128 ? 128 : kTableThreads;
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
    return cudaLaunchKernelEx(&cfg, update_tables_kernel, p);
}

}  // namespace pa
