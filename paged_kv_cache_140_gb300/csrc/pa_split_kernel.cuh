// Split decode attention over a paged cache: 16-bit caches, and 8-bit caches
// (e4m3 or int8 codes) with one scale per token and KV head.
//
// For query row q of an entry and the entry's tokens p, with code rows c_p and
// scales k_p, v_p (1 for 16-bit caches):
//     x_p = scale k_p <q, cK_p>,   out = sum_p softmax(x)_p v_p cV_p.
// An entry is a sequence (its whole context, or what follows the blocks it
// shares with its group) or a chunk of a group's sequences over their shared
// blocks; it is cut into partitions, and the partitions' states (reference,
// sum, weighted sum of V) are joined by pa_split_merge.cu.
//
// The softmax runs in base 2 with one running reference m per query row that
// serves the sum and the V product: with s_p = log2(e) x_p,
//     l = sum 2^(s_p - m),   acc = sum (2^(s_p - m) v_p) cV_p.
// m follows the maximum of s_p + log2 v_p, the exponent of the weights that
// enter the V product, less 7: the largest weight 2^(s_p - m) v_p lies between
// 2^7 and 2^15 (m is raised only when one passes 2^15) whatever the scales are.
// They go into the product as a high and a low part of the products' type: binary16
// (f16 and 8-bit caches), ~22 bits down to 2^-24, that is 2^-31 of the largest, so
// that even 2^15 tokens of the least weight lose no more than 2^-16; or, for bf16
// caches, bfloat16, 16 bits (2^-17 off at most) of any size.  2^(s_p - m) itself is then off by up to 1 / v_p,
// which 32 bits hold for every scale the cache write makes from rows below 2^60.
//
// 8-bit codes are exact in binary16 and the products run there; the query is
// scaled per row by a power of two to a largest element in [1, 2) (undone on
// the logits), so that a bfloat16 query of any size fits.
//
// What bounds it: reading the cache.  One producer warp brings ring slots in by
// TMA (boxes of up to 8 KV heads: 16 rows of one physical block of each land as
// one swizzled tile) and, for 8-bit caches, the scales, as boxes too where 4 or 8
// heads make them wide enough, else by 4-byte asynchronous copies that complete on
// the same barrier.  A slot holds one tile of 16 tokens (two for 8-bit caches) for
// each of 8 consumer warps: the box's heads times as many 16-token stages as make
// up the warps, so KV-head counts that are not a multiple of 8 keep every warp busy;
// warps that share a head keep states of their own and join them at the item's end.
// The SMs take equal shares of all slots; an item across a share's end is cut there.
//
// Measured (GB300, whole calls, join included; of the measured copy rate): 256
// 13B-shaped sequences over e4m3 codes 217 us, 0.91; 64 7B-shaped over int8 99 us,
// 0.85; 16 of 16 K to 32 K tokens, 32 heads on 8, e4m3, 127 us, 0.95.  With the math
// left out the first took 216, without the scales' loads too 202: the 3 % of bytes
// that scales are cost 7 %, as 32-byte pieces.  Tried and slower: 16 consumer warps
// (240 us against 221 at that time), one stage per slot (277), two ring slots instead
// of three (241), a warp that prefetches slots into L2 (2 ahead 220, 8 ahead 296).
// Waits are bounded (2 s) and report PA_FLAG_TIMEOUT.
#pragma once

#include <type_traits>

#include "pa_decode_common.cuh"
#include "pa_device.cuh"
#include "pa_split.h"

namespace pa {

namespace {

using namespace decode_common;

constexpr int kQueryRing = 2;

template <int D, int C, int CT>
struct SplitLayout {
    static constexpr bool k8 = CT >= kCacheE4M3;
    static constexpr int kES = k8 ? 1 : 2;
    static constexpr int kWarps = 8;                     // consumer warps
    static constexpr int kSub = k8 ? 2 : 1;              // stages per consumer warp and slot
    // Up to 4 query rows leave half of the products' 8 columns free: the weights'
    // high parts take columns 0-3 and their low parts columns 4-7 (the queries are
    // repeated there), one product in place of two.
    static constexpr bool kPaired = C <= 4;
    static constexpr int kTiles = kWarps * kSub;         // (stage, head) tiles of a slot
    static constexpr int kRowB = D * kES < 128 ? D * kES : 128;   // bytes of one box row
    static constexpr int kHalves = D * kES / kRowB;
    static constexpr int kKVBytes = kTiles * kStageTokens * D * kES;   // a slot's K (or V) rows
    static constexpr int kScaleBytes = k8 ? kTiles * kStageTokens * 4 : 0;
    static constexpr int kSlotBytes = (2 * kKVBytes + 2 * kScaleBytes + 1023) / 1024 * 1024;
    static constexpr int kThreads = (kWarps + 1) * 32;
    static constexpr int kMT = D / 16;
    static constexpr int kStateRow = D + 4;              // floats per query row of a warp's state
    static constexpr int kStateBytes = C * kStateRow * 4;
};

// One ring slot's description.
struct SlotMeta {
    int seq;         // the entry's first query sequence; < 0: no more work
    int kvh0;        // first KV head of the box
    int part;
    int flags;       // kFirst | kLast and one of kFinal, kContinued, kCut, members << 8
    int ntok;        // valid tokens from the slot's first
    uint32_t bad;    // bit 2 i (+ 1): rows 0-7 (8-15) of the slot's stage i were not loaded
    int pad[2];
};
constexpr int kFirst = 1;    // the first slot of an item (of this CTA's part of it): load the queries, reset the state
constexpr int kLast = 2;     // its last slot: write the results
constexpr int kFinal = 4;    // the item is the whole of the sequence's context
constexpr int kContinued = 8;   // the item was begun by the CTA before: the result goes to this CTA's own row
constexpr int kCut = 16;        // the CTA behind goes on with the item

__device__ __forceinline__ void arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// This thread's earlier cp.async copies arrive once on `bar` when they land
// (one of the barrier's expected arrivals).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// 2-D tiled TMA load (scales; the other heads' scales of the same tokens share
// its cache lines, so no early eviction).
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ float fast_log2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The largest weight is raised to this exponent, and the reference moved when
// one passes kWeightMax (below binary16's 65504).
constexpr float kWeightExp = 7.f, kWeightMax = 32768.f;

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
// V scales below this count as this (the cache write makes none below 2^-69),
// which bounds 2^(s_p - m) to 2^85.
constexpr float kScaleFloor = 8.470329472543003e-22f;   // 2^-70

// Four K codes (bytes 0-3) as f16 pairs (0, 1) and (2, 3).  An int8 code b is
// u - 128 for the byte u = b ^ 0x80, and 0x6400 | u is binary16 1024 + u: exact.
template <int CT>
__device__ __forceinline__ void widen_k(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (CT == kCacheE4M3) {
        e4m3x4_to_f16x2x2(w, lo, hi);
    } else {
        const uint32_t u = w ^ 0x80808080u;
        lo = __byte_perm(u, 0x64646464u, 0x4140u);
        hi = __byte_perm(u, 0x64646464u, 0x4342u);
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
    }
}

// Four V codes as f16 pairs (0, 2) and (1, 3), exactly, as K's.  (With u in their place
// and 128 sum w taken off an item's sum, 64 7B-shaped sequences took 98.2 us against 99.2,
// but a sum over values of both signs kept the roundings of 128 sum w: 2e-5 of the result
// there and 2e-4 at 16 K to 32 K tokens, against 6e-7 and 1e-6.)
template <int CT>
__device__ __forceinline__ void widen_v(uint32_t w, uint32_t &ev, uint32_t &od) {
    if constexpr (CT == kCacheE4M3) {
        e4m3x4_to_f16x2x2(prmt(w, 0x3120u), ev, od);
    } else {
        ev = (w & 0x00ff00ffu) ^ 0x64806480u;
        od = ((w >> 8) & 0x00ff00ffu) ^ 0x64806480u;
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(ev) : "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(od) : "r"(0x64806480u));
    }
}

// Sequence s's shared blocks; a length that is negative, above the bound or
// beyond the sequence's context counts as none and is reported.
__device__ __forceinline__ int shared_blocks(const SplitParams &p, int s, int ctx, bool tell) {
    const int n = __ldg(p.shared_lens + s);
    if (n < 0 || n > p.max_shared_len || n > ctx) {
        if (tell) report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
        return 0;
    }
    return n / p.block_size;
}

__device__ __forceinline__ int context_of(const SplitParams &p, int s, bool tell) {
    const int c = __ldg(p.context_lens + s);
    if (c < 0 || c > p.max_context_len) {
        if (tell) report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
        return 0;
    }
    return c;
}

// Group bounds that break the rules: from 0, never falling, the last num_seqs,
// groups of at most max_group_size.
__device__ __forceinline__ bool bad_group(const SplitParams &p, int g, int q0, int q1) {
    return q0 < 0 || q1 < q0 || q1 > p.num_seqs || q1 - q0 > p.max_group_size || (g == 0 && q0 != 0) ||
           (g == p.num_groups - 1 && q1 != p.num_seqs);
}

// Row, after p.cut_row, of query row `col` of head `head` of a box in what CTA
// `cta` of this launch continued.
__device__ __forceinline__ int cut_row_of(const SplitParams &p, uint32_t cta, int head, int col) {
    return static_cast<int>(((((p.e0 / kSplitEntries) * kSplitMaxCtas + cta) << p.log2_heads) + head) * p.cut_cols + col);
}

// Items (entry, partition, box of heads) in that order, weighed in slots: the
// boxes of one partition, whose rows lie next to one another, are read one after
// the other.  An entry without tokens weighs nothing, except where it costs the slot that writes
// its zero row.
struct ItemCursor {
    int e, len, nparts, part, grp, nslots;
    uint32_t start;
};

__device__ __forceinline__ int item_slots(int len, int part, int P, int SW) {
    const int n = len - part * P;
    const int st = n > 0 ? (min(P, n) + kStageTokens - 1) / kStageTokens : 1;
    return (st + SW - 1) / SW;
}

// Modes in which a list of one partition is the whole result.
__device__ __forceinline__ bool final_mode(int mode) { return mode == kSplitDecode || mode == kSplitWhole; }

__device__ __forceinline__ uint32_t entry_weight(int len, int mode, int ngroups, int P, int SW) {
    if (len <= 0) return final_mode(mode) ? static_cast<uint32_t>(ngroups) : 0u;
    const int full = (len - 1) / P;   // partitions before the last
    return static_cast<uint32_t>(ngroups) *
           static_cast<uint32_t>(full * ((P / kStageTokens + SW - 1) / SW) + item_slots(len, full, P, SW));
}

template <int D, int C, int CT>
__global__ void __launch_bounds__((SplitLayout<D, C, CT>::kThreads), 1)
    paged_split_kernel(const __grid_constant__ SplitParams p, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_ks,
                       const __grid_constant__ CUtensorMap tmap_vs) {
    using L = SplitLayout<D, C, CT>;
    constexpr bool k8 = L::k8;
    constexpr bool BF16 = CT == kCacheBF16;   // MMA operand type
    constexpr int SUB = L::kSub, W = L::kWarps, MT = L::kMT, KS = D / 16;
    constexpr int NE = C == 1 ? 1 : 2;        // live columns per lane (columns 2t, 2t + 1)
    using Cvt = Half2x<BF16>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int S = p.stages, E = p.entries, Hkv = p.num_kv_heads, Hq = p.num_heads;
    const int P = p.partition_size, bs = p.block_size, mode = p.mode, lg = p.log2_group;
    const int H = 1 << p.log2_heads, ngroups = Hkv >> p.log2_heads;
    const int SW = L::kTiles >> p.log2_heads;          // stages per slot
    const int nsubs = W >> p.log2_heads;               // consumer warps per head
    const int RB = min(bs, kStageTokens);              // rows per box
    const int per_stage = kStageTokens / RB;           // boxes (blocks) per stage
    const int qmember = H * D * 2 << lg;               // one sequence's query rows of a box
    constexpr int kQEntry = C * D * 2;                 // x H: one query-ring entry

    uint8_t *slots = smem;
    uint8_t *qbuf = smem + static_cast<size_t>(S) * L::kSlotBytes;
    uint8_t *xbuf = qbuf + kQueryRing * kQEntry * H;   // (W - H) warp states
    float2 *xml = reinterpret_cast<float2 *>(xbuf + (W - H) * L::kStateBytes);   // [warp][8]
    SlotMeta *meta = reinterpret_cast<SlotMeta *>(xml + W * 8);
    uint64_t *full = reinterpret_cast<uint64_t *>(meta + S);
    uint64_t *empty = full + S;
    uint64_t *qfull = empty + S;
    uint64_t *qempty = qfull + kQueryRing;
    uint64_t *xfull = qempty + kQueryRing;             // per head: the other warps' states are written
    uint64_t *xfree = xfull + 8;                       //           and have been read
    uint32_t *warp_tot = reinterpret_cast<uint32_t *>(xfree + 8);
    int *len_s = reinterpret_cast<int *>(warp_tot + 32);
    int *aux_s = len_s + E;                            // suffix: first block; prefix: sequence | members << 27;
                                                       // whole: the group's first sequence
    uint32_t *prefix = reinterpret_cast<uint32_t *>(aux_s + E);
    // Scales of 4 or 8 heads are 16 or 32 bytes per token: boxes.  Fewer are below
    // a box's least width: 4-byte copies by all lanes of the producer.
    const bool scale_boxes = k8 && p.log2_heads >= 2;

    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], k8 && !scale_boxes ? 33 : 1);
            mbar_init(&empty[i], W);
        }
        for (int i = 0; i < kQueryRing; ++i) {
            mbar_init(&qfull[i], 1);
            mbar_init(&qempty[i], W);
        }
        for (int i = 0; i < H; ++i) {
            mbar_init(&xfull[i], max(1, nsubs - 1));
            mbar_init(&xfree[i], 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&tmap_k);
        prefetch_tensormap(&tmap_v);
    }
    // Launched with programmatic dependent launch.  late_wait: the previous kernel is
    // this call's prefix kernel (or an earlier launch of this one behind it), whose
    // results are not read here, and this one waits for it only at its end.  Lengths,
    // tables, queries and K/V are read before that wait although a kernel ahead of the
    // call may have written them.  The programming model promises what earlier kernels
    // wrote to a grid that has waited itself; here every CTA of the prefix kernel waited
    // before it let dependents start, so all of that was complete and in memory before
    // this grid's first CTA began, as before any launch, and no cache of a new grid holds
    // older lines.  The workspace rows written here were last read by the join before the
    // prefix kernel.  (Waiting at the start: one long prompt 108 us against 99, 24 mixed
    // groups 141 against 129, 64 x 4 samples 266 against 254.)
    if (!p.late_wait) pdl_wait();
    pdl_launch_dependents();
    // ---- the entries' lengths ----
    const bool tell = blockIdx.x == 0;
    if (mode == kSplitWhole && tell)   // every group's bounds, the warps with the fewest entries first
        for (int g = blockDim.x - 1 - threadIdx.x; g < p.num_groups; g += blockDim.x)
            if (bad_group(p, g, __ldg(p.cu_groups + g), __ldg(p.cu_groups + g + 1)))
                report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
    for (int i = threadIdx.x; i < E; i += blockDim.x) {
        int len = 0, aux = 0;
        if (mode == kSplitPrefix) {
            const int g = (p.e0 + i) / p.chunks, ck = (p.e0 + i) % p.chunks;
            const int q0 = __ldg(p.cu_groups + g), q1 = __ldg(p.cu_groups + g + 1);
            if (bad_group(p, g, q0, q1)) {
                if (tell) report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
            } else {
                const int s0 = q0 + ck * p.chunk_seqs, m = min(p.chunk_seqs, q1 - s0);
                if (m > 0) {
                    len = shared_blocks(p, q0, context_of(p, q0, false), false) * bs;
                    aux = s0 | (m << 27);
                    for (int k = 0; tell && k < m; ++k)   // one length for all of a group
                        if (__ldg(p.shared_lens + s0 + k) != __ldg(p.shared_lens + q0))
                            report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
                }
            }
        } else {
            const int s = p.e0 + i;
            len = context_of(p, s, tell);
            if (mode == kSplitSuffix) {
                aux = shared_blocks(p, s, len, tell);
                len -= aux * bs;
            } else if (mode == kSplitWhole) {
                int a = 0, b = p.num_groups;             // the last group that starts at or before s
                while (b - a > 1) {
                    const int m = (a + b) >> 1;
                    if (__ldg(p.cu_groups + m) <= s) a = m; else b = m;
                }
                const int q0 = __ldg(p.cu_groups + a), q1 = __ldg(p.cu_groups + a + 1);
                const bool bad = bad_group(p, a, q0, q1) || q0 > s || q1 <= s;
                aux = bad ? s : q0;
                if (tell && (bad || __ldg(p.shared_lens + s) != __ldg(p.shared_lens + aux)))
                    report(p.err_flag, 0x4 /* PA_FLAG_BAD_CONTEXT_LEN */);
                shared_blocks(p, s, len, tell);
            }
        }
        len_s[i] = len;
        aux_s[i] = aux;
    }
    __syncthreads();
    {
        // prefix[i]: slots of the entries before i
        const int nthr = blockDim.x, nw = nthr >> 5;
        const int per = (E + nthr - 1) / nthr;
        const int beg = min(E, static_cast<int>(threadIdx.x) * per), end = min(E, beg + per);
        uint32_t local = 0;
        for (int i = beg; i < end; ++i) local += entry_weight(len_s[i], mode, ngroups, P, SW);
        uint32_t incl = local;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_tot[warp] = incl;
        __syncthreads();
        uint32_t run = incl - local;
        for (int w = 0; w < warp; ++w) run += warp_tot[w];
        for (int i = beg; i < end; ++i) {
            prefix[i] = run;
            run += entry_weight(len_s[i], mode, ngroups, P, SW);
        }
        if (threadIdx.x == 0) {
            uint32_t tot = 0;
            for (int w = 0; w < nw; ++w) tot += warp_tot[w];
            prefix[E] = tot;
        }
        __syncthreads();
    }
    // This CTA takes the items whose first slot lies in its equal share of the
    // slots, or (p.cut, with shares at least as long as an item) exactly its share:
    // an item across the end is continued by the next CTA, which leaves a partial
    // result of its own, named in the item's.
    const uint32_t total = prefix[E];
    const bool cut = p.cut && total >= gridDim.x * static_cast<uint32_t>((P / kStageTokens + SW - 1) / SW);
    const uint32_t lo = static_cast<uint32_t>(static_cast<uint64_t>(total) * blockIdx.x / gridDim.x);
    const uint32_t hi = static_cast<uint32_t>(static_cast<uint64_t>(total) * (blockIdx.x + 1) / gridDim.x);

    if (warp == W) {
        // ------------------------------------------------------------ producer
        const uint64_t policy =
            mode == kSplitPrefix && p.chunks > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
        ItemCursor ic{};
        auto set_entry = [&](int e) {
            ic.e = e;
            ic.len = len_s[e];
            ic.nparts = ic.len > 0 ? (ic.len + P - 1) / P : 1;
        };
        auto set_part = [&](int part) {
            ic.part = part;
            ic.nslots = item_slots(ic.len, part, P, SW);
        };
        auto advance = [&]() {
            ic.start += ic.nslots;
            if (++ic.grp < ngroups) return;
            ic.grp = 0;
            if (ic.part + 1 < ic.nparts) {
                set_part(ic.part + 1);
                return;
            }
            int e = ic.e + 1;
            while (e < E && prefix[e] == prefix[e + 1]) ++e;   // entries without work
            if (e < E) {
                set_entry(e);
                set_part(0);
            }
        };
        const bool work = lo < hi;
        if (work) {
            // the entry holding slot lo (the last with prefix <= lo), then its first item starting at or after lo
            int a = 0, b = E;
            while (b - a > 1) {
                const int m = (a + b) >> 1;
                if (prefix[m] <= lo) a = m; else b = m;
            }
            set_entry(a);
            const uint32_t pw = static_cast<uint32_t>(ngroups) * static_cast<uint32_t>((P / kStageTokens + SW - 1) / SW);
            const uint32_t off = lo - prefix[a];
            set_part(min(ic.nparts - 1, static_cast<int>(off / pw)));
            const uint32_t pstart = prefix[a] + static_cast<uint32_t>(ic.part) * pw;
            const int grp = static_cast<int>((lo - pstart + (cut ? 0 : ic.nslots - 1)) / ic.nslots);
            ic.grp = min(grp, ngroups - 1);
            ic.start = pstart + static_cast<uint32_t>(ic.grp) * ic.nslots;
            if (grp >= ngroups) advance();
        }
        // An item's sequence, members, table row and first block; its tokens and
        // the block ids of its partition, one per lane.
        int seq, members, blk0, t0, ntok, fb;
        int32_t bid;
        auto open_item = [&]() {
            int row;
            seq = row = p.e0 + ic.e;
            members = 1;
            blk0 = 0;
            if (mode == kSplitPrefix) {
                seq = aux_s[ic.e] & 0x7ffffff;
                members = aux_s[ic.e] >> 27;
                row = seq - ((p.e0 + ic.e) % p.chunks) * p.chunk_seqs;   // the group's first sequence
            } else if (mode == kSplitSuffix) {
                blk0 = aux_s[ic.e];
            }
            t0 = ic.part * P;
            ntok = max(0, min(P, ic.len - t0));
            fb = t0 / bs;
            if (mode == kSplitWhole && fb + lane < shared_blocks(p, seq, ic.len, false)) row = aux_s[ic.e];
            bid = -1;
            if (ntok > 0 && lane <= (t0 + ntok - 1) / bs - fb)
                bid = __ldg(p.block_tables + static_cast<int64_t>(row) * p.max_blocks_per_seq + blk0 + fb + lane);
        };
        int islot = 0;
        uint32_t uses = 0, items = 0;
        bool ok = true;
        auto take_slot = [&]() -> int {
            const int slot = islot;
            if (uses >= static_cast<uint32_t>(S)) {
                const uint32_t par = ((uses / S) - 1) & 1u;
                if (!mbar_try_wait(&empty[slot], par) && !mbar_wait_bounded(&empty[slot], par)) {
                    if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                    ok = false;
                }
            }
            ok = __all_sync(kFull, ok);
            if (ok) {
                islot = (islot + 1 == S) ? 0 : islot + 1;
                ++uses;
            }
            return slot;
        };
        while (ok && work && ic.start < hi) {
            const int kvh0 = ic.grp << p.log2_heads;
            open_item();
            {
                const int qi = static_cast<int>(items % kQueryRing);
                if (items >= static_cast<uint32_t>(kQueryRing)) {
                    const uint32_t par = ((items / kQueryRing) - 1) & 1u;
                    if (!mbar_try_wait(&qempty[qi], par) && !mbar_wait_bounded(&qempty[qi], par)) {
                        if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                        ok = false;
                    }
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&qfull[qi], static_cast<uint32_t>(members * qmember));
                    for (int m = 0; m < members; ++m)
                        bulk_load(qbuf + qi * kQEntry * H + m * qmember,
                                  p.q + (static_cast<int64_t>(seq + m) * Hq + (kvh0 << lg)) * D,
                                  static_cast<uint32_t>(qmember), &qfull[qi]);
                }
                ++items;
                __syncwarp();
            }
            // this CTA's slots of the item
            const int jb = cut && ic.start < lo ? static_cast<int>(lo - ic.start) : 0;
            const int je = cut ? min(ic.nslots, static_cast<int>(hi - ic.start)) : ic.nslots;
            const int kind = jb > 0               ? kContinued
                             : je < ic.nslots     ? kCut
                             : final_mode(mode) && ic.nparts == 1 ? kFinal
                                                                  : 0;
            for (int j = jb; j < je; ++j) {
                const int slot = take_slot();
                if (!ok) break;
                uint8_t *sp = slots + static_cast<size_t>(slot) * L::kSlotBytes;
                const int tok0 = t0 + j * SW * kStageTokens;                 // the slot's first position
                const int nt = max(0, min(SW * kStageTokens, t0 + ntok - tok0));
                // The slot's pieces are RB rows of one block (SW * per_stage of them, at most 32), one per lane.
                const int ptok = tok0 + lane * RB;
                const bool has = lane < SW * per_stage && lane * RB < nt;
                const int id = __shfl_sync(kFull, bid, has ? ptok / bs - fb : 0);
                const bool load = has && id >= 0 && static_cast<int64_t>(id) < p.num_blocks;
                const uint32_t loaded = __ballot_sync(kFull, load);
                uint32_t bad = __ballot_sync(kFull, has && !load);
                if (bad && lane == 0) report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
                if (bad && per_stage == 1) {   // one bit per stage -> two
                    uint32_t w = 0;
                    for (int i = 0; i < SW; ++i) w |= ((bad >> i) & 1u) * (3u << (2 * i));
                    bad = w;
                }
                const uint32_t box = static_cast<uint32_t>(RB * L::kRowB) << p.log2_heads;
                const uint32_t sbox = scale_boxes ? static_cast<uint32_t>(RB * 4) << p.log2_heads : 0u;
                if (lane == 0) {
                    SlotMeta mt;
                    mt.seq = seq;
                    mt.kvh0 = kvh0;
                    mt.part = ic.part;
                    mt.flags = (j == jb ? kFirst : 0) | (j + 1 == je ? kLast : 0) | kind | (members << 8);
                    mt.ntok = nt;
                    mt.bad = bad;
                    mt.pad[0] = mt.pad[1] = 0;
                    meta[slot] = mt;
                    mbar_arrive_expect_tx(&full[slot],
                                          static_cast<uint32_t>(__popc(loaded)) * 2u * (box * L::kHalves + sbox));
                }
                __syncwarp();
                const int z = load ? id * bs + ptok % bs : 0;               // the piece's first cache slot
                if (load) {
                    const int st = lane / per_stage, b = lane % per_stage;
                    uint8_t *dst = sp + ((static_cast<size_t>(st) * kStageTokens * D * L::kES) << p.log2_heads) + b * box;
#pragma unroll
                    for (int h = 0; h < L::kHalves; ++h) {
                        const uint32_t ho = h * per_stage * box;
                        tma_load_3d(dst + ho, &tmap_k, &full[slot], h * (L::kRowB / L::kES), z, kvh0, policy);
                        tma_load_3d(dst + L::kKVBytes + ho, &tmap_v, &full[slot], h * (L::kRowB / L::kES), z, kvh0,
                                    policy);
                    }
                }
                if constexpr (k8) {
                    // scales, [token of the slot][head of the box], K then V
                    uint8_t *ss = sp + 2 * L::kKVBytes;
                    if (scale_boxes) {
                        if (load) {
                            tma_load_2d(ss + lane * sbox, &tmap_ks, &full[slot], kvh0, z);
                            tma_load_2d(ss + L::kScaleBytes + lane * sbox, &tmap_vs, &full[slot], kvh0, z);
                        }
                    } else {
                        const int n = (SW * kStageTokens) << p.log2_heads;
                        for (int i = lane; i < n; i += 32) {
                            const int tk = i >> p.log2_heads, h = i & (H - 1), pc = tk / RB;
                            const int zz = __shfl_sync(kFull, z, pc);
                            if (!((loaded >> pc) & 1u) || tk >= nt) continue;
                            const int64_t src = static_cast<int64_t>(zz + tk % RB) * Hkv + kvh0 + h;
                            cp_async4(smem_addr(ss) + i * 4, p.k_scales + src);
                            cp_async4(smem_addr(ss) + L::kScaleBytes + i * 4, p.v_scales + src);
                        }
                        cp_async_arrive(&full[slot]);
                    }
                }
                __syncwarp();
            }
            advance();
        }
        // one more slot tells the consumers to stop
        if (ok) {
            const int slot = take_slot();
            if (ok) {
                if (lane == 0) {
                    SlotMeta mt{};
                    mt.seq = -1;
                    meta[slot] = mt;
                    arrive(&full[slot]);
                }
                if (k8 && !scale_boxes) {
                    __syncwarp();
                    arrive(&full[slot]);
                }
            }
        }
        // After a wait that gave up, let the copies still in flight land before the CTA ends.
        if (!ok) {
            for (uint32_t u = uses > static_cast<uint32_t>(S) ? uses - S : 0u; u < uses; ++u)
                mbar_wait_bounded(&full[u % S], (u / S) & 1u);
            for (uint32_t i = items > static_cast<uint32_t>(kQueryRing) ? items - kQueryRing : 0u; i < items; ++i)
                mbar_wait_bounded(&qfull[i % kQueryRing], (i / kQueryRing) & 1u);
        }
        if (p.late_wait) pdl_wait();   // the grid does not finish before the prefix kernel
        return;
    }

    // ---------------------------------------------------------------- consumers
    // Warp w takes head kvh0 + w % H and, of a slot's stages, the SUB at
    // (w / H) * SUB.  Column c of its MMAs (c < 8) is query row c % G of member
    // c / G; columns without a query hold zero queries and are never written.
    const int head = warp & (H - 1), sub = warp >> p.log2_heads;
    const int g = lane >> 2, t = lane & 3;
    const int r8 = lane & 7, j8 = lane >> 3;
    const uint32_t slots_sa = smem_addr(slots);
    const uint32_t box = static_cast<uint32_t>(RB * L::kRowB) << p.log2_heads;
    const uint32_t half_off = box * per_stage;                       // next 128-byte column block
    const uint32_t stage_off = half_off * L::kHalves;
    const uint32_t head_off = head * RB * L::kRowB;
    const uint32_t hi_off = per_stage == 1 ? 8 * L::kRowB : box;     // rows 8-15 of a stage
    // A lane's 16-byte chunk 2 i + (0 or 1) of its row sits, swizzled, at the row's
    // start + 16 ((2 i + b) ^ swz): the address for i = 0, with 32 i flipped in.
    const uint32_t swz = L::kRowB == 128 ? r8 : (r8 >> 1) & 3;
    const uint32_t off_k = head_off + (j8 & 1) * hi_off + r8 * L::kRowB + (((j8 >> 1) ^ swz) << 4);
    const uint32_t off_v = L::kKVBytes + head_off + (j8 >> 1) * hi_off + r8 * L::kRowB + (((j8 & 1) ^ swz) << 4);
    // 8-bit caches: my tokens' scales in a slot (K; V scales kScaleBytes further)
    const uint32_t scl_off = 2 * L::kKVBytes + ((((sub * SUB * kStageTokens + g) << p.log2_heads) + head) << 2);
    const uint32_t scl_8 = 32u << p.log2_heads;                      // 8 tokens further
    const uint64_t keep = l2_policy_evict_last();

    uint32_t qf[KS][2];
    float qs[2];                  // logit scale of columns 2t, 2t + 1
    float acc[MT][4], m_run[2], l_run[2];
    float mu[2];                  // the reference that weights are taken under: m_run, or 0 while there is none
    int cslot = 0;
    uint32_t cphase = 0, citems = 0;
    for (;;) {
        const int slot = cslot;
        uint8_t *sp = slots + static_cast<size_t>(slot) * L::kSlotBytes;
        const uint32_t sa = slots_sa + slot * L::kSlotBytes;
        if (!mbar_try_wait(&full[slot], cphase) && !mbar_wait_bounded(&full[slot], cphase)) {
            if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
            return;
        }
        if (++cslot == S) {
            cslot = 0;
            cphase ^= 1u;
        }
        const SlotMeta m = meta[slot];
        if (m.seq < 0) break;
        const int members = m.flags >> 8;

        if (m.flags & kFirst) {
            const int qi = static_cast<int>(citems % kQueryRing);
            const uint32_t qpar = (citems / kQueryRing) & 1u;
            ++citems;
            if (!mbar_try_wait(&qfull[qi], qpar) && !mbar_wait_bounded(&qfull[qi], qpar)) {
                if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                return;
            }
            const int gq = L::kPaired ? g & 3 : g;        // my column's query row
            const bool live = gq < (members << lg);
            const uint32_t *qw = reinterpret_cast<const uint32_t *>(qbuf + qi * kQEntry * H + (live ? gq >> lg : 0) * qmember) +
                                 ((head << lg) + (gq & ((1 << lg) - 1))) * (D / 2);
            if constexpr (!k8) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    qf[ks][0] = live ? qw[(ks * 16 + 2 * t) >> 1] : 0u;
                    qf[ks][1] = live ? qw[(ks * 16 + 2 * t + 8) >> 1] : 0u;
                }
                qs[0] = qs[1] = p.scale_log2;
            } else {
                // Dims in the order the widened K fragments arrive: step
                // 2kc + hl takes dims 32kc + 4t + 2hl (+1) and the same + 16.
                float2 f[KS][2];
                float amax = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t w = live ? qw[(32 * (ks >> 1) + 4 * t + 2 * (ks & 1) + 16 * k) >> 1] : 0u;
                        f[ks][k] = p.q_bf16 ? Half2x<true>::to_float2(w) : Half2x<false>::to_float2(w);
                        amax = fmaxf(amax, fmaxf(fabsf(f[ks][k].x), fabsf(f[ks][k].y)));
                    }
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                // 2^e <= amax < 2^(e+1), e kept where both 2^e and 2^-e are normal
                const uint32_t eb = min(max(__float_as_uint(amax) & 0x7f800000u, 0x00800000u), 0x7e800000u);
                const float inv = __uint_as_float(0x7f000000u - eb);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int k = 0; k < 2; ++k) qf[ks][k] = pack2<false>(f[ks][k].x * inv, f[ks][k].y * inv);
                const float up = __uint_as_float(eb) * p.scale_log2;
                qs[0] = __shfl_sync(kFull, up, 8 * t);        // column 2t is held by lanes of group 2t
                qs[1] = __shfl_sync(kFull, up, 8 * t + 4);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) arrive(&qempty[qi]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m_run[e] = -INFINITY;
                l_run[e] = mu[e] = 0.f;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
        }

        // My tokens of this slot.  kWhole: every one of them counts (all but a
        // list's last slot), compiled apart so that the common case carries no masks.
        const int st0 = sub * SUB;
        const int mine = m.ntok - st0 * kStageTokens;
        auto attend = [&](auto whole_tag) {
            constexpr bool kWhole = decltype(whole_tag)::value;
            const bool second = kWhole || (SUB > 1 && mine > kStageTokens);
            uint32_t smask[SUB];
            float x[SUB][4], sv[SUB][2];
#pragma unroll
            for (int hs = 0; hs < SUB; ++hs) {
                smask[hs] = 0xffffu;
                if constexpr (!kWhole) {
                    if (hs > 0 && !second) {
                        smask[hs] = 0;
                        x[hs][0] = x[hs][1] = x[hs][2] = x[hs][3] = -INFINITY;
                        sv[hs][0] = sv[hs][1] = 0.f;
                        continue;
                    }
                    const int n = mine - hs * kStageTokens;
                    uint32_t mk = n >= kStageTokens ? 0xffffu : (1u << n) - 1u;
                    const uint32_t b = (m.bad >> (2 * (st0 + hs))) & 3u;
                    mk &= ~(((b & 1u) ? 0xffu : 0u) | ((b & 2u) ? 0xff00u : 0u));
                    smask[hs] = mk;
                }
                // ---- QK: 16 tokens x 8 columns ----
                const uint32_t ka = sa + (st0 + hs) * stage_off + off_k;
                float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                if constexpr (!k8) {
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        uint32_t a[4];
                        ldsm_x4(a, (ka + (ks >> 2) * half_off) ^ ((ks & 3) << 5));
                        mma_16816<BF16>(c[ks & 1], a, qf[ks][0], qf[ks][1]);
                    }
                } else {
#pragma unroll
                    for (int kc = 0; kc < D / 32; ++kc) {
                        uint32_t a[4], lo4[4], hi4[4];
                        ldsm_x4(a, ka ^ (kc << 5));
#pragma unroll
                        for (int i = 0; i < 4; ++i) widen_k<CT>(a[i], lo4[i], hi4[i]);
                        mma_16816<false>(c[0], lo4, qf[2 * kc][0], qf[2 * kc][1]);
                        mma_16816<false>(c[1], hi4, qf[2 * kc + 1][0], qf[2 * kc + 1][1]);
                    }
                }
                const bool v_lo = kWhole || ((smask[hs] >> g) & 1u), v_hi = kWhole || ((smask[hs] >> (g + 8)) & 1u);
                float k_lo = 1.f, k_hi = 1.f;
                if constexpr (k8) {
                    // a masked token's scales may be anything: its V scale counts as 0
                    const uint8_t *lo = sp + scl_off + 2 * hs * scl_8, *hi = lo + scl_8;
                    k_lo = *reinterpret_cast<const float *>(lo);
                    k_hi = *reinterpret_cast<const float *>(hi);
                    const float a = *reinterpret_cast<const float *>(lo + L::kScaleBytes);
                    const float b = *reinterpret_cast<const float *>(hi + L::kScaleBytes);
                    sv[hs][0] = v_lo ? max_nan(a, kScaleFloor) : 0.f;
                    sv[hs][1] = v_hi ? max_nan(b, kScaleFloor) : 0.f;
                }
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    const float a = (c[0][e] + c[1][e]) * (k8 ? k_lo * qs[e] : qs[e]);
                    const float b = (c[0][2 + e] + c[1][2 + e]) * (k8 ? k_hi * qs[e] : qs[e]);
                    x[hs][e] = v_lo ? a : -INFINITY;
                    x[hs][2 + e] = v_hi ? b : -INFINITY;
                }
            }
            // Weights under the present reference: 2^(x - m) for the sum, times the V
            // scale for the product.  The reference is raised only when a weight
            // passes 2^15 (or there is none yet): one vote in the common case.
            float pw[SUB][4], w4[SUB][4];
            auto weigh = [&]() {
#pragma unroll
                for (int hs = 0; hs < SUB; ++hs)
#pragma unroll
                    for (int e = 0; e < NE; ++e)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            pw[hs][2 * k + e] = fast_exp2(x[hs][2 * k + e] - mu[e]);
                            w4[hs][2 * k + e] = k8 ? pw[hs][2 * k + e] * sv[hs][k] : pw[hs][2 * k + e];
                        }
            };
            weigh();
            bool nd = false;
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                nd = nd || m_run[e] == -INFINITY;
#pragma unroll
                for (int hs = 0; hs < SUB; ++hs) nd = nd || fmaxf(w4[hs][e], w4[hs][2 + e]) > kWeightMax;
            }
            if (__any_sync(kFull, nd)) {
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    // the largest exponent of a weight: max x + log2 of the V scale
                    float mx = -INFINITY;
#pragma unroll
                    for (int hs = 0; hs < SUB; ++hs)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            mx = fmaxf(mx, k8 ? x[hs][2 * k + e] + fast_log2(sv[hs][k]) : x[hs][2 * k + e]);
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
                    const float mn = fmaxf(m_run[e], mx - kWeightExp);
                    const float al = mn == -INFINITY ? 1.f : fast_exp2(m_run[e] - mn);
                    m_run[e] = mn;
                    mu[e] = mn == -INFINITY ? 0.f : mn;
                    l_run[e] *= al;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[mt][e] *= al;
                        acc[mt][2 + e] *= al;
                    }
                }
                weigh();
            }
#pragma unroll
            for (int hs = 0; hs < SUB; ++hs) {
                if constexpr (!kWhole)
                    if (hs > 0 && !second) continue;
#pragma unroll
                for (int e = 0; e < NE; ++e) l_run[e] += pw[hs][e] + pw[hs][2 + e];
                // weights as the PV B fragment: tokens 2t, 2t+1, 2t+8, 2t+9 of column g
                uint32_t bhi[2], blo[2];
                {
                    const int srcA = 8 * t + (g >> 1), srcB = srcA + 4;
                    float w[4];
                    w[0] = __shfl_sync(kFull, w4[hs][0], srcA);
                    w[1] = __shfl_sync(kFull, w4[hs][0], srcB);
                    w[2] = __shfl_sync(kFull, w4[hs][2], srcA);
                    w[3] = __shfl_sync(kFull, w4[hs][2], srcB);
                    if constexpr (NE == 2) {
                        const float o0 = __shfl_sync(kFull, w4[hs][1], srcA), o1 = __shfl_sync(kFull, w4[hs][1], srcB);
                        const float o2 = __shfl_sync(kFull, w4[hs][3], srcA), o3 = __shfl_sync(kFull, w4[hs][3], srcB);
                        if (g & 1) {
                            w[0] = o0;
                            w[1] = o1;
                            w[2] = o2;
                            w[3] = o3;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        bhi[k] = pack2<BF16>(w[2 * k], w[2 * k + 1]);
                        const float2 h = Cvt::to_float2(bhi[k]);
                        blo[k] = pack2<BF16>(w[2 * k] - h.x, w[2 * k + 1] - h.y);
                        if (L::kPaired && g >= 4) bhi[k] = blo[k];
                    }
                }
                const uint32_t vbase = (st0 + hs) * stage_off + L::kKVBytes;
                // V rows that are masked are zeroed first: stale slots may hold NaN
                // (not so int8 codes, which a zero weight always cancels)
                if constexpr (!kWhole && CT != kCacheInt8) {
                    if (smask[hs] != 0xffffu) {
                        constexpr int kCh = L::kRowB / 16;                  // 16-byte chunks per box row
#pragma unroll
                        for (int k = 0; k < kStageTokens * L::kHalves * kCh / 32; ++k) {
                            const int q16 = lane + 32 * k;
                            const int half = q16 / (kStageTokens * kCh), row = (q16 / kCh) % kStageTokens;
                            if (!((smask[hs] >> row) & 1u))
                                *reinterpret_cast<uint4 *>(sp + vbase + half * half_off + head_off +
                                                           (row >> 3) * hi_off + (row & 7) * L::kRowB + (q16 % kCh) * 16) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                        __syncwarp();
                    }
                }
                const uint32_t va = sa + (st0 + hs) * stage_off + off_v;
                if constexpr (!k8) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        uint32_t a[4];
                        ldsm_x4_trans(a, (va + (mt >> 2) * half_off) ^ ((mt & 3) << 5));
                        mma_16816<BF16>(acc[mt], a, bhi[0], bhi[1]);
                        if constexpr (!L::kPaired) mma_16816<BF16>(acc[mt], a, blo[0], blo[1]);
                    }
                } else {
                    // Byte pairs (dims 2g, 2g+1) of two tokens: even dims feed
                    // acc[2vc], odd dims acc[2vc+1].
#pragma unroll
                    for (int vc = 0; vc < D / 32; ++vc) {
                        uint32_t a[4], ev[4], od[4];
                        ldsm_x4_trans(a, va ^ (vc << 5));
#pragma unroll
                        for (int i = 0; i < 4; ++i) widen_v<CT>(a[i], ev[i], od[i]);
                        mma_16816<false>(acc[2 * vc], ev, bhi[0], bhi[1]);
                        if constexpr (!L::kPaired) mma_16816<false>(acc[2 * vc], ev, blo[0], blo[1]);
                        mma_16816<false>(acc[2 * vc + 1], od, bhi[0], bhi[1]);
                        if constexpr (!L::kPaired) mma_16816<false>(acc[2 * vc + 1], od, blo[0], blo[1]);
                    }
                }
            }
        };
        if (mine >= SUB * kStageTokens && m.bad == 0)
            attend(std::true_type{});
        else if (mine > 0)
            attend(std::false_type{});
        // my reads (and zeroing) of the slot are done
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&empty[slot]);

        if (!(m.flags & kLast)) continue;
        // ---- item end ----
        if constexpr (L::kPaired) {   // the low parts' columns (c + 4: lane t + 2) onto the high parts'
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    acc[mt][e] += __shfl_xor_sync(kFull, acc[mt][e], 2);
                    acc[mt][2 + e] += __shfl_xor_sync(kFull, acc[mt][2 + e], 2);
                }
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int e = 0; e < NE; ++e) l_run[e] += __shfl_xor_sync(kFull, l_run[e], o);
        if (nsubs > 1) {
            // join the states of the head's warps: the others hand theirs to the first
            const uint32_t par = (citems - 1) & 1u;      // of this item
            if (sub > 0) {
                if (citems > 1 && !mbar_try_wait(&xfree[head], par ^ 1u) && !mbar_wait_bounded(&xfree[head], par ^ 1u)) {
                    if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                    return;
                }
                float *xs = reinterpret_cast<float *>(xbuf + (warp - H) * L::kStateBytes);
#pragma unroll
                for (int e = 0; e < NE; ++e) {
                    const int c = 2 * t + e;
                    if (c >= C) continue;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        xs[c * L::kStateRow + 16 * mt + g] = acc[mt][e];
                        xs[c * L::kStateRow + 16 * mt + 8 + g] = acc[mt][2 + e];
                    }
                    if (g == 0) xml[warp * 8 + c] = make_float2(m_run[e], l_run[e]);
                }
                __syncwarp();
                if (lane == 0) arrive(&xfull[head]);
                continue;
            }
            if (!mbar_try_wait(&xfull[head], par) && !mbar_wait_bounded(&xfull[head], par)) {
                if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                return;
            }
#pragma unroll
            for (int e = 0; e < NE; ++e) {
                const int c = 2 * t + e;
                if (c >= C) continue;
                float mn = m_run[e];
                for (int k = 1; k < nsubs; ++k) mn = fmaxf(mn, xml[(warp + k * H) * 8 + c].x);
                const float al = m_run[e] == -INFINITY ? 1.f : fast_exp2(m_run[e] - mn);
                m_run[e] = mn;
                l_run[e] *= al;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    acc[mt][e] *= al;
                    acc[mt][2 + e] *= al;
                }
                for (int k = 1; k < nsubs; ++k) {
                    const float *xs = reinterpret_cast<const float *>(xbuf + (warp + (k - 1) * H) * L::kStateBytes) +
                                      c * L::kStateRow + g;
                    const float2 ml = xml[(warp + k * H) * 8 + c];
                    const float be = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - mn);
                    l_run[e] = fmaf(ml.y, be, l_run[e]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[mt][e] = fmaf(xs[16 * mt], be, acc[mt][e]);
                        acc[mt][2 + e] = fmaf(xs[16 * mt + 8], be, acc[mt][2 + e]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&xfree[head]);
        }
        const int kvh = m.kvh0 + head;
        const bool fin = (m.flags & kFinal) != 0;
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int c = 2 * t + e;
            if (c >= (members << lg)) continue;
            const int64_t sq = m.seq + (c >> lg);
            const int hq = c & ((1 << lg) - 1);
            const float sc = fin ? (l_run[e] == 0.f ? 0.f : 1.f / l_run[e]) : 1.f;
            const int64_t r =
                (m.flags & kContinued)
                    ? p.cut_row + cut_row_of(p, blockIdx.x, head, c)
                    : (((sq * Hkv + kvh) * p.max_parts + p.part_off + m.part) << lg) + hq;
            if (g == 0 && !(fin && p.ws_ml == nullptr)) {
                const bool more = (m.flags & kCut) != 0;
                st_global_hint(p.ws_ml + 4 * r,
                               make_float4(m_run[e], l_run[e], __int_as_float(fin ? kRowFinal : more ? kRowCut : 0),
                                           __int_as_float(more ? cut_row_of(p, blockIdx.x + 1, head, c) : 0)),
                               keep);
            }
            const int64_t orow = fin ? (sq * Hq + (kvh << lg) + hq) * D : r * D;
            auto put2 = [&](int d, float a, float b) {   // two consecutive elements
                if (!fin)
                    st_global_hint(p.ws_acc + orow + d, make_float2(a, b), keep);
                else if (p.out_dtype == 2)
                    *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + orow + d) = make_float2(a, b);
                else
                    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + orow + d) =
                        p.out_dtype == 1 ? pack2<true>(a, b) : pack2<false>(a, b);
            };
            auto put1 = [&](int d, float a) {
                if (!fin)
                    p.ws_acc[orow + d] = a;
                else if (p.out_dtype == 2)
                    static_cast<float *>(p.out)[orow + d] = a;
                else
                    static_cast<uint16_t *>(p.out)[orow + d] = p.out_dtype == 1 ? float_to_bf16_bits(a) : float_to_f16_bits(a);
            };
            if constexpr (k8) {
#pragma unroll
                for (int vc = 0; vc < D / 32; ++vc) {
                    put2(32 * vc + 2 * g, acc[2 * vc][e] * sc, acc[2 * vc + 1][e] * sc);
                    put2(32 * vc + 16 + 2 * g, acc[2 * vc][2 + e] * sc, acc[2 * vc + 1][2 + e] * sc);
                }
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    put1(16 * mt + g, acc[mt][e] * sc);
                    put1(16 * mt + g + 8, acc[mt][2 + e] * sc);
                }
            }
        }
    }
}

template <int D, int C, int CT>
cudaError_t launch_split_t(const SplitParams &p, const SplitMaps &m, int grid, size_t smem, cudaStream_t stream) {
    auto kern = paged_split_kernel<D, C, CT>;
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(grid), dim3(SplitLayout<D, C, CT>::kThreads), smem, stream, p, m.k, m.v, m.ks,
                      m.vs);
}

template <int D, int CT>
cudaError_t launch_split_d(const SplitParams &p, int cols, const SplitMaps &m, int grid, size_t smem,
                           cudaStream_t stream) {
    switch (cols) {
        case 1: return launch_split_t<D, 1, CT>(p, m, grid, smem, stream);
        case 2: return launch_split_t<D, 2, CT>(p, m, grid, smem, stream);
        case 4: return launch_split_t<D, 4, CT>(p, m, grid, smem, stream);
        case 8: return launch_split_t<D, 8, CT>(p, m, grid, smem, stream);
        default: return cudaErrorInvalidValue;
    }
}

template <int CT>
cudaError_t launch_split_ct(const SplitParams &p, int head_dim, int cols, const SplitMaps &m, int grid, size_t smem,
                            cudaStream_t stream) {
    if (head_dim == 128) return launch_split_d<128, CT>(p, cols, m, grid, smem, stream);
    if (head_dim == 64) return launch_split_d<64, CT>(p, cols, m, grid, smem, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

}  // namespace pa
