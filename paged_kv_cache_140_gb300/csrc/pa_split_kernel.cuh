// Split decode attention over a paged cache: 16-bit caches, 8-bit caches (e4m3 or
// int8 codes) with one scale per token and KV head, and 4-bit caches (codes of 0 to 15)
// with a scale and a zero per 64 elements of them.
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
// 4-bit codes u of group r stand for s_pr (u + z_pr), and everything but the codes is
// taken out of the products, Q_r being the sum of q's elements in the group:
//     x_p = scale sum_r s_pr (<q_r, u_pr> + z_pr Q_r),
//     acc_r = sum (2^(s_p - m) s_pr) u_pr + sum (2^(s_p - m) s_pr) z_pr.
// Each group of V has a reference of its own, so that its largest weight lies between
// 2^6 and 2^15 however much smaller its values are than its neighbour's (under one
// reference for both, codes of a group 2^-16 as large were off by 7e-5 of themselves and
// from 2^-32 on lost, their zeros not): with one query row a lane weighs one group and m is
// that group's, else a group's weights and sums are taken a power of two up (4 rows, long
// contexts 94.9 us against 92.9; 8 rows 122.1 against 121.2).  Weights of 2^-76 and less of the
// row's largest may count as none.  What the codes cost is
// said at codes4, which lane weighs what where the consumers begin.
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
// 13B-shaped sequences over e4m3 codes 212 us, 0.93; 64 7B-shaped over int8 96 us,
// 0.88; 16 of 16 K to 32 K tokens, 32 heads on 8, e4m3, 126 us, 0.96.  (Before the bookkeeping
// lost its divisions 217, 99 and 127.)  With the math
// left out the first then took 216, without the scales' loads too 202: the 3 % of bytes
// that scales are cost 7 %, as 32-byte pieces.  Tried and slower: 16 consumer warps
// (240 us against 221 at that time), one stage per slot (277), two ring slots instead
// of three (241), a warp that prefetches slots into L2 (2 ahead 220, 8 ahead 296).
//
// 4-bit codes (in a graph, join included): the 13B-shaped batch 120 us, 0.81; the long
// contexts 94.5, 0.73 (8 query heads per KV head 121, 0.57; 2 86, 0.80; 1 80, 0.87), of which 9 us
// pass before the first slot is there and 5 in the join.  Without the consumers' arithmetic, after a
// flush: 126 us of 134, 90 of 104 and, 8 heads, 95 of 128.  96 registers are what 18 warps
// leave (five on one sub-partition): at head_dim 128 the compiler spills 36, 100 and 120 bytes
// a thread with 1, 2 and 4 query rows.
// Half the bytes of 8 bits for as many products: with the 8-bit consumer's shuffles and
// conversions 198 and 129.  What it took: lanes that weigh logits of their own and codes that
// enter the products unconverted (-9 and -5 %), two teams of 8 consumers in a CTA (-17 %, long
// contexts none), three operations in place of five per eight codes (-5 %), the bookkeeping of
// slots and shares without divisions (-5 %), shares weighed with items' ends (-4 %), weights
// transposed by movmatrix (long contexts -2 %): 116 and 85.  V's sums kept small for their
// accuracy's sake took 5 and 9 % of it back, references of the groups' own 2 % of the long
// contexts'.  Tried and slower: three ring slots for each team
// instead of two (150 us against 146 after a flush, long contexts 89 against 85 in a graph: more
// requests in flight only queue), queries read from memory to make room for them, 16
// consumers on one ring (250 against 226: 96 registers and a state each to join), two sets of
// consumers that take one item's slots in turn (304 against 207).  Four producer warps for one
// team took it from 207 to 191 before its bookkeeping was made shorter.
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
    static constexpr bool k8 = CT >= kCacheE4M3;         // codes with scales
    static constexpr bool k4 = CT == kCacheInt4;
    static constexpr int kRow = k4 ? D / 2 : k8 ? D : D * 2;     // bytes of one token and head
    static constexpr int kGroups = k4 ? D / 64 : 1;      // scales of a token and head
    static constexpr int kWarps = 8;                     // consumer warps
    static constexpr int kSub = k8 ? 2 : 1;              // stages per consumer warp and slot
    // Up to 4 query rows leave half of the products' 8 columns free: the weights'
    // high parts take columns 0-3 and their low parts columns 4-7 (the queries are
    // repeated there), one product in place of two.  (4-bit codes: even and odd columns.)
    static constexpr bool kPaired = C <= 4;
    static constexpr int kTiles = kWarps * kSub;         // (stage, head) tiles of a slot
    static constexpr int kRowB = kRow < 128 ? kRow : 128;         // bytes of one box row
    static constexpr int kHalves = kRow / kRowB;
    static constexpr int kKVBytes = kTiles * kStageTokens * kRow;      // a slot's K (or V) rows
    static constexpr int kScaleBytes = k8 ? kTiles * kStageTokens * 4 * kGroups : 0;
    static constexpr int kSlotBytes = (2 * kKVBytes + 2 * kScaleBytes + 1023) / 1024 * 1024;
    // Teams of a producer and its consumers, each with a ring and a share of the slots of its
    // own.  4-bit codes: two, since one's warps are too few to hide their own latencies (with
    // 8 query rows one of 168 registers is the faster: 121 us against 165, whose 96 spill 208
    // bytes, for 16 sequences of 16 K to 32 K tokens, 64 heads on 8).
    static constexpr int kTeams = k4 && C < 8 ? 2 : 1;
    // What an item's start and end cost, in slots: 4-bit slots are short enough for shares to
    // be weighed with it (256 13B-shaped sequences: teams with 18 items of a few slots took
    // 300,000 cycles, with 5 long ones 252,000).  It counts as lying before the item's slots.
    static constexpr int kItemExtra = k4 ? 1 : 0;
    static constexpr int kThreads = kTeams * (kWarps + 1) * 32;
    static constexpr int kMT = D / 16;
    static constexpr int kStateRow = D + 4;              // floats per query row of a warp's state
    static constexpr int kStateBytes = C * kStateRow * 4;
};

// One ring slot's description.
struct alignas(16) SlotMeta {
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

// 4-bit codes enter the products as they lie in a byte: as binary16 numbers, the low four
// bits alone are n0 2^-24 (subnormal, exact), and a whole byte is (16 n1 + n0) 2^-24.
// A register of eight codes so takes three ANDs and a byte permutation and no
// conversion; n1's share is the byte's less the low bits':
//   V product: an accumulator for either, subtracted once at an item's end;
//   K product, up to 4 query rows: even columns take q0 n0 and q1 n1 + q1 n0 / 16, odd
//   ones the q1 n0 / 16 to take off (8 rows fill the columns: n1 is masked out instead).
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// The registers' codes 0 and 4 (low) and, with 1 and 5, their bytes (kBytes) or 1 and 5
// alone 16 times larger; second: codes 2, 6 and 3, 7.
template <bool kBytes>
__device__ __forceinline__ void codes4(uint32_t (&low)[4], uint32_t (&high)[4], const uint32_t (&a)[4], bool second) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = second ? __byte_perm(a[k], 0u, 0x4341u) : a[k];
        low[k] = w & 0x000f000fu;
        high[k] = kBytes && second ? w : w & (kBytes ? 0x00ff00ffu : 0x00f000f0u);
    }
}
// The same codes and bytes of V, 4 times up: a product's terms are aligned by their
// exponents, which a denormal has as high as its format's lowest, and lose what lies 24 bits
// below (whole calls' errors of 3e-6 to 4e-6 become 2e-6).  Inverted where turned has bits
// (kTurned or 0): upper halves' codes n become 15 - n.
constexpr uint32_t kTurned = 0x03fc0000u;
__device__ __forceinline__ void value_codes4(uint32_t (&low)[4], uint32_t (&high)[4], const uint32_t (&a)[4], bool second,
                                             uint32_t turned) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = second ? a[k] >> 6 : a[k] << 2;
        low[k] = (w & 0x003c003cu) ^ (turned & 0x003c003cu);
        high[k] = (w & 0x03fc03fcu) ^ turned;
    }
}
// An 8 x 8 matrix of 16-bit elements, lane (g, t) holding (g, 2t) and (g, 2t + 1), transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// N words of scale and zero, neighbours in shared memory.
template <int N>
struct Words {
    uint32_t w[N];
};
template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t *p) {
    Words<N> r;
    if constexpr (N == 1) {
        r.w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        r.w[0] = v.x;
        r.w[1] = v.y;
    }
    return r;
}
__device__ __forceinline__ float word_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float word_zero(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Weights' high parts, as many bits as binary16 has (cut off, not rounded).
__device__ __forceinline__ float high_part(float w) { return __uint_as_float(__float_as_uint(w) & 0xffffe000u); }
__device__ __forceinline__ uint32_t pack2_rz(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Query elements, in [1, 2) at the largest, are taken this much larger (16 times that
// stays below binary16's 65504), so that those 2^-24 of it still are normal numbers.
constexpr float kQ4 = 1024.f;

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
    return static_cast<int>(((((p.e0 / kSplitEntries) * p.max_shares + cta) << p.log2_heads) + head) * p.cut_cols + col);
}

// Items (entry, partition, box of heads) in that order, weighed in slots: the
// boxes of one partition, whose rows lie next to one another, are read one after
// the other.  An entry without tokens weighs nothing, except where it costs the slot that writes
// its zero row.
struct ItemCursor {
    int e, len, nparts, part, grp, nslots;
    uint32_t start;
};

// (Divisions by the partition's, the block's and the shares' number are products; slots
// hold 2^lsw stages.  With the compiler's 32- and 64-bit divisions this bookkeeping took
// 2 us of a call.)
__device__ __forceinline__ int item_slots(int len, int part, int P, int lsw) {
    const int n = len - part * P;
    const int st = n > 0 ? (min(P, n) + kStageTokens - 1) >> 4 : 1;
    return (st + (1 << lsw) - 1) >> lsw;
}

// Modes in which a list of one partition is the whole result.
__device__ __forceinline__ bool final_mode(int mode) { return mode == kSplitDecode || mode == kSplitWhole; }

// EX: what an item costs beyond its slots, in slots.
template <int EX>
__device__ __forceinline__ uint32_t entry_weight(const SplitParams &p, int len, int ngroups, int lsw) {
    if (len <= 0) return final_mode(p.mode) ? static_cast<uint32_t>(ngroups * (1 + EX)) : 0u;
    const int P = p.partition_size;
    const int full = static_cast<int>(divided(static_cast<uint32_t>(len - 1), p.part_div));   // partitions before the last
    return static_cast<uint32_t>(ngroups) *
           static_cast<uint32_t>(full * (item_slots(P, 0, P, lsw) + EX) + item_slots(len, full, P, lsw) + EX);
}

template <int D, int C, int CT>
__global__ void __launch_bounds__((SplitLayout<D, C, CT>::kThreads), 1)
    paged_split_kernel(const __grid_constant__ SplitParams p, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, const __grid_constant__ CUtensorMap tmap_ks,
                       const __grid_constant__ CUtensorMap tmap_vs) {
    using L = SplitLayout<D, C, CT>;
    constexpr bool k8 = L::k8;
    constexpr bool BF16 = CT == kCacheBF16;   // MMA operand type
    constexpr int SUB = L::kSub, W = L::kWarps, TEAMS = L::kTeams, EX = L::kItemExtra, MT = L::kMT, KS = D / 16;
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
    constexpr int kLog2Tiles = L::kTiles == 8 ? 3 : 4;
    static_assert(L::kTiles == 1 << kLog2Tiles && kStageTokens == 16, "");
    const int lsw = kLog2Tiles - p.log2_heads;
    const int nsubs = W >> p.log2_heads;               // consumer warps per head
    const int RB = min(bs, kStageTokens);              // rows per box
    const int per_stage = kStageTokens / RB;           // boxes (blocks) per stage
    const int qmember = H * D * 2 << lg;               // one sequence's query rows of a box
    constexpr int kQEntry = C * D * 2;                 // x H: one query-ring entry

    // A team's part of shared memory: ring, queries, states, slots' descriptions, barriers.
    const int team = TEAMS == 1 ? 0 : warp / (W + 1), tw = TEAMS == 1 ? warp : warp % (W + 1);
    const size_t team_slots = static_cast<size_t>(S) * L::kSlotBytes;
    const int states = L::k4 && H < W ? W : W - H;
    const size_t team_rest = kQueryRing * kQEntry * H + states * L::kStateBytes + W * 8 * sizeof(float2) +
                             S * (sizeof(SlotMeta) + 16) + (2 * kQueryRing + 16) * 8;
    uint8_t *slots = smem + team * team_slots;
    uint8_t *qbuf = smem + TEAMS * team_slots + team * team_rest;
    uint8_t *xbuf = qbuf + kQueryRing * kQEntry * H;   // warp states
    float2 *xml = reinterpret_cast<float2 *>(xbuf + states * L::kStateBytes);    // [warp][8]
    SlotMeta *meta = reinterpret_cast<SlotMeta *>(xml + W * 8);
    uint64_t *full = reinterpret_cast<uint64_t *>(meta + S);
    uint64_t *empty = full + S;
    uint64_t *qfull = empty + S;
    uint64_t *qempty = qfull + kQueryRing;
    uint64_t *xfull = qempty + kQueryRing;             // per head: the other warps' states are written
    uint64_t *xfree = xfull + 8;                       //           and have been read
    uint32_t *warp_tot = reinterpret_cast<uint32_t *>(smem + TEAMS * (team_slots + team_rest));
    int *len_s = reinterpret_cast<int *>(warp_tot + 32);
    int *aux_s = len_s + E;                            // suffix: first block; prefix: sequence | members << 27;
                                                       // whole: the group's first sequence
    uint32_t *prefix = reinterpret_cast<uint32_t *>(aux_s + E);
    // Scales of 4 or 8 heads are 16 or 32 bytes per token: boxes.  Fewer are below
    // a box's least width: 4-byte copies by all lanes of the producer.  Those of 4-bit
    // codes are 32 to 128 neighbouring bytes per head and piece: boxes too, from 128 bytes
    // on (what a box's place in shared memory has to be a multiple of), else a bulk copy each.
    constexpr int kScaleTok = 4 * L::kGroups;          // bytes of a token's scales
    const uint32_t shead = static_cast<uint32_t>(L::k4 ? RB * kScaleTok : 4);   // next head's
    const uint32_t sbox = k8 ? static_cast<uint32_t>(RB * kScaleTok) << p.log2_heads : 0u;
    const bool scale_boxes = L::k4 ? sbox >= 128u : k8 && p.log2_heads >= 2;
    const bool lane_copies = k8 && !L::k4 && !scale_boxes;
    // Heads side by side in a row of a box: 4-bit rows of 32 or 64 bytes fill 128 together
    // (a box's rows, not its bytes, are what the copies' rate goes by).
    const int log2_row_heads = L::k4 ? min(p.log2_heads, D == 128 ? 1 : 2) : 0;
    const uint32_t rowB = static_cast<uint32_t>(L::kRowB) << log2_row_heads;

    if (tw == 0) {                 // the barriers, by the lanes of a team's first warp (8 of each kind at most)
        const int i = lane & 7;
        if (lane < 8) {
            if (i < S) {
                mbar_init(&full[i], lane_copies ? 33 : 1);
                mbar_init(&empty[i], W);
            }
        } else if (lane < 16) {
            if (i < kQueryRing) {
                mbar_init(&qfull[i], 1);
                mbar_init(&qempty[i], W);
            }
        } else if (lane < 24 && i < H) {
            mbar_init(&xfull[i], L::k4 ? nsubs : max(1, nsubs - 1));
            mbar_init(&xfree[i], L::k4 ? nsubs : 1);
        }
        fence_barrier_init();
        if (lane == 0) prefetch_tensormap(&tmap_k);
        if (lane == 1) prefetch_tensormap(&tmap_v);
        if (scale_boxes && lane == 2) prefetch_tensormap(&tmap_ks);
        if (scale_boxes && lane == 3) prefetch_tensormap(&tmap_vs);
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
    // (Asking for the block tables' lines meanwhile gains nothing, tables in L2 or not.)
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
        for (int i = beg; i < end; ++i) local += entry_weight<EX>(p, len_s[i], ngroups, lsw);
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
            run += entry_weight<EX>(p, len_s[i], ngroups, lsw);
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
    const uint32_t shares = gridDim.x * TEAMS, share = blockIdx.x * TEAMS + team;
    const uint32_t full_slots = static_cast<uint32_t>(item_slots(P, 0, P, lsw) + EX);    // of a whole partition
    const bool cut = p.cut && total >= shares * full_slots;
    // total share / shares, rounded down
    const uint32_t each = divided(total, p.share_div), left = total - each * shares;
    const uint32_t lo = each * share + divided(left * share, p.share_div);
    const uint32_t hi = each * (share + 1) + divided(left * (share + 1), p.share_div);

    if (tw == W) {
        // ------------------------------------------------------------ producer
        const uint64_t policy =
            mode == kSplitPrefix && p.chunks > 1 ? l2_policy_evict_normal() : l2_policy_evict_first();
        ItemCursor ic{};
        auto set_entry = [&](int e) {
            ic.e = e;
            ic.len = len_s[e];
            ic.nparts = ic.len > 0 ? static_cast<int>(divided(static_cast<uint32_t>(ic.len + P - 1), p.part_div)) : 1;
        };
        auto set_part = [&](int part) {
            ic.part = part;
            ic.nslots = item_slots(ic.len, part, P, lsw);
        };
        auto advance = [&]() {
            ic.start += ic.nslots + EX;
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
            const uint32_t pw = static_cast<uint32_t>(ngroups) * full_slots;
            const uint32_t off = lo - prefix[a];
            set_part(min(ic.nparts - 1, static_cast<int>(off / pw)));
            const uint32_t pstart = prefix[a] + static_cast<uint32_t>(ic.part) * pw;
            const int weight = ic.nslots + EX;
            const int grp = static_cast<int>((lo - pstart + (cut ? 0 : weight - 1)) / weight);
            ic.grp = min(grp, ngroups - 1);
            ic.start = pstart + static_cast<uint32_t>(ic.grp) * weight;
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
            fb = static_cast<int>(divided(static_cast<uint32_t>(t0), p.block_div));
            if (mode == kSplitWhole && fb + lane < shared_blocks(p, seq, ic.len, false)) row = aux_s[ic.e];
            bid = -1;
            if (ntok > 0 && lane <= static_cast<int>(divided(static_cast<uint32_t>(t0 + ntok - 1), p.block_div)) - fb)
                bid = __ldg(p.block_tables + static_cast<int64_t>(row) * p.max_blocks_per_seq + blk0 + fb + lane);
        };
        // The slot's pieces are RB rows of one block (SW * per_stage of them, at most 32), one
        // per lane.  Where a piece lies in a slot, and how far its token moves from slot to slot:
        const int pieces = SW * per_stage;
        const uint32_t box = static_cast<uint32_t>(RB * L::kRowB) << p.log2_heads;
        const uint32_t piece_off = per_stage == 1 ? lane * (box * L::kHalves)
                                                  : (lane >> 1) * (2 * box * L::kHalves) + (lane & 1) * box;
        const int step_blocks = static_cast<int>(divided(SW * kStageTokens, p.block_div)), step_rows = SW * kStageTokens - step_blocks * bs;
        int islot = 0;
        uint32_t uses = 0, items = 0, phase = 1;       // phase: of the wait for a slot, once the ring has been gone round
        bool ok = true;
        auto take_slot = [&]() -> int {
            const int slot = islot;
            if (uses >= static_cast<uint32_t>(S)) {
                const uint32_t par = phase;
                if (!mbar_try_wait(&empty[slot], par) && !mbar_wait_bounded(&empty[slot], par)) {
                    if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                    ok = false;
                }
            }
            ok = __all_sync(kFull, ok);
            if (ok) {
                if (++islot == S) {
                    islot = 0;
                    phase ^= 1u;
                }
                ++uses;
            }
            return slot;
        };
        while (ok && work && ic.start < hi) {
            const int kvh0 = ic.grp << p.log2_heads;
            // this share's slots of the item
            const int jb = cut ? max(0, static_cast<int>(lo - ic.start) - EX) : 0;
            const int je = cut ? min(ic.nslots, static_cast<int>(hi - ic.start) - EX) : ic.nslots;
            if (EX > 0 && je <= 0) break;      // the share ends before the item's first slot
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
            const int kind = jb > 0               ? kContinued
                             : je < ic.nslots     ? kCut
                             : final_mode(mode) && ic.nparts == 1 ? kFinal
                                                                  : 0;
            // my piece's block (of the partition's) and its first row in it
            const int first = jb * SW * kStageTokens + (t0 - fb * bs) + lane * RB;
            int pblk = static_cast<int>(divided(static_cast<uint32_t>(first), p.block_div)), prow = first - pblk * bs;
            for (int j = jb; j < je; ++j) {
                const int slot = take_slot();
                if (!ok) break;
                uint8_t *sp = slots + static_cast<size_t>(slot) * L::kSlotBytes;
                const int nt = max(0, min(SW * kStageTokens, ntok - j * SW * kStageTokens));   // valid tokens
                const bool has = lane < pieces && lane * RB < nt;
                const int id = __shfl_sync(kFull, bid, has ? pblk : 0);
                const int row = prow;
                pblk += step_blocks;
                if ((prow += step_rows) >= bs) {
                    prow -= bs;
                    ++pblk;
                }
                const bool load = has && id >= 0 && static_cast<int64_t>(id) < p.num_blocks;
                const uint32_t loaded = __ballot_sync(kFull, load);
                uint32_t bad = __ballot_sync(kFull, has && !load);
                if (bad && lane == 0) report(p.err_flag, 0x2 /* PA_FLAG_BAD_BLOCK_ID */);
                if (bad && per_stage == 1) {   // one bit per stage -> two
                    uint32_t w = 0;
                    for (int i = 0; i < SW; ++i) w |= ((bad >> i) & 1u) * (3u << (2 * i));
                    bad = w;
                }
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
                                          static_cast<uint32_t>(__popc(loaded)) * 2u * (box * L::kHalves + (lane_copies ? 0u : sbox)));
                }
                __syncwarp();
                const int z = load ? id * bs + row : 0;                     // the piece's first cache slot
                if (load) {
                    uint8_t *dst = sp + piece_off;
#pragma unroll
                    for (int h = 0; h < L::kHalves; ++h) {
                        const uint32_t ho = h * per_stage * box;
                        tma_load_3d(dst + ho, &tmap_k, &full[slot], h * (D / L::kHalves), z, kvh0 >> log2_row_heads, policy);
                        tma_load_3d(dst + L::kKVBytes + ho, &tmap_v, &full[slot], h * (D / L::kHalves), z,
                                    kvh0 >> log2_row_heads, policy);
                    }
                }
                if constexpr (L::k4) {
                    // scales, [piece][head of the box][token][group], K then V
                    uint8_t *ss = sp + 2 * L::kKVBytes + lane * sbox;
                    if (load) {
                        const int y = id * Hkv + kvh0, x = row * L::kGroups;
                        if (scale_boxes) {
                            tma_load_2d(ss, &tmap_ks, &full[slot], x, y);
                            tma_load_2d(ss + L::kScaleBytes, &tmap_vs, &full[slot], x, y);
                        } else {
                            const int64_t src = static_cast<int64_t>(y) * bs * L::kGroups + x;
                            for (int h = 0; h < H; ++h) {
                                bulk_load(ss + h * shead, p.k_scales + src + h * bs * L::kGroups, shead, &full[slot]);
                                bulk_load(ss + L::kScaleBytes + h * shead, p.v_scales + src + h * bs * L::kGroups, shead,
                                          &full[slot]);
                            }
                        }
                    }
                } else if constexpr (k8) {
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
                if (lane_copies) {
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
    const int head = tw & (H - 1), sub = tw >> p.log2_heads;
    const int g = lane >> 2, t = lane & 3;
    const int r8 = lane & 7, j8 = lane >> 3;
    const uint32_t slots_sa = smem_addr(slots);
    const uint32_t box = static_cast<uint32_t>(RB * L::kRowB) << p.log2_heads;
    const uint32_t half_off = box * per_stage;                       // next 128-byte column block
    const uint32_t stage_off = half_off * L::kHalves;
    const int row_head = head & ((1 << log2_row_heads) - 1);         // my head's place in a row
    const uint32_t head_off = (head >> log2_row_heads) * RB * rowB;
    const uint32_t hi_off = per_stage == 1 ? 8 * rowB : box;         // rows 8-15 of a stage
    // A lane's 16-byte chunk 2 i + (0 or 1) of its row sits, swizzled, at the row's
    // start + 16 ((2 i + b) ^ swz): the address for i = 0, with 32 i flipped in.
    const uint32_t swz = rowB == 128 ? r8 : rowB == 64 ? (r8 >> 1) & 3 : (r8 >> 2) & 1;
    const uint32_t chunk0 = row_head * (L::kRowB / 16);
    const uint32_t off_k = head_off + (j8 & 1) * hi_off + r8 * rowB + (((chunk0 + (j8 >> 1)) ^ swz) << 4);
    const uint32_t off_v = L::kKVBytes + head_off + (j8 >> 1) * hi_off + r8 * rowB + (((chunk0 + (j8 & 1)) ^ swz) << 4);
    // 8-bit caches: my tokens' scales in a slot (K; V scales kScaleBytes further)
    const uint32_t scl_off = 2 * L::kKVBytes + ((((sub * SUB * kStageTokens + g) << p.log2_heads) + head) << 2);
    const uint32_t scl_8 = 32u << p.log2_heads;                      // 8 tokens further
    // 4-bit: my head's tokens of my first stage; the next stage's; 8 tokens further
    const uint32_t s4_off = 2 * L::kKVBytes + sub * SUB * per_stage * sbox + head * shead;
    const uint32_t s4_8 = per_stage == 1 ? 8 * kScaleTok : sbox, s4_st = per_stage * sbox;
    const uint64_t keep = l2_policy_evict_last();

    uint32_t qf[KS][2];
    float qs[2];                  // logit scale of columns 2t, 2t + 1
    float acc[MT][4], m_run[2], l_run[2];
    // 4-bit codes: what a lane weighs of the logits it holds (rows g and g + 8 of a stage's
    // tokens, columns 2t and 2t + 1).  Up to 4 query rows are repeated in the even columns,
    // so that every lane has logits to weigh, and each weighs one column:
    //   1 query row:  the slot's stage t & 1; its V weights for group t >> 1
    //   2 query rows: row t & 1, stage t >> 1
    //   4: row t; 8: rows 2t and 2t + 1 (both columns); one stage after the other.
    // A lane's weights are the columns 2t and 2t + 1 of the V product too, as the high and
    // low part of one (8 rows: of the two rows, the low parts in a product of their own), so
    // that its sums, references and results are of the same rows throughout.
    constexpr int NX = C == 8 ? 2 : 1, ZG = C == 1 ? 1 : L::kGroups;
    const int my_stage = C == 1 ? t & 1 : t >> 1, my_group = t >> 1;
    float qsum[L::kGroups][2];    // the sum of a group's query elements, as large as the products have them
    float zs[ZG][NX];             // the sum of weight, scale and zero
    // both groups: the power of two that a group's weights are taken up by, in acc and zs too
    constexpr bool kUp = ZG > 1;
    [[maybe_unused]] float up[ZG][NX];
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
            const int gq = !L::kPaired ? g : L::k4 ? (g >> 1) & (C - 1) : g & 3;   // my column's query row
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
            } else if constexpr (L::k4) {
                // Step 4 gr + i takes elements 8t + i and 8t + i + 4 of group gr's first
                // half and of its second; even steps meet low codes, 16 times smaller.  Up
                // to 4 rows: odd columns as said at codes4.
                uint4 w[2 * L::kGroups];
#pragma unroll
                for (int c = 0; c < 2 * L::kGroups; ++c)
                    w[c] = live ? *reinterpret_cast<const uint4 *>(qw + (32 * c + 8 * t) / 2) : make_uint4(0u, 0u, 0u, 0u);
                float f[2 * L::kGroups][8], amax = 0.f;
#pragma unroll
                for (int c = 0; c < 2 * L::kGroups; ++c) {
                    const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 x = p.q_bf16 ? Half2x<true>::to_float2(v[k]) : Half2x<false>::to_float2(v[k]);
                        f[c][2 * k] = x.x;
                        f[c][2 * k + 1] = x.y;
                        amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
                    }
                }
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
                // 2^e <= amax < 2^(e+1), e kept where 2^e and kQ4 16 2^-e are normal
                const uint32_t eb = min(max(__float_as_uint(amax) & 0x7f800000u, 0x08000000u), 0x7e800000u);
                const bool odd = L::kPaired && (g & 1);
                const float inv = __uint_as_float(0x7f000000u - eb) * kQ4;
                const float m0 = odd ? 0.f : 16.f * inv, m1 = odd ? 0.f : inv, m1low = odd ? inv : 0.f;
#pragma unroll
                for (int gr = 0; gr < L::kGroups; ++gr) {
                    float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float(&v)[8] = f[2 * gr + k];
                            qf[4 * gr + i][k] = pack2<false>(fmaf(v[i], m0, v[i + 1] * m1low), fmaf(v[i + 4], m0, v[i + 5] * m1low));
                            qf[4 * gr + i + 1][k] = pack2<false>(v[i + 1] * m1, v[i + 5] * m1);
                        }
                        // the sum of the elements: what codes of 1 would give
                        const uint32_t one[4] = {0x00010001u, 0x00010001u, 0x00010001u, 0x00010001u};
                        constexpr uint32_t kHigh = L::kPaired ? 0x00110011u : 0x00100010u;
                        const uint32_t high[4] = {kHigh, kHigh, kHigh, kHigh};
                        mma_f16(sums, one, qf[4 * gr + i]);
                        mma_f16(sums, high, qf[4 * gr + i + 1]);
                    }
                    qsum[gr][0] = L::kPaired ? sums[0] - sums[1] : sums[0];
                    qsum[gr][1] = sums[1];
                }
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr)
#pragma unroll
                    for (int e = 0; e < NX; ++e) {
                        zs[gr][e] = 0.f;
                        up[gr][e] = 1.f;
                    }
                const float logits = __uint_as_float(eb) * p.scale_log2 * (0x1p20f / kQ4);
                qs[0] = __shfl_sync(kFull, logits, 8 * t);
                qs[1] = __shfl_sync(kFull, logits, 8 * t + 4);
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
        // 4-bit codes: NS stages from st0 + first on (both where a lane weighs one of them).
        auto attend4 = [&](auto whole_tag, int first) {
            constexpr bool kWhole = decltype(whole_tag)::value;
            constexpr int NS = C <= 2 ? SUB : 1;
            const uint32_t stage = sa + (st0 + first) * stage_off;
            // ---- QK: 16 tokens x 8 columns, a group's codes apart ----
            float c[NS][L::kGroups][4];
#pragma unroll
            for (int hs = 0; hs < NS; ++hs) {
                uint32_t a[L::kGroups][4], low[4], high[4];
#pragma unroll
                for (int gr = 0; gr < L::kGroups; ++gr) {
                    ldsm_x4(a[gr], (stage + hs * stage_off + off_k) ^ (gr << 5));
                    c[hs][gr][0] = c[hs][gr][1] = c[hs][gr][2] = c[hs][gr][3] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; i += 2)
#pragma unroll
                    for (int gr = 0; gr < L::kGroups; ++gr) {
                        codes4<L::kPaired>(low, high, a[gr], i > 0);
                        mma_f16(c[hs][gr], low, qf[4 * gr + i]);
                        mma_f16(c[hs][gr], high, qf[4 * gr + i + 1]);
                    }
            }
            // ---- logits, and the scales and zeros of the weights to come ----
            float x[2][NX], vsc[2][ZG], vz[2][ZG];
            bool below = false;
            const int st = first + (NS > 1 ? my_stage : 0);          // the stage I weigh
            const uint8_t *ks = sp + s4_off + st * s4_st + g * kScaleTok, *vs = ks + L::kScaleBytes;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                // a masked token's scales may be anything: its V scales count as 0
                const bool ok = kWhole || (g + 8 * k < mine - st * kStageTokens && !((m.bad >> (2 * (st0 + st) + k)) & 1u));
                const Words<L::kGroups> kw = load_words<L::kGroups>(ks + k * s4_8), vw = load_words<L::kGroups>(vs + k * s4_8);
                float sum[NX] = {};
#pragma unroll
                for (int gr = 0; gr < L::kGroups; ++gr) {
#pragma unroll
                    for (int e = 0; e < NX; ++e) {
                        float cv[NS];
#pragma unroll
                        for (int hs = 0; hs < NS; ++hs)
                            cv[hs] = L::kPaired ? c[hs][gr][2 * k] - c[hs][gr][2 * k + 1] : c[hs][gr][2 * k + e];
                        const float one = NS > 1 && my_stage ? cv[NS - 1] : cv[0];
                        sum[e] = fmaf(word_scale(kw.w[gr]), fmaf(word_zero(kw.w[gr]), qsum[gr][e], one), sum[e]);
                    }
                }
#pragma unroll
                for (int e = 0; e < NX; ++e) x[k][e] = ok ? sum[e] * qs[e] : -INFINITY;
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr) {
                    const uint32_t w = ZG == 1 && my_group ? vw.w[L::kGroups - 1] : vw.w[gr];
                    vsc[k][gr] = ok ? word_scale(w) : 0.f;
                    vz[k][gr] = ok ? word_zero(w) : 0.f;
                    below = below || vz[k][gr] < 0.f;
                }
            }
            // Values on both sides of 0: every second token enters with its codes turned, 15 - n,
            // and its weight negative: w (n + z) = -w (15 - n) + w (z + 15).  Sums over codes
            // of one sign would grow far above the result, and the products cut off their
            // accumulators' low bits every time: 7e-5 to 3e-4 of the result after 32 K tokens,
            // 2e-6 with it at any length (13B-shaped 122 us against 116, long contexts 92 against
            // 85; with the 8s' sum taken off by products of its own 121 and 99, with all codes as
            // normal numbers 3e-7 to 2e-6, 151 and 116).  Rows of zeros have zeros of 0 and sum up
            // to 0.
            const bool turns = __any_sync(kFull, below);
            const uint32_t turned = turns ? kTurned : 0u;
            const float side = turns && (g & 1) ? -1.f : 1.f, top = turns && (g & 1) ? -15.f : 0.f;
            // ---- weights under the present references, as for 8 bits; wt: with their scales, and where
            // there is one group of them, their sides ----
            float pw[2][NX], wt[2][ZG][NX];
            auto weigh = [&]() {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int e = 0; e < NX; ++e) {
                        pw[k][e] = fast_exp2(x[k][e] - mu[e]);
#pragma unroll
                        for (int gr = 0; gr < ZG; ++gr)
                            wt[k][gr][e] = kUp ? pw[k][e] * vsc[k][gr] * up[gr][e] : pw[k][e] * (vsc[k][gr] * side);
                    }
            };
            weigh();
            bool nd = false;
#pragma unroll
            for (int e = 0; e < NX; ++e) {
                nd = nd || m_run[e] == -INFINITY;
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr) {
                    const float a = wt[0][gr][e], b = wt[1][gr][e];
                    nd = nd || (kUp ? fmaxf(a, b) : fmaxf(fabsf(a), fabsf(b))) > kWeightMax;
                }
            }
            if (__any_sync(kFull, nd)) {
                float al[ZG][NX];
#pragma unroll
                for (int e = 0; e < NX; ++e) {
                    float mx[ZG], mn = m_run[e];
#pragma unroll
                    for (int gr = 0; gr < ZG; ++gr) {
                        // (a scale that is no number makes its own group's sums such, not the reference)
                        mx[gr] = fmaxf(x[0][e] + fast_log2(fmaxf(vsc[0][gr], kScaleFloor)),
                                       x[1][e] + fast_log2(fmaxf(vsc[1][gr], kScaleFloor)));
#pragma unroll
                        for (int o = C == 1 ? 1 : C == 2 ? 2 : 4; o < 32; o <<= 1)
                            if (C != 1 || L::kGroups == 1 || o != 2) mx[gr] = fmaxf(mx[gr], __shfl_xor_sync(kFull, mx[gr], o));
                        mn = fmaxf(mn, mx[gr] - kWeightExp);
                    }
                    const float fall = m_run[e] - mn;
                    l_run[e] *= mn == -INFINITY ? 1.f : fast_exp2(fall);
#pragma unroll
                    for (int gr = 0; gr < ZG; ++gr) {
                        float rise = 0.f;
                        if constexpr (kUp) {
                            // the group's own reference, m less the exponent it is taken up by, never falls
                            const float had = static_cast<float>(static_cast<int>(__float_as_uint(up[gr][e]) >> 23) - 127);
                            const float ref = fmaxf(m_run[e] - had, mx[gr] - kWeightExp);
                            const float has = fminf(fmaxf(floorf(mn - ref), 0.f), 126.f);    // (0 while there is no reference)
                            up[gr][e] = __uint_as_float(static_cast<uint32_t>(127 + static_cast<int>(has)) << 23);
                            rise = has - had;
                        }
                        al[gr][e] = mn == -INFINITY ? 1.f : fast_exp2(fall + rise);
                        zs[gr][e] *= al[gr][e];
                    }
                    m_run[e] = mn;
                    mu[e] = mn == -INFINITY ? 0.f : mn;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[mt][e] *= al[kUp ? mt / 4 : 0][C == 8 ? e & (NX - 1) : 0];
                weigh();
            }
            // ---- those as binary16 parts: the high and low part of one column (8 rows: the two
            // columns' high parts, and their low ones) ----
            uint32_t ph[2][ZG];
            [[maybe_unused]] uint32_t pl[2][ZG];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int e = 0; e < NX; ++e) l_run[e] += pw[k][e];
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr) {
                    float(&w)[NX] = wt[k][gr];
#pragma unroll
                    for (int e = 0; e < NX; ++e) {
                        if constexpr (kUp) w[e] *= side;
                        zs[gr][e] = fmaf(w[e], fmaf(vz[k][gr], side, top), zs[gr][e]);
                    }
                    if constexpr (L::kPaired) {
                        ph[k][gr] = pack2_rz(w[0], w[0] - high_part(w[0]));
                    } else {
                        ph[k][gr] = pack2_rz(w[0], w[NX - 1]);
                        pl[k][gr] = pack2_rz(w[0] - high_part(w[0]), w[NX - 1] - high_part(w[NX - 1]));
                    }
                }
            }
            // ---- PV: the weights transposed to tokens 2t, 2t + 1, 2t + 8, 2t + 9 of column g ----
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr) {
                    ph[k][gr] = transposed(ph[k][gr]);
                    if constexpr (!L::kPaired) pl[k][gr] = transposed(pl[k][gr]);
                }
#pragma unroll
            for (int hs = 0; hs < NS; ++hs) {
#pragma unroll
                for (int gr = 0; gr < L::kGroups; ++gr) {
                    // (up to 2 rows: the columns made for this stage and group)
                    const bool of = C == 1 ? (g >> 1) == hs + 2 * gr : C == 2 ? (g >> 2) == hs : true;
                    uint32_t a[4], low[4], high[4], w[2];
                    ldsm_x4_trans(a, (stage + hs * stage_off + off_v) ^ (gr << 5));
#pragma unroll
                    for (int k = 0; k < 2; ++k) w[k] = of ? ph[k][ZG == 1 ? 0 : gr] : 0u;
#pragma unroll
                    for (int i = 0; i < 4; i += 2) {
                        value_codes4(low, high, a, i > 0, turned);
                        mma_f16(acc[4 * gr + i], low, w);
                        mma_f16(acc[4 * gr + i + 1], high, w);
                        if constexpr (!L::kPaired) {
                            const uint32_t wl[2] = {pl[0][gr], pl[1][gr]};
                            mma_f16(acc[4 * gr + i], low, wl);
                            mma_f16(acc[4 * gr + i + 1], high, wl);
                        }
                    }
                }
            }
        };
        auto consume = [&](auto whole_tag) {
            if constexpr (!L::k4) {
                attend(whole_tag);
            } else if constexpr (C <= 2) {
                attend4(whole_tag, 0);
            } else {
#pragma unroll 1
                for (int i = 0; i < SUB; ++i) attend4(whole_tag, i);
            }
        };
        if (mine >= SUB * kStageTokens && m.bad == 0)
            consume(std::true_type{});
        else if (mine > 0)
            consume(std::false_type{});
        // my reads (and zeroing: not of 4-bit slots) of the slot are done
        if constexpr (!L::k4) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&empty[slot]);

        if (!(m.flags & kLast)) continue;
        // ---- item end ----
        if constexpr (L::k4) {
            // sums over low codes and over bytes: their powers of two off, the bytes' low codes too
#pragma unroll
            for (int mt = 0; mt < MT; mt += 2)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[mt + 1][e] = (acc[mt + 1][e] - acc[mt][e]) * 0x1p18f;
                    acc[mt][e] *= 0x1p22f;
                }
            // sums over the lanes that weighed for one row
            auto total = [&](float v, int first) {
                if constexpr (C == 1) v += __shfl_xor_sync(kFull, v, 1);
                if constexpr (C == 2) v += __shfl_xor_sync(kFull, v, 2);
#pragma unroll
                for (int o = 4; o < first; o <<= 1) v += __shfl_xor_sync(kFull, v, o);
                return v;
            };
#pragma unroll
            for (int e = 0; e < NX; ++e) {
                l_run[e] = total(l_run[e], 32);
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr) zs[gr][e] = total(zs[gr][e], 32);    // the zeros' share of a group's elements
            }
            const bool fin = (m.flags & kFinal) != 0;
            // What takes a group's sums back to the row's reference.  Two groups weighed by lanes
            // apart: the larger reference and the sum under it, but for whole results, which
            // need none in common.
            [[maybe_unused]] float down[ZG][NX];
            constexpr bool kApart = C == 1 && L::kGroups == 2;
            if constexpr (kUp) {
#pragma unroll
                for (int gr = 0; gr < ZG; ++gr)
#pragma unroll
                    for (int e = 0; e < NX; ++e) down[gr][e] = __uint_as_float(0x7f000000u - __float_as_uint(up[gr][e]));
            } else if constexpr (kApart) {
                down[0][0] = 1.f;
                if (!fin || nsubs > 1) {
                    const float om = __shfl_xor_sync(kFull, m_run[0], 2), ol = __shfl_xor_sync(kFull, l_run[0], 2);
                    if (om > m_run[0]) {
                        down[0][0] = fast_exp2(m_run[0] - om);
                        m_run[0] = om;
                        l_run[0] = ol;
                    }
                }
            }
            // My results, quads of neighbouring elements 4g .. 4g + 3 of a group's halves:
            // 1 row: those of group t >> 1, else of every group.
            constexpr int NQ = C == 1 ? 2 : 2 * L::kGroups;
            auto quad = [&](int e, int i) {
                const int gr = i >> 1, r = 2 * (i & 1);
                float q[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    auto part = [&](int mt) { return C == 8 ? acc[mt][r + e] : acc[mt][r] + acc[mt][r + 1]; };
                    float v = part(4 * gr + j);
                    if constexpr (C == 1 && L::kGroups == 2)
                        if (my_group) v = part(4 + j);
                    q[j] = total(v, 4) + zs[gr][e];
                    if constexpr (kUp || kApart) q[j] *= down[gr][e];
                }
                return make_float4(q[0], q[1], q[2], q[3]);
            };
            auto element = [&](int i) { return (C == 1 ? 64 * my_group + 32 * i : 64 * (i >> 1) + 32 * (i & 1)) + 4 * g; };
            const bool writes = C == 1 ? (t & 1) == 0 && my_group < L::kGroups : C == 2 ? t < 2 : true;
            auto row_of = [&](int e) { return C == 8 ? 2 * t + e : t & (C - 1); };
            const bool tells = g == 0 && (C == 1 ? t == 0 : writes);
            const int kvh = m.kvh0 + head;
            // A row's reference and sum, and quads of it, into the output or a row of the workspace.
            auto row_at = [&](int c) -> int64_t {
                return (m.flags & kContinued)
                           ? p.cut_row + cut_row_of(p, share, head, c)
                           : (((static_cast<int64_t>(m.seq) * Hkv + kvh) * p.max_parts + p.part_off + m.part) << lg) + c;
            };
            auto tell_row = [&](int c, float ref, float l) {
                if (fin && p.ws_ml == nullptr) return;
                const bool more = (m.flags & kCut) != 0;
                st_global_hint(p.ws_ml + 4 * row_at(c),
                               make_float4(ref, l, __int_as_float(fin ? kRowFinal : more ? kRowCut : 0),
                                           __int_as_float(more ? cut_row_of(p, share + 1, head, c) : 0)),
                               keep);
            };
            auto put = [&](int64_t at, float4 q, float sc) {
                if (!fin) {
                    st_global_hint(p.ws_acc + at, q, keep);
                    return;
                }
                q = make_float4(q.x * sc, q.y * sc, q.z * sc, q.w * sc);
                if (p.out_dtype == 2)
                    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = q;
                else
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
                        p.out_dtype == 1 ? make_uint2(pack2<true>(q.x, q.y), pack2<true>(q.z, q.w))
                                         : make_uint2(pack2<false>(q.x, q.y), pack2<false>(q.z, q.w));
            };
            auto out_at = [&](int c) {
                return fin ? (static_cast<int64_t>(m.seq) * Hq + (kvh << lg) + c) * D : row_at(c) * D;
            };
            if (nsubs == 1) {
#pragma unroll
                for (int e = 0; e < NX; ++e) {
                    const int c = row_of(e);
                    const float l = l_run[e], sc = l == 0.f ? 0.f : 1.f / l;
                    if (tells) tell_row(c, m_run[e], l);
                    const int64_t at = out_at(c);
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        const float4 q = quad(e, i);
                        if (writes) put(at + element(i), q, sc);
                    }
                }
                continue;
            }
            // Warps that share a head: all put their states into shared memory, and each joins its
            // share of the rows' quads.
            const uint32_t par = (citems - 1) & 1u;          // of this item
            if (citems > 1 && !mbar_try_wait(&xfree[head], par ^ 1u) && !mbar_wait_bounded(&xfree[head], par ^ 1u)) {
                if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                return;
            }
            {
                float *xs = reinterpret_cast<float *>(xbuf + tw * L::kStateBytes);
#pragma unroll
                for (int e = 0; e < NX; ++e) {
#pragma unroll
                    for (int i = 0; i < NQ; ++i) {
                        const float4 q = quad(e, i);
                        if (writes) *reinterpret_cast<float4 *>(xs + row_of(e) * L::kStateRow + element(i)) = q;
                    }
                    if (tells) xml[tw * 8 + row_of(e)] = make_float2(m_run[e], l_run[e]);
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&xfull[head]);
            if (!mbar_try_wait(&xfull[head], par) && !mbar_wait_bounded(&xfull[head], par)) {
                if (lane == 0) report(p.err_flag, 0x10 /* PA_FLAG_TIMEOUT */);
                return;
            }
            for (int i = sub * 32 + lane; i < C * D / 4; i += nsubs * 32) {
                const int c = i / (D / 4), d = i % (D / 4) * 4;
                float ref = -INFINITY, l = 0.f;
                for (int k = 0; k < nsubs; ++k) ref = fmaxf(ref, xml[(head + k * H) * 8 + c].x);
                float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int k = 0; k < nsubs; ++k) {
                    const float2 ml = xml[(head + k * H) * 8 + c];
                    const float be = ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - ref);
                    const float4 x =
                        *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(xbuf + (head + k * H) * L::kStateBytes) +
                                                          c * L::kStateRow + d);
                    l = fmaf(ml.y, be, l);
                    q = make_float4(fmaf(x.x, be, q.x), fmaf(x.y, be, q.y), fmaf(x.z, be, q.z), fmaf(x.w, be, q.w));
                }
                if (d == 0) tell_row(c, ref, l);
                put(out_at(c) + d, q, l == 0.f ? 0.f : 1.f / l);
            }
            __syncwarp();
            if (lane == 0) arrive(&xfree[head]);
            continue;
        }
        if constexpr (!L::k4) {
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
                    float *xs = reinterpret_cast<float *>(xbuf + (tw - H) * L::kStateBytes);
#pragma unroll
                    for (int e = 0; e < NE; ++e) {
                        const int c = 2 * t + e;
                        if (c >= C) continue;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            xs[c * L::kStateRow + 16 * mt + g] = acc[mt][e];
                            xs[c * L::kStateRow + 16 * mt + 8 + g] = acc[mt][2 + e];
                        }
                        if (g == 0) xml[tw * 8 + c] = make_float2(m_run[e], l_run[e]);
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
                    for (int k = 1; k < nsubs; ++k) mn = fmaxf(mn, xml[(tw + k * H) * 8 + c].x);
                    const float al = m_run[e] == -INFINITY ? 1.f : fast_exp2(m_run[e] - mn);
                    m_run[e] = mn;
                    l_run[e] *= al;
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        acc[mt][e] *= al;
                        acc[mt][2 + e] *= al;
                    }
                    for (int k = 1; k < nsubs; ++k) {
                        const float *xs = reinterpret_cast<const float *>(xbuf + (tw + (k - 1) * H) * L::kStateBytes) +
                                          c * L::kStateRow + g;
                        const float2 ml = xml[(tw + k * H) * 8 + c];
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
                        ? p.cut_row + cut_row_of(p, share, head, c)
                        : (((sq * Hkv + kvh) * p.max_parts + p.part_off + m.part) << lg) + hq;
                if (g == 0 && !(fin && p.ws_ml == nullptr)) {
                    const bool more = (m.flags & kCut) != 0;
                    st_global_hint(p.ws_ml + 4 * r,
                                   make_float4(m_run[e], l_run[e], __int_as_float(fin ? kRowFinal : more ? kRowCut : 0),
                                               __int_as_float(more ? cut_row_of(p, share + 1, head, c) : 0)),
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
