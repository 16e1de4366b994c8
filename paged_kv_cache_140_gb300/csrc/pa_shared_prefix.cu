// Attention of a group's query rows over the prefix they share, on the
// fifth-generation tensor cores: partial softmax states only.
//
// For group g, KV head h and the n G query rows of its n sequences (G query
// heads each), over the group's L shared tokens (whole blocks, reached through
// its first member's block table):
//     s_rp = scale log2(e) <q_r, K_p>,  m_r ~ max_p s_rp - 7,
//     l_r = sum_p 2^(s_rp - m_r),  acc_r = sum_p 2^(s_rp - m_r) V_p,
// written as partial results that pa_split_merge.cu joins with those of the
// sequences' private parts.  There is no causal mask: every row sees every
// shared token, which is what makes the product dense.
//
// What bounds it: with 128 rows per K/V tile the tensor cores (2 x 128 x 128 x D
// products per tile, half as many again for bfloat16, whose weights go in as a
// high and a low part; binary16 weights are rounded once, 11 bits, and summed as
// rounded), with few rows the K/V loads.  A unit is a query tile of 128 rows or a pair
// of them, a KV head and a range of tokens; the range is chosen by the host so that
// the units fill the SMs in whole waves.
//
// Groups of up to 128 rows (NS = 1): one stream per CTA, a query tile over every K/V
// tile of the range, and two CTAs per SM, so that one's start, end and softmax run
// under the other's loads and products.  Its 128 registers a thread hold 32 scores of a
// row at a time.
// Larger groups (NS = 2): pairs of tiles, one CTA per SM with two streams, X = A and B,
// each with its own scores and output in tensor memory, so that one stream's softmax
// runs under the other's products:
//   two query tiles: stream X is query tile X, both over every K/V tile loaded
//                    (each byte brought in feeds 256 rows);
//   one query tile (the odd last, or a smaller group): the streams take the range's
//                    first and second half of the K/V tiles, with the same queries,
//                    and write two partials.
// Per stream and K/V tile: S = Q K^T (tcgen05.mma from shared memory), softmax by
// one thread per row (NS = 2: its 128 scores in registers; the output rescaled only
// when the maximum grows by more than 2^8), weights back over S in four chunks of 32
// keys released one by one, O += P V (P from tensor memory).
//
// Warps: four per stream for softmax and output, then one that loads K tiles, one that
// issues the products and one that loads V tiles (TMA, one box per block and 64
// columns): 7 or 11.  Warps whose rows are all past the group's end skip the softmax.
// Every wait is bounded (2 s) and reports PA_FLAG_TIMEOUT.
#include <math_constants.h>

#include "pa.h"
#include "pa_shared_prefix.h"
#include "pa_split_kernel.cuh"
#include "pa_umma.cuh"

namespace pa {

namespace {

constexpr int kTile = kSharedTile;
constexpr int kRegion = kTile * 128;     // 128 rows x 128 bytes: one swizzled operand region
// NS streams: S/P of stream X in tensor-memory columns 128 X, O of X behind them.
template <int NS> struct Streams {
    static constexpr uint32_t kCols = 256 * NS, kColO = 128 * NS;
    static constexpr int kWarpK = 4 * NS, kWarpMma = kWarpK + 1, kWarpV = kWarpK + 2;
    static constexpr int kThreads = (4 * NS + 3) * 32;
    static constexpr int kCtas = 3 - NS;     // per SM
};
constexpr int kChunks = 4;
constexpr int kMaxRing = 4;
constexpr uint64_t kWaitLimitNs = 2000000000ull;

// K and V tiles in flight, each: what fits next to the query tiles (two streams:
// two of them and one CTA per SM; one stream: one and two CTAs).
template <int D, int NS> constexpr int kSharedRing = (D == 128 ? 1 : 2) * NS;
template <int D, int NS> constexpr size_t kSharedSmem = 1024 + static_cast<size_t>(D / 64) * kRegion * (NS + 2 * kSharedRing<D, NS>);

struct PrefixShared {
    uint64_t q_full;
    uint64_t k_full[kMaxRing], k_empty[kMaxRing], v_full[kMaxRing], v_empty[kMaxRing];
    uint64_t s_full[2], p_full[2][kChunks];
    uint64_t zeroed;                     // the rows past the prefix in the last V tile are zero
    uint64_t done;
    uint32_t tmem_base;
    int abort, bad;
    int group, local, sums[Streams<2>::kThreads / 32];   // find_unit
    int held;                            // padded lists: tensor memory is held, the barriers have been used
    int64_t listed, next;                //               units that there are, the CTA's next
};

// Bounded wait that also gives up once another thread has aborted the CTA.
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, PrefixShared &sh, int *err_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 0;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 63u) {
            if (*reinterpret_cast<volatile int *>(&sh.abort)) return false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *reinterpret_cast<volatile int *>(&sh.abort) = 1;
                report(err_flag, PA_FLAG_TIMEOUT);
                return false;
            }
        }
    }
}

// The warp goes on only if all its lanes saw the phase complete.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, PrefixShared &sh, int *err_flag) {
    return __all_sync(kFull, wait_bar(bar, parity, sh, err_flag));
}

__device__ __forceinline__ void mbar_inval(uint64_t *bar) {
    asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred P;\n\t"
        "elect.sync _|P, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, P;\n\t}"
        : "=r"(r));
    return r != 0;
}

// 3-D tiled TMA load without an L2 hint (the other query tiles and KV ranges of
// the group read the same blocks).
__device__ __forceinline__ void tma_load(void *dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_addr(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// Pairs of fp32 values in one 64-bit register.
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unf2(uint64_t r) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(r));
    return v;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A loader warp's view of the block table: 32 entries, one per lane, the next 32
// already requested (128 / bs divides 32, so no tile straddles two groups).
struct TableWindow {
    const int32_t *table;
    int needed;          // entries that may be read
    int base = -64;
    int32_t cur = -1, nxt = -1;
    __device__ int32_t fetch(int b, int lane) const { return b + lane < needed ? __ldg(table + b + lane) : -1; }
    // Block id of entry `entry + i` (entry: a tile's first entry).
    __device__ int32_t id_for(int entry, int i, int lane) {
        const int b = entry & ~31;
        if (b != base) {
            cur = b == base + 32 ? nxt : fetch(b, lane);
            nxt = fetch(b + 32, lane);
            base = b;
        }
        return __shfl_sync(kFull, cur, (entry & 31) + i);
    }
};

// One K or V tile (its blocks that hold tokens below `len`).
template <int R>
__device__ __forceinline__ void load_tile(TableWindow &win, int tile, int bs, int len, int kvh, int64_t num_blocks,
                                          uint8_t *dst, const CUtensorMap *map, uint64_t *full, int lane,
                                          PrefixShared &sh, int *err_flag) {
    const int nb = (min(len, (tile + 1) * kTile) - tile * kTile + bs - 1) / bs;
    const int32_t id = win.id_for(tile * (kTile / bs), lane < nb ? lane : 0, lane);
    const bool ok = lane < nb && id >= 0 && static_cast<int64_t>(id) < num_blocks;
    const uint32_t okmask = __ballot_sync(kFull, ok);
    if (lane == 0) {
        if (__popc(okmask) != nb) {
            report(err_flag, PA_FLAG_BAD_BLOCK_ID);
            sh.bad = 1;
        }
        mbar_arrive_expect_tx(full, static_cast<uint32_t>(__popc(okmask)) * bs * 128u * R);
    }
    __syncwarp();
    if (ok) {
#pragma unroll
        for (int r = 0; r < R; ++r) tma_load(dst + r * kRegion + lane * bs * 128, map, full, r * 64, kvh, id * bs);
    }
}

__device__ __forceinline__ int group_shared_blocks(const SplitParams &p, int q0) {
    return shared_blocks(p, q0, context_of(p, q0, false), false);
}

// Unit n of those that the groups really have, in order: its group and its number
// among the group's units; sh.listed: how many units there are.  (A group that breaks the rules
// counts as one unit, which reports it.)  All threads of the CTA.
__device__ __forceinline__ void find_unit(const SplitParams &p, int64_t n, int tile_seqs, int unit_tokens, PrefixShared &sh,
                                          int &group, int &local) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int64_t total = 0;
    for (int g0 = 0; g0 < p.num_groups; g0 += blockDim.x) {
        const int g = g0 + threadIdx.x;
        int units = 0;
        if (g < p.num_groups) {
            const int q0 = __ldg(p.cu_groups + g), q1 = __ldg(p.cu_groups + g + 1);
            if (bad_group(p, g, q0, q1)) {
                units = 1;
            } else if (q0 < q1) {
                const int len = group_shared_blocks(p, q0) * p.block_size;
                units = (q1 - q0 + tile_seqs - 1) / tile_seqs * ((len + unit_tokens - 1) / unit_tokens) * p.num_kv_heads;
            }
        }
        int incl = units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) sh.sums[warp] = incl;
        __syncthreads();
        int64_t before = total + incl - units;
        for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) {
            if (w < warp) before += sh.sums[w];
            total += sh.sums[w];
        }
        if (n >= before && n < before + units) {
            sh.group = g;
            sh.local = static_cast<int>(n - before);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) sh.listed = total;
    __syncthreads();
    group = sh.group;
    local = sh.local;
}

// One unit: the CTA's only one (kOnly), or one of several.  `begun`: an earlier one used
// the barriers and left the tensor memory held; `more`: another follows.
template <int D, bool BF16, int NS, bool kOnly>
__device__ __forceinline__ void prefix_unit(const SplitParams &p, PrefixShared &sh, uint8_t *base, int g, int pi, int kvh,
                                            int range, int unit_tokens, bool &begun, bool more, const CUtensorMap &tq,
                                            const CUtensorMap &tk, const CUtensorMap &tv) {
    constexpr int R = D / 64;               // 128-byte regions per row
    constexpr int kOp = R * kRegion;        // one 128-row operand tile
    constexpr int NR = kSharedRing<D, NS>;
    using W = Streams<NS>;
    constexpr uint32_t kColS = 0, kColO = W::kColO;
    constexpr int kKSteps = D / 16;
    constexpr int kPVSteps = kTile / 16;
    constexpr uint32_t kIdescQK = umma::idesc_f16(BF16, kTile, kTile, false);
    constexpr uint32_t kIdescPV = umma::idesc_f16(BF16, kTile, D, true);

    uint8_t *sQ = base, *sK = sQ + NS * kOp, *sV = sK + NR * kOp;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int lg = p.log2_group, G = 1 << lg;
    const int TT = kTile >> lg;             // sequences per query tile
    const int q0 = __ldg(p.cu_groups + g), q1 = __ldg(p.cu_groups + g + 1);
    const bool first = pi == 0 && kvh == 0 && range == 0;
    if (bad_group(p, g, q0, q1)) {
        if (first && threadIdx.x == 0) report(p.err_flag, PA_FLAG_BAD_CONTEXT_LEN);
        return;
    }
    if (q0 == q1) return;
    if (first) {   // one length for all of a group
        const int n0 = __ldg(p.shared_lens + q0);
        for (int s = q0 + threadIdx.x; s < q1; s += blockDim.x)
            if (__ldg(p.shared_lens + s) != n0) report(p.err_flag, PA_FLAG_BAD_CONTEXT_LEN);
    }
    const int len = group_shared_blocks(p, q0) * p.block_size;
    const int t0 = range * unit_tokens, tA = pi * NS * TT;  // first token, first sequence of the group
    if (t0 >= len || tA >= q1 - q0) return;
    const int n_seq = NS == 1 ? min(TT, q1 - q0 - tA) : q1 - q0 - tA;   // sequences from this unit's first on
    const bool duo = NS == 2 && n_seq > TT;                 // two query tiles
    const int end = min(len, t0 + unit_tokens);
    const int tile0 = t0 / kTile;
    const int nt = (end - t0 + kTile - 1) / kTile;          // K/V tiles of the range
    const int nA = duo || NS == 1 ? nt : (nt + 1) / 2, nB = duo ? nt : nt - nA;
    // The last tile reaches past the prefix: its V rows there, not loaded, are
    // zeroed before a product reads them (0 x NaN).
    const bool zero_tail = (end - t0) % kTile != 0;
    const int zx = nB > 0 ? 1 : 0;                          // the stream that zeroes them

    if (threadIdx.x == 0) {
        if (begun) {
            for (uint64_t *bar = &sh.q_full; bar <= &sh.done; ++bar) mbar_inval(bar);
        }
        mbar_init(&sh.q_full, 1);
        for (int i = 0; i < NR; ++i) {
            mbar_init(&sh.k_full[i], 1);
            mbar_init(&sh.k_empty[i], 1);
            mbar_init(&sh.v_full[i], 1);
            mbar_init(&sh.v_empty[i], 1);
        }
        for (int i = 0; i < NS; ++i) {
            mbar_init(&sh.s_full[i], 1);
            for (int c = 0; c < kChunks; ++c) mbar_init(&sh.p_full[i][c], 128);
        }
        mbar_init(&sh.zeroed, 128);
        mbar_init(&sh.done, 1);
        sh.abort = 0;
        sh.bad = 0;
        fence_barrier_init();
    }
    if (!begun && warp == W::kWarpMma) {
        umma::tmem_alloc(smem_addr(&sh.tmem_base), W::kCols);
        umma::tmem_relinquish();
    }
    begun = true;
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = sh.tmem_base;

    // K/V tile number (in load order) of stream x's i-th tile, and back
    auto seqno = [&](int x, int i) { return duo || NS == 1 ? i : i < nB ? 2 * i + x : nB + i; };

    if (warp == W::kWarpK || warp == W::kWarpV) {
        // ---------------------------------------------------- TMA loaders
        const bool is_k = warp == W::kWarpK;
        const CUtensorMap *map = is_k ? &tk : &tv;
        uint64_t *full = is_k ? sh.k_full : sh.v_full;
        uint64_t *empty = is_k ? sh.k_empty : sh.v_empty;
        uint8_t *ring = is_k ? sK : sV;
        if (lane == 0) {
            prefetch_tensormap(map);
            if (is_k) {
                prefetch_tensormap(&tq);
                mbar_arrive_expect_tx(&sh.q_full, kOp * (duo ? 2 : 1));
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    tma_load(sQ + r * kRegion, &tq, &sh.q_full, r * 64, kvh * G, q0 + tA);
                    if (duo) tma_load(sQ + kOp + r * kRegion, &tq, &sh.q_full, r * 64, kvh * G, q0 + tA + TT);
                }
            }
        }
        const int32_t *table = p.block_tables + static_cast<int64_t>(q0) * p.max_blocks_per_seq;
        TableWindow winA{table, len / p.block_size}, winB{table, len / p.block_size};
        int issued = 0;
        for (int s = 0; s < nt; ++s) {
            const int st = s % NR;
            if (s >= NR && !warp_wait(&empty[st], ((s / NR) - 1) & 1, sh, p.err_flag)) break;
            const bool inB = NS == 2 && !duo && s < 2 * nB && (s & 1);
            const int tile = tile0 + (duo || NS == 1 ? s : inB ? nA + (s >> 1) : s < 2 * nB ? s >> 1 : s - nB);
            load_tile<R>(inB ? winB : winA, tile, p.block_size, end, kvh, p.num_blocks, ring + st * kOp, map, &full[st],
                         lane, sh, p.err_flag);
            ++issued;
        }
        // On an abort, let the copies still in flight land before the CTA exits.
        if (lane == 0 && *reinterpret_cast<volatile int *>(&sh.abort)) {
            for (int s = max(0, issued - NR); s < issued; ++s)
                mbar_wait_bounded(&full[s % NR], (s / NR) & 1, kWaitLimitNs);
            if (is_k) mbar_wait_bounded(&sh.q_full, 0, kWaitLimitNs);
        }
    } else if (warp == W::kWarpMma) {
        // ------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t qd0 = umma::desc_sw128(smem_addr(sQ), 16, 1024);
        const uint64_t kd0 = umma::desc_sw128(smem_addr(sK), 16, 1024);
        const uint64_t vd0 = umma::desc_sw128(smem_addr(sV), kRegion, 1024);
        constexpr uint32_t kOpDesc = kOp >> 4;
        const int nx[2] = {nA, nB};
        bool ok = warp_wait(&sh.q_full, 0, sh, p.err_flag);
        auto qk = [&](int x, int i) -> bool {   // S_x = Q_x K^T
            const int s = seqno(x, i), st = s % NR;
            if (!warp_wait(&sh.k_full[st], (s / NR) & 1, sh, p.err_flag)) return false;
            umma::fence_after_sync();
            const uint64_t qd = qd0 + (duo ? static_cast<uint32_t>(x) * kOpDesc : 0u);
            const uint64_t kd = kd0 + static_cast<uint32_t>(st) * kOpDesc;
            const uint32_t ts = tmem + kColS + 128u * x;
            if (leader) {
#pragma unroll
                for (int k = 0; k < kKSteps; ++k) {
                    constexpr uint32_t kRegDesc = kRegion >> 4;
                    const uint32_t off = (k >> 2) * kRegDesc + (k & 3) * 2;
                    umma::mma_ss(ts, qd + off, kd + off, kIdescQK, k > 0 ? 1u : 0u);
                }
                umma::commit(smem_addr(&sh.s_full[x]));
                if (!duo || x == 1) umma::commit(smem_addr(&sh.k_empty[st]));
            }
            __syncwarp();
            return true;
        };
        if (ok) ok = qk(0, 0);
        if (ok && nx[1] > 0) ok = qk(1, 0);
        for (int i = 0; ok && i < nA; ++i) {
            for (int x = 0; ok && x < NS; ++x) {
                if (i >= nx[x]) continue;
                const int s = seqno(x, i), st = s % NR;
                if (zero_tail && i == nx[x] - 1 && (duo || x == zx) && !warp_wait(&sh.zeroed, 0, sh, p.err_flag)) {
                    ok = false;
                    break;
                }
                if (!warp_wait(&sh.v_full[st], (s / NR) & 1, sh, p.err_flag)) {
                    ok = false;
                    break;
                }
                const uint64_t vd = vd0 + static_cast<uint32_t>(st) * kOpDesc;
                const uint32_t tP = tmem + kColS + 128u * x, tO = tmem + kColO + 128u * x;
                const uint32_t acc0 = i > 0 ? 1u : 0u;
#pragma unroll
                for (int c = 0; c < kChunks; ++c) {
                    if (!warp_wait(&sh.p_full[x][c], i & 1, sh, p.err_flag)) {
                        ok = false;
                        break;
                    }
                    umma::fence_after_sync();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < kPVSteps / kChunks; ++kk) {
                            const int k = (kPVSteps / kChunks) * c + kk;
                            const uint32_t pk = tP + 32u * (k >> 1) + 8u * (k & 1);
                            umma::mma_ts(tO, pk, vd + static_cast<uint32_t>(k * (2048 >> 4)), kIdescPV,
                                         (c > 0 || kk > 0) ? 1u : acc0);
                            if constexpr (BF16)
                                umma::mma_ts(tO, pk + 16u, vd + static_cast<uint32_t>(k * (2048 >> 4)), kIdescPV, 1u);
                        }
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (leader && (!duo || x == 1)) umma::commit(smem_addr(&sh.v_empty[st]));
                __syncwarp();
                if (i + 1 < nx[x]) ok = qk(x, i + 1);
            }
        }
        if (leader) {
            umma::commit(smem_addr(&sh.done));
            mbar_wait_bounded(&sh.done, 0, kWaitLimitNs);
            // the last arrivals on these, which nobody else waits for, before the barriers are set up again
            for (int st = 0; more && ok && st < min(NR, nt); ++st) {
                const uint32_t par = ((nt - 1 - st) / NR) & 1;
                ok = mbar_wait_bounded(&sh.k_empty[st], par, kWaitLimitNs) &&
                     mbar_wait_bounded(&sh.v_empty[st], par, kWaitLimitNs);
            }
            if (!ok) *reinterpret_cast<volatile int *>(&sh.abort) = 1;
        }
        __syncwarp();
    } else {
        // -------------------------------------------- softmax and output
        const int x = NS == 2 ? (warp >> 2) & 1 : 0, q4 = warp & 3;
        const int row = 32 * q4 + lane;                     // of the query tile
        const int rows = (duo ? min(TT, n_seq - x * TT) : n_seq) << lg;
        const bool live = 32 * q4 < rows;                   // some row of this warp is a query
        const int n = x == 0 ? nA : nB;
        const uint32_t lane_off = static_cast<uint32_t>(32 * q4) << 16;
        const uint32_t tS = tmem + kColS + 128u * x + lane_off;
        const uint32_t tO = tmem + kColO + 128u * x + lane_off;
        // (a scale of 0 keeps the masked -inf and makes every other logit 0 to 32 bits)
        const float sl = p.scale_log2 == 0.f ? 1e-30f : p.scale_log2;
        const uint64_t sl2 = f2(sl, sl);
        float m_run = -CUDART_INF_F, l_run = 0.f;
        bool ok = true;
        for (int j = 0; j < n; ++j) {
            if (!warp_wait(&sh.s_full[x], j & 1, sh, p.err_flag)) {
                ok = false;
                break;
            }
            umma::fence_after_sync();
            const int tile = tile0 + (!duo && x == 1 ? nA : 0) + j;
            const int lim = end - tile * kTile;             // the tile's tokens below `lim` exist
            if (lim < kTile && x == zx) {
                const int s = seqno(x, j), st = s % NR;
                if (!warp_wait(&sh.v_full[st], (s / NR) & 1, sh, p.err_flag)) {
                    ok = false;
                    break;
                }
                if (row >= lim) {
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        uint4 *d = reinterpret_cast<uint4 *>(sV + st * kOp + r * kRegion + row * 128);
#pragma unroll
                        for (int i = 0; i < 8; ++i) d[i] = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                fence_proxy_async_smem();
                arrive(&sh.zeroed);
            }
            if (!live) {   // these rows' products are never read
                umma::fence_before_sync();
#pragma unroll
                for (int c = 0; c < kChunks; ++c) arrive(&sh.p_full[x][c]);
                continue;
            }
            // Two streams: the row's 128 scores stay in registers.  One stream, two
            // CTAs per SM and so 128 registers: they are read twice, 32 at a time,
            // for the maximum and for the weights.
            constexpr int kHeld = NS == 2 ? kTile : 32;
            uint32_t v[kHeld];
            auto mask = [&](uint32_t *w, int c) {        // columns 32 c .. of the last tile
                if (lim < kTile) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (32 * c + i >= lim) w[i] = 0xff800000u;     // -inf
                }
            };
            float mx;
            if constexpr (NS == 2) {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    umma::ld_32x32b_x32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v + 32 * c));
                umma::wait_ld();
#pragma unroll
                for (int c = 0; c < kChunks; ++c) mask(v + 32 * c, c);
                float a[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) a[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[k + 8]));
#pragma unroll
                for (int i = 1; i < kTile / 16; ++i)
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        a[k] = max3(a[k], __uint_as_float(v[16 * i + k]), __uint_as_float(v[16 * i + 8 + k]));
                mx = max3(max3(a[0], a[1], a[2]), max3(a[3], a[4], a[5]), fmaxf(a[6], a[7]));
            } else {
                mx = -CUDART_INF_F;
                uint32_t w[32];
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {   // two loads in flight
                    umma::ld_32x32b_x32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v));
                    umma::ld_32x32b_x32(tS + 32 * c + 32, w);
                    umma::wait_ld();
                    mask(v, c);
                    mask(w, c + 1);
#pragma unroll
                    for (int i = 0; i < 32; ++i) mx = max3(mx, __uint_as_float(v[i]), __uint_as_float(w[i]));
                }
            }
            const float x_tile = mx * sl;
            // The reference is 2^7 below the maximum it was set by and moves when that
            // grows by more than 2^8: binary16 weights reach 2^15 and end at 2^-24,
            // 2^-31 of the largest.
            const bool need = x_tile > m_run + (kWeightExp + 8.f);
            if (__any_sync(kFull, need)) {
                // O already holds tile j-1: its product preceded this tile's QK in issue order
                const float m_new = x_tile - kWeightExp;
                const float f = need ? fast_exp2(m_run - m_new) : 1.f;
                if (j > 0) {
                    const uint64_t f2x = f2(f, f);
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        umma::ld_32x32b_x16(tO + 16 * c, o);
                        umma::wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float2 w =
                                unf2(mul2(f2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), f2x));
                            o[2 * i] = __float_as_uint(w.x);
                            o[2 * i + 1] = __float_as_uint(w.y);
                        }
                        umma::st_32x32b_x16(tO + 16 * c, o);
                    }
                }
                if (need) {
                    l_run *= f;
                    m_run = m_new;
                }
            }
            // weights 2^(s - m) as 16-bit pairs over their own S columns
            const float mref = m_run == -CUDART_INF_F ? 0.f : m_run;
            const uint64_t nm2 = f2(-mref, -mref);
            uint64_t acc0 = f2(0.f, 0.f), acc1 = f2(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < kChunks; ++c) {
                constexpr bool kReload = NS == 1;
                if constexpr (kReload) {
                    umma::ld_32x32b_x32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(v));
                    umma::wait_ld();
                    mask(v, c);
                }
                const uint32_t *vc = v + (kReload ? 0 : 32 * c);
                uint32_t hi[16];
                [[maybe_unused]] uint32_t lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 xv =
                        unf2(fma2(f2(__uint_as_float(vc[2 * i]), __uint_as_float(vc[2 * i + 1])), sl2, nm2));
                    const float p0 = fast_exp2(xv.x), p1 = fast_exp2(xv.y);
                    hi[i] = pack2<BF16>(p0, p1);
                    const float2 hv = Half2x<BF16>::to_float2(hi[i]);
                    // the sum takes what the product takes: the rounded weight, or (two parts) the weight
                    uint64_t term;
                    if constexpr (BF16) {
                        const float2 lv = unf2(sub2(f2(p0, p1), f2(hv.x, hv.y)));
                        lo[i] = pack2<true>(lv.x, lv.y);
                        term = f2(p0, p1);
                    } else {
                        term = f2(hv.x, hv.y);
                    }
                    if (i & 1) acc1 = add2(acc1, term); else acc0 = add2(acc0, term);
                }
                umma::st_32x32b_x16(tS + 32 * c, hi);
                if constexpr (BF16) umma::st_32x32b_x16(tS + 32 * c + 16, lo);
                umma::wait_st();
                umma::fence_before_sync();
                arrive(&sh.p_full[x][c]);
            }
            const float2 acc = unf2(add2(acc0, acc1));
            l_run += acc.x + acc.y;
        }
        // `done` completes once every product of the CTA has.
        if (ok && live && warp_wait(&sh.done, 0, sh, p.err_flag)) {
            umma::fence_after_sync();
            const bool bad = *reinterpret_cast<volatile int *>(&sh.bad) != 0;
            const bool none = n == 0 || bad;                // nothing to add: an empty partial
            const int64_t sq = q0 + tA + (duo ? x * TT : 0) + (row >> lg);
            const int64_t at = (sq * p.num_kv_heads + kvh) * p.max_parts + NS * range;
            const int hq = row & (G - 1);
            if (row < rows) {
                const int64_t mine = ((at + (duo ? 0 : x)) << lg) + hq;
                *reinterpret_cast<float4 *>(p.ws_ml + 4 * mine) =
                    none ? make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f) : make_float4(m_run, l_run, 0.f, 0.f);
                if (duo)   // two query tiles write one partial per range
                    *reinterpret_cast<float4 *>(p.ws_ml + 4 * (((at + 1) << lg) + hq)) =
                        make_float4(-CUDART_INF_F, 0.f, 0.f, 0.f);
            }
            if (!none) {
                float *dst = p.ws_acc + (((at + (duo ? 0 : x)) << lg) + hq) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    umma::ld_32x32b_x32(tO + 32 * c, o);
                    umma::wait_ld();
                    if (row < rows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<uint4 *>(dst + 32 * c + 4 * i) =
                                make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                }
            }
        }
    }

    umma::fence_before_sync();
    __syncthreads();
    if (kOnly && warp == W::kWarpMma) {
        umma::fence_after_sync();
        umma::tmem_dealloc(tmem, W::kCols);
    }
}

// kPadded: the list of groups is padded with empty ones; the grid's CTAs take the
// units that there really are in turn.
template <int D, bool BF16, int NS, bool kPadded>
__global__ void __launch_bounds__(Streams<NS>::kThreads, Streams<NS>::kCtas)
    shared_prefix_kernel(const __grid_constant__ SplitParams p, int tiles, int unit_tokens, int units_per_list,
                         const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                         const __grid_constant__ CUtensorMap tv) {
    using W = Streams<NS>;
    __shared__ PrefixShared sh;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // Units in this order: the query tiles (pairs of them) of one K/V range run next to each other (L2).
    if constexpr (!kPadded) {
        int u = blockIdx.x;
        const int pi = u % tiles;
        u /= tiles;
        const int kvh = u % p.num_kv_heads;
        u /= p.num_kv_heads;
        const int range = u % units_per_list, g = u / units_per_list;
        pdl_wait();
        pdl_launch_dependents();
        bool begun = false;
        prefix_unit<D, BF16, NS, true>(p, sh, base, g, pi, kvh, range, unit_tokens, begun, false, tq, tk, tv);
    } else {
        const int tile_seqs = NS * (kTile >> p.log2_group);
        pdl_wait();
        pdl_launch_dependents();
        if (blockIdx.x == 0)   // groups without whole shared blocks: one length for all of each, as the units check
            for (int g = threadIdx.x; g < p.num_groups; g += blockDim.x) {
                const int q0 = __ldg(p.cu_groups + g), q1 = __ldg(p.cu_groups + g + 1);
                if (bad_group(p, g, q0, q1) || q0 == q1 || group_shared_blocks(p, q0) > 0) continue;
                for (int s = q0 + 1; s < q1; ++s)
                    if (__ldg(p.shared_lens + s) != __ldg(p.shared_lens + q0)) report(p.err_flag, PA_FLAG_BAD_CONTEXT_LEN);
            }
        if (threadIdx.x == 0) sh.held = 0;
        // What an iteration needs comes out of shared memory again: kept in registers across
        // the unit it makes the softmax spill (8,192 tokens before 256 sequences, 255 of 256
        // groups empty: 101 us, with it 111; without the empty groups 99).
        volatile PrefixShared &now = sh;
#pragma unroll 1
        for (int64_t n = blockIdx.x;; n = now.next) {
            int g, local;
            find_unit(p, n, tile_seqs, unit_tokens, sh, g, local);
            const int64_t listed = now.listed;
            if (n >= listed) break;
            if (threadIdx.x == 0) sh.next = n + gridDim.x;
            // (a group that breaks the rules: any query tile)
            const int have = max(1, (__ldg(p.cu_groups + g + 1) - __ldg(p.cu_groups + g) + tile_seqs - 1) / tile_seqs);
            bool held = now.held != 0;
            uint8_t *b = base;
            asm volatile("" : "+l"(b));
            prefix_unit<D, BF16, NS, false>(p, sh, b, g, local % have, local / have % p.num_kv_heads,
                                     local / have / p.num_kv_heads, unit_tokens, held, n + gridDim.x < listed, tq, tk, tv);
            if (threadIdx.x == 0) sh.held = held;
            __syncthreads();
            if ((now.held && now.abort) || now.next >= now.listed) break;
        }
        __syncthreads();
        if (now.held && (threadIdx.x >> 5) == W::kWarpMma) {
            umma::fence_after_sync();
            umma::tmem_dealloc(sh.tmem_base, W::kCols);
        }
    }
}

template <int D, bool BF16, int NS>
cudaError_t launch_t(const SplitParams &p, int grid, bool padded, int tiles, int unit_tokens, int units_per_list,
                     const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv, cudaStream_t stream) {
    auto kern = padded ? shared_prefix_kernel<D, BF16, NS, true> : shared_prefix_kernel<D, BF16, NS, false>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(kSharedSmem<D, NS>));
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(static_cast<unsigned>(grid)), dim3(Streams<NS>::kThreads), kSharedSmem<D, NS>, stream, p,
                      tiles, unit_tokens, units_per_list, tq, tk, tv);
}

template <int D>
cudaError_t launch_d(const SplitParams &p, bool bf16, bool pairs, int grid, bool padded, int tiles, int unit_tokens,
                     int units_per_list, const CUtensorMap &tq, const CUtensorMap &tk, const CUtensorMap &tv,
                     cudaStream_t stream) {
    if (pairs)
        return bf16 ? launch_t<D, true, 2>(p, grid, padded, tiles, unit_tokens, units_per_list, tq, tk, tv, stream)
                    : launch_t<D, false, 2>(p, grid, padded, tiles, unit_tokens, units_per_list, tq, tk, tv, stream);
    return bf16 ? launch_t<D, true, 1>(p, grid, padded, tiles, unit_tokens, units_per_list, tq, tk, tv, stream)
                : launch_t<D, false, 1>(p, grid, padded, tiles, unit_tokens, units_per_list, tq, tk, tv, stream);
}

}  // namespace

size_t shared_prefix_smem(int head_dim) { return head_dim == 128 ? kSharedSmem<128, 2> : kSharedSmem<64, 2>; }

cudaError_t launch_shared_prefix(const SplitParams &p, int head_dim, bool bf16, bool pairs, int grid, bool padded, int tiles,
                                 int unit_tokens, int units_per_list, const CUtensorMap &tq, const CUtensorMap &tk,
                                 const CUtensorMap &tv, cudaStream_t stream) {
    auto launch = head_dim == 128 ? launch_d<128> : launch_d<64>;
    return launch(p, bf16, pairs, grid, padded, tiles, unit_tokens, units_per_list, tq, tk, tv, stream);
}

}  // namespace pa
