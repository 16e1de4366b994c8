// Norms of queries and keys, the rotation to their positions, and the write of keys
// and values into the paged cache, in one pass.
//
// A row x of D elements (one token, one head):
//     y = x w / sqrt(mean x^2 + eps)                  (queries and keys, where a weight is given)
//     (a, b) -> m (a cos - b sin, b cos + a sin)      (queries and keys: pair i of the first 2F elements)
// with the angle position * f_i, a pair being the elements (i, i + F) or, interleaved,
// (2i, 2i + 1).  Nothing is rounded between the steps; rows come out in the inputs'
// type, or as codes of the cache's (pa_quant_codes.cuh).
//
// The angle is taken in turns, in integer arithmetic: with f_i / 2 pi = F_i 2^-64, position * F_i
// modulo 2^64 is the fraction of a turn, off by position times F_i's error.  32-bit positions of
// frequencies below 2 have F_i to 64 bits (2^-32 of a turn off at most), others, in a loop of their
// own, to 128, so that any position and any frequency allowed is right to 2^-42 of a turn.
// (64 bits everywhere: 185 2^-24 off at position 2^45, f = 1, and 743 2^-24 at 2^30, f = 2^19; 128
// everywhere: 8,192 tokens 39.5 us against 37.8, 256 5.8 against 5.2.)  sincospif of the
// fraction is good to a few 2^-24.
//
// Bound by memory: every row is read once and written once.  D / 8 lanes take a row,
// 8 elements each; with the pairs half a row apart those are 4 and their 4 partners,
// so that no element changes lanes.  A CTA takes one or four tokens' rows, its threads
// first make the tokens' sines and cosines (once per token, not per head: 40 heads
// share them), while each lane's first rows are on their way.
//
// Measured (GB300, in a graph): 8,192 tokens of 32 query and 8 KV heads of 128, bf16, with
// norms 37.2 us, 0.81 of the measured copy rate (34.6 without norms, 136 for four times the
// tokens, 0.89; copying as many bytes takes 31); 256 tokens of 40 + 40 heads 5.1 us; 4 tokens
// of 4 + 4 heads 1.9.  Into 8-bit caches the first takes 51.5 (0.54) and into a 4-bit one 72
// (0.37), bound by their operations: 37 and 52 M warp instructions against 28 M, at 122
// registers, four CTAs an SM.  Steps: rows of any token to any lane 64 us; a row of four tokens
// at a time 43; their four sums of squares reduced together (9 shuffles in place of 16) 41;
// CTAs of 128 threads 38; value rows stored as they were read 37.2.  Eight tokens at a time
// take 52.
#include <type_traits>

#include "pa_decode_common.cuh"
#include "pa_device.cuh"
#include "pa_f32x2.cuh"
#include "pa_quant_codes.cuh"
#include "pa_step_ops.h"

namespace pa {

namespace {

using decode_common::launch_pdl;

constexpr int kRopeThreads = 128;
constexpr int kRopeTokens = 4;       // tokens of a CTA at most

// f / 2 pi and position * f / 2 pi, as fractions of 2^64 (whole turns dropped).  |f| = M 2^(e - 1086)
// with M's top bit set, and 1 / 2 pi = C 2^-130, C = floor(2^128 2 / pi).
constexpr uint64_t kTurnHigh = 0xa2f9836e4e441529ull, kTurnLow = 0xfc2757d1f534ddc0ull;
__device__ __forceinline__ uint64_t mantissa(uint64_t bits) {
    return ((bits & 0xfffffffffffffull) | 0x10000000000000ull) << 11;
}
__device__ __forceinline__ int exponent(uint64_t bits) { return static_cast<int>((bits >> 52) & 0x7ff); }
// For |f| < 2 (others: some number).
__device__ __forceinline__ uint64_t turn_fraction(uint64_t bits) {
    const int e = exponent(bits);
    uint64_t t = __umul64hi(mantissa(bits), kTurnHigh + 1) >> ((1024 - e) & 63);      // (C's 64 bits, rounded)
    if (e <= 960) t = 0;
    return bits >> 63 ? 0 - t : t;
}
__device__ __forceinline__ uint64_t far_turn(int64_t position, uint64_t bits) {
    const int sh = exponent(bits) - 1024;
    if (sh <= -128 || sh >= 64) return 0;
    const uint64_t M = mantissa(bits), p = static_cast<uint64_t>(position < 0 ? 0 - static_cast<uint64_t>(position) : position);
    const unsigned __int128 h = static_cast<unsigned __int128>(M) * kTurnHigh + __umul64hi(M, kTurnLow);
    const unsigned __int128 F = sh >= 0 ? h << sh : h >> -sh;
    const uint64_t t = p * static_cast<uint64_t>(F >> 64) + __umul64hi(p, static_cast<uint64_t>(F));
    return (position < 0) != (bits >> 63 != 0) ? 0 - t : t;
}

// Of a fraction of a turn.
__device__ __forceinline__ float2 cos_sin(uint64_t turn, float factor) {
    float s, c;
    sincospif(__ll2float_rn(static_cast<int64_t>(turn)) * 0x1p-63f, &s, &c);
    return make_float2(c * factor, s * factor);
}

// Sums over the LPR lanes of a row, of one value or of four at once: with four, halves and
// then quarters of the lanes go on with two and then one of them, and every lane looks up all
// four at the end.  Both add lanes LPR / 2 apart first, then LPR / 4 and so on to neighbours: a
// token's bytes do not depend on how many others are in the call.  `then`: applied to a sum
// once per lane that holds it.
template <int LPR, typename Then>
__device__ __forceinline__ void row_sums(float (&v)[1], int, uint32_t lanes, Then then) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) v[0] += __shfl_xor_sync(lanes, v[0], o);
    v[0] = then(v[0]);
}
template <int LPR, typename Then>
__device__ __forceinline__ void row_sums(float (&v)[4], int l, uint32_t lanes, Then then) {
    const bool upper = l & (LPR / 2), odd = l & (LPR / 4);
    float a = upper ? v[2] : v[0], b = upper ? v[3] : v[1];
    a += __shfl_xor_sync(lanes, upper ? v[0] : v[2], LPR / 2);
    b += __shfl_xor_sync(lanes, upper ? v[1] : v[3], LPR / 2);
    float c = odd ? b : a;
    c += __shfl_xor_sync(lanes, odd ? a : b, LPR / 4);
#pragma unroll
    for (int o = LPR / 8; o > 0; o >>= 1) c += __shfl_xor_sync(lanes, c, o);
    c = then(c);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = __shfl_sync(lanes, c, (k & 2 ? LPR / 2 : 0) + (k & 1 ? LPR / 4 : 0), LPR);
}

// Codes of a row's eight values (four at elements oa, four at ob) into the cache.
template <int D>
__device__ __forceinline__ void write_codes(const RopeParams &p, int kind, int kv, const float (&y)[8], int oa, int ob, int l,
                                            int head, int64_t slot, uint32_t lanes) {
    const int64_t row = slot * p.hkv + head;
    uint8_t *base = static_cast<uint8_t *>(p.cache[kv]);
    if (kind == kRopeInt4) {
        float lo[D / kGroup4], hi[D / kGroup4];
        const int ga = oa / kGroup4, gb = ob / kGroup4;
        uint32_t m = 0;
#pragma unroll
        for (int g = 0; g < D / kGroup4; ++g) {
            lo[g] = INFINITY;
            hi[g] = -INFINITY;
            uint32_t mg = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if ((i < 4 ? ga : gb) == g) {
                    lo[g] = fminf(lo[g], y[i]);
                    hi[g] = fmaxf(hi[g], y[i]);
                    mg = max(mg, __float_as_uint(y[i]) & 0x7fffffffu);
                }
            if (mg >= 0x7f800000u) m |= 1u << g;
        }
#pragma unroll
        for (int o = 1; o < D / 8; o <<= 1) {
            m |= __shfl_xor_sync(lanes, m, o);
#pragma unroll
            for (int g = 0; g < D / kGroup4; ++g) {
                lo[g] = fminf(lo[g], __shfl_xor_sync(lanes, lo[g], o));
                hi[g] = fmaxf(hi[g], __shfl_xor_sync(lanes, hi[g], o));
            }
        }
        Group4 q[D / kGroup4];
#pragma unroll
        for (int g = 0; g < D / kGroup4; ++g) q[g] = group4(lo[g], hi[g], !((m >> g) & 1u));
        auto of = [&](int g) {
            const Group4 &a = q[0], &b = q[D / kGroup4 - 1];
            return Group4{g ? b.inv : a.inv, g ? b.zero : a.zero, g ? b.word : a.word};
        };
        const Group4 qa = of(ga), qb = of(gb);
        const bool fa = !((m >> ga) & 1u), fb = !((m >> gb) & 1u);
        const uint32_t ca = code4x4(y[0], y[1], y[2], y[3], qa), cb = code4x4(y[4], y[5], y[6], y[7], qb);
        uint8_t *o = base + row * (D / 2);
        *reinterpret_cast<uint16_t *>(o + oa / 2) = static_cast<uint16_t>(fa ? ca : 0u);
        *reinterpret_cast<uint16_t *>(o + ob / 2) = static_cast<uint16_t>(fb ? cb : 0u);
        if (l < D / kGroup4) {
            const uint32_t s = static_cast<uint32_t>(slot), blk = s / p.bs;
            static_cast<uint32_t *>(p.scales[kv])[word_row(blk, s - blk * p.bs, head, p.hkv, p.bs) * (D / kGroup4) + l] =
                of(l).word;
        }
        return;
    }
    uint32_t code[2];
    if (kind == kRopeE4M3) {
        const float s = p.scale[kv];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            code[h] = f32x2_to_e4m3x2(__fdiv_rn(y[4 * h], s), __fdiv_rn(y[4 * h + 1], s)) |
                      (f32x2_to_e4m3x2(__fdiv_rn(y[4 * h + 2], s), __fdiv_rn(y[4 * h + 3], s)) << 16);
    } else {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(y[i]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < D / 8; o <<= 1) m = max(m, __shfl_xor_sync(lanes, m, o));
        const bool finite = m < 0x7f800000u;      // (a NaN is above infinity)
        const float top = kind == kRopeRows ? 448.f : 127.f;
        const float amax = fmaxf(finite ? __uint_as_float(m) : 0.f, kAmaxFloor), inv = __fdiv_rn(top, amax);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float v0 = __fmul_rn(y[4 * h], inv), v1 = __fmul_rn(y[4 * h + 1], inv);
            const float v2 = __fmul_rn(y[4 * h + 2], inv), v3 = __fmul_rn(y[4 * h + 3], inv);
            code[h] = kind == kRopeRows ? f32x2_to_e4m3x2(v0, v1) | (f32x2_to_e4m3x2(v2, v3) << 16) : int8x4(v0, v1, v2, v3);
            if (!finite) code[h] = 0u;
        }
        if (l == 0) static_cast<float *>(p.scales[kv])[row] = finite ? __fdiv_rn(amax, top) : __uint_as_float(kNanBits);
    }
    *reinterpret_cast<uint32_t *>(base + row * D + oa) = code[0];
    *reinterpret_cast<uint32_t *>(base + row * D + ob) = code[1];
}

// (e0 e1)(e2 e3)(e4 e5)(e6 e7) -> (e0 e2)(e4 e6)(e1 e3)(e5 e7), and back.
__device__ __forceinline__ void part_pairs(uint32_t (&x)[4]) {
    const uint32_t a = __byte_perm(x[0], x[1], 0x5410u), b = __byte_perm(x[2], x[3], 0x5410u);
    const uint32_t c = __byte_perm(x[0], x[1], 0x7632u), d = __byte_perm(x[2], x[3], 0x7632u);
    x[0] = a;
    x[1] = b;
    x[2] = c;
    x[3] = d;
}
__device__ __forceinline__ void join_pairs(uint32_t (&x)[4]) {
    const uint32_t a = __byte_perm(x[0], x[2], 0x5410u), b = __byte_perm(x[0], x[2], 0x7632u);
    const uint32_t c = __byte_perm(x[1], x[3], 0x5410u), d = __byte_perm(x[1], x[3], 0x7632u);
    x[0] = a;
    x[1] = b;
    x[2] = c;
    x[3] = d;
}

// A CTA takes TB tokens and rows_per of their rows: a group of lanes takes a row (query,
// key or value of one head) of all TB tokens at a time, the next row's loads under way.
template <int D, bool BF16, bool QUANT, int TB>
__global__ void __launch_bounds__(kRopeThreads)
    rope_and_cache_kernel(const __grid_constant__ RopeParams p, int rows_per, int kind) {
    constexpr int LPR = D / 8, RG = kRopeThreads / LPR;
    __shared__ __align__(16) float cos_t[TB][D / 2], sin_t[TB][D / 2], neg_t[TB][D / 2];   // (neg: less the sine)
    __shared__ int64_t slot_t[TB];
    pdl_wait();
    pdl_launch_dependents();
    const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR;
    const uint32_t lanes = ((1u << LPR) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB;
    const int nt = static_cast<int>(min(static_cast<int64_t>(TB), p.num_tokens - t0));
    const int R = p.hq + 2 * p.hkv, r1 = min(R, static_cast<int>(blockIdx.y + 1) * rows_per);
    const int half = p.rot / 2;
    const bool turned = 4 * l < half;             // my elements of a query or key are turned

    // Row r of a token: 0 query, 1 key, 2 value, and the head; my elements' places in it.
    auto which = [&](int r) { return r < p.hq ? 0 : r < p.hq + p.hkv ? 1 : 2; };
    auto head_of = [&](int r, int w) { return w == 0 ? r : w == 1 ? r - p.hq : r - p.hq - p.hkv; };
    auto apart = [&](int w) { return w < 2 && turned && !p.interleaved; };
    uint32_t x[TB][4], nx[TB][4];
    auto load = [&](int r, uint32_t (&v)[TB][4]) {
        const int w = which(r);
        const uint16_t *s = p.src[w] + t0 * p.stride[w] + static_cast<int64_t>(head_of(r, w)) * D;
        const bool two = apart(w);
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            if (k < nt) {
                if (two) {
                    const uint2 a = *reinterpret_cast<const uint2 *>(s + 4 * l);
                    const uint2 b = *reinterpret_cast<const uint2 *>(s + half + 4 * l);
                    v[k][0] = a.x; v[k][1] = a.y; v[k][2] = b.x; v[k][3] = b.y;
                } else {
                    const uint4 u = *reinterpret_cast<const uint4 *>(s + 8 * l);
                    v[k][0] = u.x; v[k][1] = u.y; v[k][2] = u.z; v[k][3] = u.w;
                }
            }
            s += p.stride[w];
        }
    };
    int r = blockIdx.y * rows_per + grp;
    if (r < r1) load(r, x);
    bool far = false;
    auto angles = [&](auto far_tag) {
        for (int i = threadIdx.x; i < nt * half; i += kRopeThreads) {
            const int tok = TB == 1 ? 0 : i / half, k = i - tok * half;
            const int64_t position = __ldg(p.positions + t0 + tok);
            const uint64_t f = static_cast<uint64_t>(__double_as_longlong(__ldg(p.inv_freq + k)));
            const bool is_far = position != static_cast<int32_t>(position) || exponent(f) >= 1024;
            uint64_t turn;
            if constexpr (decltype(far_tag)::value) {
                if (!is_far) continue;
                turn = far_turn(position, f);
            } else {
                turn = static_cast<uint64_t>(position) * turn_fraction(f);
                far = far || is_far;
            }
            const float2 cs = cos_sin(turn, p.factor);
            cos_t[tok][k] = cs.x;
            sin_t[tok][k] = cs.y;
            neg_t[tok][k] = -cs.y;
        }
    };
    angles(std::false_type{});
    if (far) angles(std::true_type{});      // those that are, once more
    if (threadIdx.x < nt) {
        int64_t s = __ldg(p.slots + t0 + threadIdx.x);
        if (s >= p.num_slots) {
            report(p.err_flag, 0x1 /* PA_FLAG_BAD_SLOT */);
            s = -1;
        }
        slot_t[threadIdx.x] = s;
    }
    __syncthreads();
    for (; r < r1; r += RG) {
        if (r + RG < r1) load(r + RG, nx);
        const int w = which(r), head = head_of(r, w);
        const bool turns = w < 2 && turned, pairs = turns && p.interleaved, two = apart(w);
        const int oa = two ? 4 * l : 8 * l, ob = two ? half + 4 * l : 8 * l + 4;
        const bool norm = w < 2 && p.weight[w] != nullptr;
        F2 wt[4];
        if (norm) {
            const uint2 wa = __ldg(reinterpret_cast<const uint2 *>(p.weight[w] + oa));
            const uint2 wb = __ldg(reinterpret_cast<const uint2 *>(p.weight[w] + ob));
            uint32_t u[4] = {wa.x, wa.y, wb.x, wb.y};
            if (pairs) part_pairs(u);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Half2x<BF16>::to_float2(u[j]);
                wt[j] = f2(f.x, f.y);
            }
        }
        float size[TB];               // 1 / sqrt(mean x^2 + eps)
        if (norm) {
#pragma unroll
            for (int k = 0; k < TB; ++k) {
                F2 s = f2(0.f, 0.f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = Half2x<BF16>::to_float2(x[k][j]);
                    const F2 y = f2(f.x, f.y);
                    s = fma2(y, y, s);
                }
                const float2 ss = both(s);
                size[k] = ss.x + ss.y;
            }
            row_sums<LPR>(size, l, lanes, [&](float s) { return rsqrtf(s * (1.f / D) + p.eps); });
        }
        // where the row goes: the query's output, or from where slots are counted in the cache
        uint16_t *const base = w == 0 ? p.out_q + (t0 * p.hq + head) * D
                                      : static_cast<uint16_t *>(p.cache[w - 1]) + static_cast<int64_t>(head) * D;
        const int64_t row = static_cast<int64_t>(w == 0 ? p.hq : p.hkv) * D;
        const bool as_it_is = !QUANT && w == 2;       // values: bits of a NaN too
        if (as_it_is) {
#pragma unroll
            for (int k = 0; k < TB; ++k)
                if (k < nt && slot_t[k] >= 0)
                    *reinterpret_cast<uint4 *>(base + slot_t[k] * row + oa) = make_uint4(x[k][0], x[k][1], x[k][2], x[k][3]);
        }
#pragma unroll
        for (int k = 0; k < TB; ++k) {
            if (k >= nt || as_it_is) break;
            if (pairs) part_pairs(x[k]);
            F2 y[4];                      // turned lanes: elements (a0 a1)(a2 a3) and their partners (b0 b1)(b2 b3)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = Half2x<BF16>::to_float2(x[k][j]);
                y[j] = f2(f.x, f.y);
            }
            if (norm) {
                const F2 s2 = f2(size[k], size[k]);
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = y[j] * (s2 * wt[j]);
            }
            if (turns) {
                const float4 c = *reinterpret_cast<const float4 *>(&cos_t[k][4 * l]);
                const float4 s = *reinterpret_cast<const float4 *>(&sin_t[k][4 * l]);
                const float4 n = *reinterpret_cast<const float4 *>(&neg_t[k][4 * l]);
                const F2 cc[2] = {f2(c.x, c.y), f2(c.z, c.w)}, sn[2] = {f2(s.x, s.y), f2(s.z, s.w)};
                const F2 ng[2] = {f2(n.x, n.y), f2(n.z, n.w)};
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const F2 a = y[j], b = y[j + 2];
                    y[j] = fma2(b, ng[j], a * cc[j]);
                    y[j + 2] = fma2(a, sn[j], b * cc[j]);
                }
            }
            const int64_t slot = slot_t[k];
            if (QUANT && w > 0) {
                const float2 v0 = both(y[0]), v1 = both(y[1]), v2 = both(y[2]), v3 = both(y[3]);
                float z[8] = {v0.x, v0.y, v1.x, v1.y, v2.x, v2.y, v3.x, v3.y};
                if (pairs) {          // back into the row's order
                    z[1] = v2.x;
                    z[2] = v0.y;
                    z[3] = v2.y;
                    z[4] = v1.x;
                    z[5] = v3.x;
                    z[6] = v1.y;
                }
                if (slot >= 0) write_codes<D>(p, kind, w - 1, z, oa, ob, l, head, slot, lanes);
                continue;
            }
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = both(y[j]);
                h[j] = pack2<BF16>(f.x, f.y);
            }
            if (pairs) join_pairs(h);
            uint16_t *const out = base + (w == 0 ? k : slot) * row;
            if (w == 0 || slot >= 0) {
                if (two) {
                    *reinterpret_cast<uint2 *>(out + oa) = make_uint2(h[0], h[1]);
                    *reinterpret_cast<uint2 *>(out + ob) = make_uint2(h[2], h[3]);
                } else {
                    *reinterpret_cast<uint4 *>(out + oa) = make_uint4(h[0], h[1], h[2], h[3]);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < TB; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) x[k][j] = nx[k][j];
    }
}

template <int D, bool BF16, bool QUANT>
cudaError_t rope_q(const RopeParams &p, int kind, int sms, cudaStream_t stream) {
    constexpr int RG = kRopeThreads / (D / 8);
    const int R = p.hq + 2 * p.hkv;
    // Four tokens to a CTA from 128 rows an SM on (800 tokens of 32 + 8 heads 5.6 us, one by one
    // 7.3; 256 tokens 3.6, one by one 3.4).  A token's rows are spread over CTAs while the GPU has
    // fewer than four an SM, in whole rounds of a CTA's groups of lanes (64 + 8 heads, 800 tokens:
    // 7.3 us, cut by halves 9.1).
    const bool many = p.num_tokens * R >= static_cast<int64_t>(128) * sms;
    const int64_t blocks = many ? (p.num_tokens + kRopeTokens - 1) / kRopeTokens : p.num_tokens;
    const int rounds = (R + RG - 1) / RG;
    const int64_t want = (4 * sms + blocks - 1) / blocks;
    const int rows = (want < rounds ? static_cast<int>(rounds / want) : 1) * RG;
    const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>((R + rows - 1) / rows));
    if (many) return launch_pdl(rope_and_cache_kernel<D, BF16, QUANT, kRopeTokens>, grid, dim3(kRopeThreads), 0, stream, p, rows, kind);
    return launch_pdl(rope_and_cache_kernel<D, BF16, QUANT, 1>, grid, dim3(kRopeThreads), 0, stream, p, rows, kind);
}

template <int D, bool BF16>
cudaError_t rope_t(const RopeParams &p, int kind, int sms, cudaStream_t stream) {
    return kind == kRopeHalf ? rope_q<D, BF16, false>(p, kind, sms, stream) : rope_q<D, BF16, true>(p, kind, sms, stream);
}

}  // namespace

cudaError_t launch_rope_and_cache(const RopeParams &p, int head_dim, bool bf16, int kind, int sms, cudaStream_t stream) {
    if (head_dim == 128) return bf16 ? rope_t<128, true>(p, kind, sms, stream) : rope_t<128, false>(p, kind, sms, stream);
    return bf16 ? rope_t<64, true>(p, kind, sms, stream) : rope_t<64, false>(p, kind, sms, stream);
}

}  // namespace pa
