// The codes and scales of the quantised caches, from a row's extremes: shared by
// the cache write (pa_quant_ops.cu) and the rotation that writes into a cache
// (pa_rope.cu), so that both make the same bytes of the same 32-bit values.
#pragma once

#include "pa_device.cuh"
#include "pa_f32x2.cuh"

namespace pa {

constexpr float kAmaxFloor = 8.673617379884035e-19f;   // 2^-60
constexpr uint32_t kNanBits = 0x7fc00000u;

// Values per group of a 4-bit row, which has a scale and a zero of its own.
constexpr int kGroup4 = 64;

// Four values -> four int8 codes.  v + 1.5 * 2^23 holds round(v) (nearest,
// ties to even) in its low bits for |v| < 2^22.
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
    constexpr float k = 12582912.f;
    const uint32_t ia = __float_as_uint(__fadd_rn(a, k)), ib = __float_as_uint(__fadd_rn(b, k));
    const uint32_t ic = __float_as_uint(__fadd_rn(c, k)), id = __float_as_uint(__fadd_rn(d, k));
    return __byte_perm(__byte_perm(ia, ib, 0x0040u), __byte_perm(ic, id, 0x0040u), 0x5410u);
}

// Where the (scale, zero) words of a 4-bit row lie, in rows: [block][head][token][group].
__device__ __forceinline__ int64_t word_row(int64_t block, int offset, int head, int hkv, int bs) {
    return (block * hkv + head) * bs + offset;
}

// A group of 4-bit codes: x stands for s (u + z), s and z bfloat16.  The codes are
// chosen for the rounded s and z: a range that s falls short of by its rounding, 2^-8,
// costs a sixteenth of a code; z's rounding a thirty-second where a group is spread about
// zero (|z| of 7.5), half a code where |z| is 2^8 and one just above.  |z| goes no
// further, since s is at least 2^-8 of the largest magnitude.
struct Group4 {
    float inv, zero;     // 1 / s and z
    uint32_t word;       // s in the low half, z in the high half
};

// Quotients correctly rounded by one step on an approximate one (P. Markstein, "Computation
// of elementary functions on the IBM RISC System/6000 processor", 1990): with inv the
// correctly rounded 1 / b, q = a inv and the exact remainder r = a - b q, the quotient is
// q + r inv, rounded once.  (Checked against IEEE division: every s, 2^28 pairs (min, s), as
// many d / 7.5.)
__device__ __forceinline__ float quotient(float a, float b, float inv) {
    const float q = __fmul_rn(a, inv);
    return __fmaf_rn(__fmaf_rn(-b, q, a), inv, q);
}
// 1 / s for a bfloat16 s of 2^-60 to 2^125, correctly rounded: one step on an approximation.
__device__ __forceinline__ float inverse(float s) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return __fmaf_rn(__fmaf_rn(-s, r, 1.f), r, r);
}

__device__ __forceinline__ Group4 group4(float lo, float hi, bool finite) {
    // (halves: the range of values of both signs may pass the largest float)
    const float step = quotient(__fsub_rn(__fmul_rn(0.5f, hi), __fmul_rn(0.5f, lo)), 7.5f, 0.13333333333f);
    const float s = fmaxf(fmaxf(step, __fmul_rn(fmaxf(hi, -lo), 0.00390625f)), kAmaxFloor);
    const uint32_t sb = float_to_bf16_bits(s);
    const float sf = __uint_as_float(sb << 16);
    Group4 g;
    g.inv = inverse(sf);
    const uint32_t zb = float_to_bf16_bits(quotient(lo, sf, g.inv));
    g.zero = __uint_as_float(zb << 16);
    g.word = finite ? sb | (zb << 16) : kNanBits >> 16;
    return g;
}

// The codes of x0 and x1 in the low and high half.  The roundings of s and z leave
// x (1 / s) - z within a few codes of 0 and 15, so that the rounded value (in the low bits
// once 1.5 2^23 is added) is cut off there as a 16-bit number.
__device__ __forceinline__ uint32_t codes4_pair(float x0, float x1, const Group4 &g) {
    constexpr float k = 12582912.f;
    // (the products one by one: a packed one and the sum behind it come out as one rounding)
    const float2 y = both(f2(__fmul_rn(x0, g.inv), __fmul_rn(x1, g.inv)) + f2(-g.zero, -g.zero) + f2(k, k));
    uint32_t v = __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x5410u);
    asm("max.s16x2 %0, %0, %1;" : "+r"(v) : "r"(0u));
    asm("min.s16x2 %0, %0, %1;" : "+r"(v) : "r"(0x000f000fu));
    return v;
}
// Eight codes, the first in the lowest bits; four codes as two bytes.
__device__ __forceinline__ uint32_t code4x8(const float *x, const Group4 &g) {
    return codes4_pair(x[0], x[4], g) + codes4_pair(x[1], x[5], g) * 16u + codes4_pair(x[2], x[6], g) * 256u +
           codes4_pair(x[3], x[7], g) * 4096u;
}
__device__ __forceinline__ uint32_t code4x4(float x0, float x1, float x2, float x3, const Group4 &g) {
    const uint32_t v = codes4_pair(x0, x2, g) + codes4_pair(x1, x3, g) * 16u;     // bytes 0 and 2
    return __byte_perm(v, 0u, 0x4420u);
}

// Packed minimum and maximum of 16-bit values, NaN where either is.
template <bool BF16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF16)
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <bool BF16>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (BF16)
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

}  // namespace pa
