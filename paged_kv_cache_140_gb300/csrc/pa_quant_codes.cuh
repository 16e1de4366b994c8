// The codes and scales of the quantised caches, from a row's extremes: shared by
// the cache write (pa_quant_ops.cu) and the rotation that writes into a cache
// (pa_rope.cu), so that both make the same bytes of the same 32-bit values.
#pragma once

#include "pa_device.cuh"

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

__device__ __forceinline__ Group4 group4(float lo, float hi, bool finite) {
    // (halves: the range of values of both signs may pass the largest float)
    const float step = __fdiv_rn(__fsub_rn(__fmul_rn(0.5f, hi), __fmul_rn(0.5f, lo)), 7.5f);
    const float s = fmaxf(fmaxf(step, __fmul_rn(fmaxf(hi, -lo), 0.00390625f)), kAmaxFloor);
    const uint32_t sb = float_to_bf16_bits(s);
    const float sf = __uint_as_float(sb << 16);
    const uint32_t zb = float_to_bf16_bits(__fdiv_rn(lo, sf));
    Group4 g;
    g.inv = __fdiv_rn(1.f, sf);
    g.zero = __uint_as_float(zb << 16);
    g.word = finite ? sb | (zb << 16) : kNanBits >> 16;
    return g;
}

// The code of x in the low four bits (those above the low byte are not zero).
__device__ __forceinline__ uint32_t code4(float x, const Group4 &g) {
    const float y = __fsub_rn(__fmul_rn(x, g.inv), g.zero);
    return __float_as_uint(__fadd_rn(fminf(fmaxf(y, 0.f), 15.f), 12582912.f));
}
// Two codes as one byte (the low byte of the result).
__device__ __forceinline__ uint32_t code4x2(float x0, float x1, const Group4 &g) {
    return code4(x0, g) + (code4(x1, g) << 4);
}
__device__ __forceinline__ uint32_t code4x8(const float *x, const Group4 &g) {
    return __byte_perm(__byte_perm(code4x2(x[0], x[1], g), code4x2(x[2], x[3], g), 0x0040u),
                       __byte_perm(code4x2(x[4], x[5], g), code4x2(x[6], x[7], g), 0x0040u), 0x5410u);
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
