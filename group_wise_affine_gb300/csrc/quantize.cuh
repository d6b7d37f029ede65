// One group of 64 values quantized by eight lanes, eight values each: the
// affine rule of the weight quantizer, shared with the KV cache.
#pragma once

#include "common.cuh"

namespace gwa {

// v: this lane's eight bf16 values (widened) of a group held by eight
// consecutive lanes; every lane of the warp takes part.  q: their codes;
// scale and bias (bf16 bits) are the same on the group's eight lanes.
template <int BITS>
__device__ __forceinline__ void quantize_group8(const float (&v)[8],
                                                uint32_t (&q)[8],
                                                uint16_t &sbits,
                                                uint16_t &bbits) {
    constexpr uint32_t QMAX = (1u << BITS) - 1u;
    float lo = v[0], hi = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fminf(lo, v[i]);
        hi = fmaxf(hi, v[i]);
    }
#pragma unroll
    for (int m = 1; m < 8; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    lo = lo + 0.0f;  // a zero minimum is stored as +0
    sbits = f32_to_bf16_bits(__fdiv_rn(hi - lo, (float)QMAX));
    const float s = bf16_bits_to_f32(sbits);
    // The code is rint of the correctly rounded quotient d / s.  A
    // product with the correctly rounded reciprocal is within
    // 1.5 * 2^-23 * d/s (<= 4.6e-5, d/s <= ~257) of that quotient, so its
    // rounding can differ only when it lies within that distance of a
    // half-integer (about one input in 10^4); a lane holding such an
    // input redoes its eight codes by the division, which gives the same
    // codes for the others.  Subnormal scales (a reciprocal that may
    // overflow) always divide.
    const bool fast = s >= 1.17549435e-38f;
    const float r = fast ? __frcp_rn(s) : 0.0f;
    float emax = 0.0f;  // the largest distance of a product from an integer
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float d = v[i] - lo;  // >= 0, as in the reading
        const float t = d * r;
        // t + 1.5 * 2^23 rounds t to an integer, ties to even, into
        // the low mantissa bits (0 <= t < 2^22)
        const float tt = t + 12582912.0f;
        emax = fmaxf(emax, fabsf(t - (tt - 12582912.0f)));
        q[i] = min(__float_as_uint(tt) - 0x4b400000u, QMAX);
    }
    // a product within reach of a half-integer, or no usable reciprocal:
    // all eight codes again by the division (rare; uniform per lane)
    if (!fast || emax > 0.5f - 0x1p-12f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = v[i] - lo;
            uint32_t c = 0u;
            if (s != 0.0f) {
                const float tx = rintf(__fdiv_rn(d, s));
                c = tx <= 0.0f ? 0u : tx >= (float)QMAX ? QMAX : (uint32_t)tx;
            }
            q[i] = c;
        }
    }
    bbits = (uint16_t)(__float_as_uint(lo) >> 16);
}

// The same codes for four lanes of 16 values each (eight words of two bf16),
// packed into the words they fill, lowest bits first: a group's own work is
// shared by twice as many values, and no lane divides.  Values that come as
// bf16 lie on a coarse grid and hit half-integers in a few groups of a hundred
// (a scale of few bits divides them exactly), so that most warps would have a
// lane on the dividing path above.  Here the quotient itself is rounded
// correctly: the product with the correctly rounded reciprocal, corrected
// twice by its remainder, the first time to within an ulp, the second time to
// the rounded quotient (Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990).  The remainders are exact while
// 2^-24 of the scale's own last place is: scales below 2^-100 divide.
template <int BITS>
__device__ __forceinline__ void quantize_group16(const uint32_t (&v)[8],
                                                 uint32_t (&word)[BITS / 2],
                                                 uint16_t &sbits,
                                                 uint16_t &bbits) {
    constexpr uint32_t QMAX = (1u << BITS) - 1u;
    constexpr int PER = 32 / BITS;  // codes of a word
    // what a word has in excess when its codes' sums with 1.5 * 2^23 are
    // added up as they are
    constexpr uint32_t EXCESS = 0x4b400000u * (0xffffffffu / QMAX);
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16_lo(v[i]);
        x[2 * i + 1] = bf16_hi(v[i]);
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    lo = lo + 0.0f;  // a zero minimum is stored as +0
    sbits = f32_to_bf16_bits(__fdiv_rn(hi - lo, (float)QMAX));
    bbits = (uint16_t)(__float_as_uint(lo) >> 16);
    const float s = bf16_bits_to_f32(sbits);
    if (s >= 0x1p-100f) {
        // (an infinite scale, r = 0: zero for finite values, the largest
        // code for the others, as above)
        const float r = __frcp_rn(s), b = r > 0.f ? -s : 0.f;
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) word[j] = 0u - EXCESS;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float d = x[i] - lo;
            float t = d * r;
            t = fmaf(fmaf(b, t, d), r, t);
            t = fmaf(fmaf(b, t, d), r, t);
            // rounded to an integer, ties to even, into the low bits
            const float tt = fminf(t, (float)QMAX) + 12582912.0f;
            word[i / PER] += __float_as_uint(tt) << (BITS * (i % PER));
        }
    } else {
#pragma unroll
        for (int j = 0; j < BITS / 2; ++j) word[j] = 0u;
        if (s != 0.0f)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float t = rintf(__fdiv_rn(x[i] - lo, s));
                const uint32_t c = t <= 0.0f ? 0u : t >= (float)QMAX ? QMAX : (uint32_t)t;
                word[i / PER] |= c << (BITS * (i % PER));
            }
    }
}

// Eight codes as the packed words they fill, lowest bits first.
__device__ __forceinline__ uint32_t pack_u4(const uint32_t (&q)[8]) {
    uint32_t word = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) word |= q[i] << (4 * i);
    return word;
}
__device__ __forceinline__ uint2 pack_u8(const uint32_t (&q)[8]) {
    return make_uint2(q[0] | (q[1] << 8) | (q[2] << 16) | (q[3] << 24),
                      q[4] | (q[5] << 8) | (q[6] << 16) | (q[7] << 24));
}

}  // namespace gwa
