// What sampling (sample.cu) and the verification of drafted tokens
// (verify.cu) share: whole-number masses, sums over warps and clusters, and
// what a row's filters keep.
#pragma once

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "mma.cuh"

namespace gwa {

using u64 = unsigned long long;

// A row's weights.
struct SmRow {
    float top, per;
    // base-2 exponent of a logit's mass relative to the largest's: <= 0; for
    // a NaN NaN, for -inf -inf or (infinite T) NaN
    __device__ __forceinline__ float expo(float x) const {
        return x == top ? 0.f : __fmul_rn(__fsub_rn(x, top), per);
    }
    // floor(2^40 exp2f(y)): the 24-bit significand shifted by the exponent.
    // From -44 to 0 exp2f gives ex2's value (checked for every float there);
    // below -40 the shifts leave zero, and so they do for a NaN, whose counts
    // all lie past 31.
    static __device__ __forceinline__ u64 mass_of(float y) { return whole(ex2(y)); }
    // floor(2^40 t), t >= 0
    static __device__ __forceinline__ u64 whole(float t) {
        const uint32_t b = __float_as_uint(t), e = b >> 23, m = (b & 0x7fffffu) | 0x800000u;
        return ((u64)shr(m, 142u - e) << 32) | (shl(m, e - 110u) | shr(m, 110u - e));
    }
    // exp2f(y), and for a NaN zero: the mass times 2^-40, before its floor.
    static __device__ __forceinline__ float part_of(float y) { return fmaxf(ex2(y), 0.f); }
    __device__ __forceinline__ u64 mass(float x) const { return mass_of(expo(x)); }
    // (zero past 31)
    static __device__ __forceinline__ uint32_t shl(uint32_t v, uint32_t n) {
        uint32_t r;
        asm("shl.b32 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(n));
        return r;
    }
    static __device__ __forceinline__ uint32_t shr(uint32_t v, uint32_t n) {
        uint32_t r;
        asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(n));
        return r;
    }
};

// Of a warp's 32 lanes: the sums up to and with one's own.
template <typename T>
__device__ __forceinline__ T warp_scan(T v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T w = __shfl_up_sync(0xffffffffu, v, o);
        if ((int)(threadIdx.x & 31) >= o) v += w;
    }
    return v;
}
// A sum of masses, each from its part t = exp2f(y), without a shift: 8 + t
// rounded towards zero holds the mass's upper 21 bits at the end of its
// significand, 2^-17 plus what is left of t its lower 20.  The words are
// added as they are and the constants taken off at the end; up to 2048 masses
// a thread (of 2^19 tokens on 1024 threads at most 512).
struct MassSum {
    uint32_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(float t) {
        const float s = __fadd_rz(t, 8.f);
        hi += __float_as_uint(s);
        lo += __float_as_uint(__fadd_rz(__fsub_rn(t, __fsub_rn(s, 8.f)), 0x1p-17f));
    }
    __device__ __forceinline__ u64 total(uint32_t count) const {
        return ((u64)(hi - count * __float_as_uint(8.f)) << 20) +
               (u64)(uint32_t)(lo - count * __float_as_uint(0x1p-17f));
    }
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// floor(total f) for f in [0, 1): the float's significand times the total,
// shifted (64-bit floating point takes thousands of cycles here).
__device__ __forceinline__ u64 part(u64 total, float f) {
    const uint32_t b = __float_as_uint(fmaxf(f, 0.f));
    const u64 m = (b & 0x7fffffu) | (b >> 23 ? 0x800000u : 0u);
    const int sh = 150 - max((int)(b >> 23), 1);  // f = m 2^-sh, sh >= 24
    const u64 lo = total * m, hi = __umul64hi(total, m);
    return sh < 64 ? lo >> sh | hi << (64 - sh) : sh < 128 ? hi >> (sh - 64) : 0;
}
// The mass at which a random number falls.
__device__ __forceinline__ u64 drawn_at(u64 total, float u) {
    return u >= 1.f ? total - 1 : part(total, u);
}
// A token's share of the kept (rounded three times).
__device__ __forceinline__ float share(u64 w, u64 total) {
    return __fdiv_rn(__ull2float_rn(w), __ull2float_rn(total));
}

// What a row's filters keep: the logits above cut_x, and its equals up to
// token cut_idx, of a mass of at least `least`; their masses' sum.
struct SmPlan {
    float top, per, cut_x;
    uint32_t cut_idx;
    u64 least, total;
    __device__ __forceinline__ u64 kept(float x, uint32_t token) const {
        // (nothing below cut_x, -inf and NaN among it)
        if (!(x > cut_x || (x == cut_x && token <= cut_idx))) return 0;
        const u64 w = SmRow{top, per}.mass(x);
        return w >= least ? w : 0;
    }
    // its part, zero where it is not kept.  least_t: least times 2^-40 (a float
    // holds it: it comes from one)
    __device__ __forceinline__ float part(float x, uint32_t token, float least_t) const {
        const float t = SmRow::part_of(SmRow{top, per}.expo(x));
        const bool in = x > cut_x || (x == cut_x && token <= cut_idx);
        return in && t >= least_t ? t : 0.f;
    }
};

// The sequence that a token belongs to (-1: none), its first token and the one
// behind its last; for a whole warp, whose lanes search 32 entries of the
// non-decreasing q_start at a time.
struct SmSeq {
    int seq, first, next;
};
__device__ __forceinline__ SmSeq sm_sequence(const int32_t *q_start, int batch, int64_t tok) {
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    int lo = 0, n = batch + 1;  // the answer's entry lies in [lo, lo + n)
    while (true) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const bool in = lane * step < n;
        const int start = in ? q_start[i] : 0;
        const int next = in && step == 1 && i < batch ? q_start[i + 1] : 0;
        const int c = __popc(__ballot_sync(FULL, in && start <= tok));
        if (c == 0) return {-1, 0, 0};
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
        if (step > 1) continue;
        if (lo >= batch) return {-1, 0, 0};
        return {lo, __shfl_sync(FULL, start, c - 1), __shfl_sync(FULL, next, c - 1)};
    }
}

}  // namespace gwa
