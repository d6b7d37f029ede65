// One token a row from logits under temperature, top-k, top-p and min-p, by
// the row's given random number: the step that ends a decode step (the pages'
// server samples its tokens, "Sanctum-MLX", server diagram; they print no
// rule, so the rule here is this library's reading, stated in gwa.h).
//
// Whole-number masses.  Token i's mass is w_i = floor(2^40 exp2((x_i - max)
// * log2(e) / T)), a 64-bit integer, and every sum of masses is an integer
// sum.  Integer sums do not depend on their order, so the token does not
// depend on how the row is split over threads and CTAs, nor on the order in
// which their atomics arrive; a floating sum would move the drawn token
// wherever the random number lies within its rounding of a boundary.  Masses
// below 2^-40 of the likeliest token's are dropped, at most 2^-21 of the
// whole at 2^19 tokens.
//
// The kept tokens are a prefix of the order (logit descending, index
// ascending).  Three ways to them, each exact:
//   top-k of up to 512: the step of exponent in which the k-th largest of the
//     threads' maxima lies bounds the k-th token from below; the tokens above
//     the bound (a few more than k) are gathered, sorted and drawn from by one
//     CTA.  No token but the maxima is counted.
//   no top-k: with the row's total mass known, a token below (total - goal) /
//     V cannot be among the first that reach top-p's goal, nor one below
//     min-p's mass be kept; if 2048 tokens or fewer are left they go the same
//     way.
//   otherwise: a histogram over 2048 equal steps of the base-2 exponent y
//     between the row's smallest value (or 2^-41, whose masses are zero) and
//     its largest, which serves top-k and top-p alike; then the tokens of the
//     one step that holds the cut are gathered and ranked by one CTA.  Steps
//     of y spread the tokens of a real row over many counters (the high bits
//     of the logits put most of them on a handful, whose atomics then queue).
//     A step that holds more than 2048 tokens (equal or clustered logits) is
//     searched digit by digit on order-preserving integer keys instead.  The
//     cut is one logit and one index, and a last pass draws.
//
// A row belongs to a cluster of CTAs.  Each keeps its slice of the row in
// shared memory, read from HBM once; histograms and sums are joined through
// distributed shared memory, each CTA adding up a share of the steps and
// handing it to all.  One launch per call.  The cluster is the smallest that
// holds the row, made larger while the rows leave SMs idle.
//
// Bound: instructions and the latency of a dozen barriers.  The logits are
// read once (256 rows of 151669 bf16, 78 MB, 11.5 us of HBM bandwidth; a CTA
// loads its 150 KB slice in 7.5 thousand cycles, near that rate), then a row
// with top-k takes about 30 thousand cycles more (bound 11, gather 11, sort
// and draw 12), one with top-p alone and a flat distribution 110 (masses 14,
// histogram 45, ranking and the last pass 45), and nothing of the next row is
// loaded meanwhile: 101 us for those rows with filters of all kinds, 16 us for
// one row of 131072 fp32 on 16 CTAs.
//
// With PLAN the same passes end before the draw, and leave the cut and the sum
// (of a row cut by top-p alone the sum is known with the cut: no last pass).
#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "sample.cuh"

namespace gwa {

constexpr int kSmThreads = 1024;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmBins = 2048;
constexpr int kSmList = 2048;  // tokens that one CTA ranks
// top-k of up to this goes by the threads' maxima: at half as many as a CTA's
// threads the bound lets about 1.4 k tokens through, and 2048 hold them (256 x
// 151669 rows with filters of all kinds: 173 us with it, 231 without)
constexpr int kSmShort = kSmThreads / 2;
constexpr int kSmMaxCluster = 16;
constexpr int64_t kSmSliceBytes = 152 * 1024;

// Logits as order-preserving keys; 0 is below every logit (no token there),
// NaN counts as -inf and -0 as +0.
template <bool BF16>
struct SmKey;
template <>
struct SmKey<true> {
    using Raw = uint16_t;
    using Key = uint16_t;
    static constexpr int PASSES = 2, BITS = 16;
    static __device__ __forceinline__ Key make(Raw r) {
        uint32_t u = r;
        if ((u & 0x7fffu) > 0x7f80u) u = 0xff80u;
        if (u == 0x8000u) u = 0u;
        return (Key)(u & 0x8000u ? 0xffffu & ~u : u | 0x8000u);
    }
    static __device__ __forceinline__ float value(Key k) {
        const uint32_t u = k & 0x8000u ? k & 0x7fffu : 0xffffu & ~(uint32_t)k;
        return __uint_as_float(u << 16);
    }
    static __device__ __forceinline__ int shift(int pass) { return pass == 0 ? 8 : 0; }
    static __device__ __forceinline__ int width(int) { return 8; }
};
template <>
struct SmKey<false> {
    using Raw = uint32_t;
    using Key = uint32_t;
    static constexpr int PASSES = 3, BITS = 32;
    static __device__ __forceinline__ Key make(Raw u) {
        if ((u & 0x7fffffffu) > 0x7f800000u) u = 0xff800000u;
        if (u == 0x80000000u) u = 0u;
        return u & 0x80000000u ? ~u : u | 0x80000000u;
    }
    static __device__ __forceinline__ float value(Key k) {
        return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
    }
    static __device__ __forceinline__ int shift(int pass) {
        return pass == 0 ? 21 : pass == 1 ? 10 : 0;
    }
    static __device__ __forceinline__ int width(int pass) { return pass == 2 ? 10 : 11; }
};

// Shared memory besides the slice.
struct SmShared {
    uint32_t cnt[kSmBins], lo[kSmBins], hi[kSmBins];  // this CTA's histogram
    uint32_t all_cnt[kSmBins];                        // the cluster's
    u64 all_mass[kSmBins];
    // gathered tokens (in rank 0), see list_key; partial sums of join
    u64 list[kSmList];
    u64 x_mass[kSmMaxCluster];      // one value from every CTA
    float x_top[kSmMaxCluster], x_low[kSmMaxCluster];
    uint32_t x_word[kSmMaxCluster];
    u64 w_mass[kSmWarps], t_mass[kSmWarps];  // one value from every warp
    uint32_t w_word[kSmWarps], t_cnt[kSmWarps];
    float w_top[kSmWarps], w_low[kSmWarps];
    uint32_t list_n;                // gathered so far (in rank 0)
    // what a search settled on
    uint32_t f_bin, f_above_cnt;
    u64 f_above_mass;
    float cut_x;
    uint32_t cut_idx;
    u64 cut_mass;                   // of a step's tokens up to the cut
};

template <bool BF16>
struct Sampler {
    using K = SmKey<BF16>;
    using Raw = typename K::Raw;
    static constexpr int PER = 16 / sizeof(Raw);  // logits of a 16-byte chunk
    SmShared &sh;
    const Raw *raw;   // the slice; element e is token base + e
    int first, last;  // its elements [first, last)
    int64_t base;
    int cl, rank;
    SmRow row;
    float steps;      // histogram steps per unit of y

    // NaN as -inf
    __device__ __forceinline__ float value(int e) const {
        const float x = __uint_as_float(BF16 ? (uint32_t)raw[e] << 16 : (uint32_t)raw[e]);
        return x == x ? x : -INFINITY;
    }
    // The logits of chunk j (-inf outside the slice).
    __device__ __forceinline__ void load(int j, float (&x)[PER]) const {
        const uint4 c = *reinterpret_cast<const uint4 *>(raw + j * PER);
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int i = 0; i < PER; ++i)
            x[i] = BF16 ? (i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2])) : __uint_as_float(w[i % 4]);
    }
    // Ascending in the order of the tokens: logit downwards, then index.
    static __device__ __forceinline__ u64 list_key(float x, uint32_t idx) {
        return ((u64)~SmKey<false>::make(__float_as_uint(x)) << 32) | idx;
    }
    __device__ __forceinline__ int bin_of(float x) const {
        // NaN and -inf (and everything past the range) in the last step
        const float t = fminf(-row.expo(x) * steps, (float)(kSmBins - 1));
        return x == -INFINITY ? kSmBins - 1 : (int)t;
    }

    // The cluster's sum of one value from every CTA, and the lower ranks'.
    __device__ u64 cluster_total(u64 v, u64 &before) {
        if (threadIdx.x < (unsigned)cl) *cluster_ptr(&sh.x_mass[rank], threadIdx.x) = v;
        cluster_sync_all();
        u64 t = 0;
        before = 0;
        for (int r = 0; r < cl; ++r) {
            if (r < rank) before += sh.x_mass[r];
            t += sh.x_mass[r];
        }
        return t;
    }

    // The cluster's sum of a value from every thread.
    __device__ u64 sum_all(u64 v) {
        v = warp_sum64(v);
        if ((threadIdx.x & 31) == 0) sh.w_mass[threadIdx.x / 32] = v;
        sync_all();  // (x_mass is read, too)
        u64 before;
        v = cluster_total(warp_sum64(sh.w_mass[threadIdx.x & 31]), before);
        __syncthreads();
        return v;
    }

    __device__ __forceinline__ void add(uint32_t bin, bool count, u64 w) {
        if (count) atomicAdd(&sh.cnt[bin], 1u);
        if (w) {
            // 64-bit sum from two 32-bit words: the carry shows in the old one
            const uint32_t wl = (uint32_t)w;
            const uint32_t old = atomicAdd(&sh.lo[bin], wl);
            const uint32_t up = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
            if (up) atomicAdd(&sh.hi[bin], up);
        }
    }
    __device__ void clear(int bins) {
        for (int i = threadIdx.x; i < bins; i += kSmThreads) sh.cnt[i] = sh.lo[i] = sh.hi[i] = 0;
        __syncthreads();
    }
    // The logits of a step, a step wider on either side.
    __device__ __forceinline__ float x_high(int bin) const {
        return steps > 0.f && bin > 1 ? x_above((float)(1 - bin) / steps) : INFINITY;
    }
    __device__ __forceinline__ float x_low(int bin) const {
        return steps > 0.f && bin < kSmBins - 1 ? x_below(-(float)(bin + 2) / steps) : -INFINITY;
    }
    __device__ __forceinline__ void sync_all() {
        if (cl > 1)
            cluster_sync_all();
        else
            __syncthreads();
    }
    // Adds the CTAs' histograms up, a share of the bins each, and hands the
    // sums to all (masses: or the counts only).  A warp reads, and writes, consecutive bins of one CTA;
    // groups of threads take different CTAs.
    __device__ void join(int bins, bool masses) {
        const int tid = threadIdx.x;
        if (cl == 1) {
            __syncthreads();
            for (int b = tid; b < bins; b += kSmThreads) {
                sh.all_cnt[b] = sh.cnt[b];
                sh.all_mass[b] = (u64)sh.lo[b] + ((u64)sh.hi[b] << 32);
            }
            __syncthreads();
            return;
        }
        cluster_sync_all();
        const int share = bins / cl, groups = min(cl, kSmThreads / share);
        const int b = tid % share, g = tid / share, bin = rank * share + b;
        uint32_t *const pc = reinterpret_cast<uint32_t *>(sh.list + kSmThreads);  // after the masses
        uint32_t c = 0;
        u64 m = 0;
        if (g < groups) {
            for (int r = g; r < cl; r += groups) {
                c += *cluster_ptr(&sh.cnt[bin], r);
                if (masses)
                    m += (u64)*cluster_ptr(&sh.lo[bin], r) + ((u64)*cluster_ptr(&sh.hi[bin], r) << 32);
            }
            pc[tid] = c;
            sh.list[tid] = m;
        }
        __syncthreads();
        if (g < groups) {
            c = 0;
            m = 0;
            for (int k = 0; k < groups; ++k) {
                c += pc[k * share + b];
                m += sh.list[k * share + b];
            }
            for (int r = g; r < cl; r += groups) {
                *cluster_ptr(&sh.all_cnt[bin], r) = c;
                if (masses) *cluster_ptr(&sh.all_mass[bin], r) = m;
            }
        }
        cluster_sync_all();
    }
    // The bin where the count, or the mass, first reaches `goal`, walking the
    // bins upwards (or down from the last); `goal` of 0 with share >= 0 is
    // that share of the total (at least 1).  Returns the goal; f_* are set.
    __device__ u64 locate(int bins, bool down, bool mass, u64 goal, float share) {
        const int per = (bins + kSmThreads - 1) / kSmThreads;
        u64 sum = 0;
        uint32_t cn = 0;
        for (int j = 0; j < per; ++j) {
            const int b = threadIdx.x * per + j;
            if (b < bins) {
                sum += sh.all_mass[down ? bins - 1 - b : b];
                cn += sh.all_cnt[down ? bins - 1 - b : b];
            }
        }
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        const u64 im = warp_scan(sum);
        const uint32_t ic = warp_scan(cn);
        if (lane == 31) {
            sh.t_mass[warp] = im;
            sh.t_cnt[warp] = ic;
        }
        __syncthreads();
        const u64 wm = warp_scan(sh.t_mass[lane]);
        const uint32_t wc = warp_scan(sh.t_cnt[lane]);
        u64 bm = im - sum + __shfl_sync(0xffffffffu, wm, max(warp - 1, 0)) * (warp > 0);
        uint32_t bc = ic - cn + __shfl_sync(0xffffffffu, wc, max(warp - 1, 0)) * (warp > 0);
        if (share >= 0.f) goal = share_of(__shfl_sync(0xffffffffu, wm, 31), share);
        for (int j = 0; j < per; ++j) {
            const int k = threadIdx.x * per + j, b = down ? bins - 1 - k : k;
            if (k >= bins) break;
            const u64 m = sh.all_mass[b];
            const uint32_t c = sh.all_cnt[b];
            const u64 at = mass ? bm : bc, v = mass ? m : c;
            if (at < goal && goal <= at + v) {
                sh.f_bin = b;
                sh.f_above_mass = bm;
                sh.f_above_cnt = bc;
            }
            bm += m;
            bc += c;
        }
        __syncthreads();
        return goal;
    }

    // Gathers, in rank 0 and in any order, the tokens that pass in(x, token);
    // those outside [x_lo, x_hi] are known not to.  Returns how many there
    // are; the list holds the first kSmList of them.  Every CTA fills its own
    // list (an atomic on another CTA's counter takes most of a microsecond),
    // which then goes to rank 0 behind the lower ranks'.
    template <class In>
    __device__ uint32_t gather(float x_lo, float x_hi, In in) {
        if (threadIdx.x == 0) sh.list_n = 0;
        __syncthreads();
        for (int j = threadIdx.x; j < (last + PER - 1) / PER; j += kSmThreads) {
            float x[PER];
            load(j, x);
            uint32_t hits = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (!(x[i] < x_lo) && !(x[i] > x_hi)) hits |= 1u << i;
            for (; hits; hits &= hits - 1) {
                const int e = j * PER + __ffs(hits) - 1;
                const float v = value(e);
                if (e < first || e >= last || !in(v, (uint32_t)(base + e))) continue;
                const uint32_t at = atomicAdd(&sh.list_n, 1u);
                if (at < kSmList) sh.list[at] = list_key(v, (uint32_t)(base + e));
            }
        }
        __syncthreads();
        const uint32_t own = sh.list_n;
        if (cl == 1) return own;
        if (threadIdx.x < cl) *cluster_ptr(&sh.x_word[rank], threadIdx.x) = own;
        cluster_sync_all();
        uint32_t before = 0, n = 0;
        for (int r = 0; r < cl; ++r) {
            if (r < rank) before += sh.x_word[r];
            n += sh.x_word[r];
        }
        if (rank > 0) {
            u64 *const list = cluster_ptr(sh.list, 0);
            for (uint32_t i = threadIdx.x; i < own && before + i < kSmList; i += kSmThreads)
                list[before + i] = sh.list[i];
        }
        cluster_sync_all();
        return n;
    }
    // The logit whose exponent is y, or a little below (above) it.
    __device__ __forceinline__ float x_below(float y) const {
        const float x = __fadd_rd(row.top, __fdiv_rd(y, row.per));
        return x == x ? x : -INFINITY;
    }
    __device__ __forceinline__ float x_above(float y) const {
        const float x = __fadd_ru(row.top, __fdiv_ru(y, row.per));
        return x == x ? x : INFINITY;
    }
    // Sorts the list's first `total` words upwards (this CTA's; bitonic, a
    // pair of words a thread and step, by as many warps as that takes).  A
    // warp's 32 pairs at a distance of up to 32 are 64 neighbouring words, so
    // those steps wait for the warp only.
    __device__ void sort(int total) {
        int size = 64;
        while (size < total) size *= 2;
        for (int i = total + threadIdx.x; i < size; i += kSmThreads) sh.list[i] = ~0ull;
        __syncthreads();
        const int i = threadIdx.x;
        if (i < size / 2)
            for (int k = 2; k <= size; k *= 2)
                for (int d = k / 2; d > 0; d /= 2) {
                    const int a = 2 * i - (i & (d - 1)), b = a + d;
                    const u64 x = sh.list[a], y = sh.list[b];
                    if ((x > y) == ((a & k) == 0)) {
                        sh.list[a] = y;
                        sh.list[b] = x;
                    }
                    if (size > 64 && (d > 32 || (d == 1 && k >= 64)))
                        asm volatile("bar.sync 1, %0;" ::"r"(size / 2) : "memory");
                    else
                        __syncwarp();
                }
        __syncthreads();
    }
    // The lower threads' sum of v in this CTA, and all threads'.
    __device__ u64 scan(u64 v, u64 &total) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        const u64 incl = warp_scan(v);
        __syncthreads();
        if (lane == 31) sh.t_mass[warp] = incl;
        __syncthreads();
        const u64 wm = warp_scan(sh.t_mass[lane]);
        total = __shfl_sync(0xffffffffu, wm, 31);
        return incl - v + __shfl_sync(0xffffffffu, wm, max(warp - 1, 0)) * (warp > 0);
    }
    static constexpr int PT = kSmList / kSmThreads;  // list words of a thread, side by side

    // ---- a whole draw from a sorted list that holds the row's first tokens
    // (this CTA's): its first n, of those as many as reach `goal` (0: the
    // share tp of the n), of those the masses of at least `least`
    __device__ void draw(int n, u64 goal, float tp, u64 least, float u, int32_t *token, float *prob) {
        u64 own[PT], sum = 0, total;
        uint32_t idx[PT];
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int i = threadIdx.x * PT + j;
            own[j] = i < n ? row.mass(SmKey<false>::value(~(uint32_t)(sh.list[i] >> 32))) : 0;
            idx[j] = i < n ? (uint32_t)sh.list[i] : 0u;
            sum += own[j];
        }
        u64 before = scan(sum, total);
        if (goal == 0) goal = tp < 1.f ? share_of(total, tp) : ~0ull;
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int i = threadIdx.x * PT + j;
            const bool keep = before < goal && own[j] >= least;
            before += own[j];
            // by token from here on: 19 bits of it, 41 of mass
            if (i < n) sh.list[i] = ((u64)idx[j] << 41) | (keep ? own[j] : 0);
        }
        sort(n);
        sum = 0;
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int i = threadIdx.x * PT + j;
            const u64 w = i < n ? sh.list[i] : 0;
            own[j] = w & ((1ull << 41) - 1);
            idx[j] = (uint32_t)(w >> 41);
            sum += own[j];
        }
        before = scan(sum, total);
        const u64 at = drawn_at(total, u);
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            if (before <= at && at < before + own[j]) {
                *token = (int32_t)idx[j];
                if (prob) *prob = share(own[j], total);
            }
            before += own[j];
        }
    }
    // What top-p has to reach, and where a random number falls.
    static __device__ __forceinline__ u64 share_of(u64 total, float tp) {
        const u64 goal = part(total, tp);
        return goal < 1 ? 1 : goal;
    }

    // ---- what that draw would keep
    __device__ void plan(int n, u64 goal, float tp, u64 least, SmPlan *out) {
        u64 own[PT], sum = 0, total;
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            const int i = threadIdx.x * PT + j;
            own[j] = i < n ? row.mass(SmKey<false>::value(~(uint32_t)(sh.list[i] >> 32))) : 0;
            sum += own[j];
        }
        u64 before = scan(sum, total), kept = 0, count = 0;
        if (goal == 0) goal = tp < 1.f ? share_of(total, tp) : ~0ull;
#pragma unroll
        for (int j = 0; j < PT; ++j) {
            if ((int)threadIdx.x * PT + j < n && before < goal && own[j] >= least) {
                kept += own[j];
                ++count;
            }
            before += own[j];
        }
        scan(kept, total);
        u64 tokens;
        scan(count, tokens);
        if (threadIdx.x == 0) {
            const u64 last = sh.list[max((int)tokens, 1) - 1];  // (the first is always kept)
            *out = SmPlan{row.top, row.per, SmKey<false>::value(~(uint32_t)(last >> 32)), (uint32_t)last,
                          least, total};
        }
    }

    // ---- the cut among the tokens of histogram step `bin` that lie above
    // (x, idx): their first `want` (by count), or as many as reach `want`
    // (by mass).  Leaves the last kept token in cut_x, cut_idx, and the mass of
    // the kept in cut_mass.
    __device__ void refine(int bin, bool mass, u64 want, bool cut, float cut_x, uint32_t cut_idx) {
        auto in = [&](float x, uint32_t idx) {
            return bin_of(x) == bin && (!cut || x > cut_x || (x == cut_x && idx <= cut_idx));
        };
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        const uint32_t n = gather(x_low(bin), x_high(bin), in);
        if (n <= kSmList) {
            if (rank == 0) {
                // in order, and counted up
                sort((int)n);
                u64 own[PT], sum = 0, kept = 0, total;
                float x[PT];
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    const int i = threadIdx.x * PT + j;
                    x[j] = i < n ? SmKey<false>::value(~(uint32_t)(sh.list[i] >> 32)) : 0.f;
                    own[j] = i >= n ? 0 : mass ? row.mass(x[j]) : 1;
                    sum += own[j];
                    if (!mass && (u64)i < min((u64)n, want)) kept += row.mass(x[j]);
                }
                u64 before = scan(sum, total);
#pragma unroll
                for (int j = 0; j < PT; ++j) {
                    if (before < want && want <= before + own[j])
                        for (int r = 0; r < cl; ++r) {
                            *cluster_ptr(&sh.cut_x, r) = x[j];
                            *cluster_ptr(&sh.cut_idx, r) = (uint32_t)sh.list[threadIdx.x * PT + j];
                            if (mass) *cluster_ptr(&sh.cut_mass, r) = before + own[j];
                        }
                    before += own[j];
                }
                if (!mass) {
                    scan(kept, total);
                    if (threadIdx.x < cl) *cluster_ptr(&sh.cut_mass, threadIdx.x) = total;
                }
            }
            sync_all();
            return;
        }
        // too many: digit by digit on integer keys
        uint32_t prefix = 0;
        int done = 0;
        u64 above = 0;
        for (int pass = 0; pass < K::PASSES; ++pass) {
            const int sft = K::shift(pass), wid = K::width(pass), bins = 1 << wid;
            if (pass == 0) save();
            clear(bins);
            for (int e = first + threadIdx.x; e < last; e += kSmThreads) {
                const float x = value(e);
                if (!in(x, (uint32_t)(base + e))) continue;
                const uint32_t k = K::make(raw[e]);
                if (done && (k >> (K::BITS - done)) != prefix) continue;
                add((k >> sft) & (bins - 1), !mass, mass ? row.mass(x) : 0);
            }
            join(bins, mass);
            locate(bins, true, mass, want - above, -1.f);
            prefix = (prefix << wid) | sh.f_bin;
            above += mass ? sh.f_above_mass : sh.f_above_cnt;
            done += wid;
            __syncthreads();
        }
        // the cut's key; of its equals, so many by index
        const float x = K::value((typename K::Key)prefix);
        const u64 left = want - above;
        const u64 own = mass ? row.mass(x) : 1;
        const u64 nth = (left + own - 1) / own;  // 1-based
        const int run = ((last - first + kSmWarps - 1) / kSmWarps + 31) & ~31;
        const int a = first + warp * run, b = min(last, a + run);
        uint32_t c = 0;
        for (int e0 = a; e0 < b; e0 += 32) {
            const int e = e0 + lane;
            c += __popc(__ballot_sync(0xffffffffu, e < b && value(e) == x && in(x, (uint32_t)(base + e))));
        }
        if (lane == 0) sh.w_word[warp] = c;
        __syncthreads();
        u64 mine = 0, before = 0, at = 0;
        for (int w = 0; w < kSmWarps; ++w) {
            if (w < warp) at += sh.w_word[w];
            mine += sh.w_word[w];
        }
        cluster_total(mine, before);
        at += before;
        if (at < nth && nth <= at + c)
            for (int e0 = a; e0 < b; e0 += 32) {
                const int e = e0 + lane;
                const bool eq = e < b && value(e) == x && in(x, (uint32_t)(base + e));
                const unsigned m = __ballot_sync(0xffffffffu, eq);
                if (eq && at + __popc(m & ((1u << lane) - 1u)) + 1 == nth)
                    for (int r = 0; r < cl; ++r) {
                        *cluster_ptr(&sh.cut_x, r) = x;
                        *cluster_ptr(&sh.cut_idx, r) = (uint32_t)(base + e);
                    }
                at += __popc(m);
            }
        cluster_sync_all();
        if (mass) {
            if (threadIdx.x == 0) sh.cut_mass = above + nth * own;
        } else {
            // the mass of the kept
            const float cx = sh.cut_x;
            const uint32_t ci = sh.cut_idx;
            u64 kept = 0;
            for (int e = first + threadIdx.x; e < last; e += kSmThreads) {
                const float v = value(e);
                if ((v > cx || (v == cx && (uint32_t)(base + e) <= ci)) && in(v, (uint32_t)(base + e)))
                    kept += row.mass(v);
            }
            kept = warp_sum64(kept);
            if (lane == 0) sh.w_mass[warp] = kept;
            __syncthreads();
            kept = 0;
            for (int w = 0; w < kSmWarps; ++w) kept += sh.w_mass[w];
            kept = cluster_total(kept, before);
            if (threadIdx.x == 0) sh.cut_mass = kept;
        }
        restore();
    }
    // The steps' sums, over a search by digits on the same arrays: a few a
    // thread.
    u64 kept_m[kSmBins / kSmThreads];
    uint32_t kept_c[kSmBins / kSmThreads];
    __device__ void save() {
#pragma unroll
        for (int i = 0; i < kSmBins / kSmThreads; ++i) {
            kept_m[i] = sh.all_mass[threadIdx.x + i * kSmThreads];
            kept_c[i] = sh.all_cnt[threadIdx.x + i * kSmThreads];
        }
        cluster_sync_all();
    }
    __device__ void restore() {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kSmBins / kSmThreads; ++i) {
            sh.all_mass[threadIdx.x + i * kSmThreads] = kept_m[i];
            sh.all_cnt[threadIdx.x + i * kSmThreads] = kept_c[i];
        }
        __syncthreads();
    }
};

// PLAN: not a token, but what each row's filters keep (SmPlan), of the target
// rows and behind them the draft rows of a batch of sequences.
template <bool BF16, bool PLAN>
__global__ void __launch_bounds__(kSmThreads, 1) sample_kernel(SampleParams p, int cl, bool in_turn) {
    using S = Sampler<BF16>;
    using Raw = typename S::Raw;
    constexpr int PER = S::PER;
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ __align__(16) unsigned char sm_raw[];
    SmShared &sh = *reinterpret_cast<SmShared *>(sm_raw);
    Raw *slice = reinterpret_cast<Raw *>(sm_raw + ((sizeof(SmShared) + 15) / 16) * 16);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int rank = cl > 1 ? (int)cluster_rank() : 0;
    int64_t r = blockIdx.x / cl;
    if (tid == 0) pdl_launch_dependents();
    pdl_wait_primary();

    if (in_turn) {
        // the row of this place in the order of the classes: top-p without a
        // short top-k, other draws, greedy rows
        int cls = 3;
        if (tid < p.rows) {
            const int f = PLAN && tid >= p.targets ? tid - (int)p.targets : tid;
            const int k = p.top_k ? p.top_k[f] : 0;
            cls = p.temperature && !(p.temperature[f] > 0.f)        ? 2
                  : k > 0 && k <= kSmShort                          ? 1
                  : p.top_p && p.top_p[f] < 1.f                     ? 0
                                                                    : 1;
        }
        const u64 one = cls < 3 ? 1ull << (16 * cls) : 0;  // three counts in a word
        const u64 incl = warp_scan(one);
        if (lane == 31) sh.t_mass[warp] = incl;
        __syncthreads();
        const u64 wm = warp_scan(sh.t_mass[lane]), all = __shfl_sync(FULL, wm, 31);
        u64 place = incl - one + __shfl_sync(FULL, wm, max(warp - 1, 0)) * (warp > 0);
        place = (place >> (16 * cls)) & 0xffffu;
        if (cls > 0) place += all & 0xffffu;
        if (cls > 1) place += (all >> 16) & 0xffffu;
        if (cls < 3 && (int64_t)place == r) sh.list_n = tid;
        __syncthreads();
        r = sh.list_n;
        __syncthreads();
    }

    const bool draft = PLAN && r >= p.targets;
    const int64_t fr = draft ? r - p.targets : r;  // the row of the filters
    if constexpr (PLAN) {
        // A row of no sequence, and a draft's without a token behind it: its plan
        // is not read, and of the draft's nor is the row, which need not be there
        // (every warp finds out for itself; the whole cluster leaves)
        const SmSeq q = sm_sequence(p.q_start, p.batch, fr);
        if (q.seq < 0 || (draft && fr + 1 >= min((int64_t)q.next, p.targets))) return;
    }

    // (waited for before the first word goes to another CTA: all of the
    // cluster run by then)
    if (cl > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");

    // ---- this CTA's slice; chunks start on 16 bytes of the input, so the
    // slice starts at element `mis` of its first chunk
    const int64_t per_cta = (p.V + cl - 1) / cl;
    const int64_t lo = min(p.V, rank * per_cta), hi = min(p.V, lo + per_cta);
    const Raw *src = draft ? static_cast<const Raw *>(p.draft) + fr * p.draft_stride + lo
                           : static_cast<const Raw *>(p.logits) + r * p.stride + lo;
    const int len = (int)(hi - lo);
    const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(Raw));
    const int chunks = (len + mis + PER - 1) / PER;
    float top = -INFINITY, low = INFINITY;  // low: the smallest finite logit
    auto see = [&](Raw v) {
        const float x = BF16 ? __uint_as_float((uint32_t)v << 16) : __uint_as_float((uint32_t)v);
        top = fmaxf(top, x);
        low = fminf(low, x == -INFINITY ? INFINITY : x);
    };
    auto whole = [&](int j) { return j * PER >= mis && (j + 1) * PER - mis <= len; };
    for (int j0 = tid; j0 < chunks; j0 += 4 * kSmThreads) {
        uint4 c[4];  // four loads in flight
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (const int j = j0 + k * kSmThreads; whole(j))
                c[k] = *reinterpret_cast<const uint4 *>(src + (j * PER - mis));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * kSmThreads;
            if (whole(j)) {
                const uint32_t w[4] = {c[k].x, c[k].y, c[k].z, c[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (BF16) {
                        see((Raw)(w[i] & 0xffffu));
                        see((Raw)(w[i] >> 16));
                    } else {
                        see(w[i]);
                    }
                }
                *reinterpret_cast<uint4 *>(slice + j * PER) = c[k];
            } else if (j < chunks) {  // an end of the slice; -inf outside it
                for (int e = j * PER; e < (j + 1) * PER; ++e) {
                    const Raw v = e >= mis && e < mis + len ? src[e - mis]
                                                            : (Raw)(BF16 ? 0xff80u : 0xff800000u);
                    see(v);
                    slice[e] = v;
                }
            }
        }
    }
    const float mine_top = top;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        low = fminf(low, __shfl_xor_sync(FULL, low, o));
    }
    if (lane == 0) {
        sh.w_top[warp] = top;
        sh.w_low[warp] = low;
    }
    __syncthreads();
    top = sh.w_top[lane];
    low = sh.w_low[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        top = fmaxf(top, __shfl_xor_sync(FULL, top, o));
        low = fminf(low, __shfl_xor_sync(FULL, low, o));
    }
    if (cl > 1) {
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        if (tid < cl) {
            *cluster_ptr(&sh.x_top[rank], tid) = top;
            *cluster_ptr(&sh.x_low[rank], tid) = low;
        }
        cluster_sync_all();
        for (int c = 0; c < cl; ++c) {
            top = fmaxf(top, sh.x_top[c]);
            low = fminf(low, sh.x_low[c]);
        }
    }
    if (top == -INFINITY) {  // nothing to draw (the whole cluster leaves)
        if (PLAN) {
            if (rank == 0 && tid == 0) p.plan[r] = SmPlan{top, 0.f, INFINITY, 0, 0, 0};
        } else if (rank == 0 && tid == 0) {
            p.token[r] = -1;
            if (p.prob) p.prob[r] = 0.f;
        }
        return;
    }

    const float T = p.temperature ? p.temperature[fr] : 1.f;
    const int kq = p.top_k ? p.top_k[fr] : 0;
    const float tp = p.top_p ? p.top_p[fr] : 1.f;
    const float mp = p.min_p ? p.min_p[fr] : 0.f;
    const float u = PLAN ? 0.f : p.u[r];
    const bool greedy = !(T > 0.f);
    S s{sh, slice, mis, mis + len, lo - mis, cl, rank, {top, 0.f}, 0.f};
    s.row.per = __fmul_rn(__fdiv_rn(1.f, T), 1.4426950408889634f);

    if (greedy) {
        // the first of the largest
        if (tid == 0) sh.list_n = 0xffffffffu;
        s.sync_all();
        for (int j = tid; j < chunks; j += kSmThreads) {
            float x[PER];
            s.load(j, x);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                if (x[i] == top)
                    atomicMin(cluster_ptr(&sh.list_n, 0), (uint32_t)(s.base + j * PER + i));
            }
        }
        s.sync_all();
        if (PLAN) {
            if (rank == 0 && tid == 0) p.plan[r] = SmPlan{top, 0.f, top, sh.list_n, 0, 1ull << 40};
        } else if (rank == 0 && tid == 0) {
            p.token[r] = (int32_t)sh.list_n;
            if (p.prob) p.prob[r] = 1.f;
        }
        return;
    }
    const u64 least = mp > 0.f ? __float2ull_rz(fminf(mp, 1.f) * 1099511627776.f) : 0;

    // ---- the cut: kept are logits above cut_x, and its equals up to cut_idx
    bool cut = false;
    float cut_x = 0.f;
    uint32_t cut_idx = 0;
    const bool by_k = kq > 0 && kq < p.V, by_p = tp < 1.f;
    if (by_k || by_p) {
        const float range = fminf(41.f, low < top ? -s.row.expo(low) : 0.f);
        s.steps = range > 0.f ? fminf((float)kSmBins / range, 1e30f) : 0.f;
    }
    if (by_k && kq <= kSmShort) {
        s.clear(kSmBins);
        if (tid == 0) sh.f_bin = kSmBins - 1;
        if (mine_top > -INFINITY) s.add(s.bin_of(mine_top), true, 0);
        s.join(kSmBins, false);
        s.locate(kSmBins, false, false, (u64)kq, -1.f);
        const int bin = sh.f_bin;
        const uint32_t n = s.gather(s.x_low(bin), INFINITY, [&](float x, uint32_t) {
            return x > -INFINITY && s.bin_of(x) <= bin;
        });
        if (n <= kSmList) {
            if (rank == 0) {
                s.sort((int)n);
                if (PLAN)
                    s.plan(min((int)n, kq), 0, tp, least, p.plan + r);
                else
                    s.draw(min((int)n, kq), 0, tp, least, u, p.token + r, p.prob ? p.prob + r : nullptr);
            }
            return;
        }
    }
    u64 goal_p = 0, prune = 0;
    float x_prune = -INFINITY;
    if (!by_k && (by_p || least > 0)) {
        MassSum sum;
        int n = 0;
        for (int j = tid; j < chunks; j += kSmThreads, n += PER) {
            float x[PER];
            s.load(j, x);
#pragma unroll
            for (int i = 0; i < PER; ++i) sum.add(SmRow::part_of(s.row.expo(x[i])));
        }
        const u64 total = s.sum_all(sum.total(n));
        if (by_p) {
            goal_p = S::share_of(total, tp);
            prune = (total - goal_p) / (u64)p.V;
        }
        const u64 thr = max(least, prune + 1);
        // (its logit, 0.01 of y below: the rounding of log2, of the exponent and
        // of the way back)
        const float x_thr = s.x_below(__log2f((float)thr) - 40.01f);
        x_prune = s.x_below(__log2f((float)(prune + 1)) - 40.01f);
        n = 0;
        for (int j = tid; j < chunks; j += kSmThreads) {
            float x[PER];
            s.load(j, x);
#pragma unroll
            for (int i = 0; i < PER; ++i) n += x[i] >= x_thr;
        }
        if (s.sum_all((u64)n) <= kSmList) {
            n = (int)s.gather(x_thr, INFINITY, [&](float x, uint32_t) { return s.row.mass(x) >= thr; });
            if (rank == 0) {
                s.sort(n);
                if (PLAN)
                    s.plan(n, goal_p, tp, least, p.plan + r);
                else
                    s.draw(n, goal_p, tp, least, u, p.token + r, p.prob ? p.prob + r : nullptr);
            }
            return;
        }
    }
    if (by_k || by_p) {
        s.clear(kSmBins);
        for (int j = tid; j < chunks; j += kSmThreads) {
            float x[PER];
            s.load(j, x);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = j * PER + i;
                if (e < mis || e >= mis + len) continue;
                // (counts only for top-k, masses only for top-p and above its
                // floor)
                if (!by_k && x[i] < x_prune) continue;
                const float y = s.row.expo(x[i]);
                const u64 w = by_p ? SmRow::mass_of(y) : 0;
                if (!by_k && w <= prune) continue;
                // (-inf, and NaN, in the last step)
                const int bin = x[i] == -INFINITY ? kSmBins - 1
                                                  : (int)fminf(-y * s.steps, (float)(kSmBins - 1));
                s.add(bin, by_k, w);
            }
        }
        s.join(kSmBins, by_p);
        if (by_k) {
            s.locate(kSmBins, false, false, (u64)kq, -1.f);
            const int bin = sh.f_bin;
            const u64 want = (u64)kq - sh.f_above_cnt;
            __syncthreads();
            s.refine(bin, false, want, false, 0.f, 0);
            cut = true;
            cut_x = sh.cut_x;
            cut_idx = sh.cut_idx;
            if (by_p) {
                // what top-p goes by: the steps above, and of this one the kept
                for (int i = tid; i < kSmBins; i += kSmThreads)
                    if (i >= bin) sh.all_mass[i] = i == bin ? sh.cut_mass : 0;
                __syncthreads();
            }
        }
        if (by_p) {
            const u64 goal = s.locate(kSmBins, false, true, goal_p, by_k ? fmaxf(tp, 0.f) : -1.f);
            const int bin = sh.f_bin;
            const u64 above = sh.f_above_mass;
            __syncthreads();
            s.refine(bin, true, goal - above, cut, cut_x, cut_idx);
            cut = true;
            cut_x = sh.cut_x;
            cut_idx = sh.cut_idx;
            if (PLAN && least == 0) {  // all below the cut is counted
                if (rank == 0 && tid == 0)
                    p.plan[r] = SmPlan{top, s.row.per, cut_x, cut_idx, 0, above + sh.cut_mass};
                return;
            }
        }
    }
    // ---- the kept masses: a warp takes a run of whole 32-token steps, in
    // index order
    const int run = (((len + mis) + kSmWarps - 1) / kSmWarps + 31) & ~31;
    const int a = warp * run, b = min(mis + len, a + run);
    auto kept_of = [&](int e, float x) -> u64 {
        if (cut && !(x > cut_x || (x == cut_x && (uint32_t)(s.base + e) <= cut_idx))) return 0;
        const u64 w = s.row.mass(x);
        return w >= least ? w : 0;
    };
    auto kept = [&](int e) { return e >= mis && e < b ? kept_of(e, s.value(e)) : 0; };
    // (floor(t 2^40) >= least where t >= least 2^-40, which a float holds:
    // least comes from one)
    const float least_t = (float)least * 0x1p-40f, floor_x = cut ? cut_x : -INFINITY;
    MassSum sum;
    int n = 0;
    u64 mine = 0;
    for (int j = a / PER + lane; j * PER < b; j += 32, n += PER) {
        float x[PER];
        s.load(j, x);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float t = SmRow::part_of(s.row.expo(x[i]));
            sum.add(x[i] > floor_x && t >= least_t ? t : 0.f);
            if (cut && x[i] == cut_x) mine += kept_of(j * PER + i, x[i]);
        }
    }
    mine += sum.total(n);
    mine = warp_sum64(mine);
    __syncthreads();
    if (lane == 0) sh.w_mass[warp] = mine;
    __syncthreads();
    const u64 wm = warp_scan(sh.w_mass[lane]), cta = __shfl_sync(FULL, wm, 31);
    const u64 warp_before = __shfl_sync(FULL, wm, max(warp - 1, 0)) * (warp > 0);
    u64 cta_before;
    cluster_sync_all();  // x_mass may still be read
    const u64 all = s.cluster_total(cta, cta_before);
    if constexpr (PLAN) {
        if (rank == 0 && tid == 0)
            p.plan[r] = SmPlan{top, s.row.per, floor_x, cut ? cut_idx : 0xffffffffu, least, all};
        return;
    }
    // the first token whose running mass passes u * all 
    const u64 goal = drawn_at(all, u);
    const u64 start = cta_before + warp_before;
    if (goal >= start && goal < start + mine) {
        u64 at = start;
        for (int e0 = a; e0 < b; e0 += 32) {
            const u64 w = kept(e0 + lane);
            const u64 sum = warp_sum64(w);
            if (goal >= at + sum) {
                at += sum;
                continue;
            }
            u64 incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(FULL, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned past = __ballot_sync(FULL, at + incl > goal);
            if (lane == __ffs(past) - 1) {
                p.token[r] = (int32_t)(s.base + e0 + lane);
                if (p.prob) p.prob[r] = share(w, all);
            }
            break;
        }
    }
}


cudaError_t allow_wide_clusters(const void *kernel) {
    static std::mutex mu;
    static std::set<std::pair<int, const void *>> done;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lk(mu);
    if (done.count({dev, kernel})) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.insert({dev, kernel});
    return e;
}

template <bool BF16, bool PLAN>
static cudaError_t launch_sample_t(const SampleParams &p, cudaStream_t st) {
    constexpr int esz = BF16 ? 2 : 4;
    const void *kfn = reinterpret_cast<const void *>(sample_kernel<BF16, PLAN>);
    constexpr size_t head = ((sizeof(SmShared) + 15) / 16) * 16;
    int cl = 1;
    while (cl < kSmMaxCluster && (p.V + cl - 1) / cl * esz > kSmSliceBytes) cl *= 2;
    while (cl < kSmMaxCluster && p.rows * cl * 2 <= num_sms() && p.V / (2 * cl) >= 2048) cl *= 2;
    const size_t smem = head + ((size_t)((p.V + cl - 1) / cl) * esz + 48) / 16 * 16;
    cudaError_t e = allow_smem(kfn, (int)(head + kSmSliceBytes + 48));
    if (e == cudaSuccess) e = allow_wide_clusters(kfn);
    if (e != cudaSuccess) return e;
    // Rows differ in work by ten: where they take more than one wave, the
    // heavy ones go first (256 x 151669 bf16, filters of all kinds: 130 us in
    // the rows' order, 101 so); for a row a thread at most.
    const bool in_turn = p.rows * cl > num_sms() && p.rows <= kSmThreads;
    return launch_pdl_cluster(kfn, (unsigned)(p.rows * cl), (unsigned)cl, kSmThreads, smem, st, p, cl, in_turn);
}

cudaError_t launch_sample(const SampleParams &p, bool bf16, cudaStream_t st) {
    return bf16 ? launch_sample_t<true, false>(p, st) : launch_sample_t<false, false>(p, st);
}

cudaError_t launch_sample_plan(const SampleParams &p, bool bf16, cudaStream_t st) {
    return bf16 ? launch_sample_t<true, true>(p, st) : launch_sample_t<false, true>(p, st);
}

}  // namespace gwa
