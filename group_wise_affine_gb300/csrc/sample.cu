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
// ascending): all logits above a cut, and the first n that equal it.  The
// cut is found digit by digit on order-preserving integer keys of the
// logits (16 bits for bf16, 32 for fp32) with a histogram per digit, of
// counts for top-k and of masses for top-p.
//
// A row belongs to a cluster of CTAs.  Each keeps its slice of the row in
// shared memory as keys, read from HBM once; histograms and sums are joined
// through distributed shared memory, each CTA adding up a share of the bins
// and handing it to all.  One launch per call.  The cluster is the smallest
// that holds the row, made larger while the rows leave SMs idle.
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"

namespace gwa {

constexpr int kSmThreads = 512;
constexpr int kSmWarps = kSmThreads / 32;
constexpr int kSmBins = 2048;
constexpr int kSmMaxCluster = 16;
constexpr int64_t kSmSliceBytes = 160 * 1024;

using u64 = unsigned long long;

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

// Shared memory besides the keys.  `mine` is filled by this CTA, `all` by
// every CTA of the cluster.
struct SmShared {
    uint32_t cnt[kSmBins], lo[kSmBins], hi[kSmBins];  // this CTA's histogram
    uint32_t all_cnt[kSmBins];
    u64 all_mass[kSmBins];
    u64 x_mass[kSmMaxCluster];   // one value from every CTA
    uint32_t x_word[kSmMaxCluster];
    u64 w_mass[kSmWarps];        // one value from every warp
    uint32_t w_word[kSmWarps];
    u64 t_mass[kSmThreads / 32 + 1];
    uint32_t t_cnt[kSmThreads / 32 + 1];
    // the digit a search settled on
    uint32_t f_digit, f_count;
    u64 f_above_mass;
    uint32_t f_above_cnt;
};

template <typename T>
__device__ __forceinline__ T *cluster_ptr(T *local, uint32_t rank) {
    u64 a;
    asm volatile("mapa.u64 %0, %1, %2;" : "=l"(a) : "l"(reinterpret_cast<u64>(local)), "r"(rank));
    return reinterpret_cast<T *>(a);
}

// A row's weights.
struct SmRow {
    float top, per;
    __device__ __forceinline__ u64 mass(float x) const {
        if (x == -INFINITY) return 0;
        const float y = x == top ? 0.f : __fmul_rn(__fsub_rn(x, top), per);
        const float e = exp2f(y);
        return e <= 1.f ? __float2ull_rz(e * 1099511627776.f) : 0;
    }
};

__device__ __forceinline__ u64 warp_sum64(u64 v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <bool BF16>
struct Sampler {
    using K = SmKey<BF16>;
    using Key = typename K::Key;
    SmShared &sh;
    Key *keys;
    int n;          // keys of this CTA, a multiple of 8, padding (0) included
    int cl, rank;
    SmRow row;

    // The digit search: the cut where the summed counts (MASS false) or
    // masses reach `goal` from the top, over keys >= floor (keys equal to it
    // taken floor_n times by rank 0).  Returns the cut's key; `above` is what
    // lies above it, `count` the keys equal to it.
    template <bool MASS>
    __device__ Key search(u64 goal, bool whole_goal, float frac, Key floor_key, uint32_t floor_n,
                          u64 &above, uint32_t &count) {
        uint32_t prefix = 0;
        int done = 0;  // bits settled
        above = 0;
        for (int pass = 0; pass < K::PASSES; ++pass) {
            const int sft = K::shift(pass), wid = K::width(pass), bins = 1 << wid;
            for (int i = threadIdx.x; i < bins; i += kSmThreads) {
                sh.cnt[i] = 0;
                if (MASS) sh.lo[i] = sh.hi[i] = 0;
            }
            __syncthreads();
            auto add = [&](uint32_t bin, uint32_t c, u64 w) {
                atomicAdd(&sh.cnt[bin], c);
                if (MASS) {
                    const uint32_t wl = (uint32_t)w;
                    const uint32_t old = atomicAdd(&sh.lo[bin], wl);
                    const uint32_t up = (uint32_t)(w >> 32) + (old + wl < old ? 1u : 0u);
                    if (up) atomicAdd(&sh.hi[bin], up);
                }
            };
            for (int i = threadIdx.x; i < n; i += kSmThreads) {
                const uint32_t k = keys[i];
                if (k <= floor_key) continue;
                if (done && (k >> (K::BITS - done)) != prefix) continue;
                const u64 w = MASS ? row.mass(K::value((Key)k)) : 0;
                if (MASS && w == 0) continue;
                add((k >> sft) & (bins - 1), 1u, w);
            }
            if (rank == 0 && threadIdx.x == 0 && floor_n &&
                (!done || ((uint32_t)floor_key >> (K::BITS - done)) == prefix)) {
                const u64 w = MASS ? row.mass(K::value(floor_key)) * floor_n : 0;
                add(((uint32_t)floor_key >> sft) & (bins - 1), floor_n, w);
            }
            // join: each CTA adds a share of the bins and hands it to all
            cluster_sync_all();
            const int share = bins / cl;
            for (int j = threadIdx.x; j < share; j += kSmThreads) {
                const int bin = rank * share + j;
                uint32_t c = 0;
                u64 m = 0;
                for (int r = 0; r < cl; ++r) {
                    c += *cluster_ptr(&sh.cnt[bin], r);
                    if (MASS)
                        m += (u64)*cluster_ptr(&sh.lo[bin], r) +
                             ((u64)*cluster_ptr(&sh.hi[bin], r) << 32);
                }
                for (int r = 0; r < cl; ++r) {
                    *cluster_ptr(&sh.all_cnt[bin], r) = c;
                    if (MASS) *cluster_ptr(&sh.all_mass[bin], r) = m;
                }
            }
            cluster_sync_all();
            // from the top: thread i holds bins top - per*i ..
            const int per = bins > kSmThreads ? bins / kSmThreads : 1;
            u64 sum = 0;
            const int hi_bin = bins - 1 - threadIdx.x * per;
            for (int j = 0; j < per; ++j)
                if (hi_bin - j >= 0)
                    sum += MASS ? sh.all_mass[hi_bin - j] : (u64)sh.all_cnt[hi_bin - j];
            u64 incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
                if ((int)(threadIdx.x & 31) >= o) incl += v;
            }
            if ((threadIdx.x & 31) == 31) sh.t_mass[threadIdx.x / 32] = incl;
            __syncthreads();
            u64 before = incl - sum, total = 0;
            for (int w = 0; w < kSmWarps; ++w) {
                if (w < (int)(threadIdx.x / 32)) before += sh.t_mass[w];
                total += sh.t_mass[w];
            }
            if (pass == 0 && !whole_goal) {
                // a share of everything; at least the first token
                goal = (u64)((double)total * (double)frac);
                if (goal < 1) goal = 1;
            }
            const u64 left = goal - above;  // within this prefix, >= 1
            if (before < left && left <= before + sum) {
                u64 a = before;
                for (int j = 0; j < per; ++j) {
                    const u64 v = MASS ? sh.all_mass[hi_bin - j] : (u64)sh.all_cnt[hi_bin - j];
                    if (left <= a + v) {
                        sh.f_digit = hi_bin - j;
                        sh.f_above_mass = a;
                        sh.f_count = sh.all_cnt[hi_bin - j];
                        break;
                    }
                    a += v;
                }
            }
            __syncthreads();
            prefix = (prefix << wid) | sh.f_digit;
            above += sh.f_above_mass;
            count = sh.f_count;
            done += wid;
        }
        goal_ = goal;
        return (Key)prefix;
    }
    u64 goal_;

    // Sum over the cluster of one value from every CTA, and the sum of the
    // lower ranks'.
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
};

template <bool BF16>
__global__ void __launch_bounds__(kSmThreads, 1) sample_kernel(SampleParams p, int cl) {
    using K = SmKey<BF16>;
    using Key = typename K::Key;
    using Raw = typename K::Raw;
    constexpr int PER = 16 / sizeof(Raw);  // logits of a 16-byte chunk
    extern __shared__ __align__(16) unsigned char sm_raw[];
    SmShared &sh = *reinterpret_cast<SmShared *>(sm_raw);
    Key *keys = reinterpret_cast<Key *>(sm_raw + ((sizeof(SmShared) + 15) / 16) * 16);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int rank = cl > 1 ? (int)cluster_rank() : 0;
    const int64_t r = blockIdx.x / cl;
    if (tid == 0) pdl_launch_dependents();
    pdl_wait_primary();

    // ---- this CTA's slice as keys; chunks start on 16 bytes of the input
    const int64_t per_cta = (p.V + cl - 1) / cl;
    const int64_t lo = min(p.V, rank * per_cta), hi = min(p.V, lo + per_cta);
    const Raw *src = static_cast<const Raw *>(p.logits) + r * p.stride + lo;
    const int len = (int)(hi - lo);
    const int mis = (int)((reinterpret_cast<uintptr_t>(src) & 15) / sizeof(Raw));
    const int chunks = (len + mis + PER - 1) / PER;
    uint32_t top_key = 0;
    for (int j = tid; j < chunks; j += kSmThreads) {
        const int e0 = j * PER - mis;
        Raw v[PER];
        Key k[PER];
        if (e0 >= 0 && e0 + PER <= len) {
            *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(src + e0);
#pragma unroll
            for (int i = 0; i < PER; ++i) k[i] = K::make(v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                k[i] = e0 + i >= 0 && e0 + i < len ? K::make(src[e0 + i]) : (Key)0;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) top_key = max(top_key, (uint32_t)k[i]);
        *reinterpret_cast<uint4 *>(keys + j * PER) = *reinterpret_cast<uint4 *>(k);
    }
    const int n = chunks * PER;
    top_key = __reduce_max_sync(0xffffffffu, top_key);
    if (lane == 0) sh.w_word[warp] = top_key;
    __syncthreads();
    for (int w = 0; w < kSmWarps; ++w) top_key = max(top_key, sh.w_word[w]);
    // every CTA of the cluster runs: its shared memory may be written
    cluster_sync_all();
    if (tid < cl) *cluster_ptr(&sh.x_word[rank], tid) = top_key;
    cluster_sync_all();
    for (int c = 0; c < cl; ++c) top_key = max(top_key, sh.x_word[c]);

    const float T = p.temperature ? p.temperature[r] : 1.f;
    const int kq = p.top_k ? p.top_k[r] : 0;
    const float tp = p.top_p ? p.top_p[r] : 1.f;
    const float mp = p.min_p ? p.min_p[r] : 0.f;
    const float u = p.u[r];
    SmRow row;
    row.top = K::value((Key)top_key);
    row.per = __fmul_rn(__fdiv_rn(1.f, T), 1.4426950408889634f);
    const bool none = row.top == -INFINITY, greedy = !(T > 0.f);

    Sampler<BF16> s{sh, keys, n, cl, rank, row, 0};
    // the cut: keys above it are kept, and the first cut_n equal to it
    Key cut = (Key)0;
    uint32_t cut_n = 0;
    bool limited = false;
    u64 dummy = 0;
    if (none) {
        if (rank == 0 && tid == 0) {
            p.token[r] = -1;
            if (p.prob) p.prob[r] = 0.f;
        }
        return;  // the whole cluster returns; nothing remote is in flight
    }
    if (greedy) {
        cut = (Key)top_key;
        cut_n = 1;
        limited = true;
    } else {
        if (kq > 0 && kq < p.V) {
            u64 above;
            uint32_t count;
            cut = s.template search<false>((u64)kq, true, 0.f, (Key)0, 0, above, count);
            cut_n = (uint32_t)((u64)kq - above);
            limited = cut_n < count;
        }
        if (tp < 1.f) {
            u64 above;
            uint32_t count;
            const Key c = s.template search<true>(0, false, fmaxf(tp, 0.f), cut, cut_n, above, count);
            const u64 w = row.mass(K::value(c));
            const uint32_t cn = (uint32_t)((s.goal_ - above + w - 1) / w);
            limited = c == cut && cut_n ? limited || cn < cut_n : cn < count;
            cut = c;
            cut_n = cn;
        }
    }
    const u64 least = !greedy && mp > 0.f
                          ? __float2ull_rz(fminf(mp, 1.f) * 1099511627776.f) : 0;
    const bool has_cut = cut_n > 0;
    // a warp takes a run of whole 32-key steps, in index order
    const int steps = (n + 31) / 32;
    const int s0 = (int)((int64_t)steps * warp / kSmWarps);
    const int s1 = (int)((int64_t)steps * (warp + 1) / kSmWarps);
    u64 eq_before = 0;  // keys equal to the cut before this warp's run
    if (limited) {
        uint32_t c = 0;
        for (int st = s0; st < s1; ++st) {
            const int i = st * 32 + lane;
            c += __popc(__ballot_sync(0xffffffffu, i < n && keys[i] == cut));
        }
        if (lane == 0) sh.w_word[warp] = c;
        __syncthreads();
        u64 mine = 0, before;
        for (int w = 0; w < kSmWarps; ++w) {
            if (w < warp) eq_before += sh.w_word[w];
            mine += sh.w_word[w];
        }
        cluster_sync_all();  // x_mass may still be read
        s.cluster_total(mine, before);
        eq_before += before;
        __syncthreads();
    }
    auto kept = [&](int i, u64 &eq) -> u64 {  // i < n or not: every lane calls
        const Key k = i < n ? keys[i] : (Key)0;
        bool in = !has_cut || k > cut;
        if (has_cut) {
            const unsigned m = __ballot_sync(0xffffffffu, k == cut);
            if (k == cut)
                in = !limited || eq + __popc(m & ((1u << lane) - 1u)) < cut_n;
            eq += __popc(m);
        }
        if (!in || k == 0) return 0;
        const u64 w = greedy ? 1 : row.mass(K::value(k));
        return w >= least ? w : 0;
    };
    u64 mine = 0, eq = eq_before;
    for (int st = s0; st < s1; ++st) mine += kept(st * 32 + lane, eq);
    mine = warp_sum64(mine);
    if (lane == 0) sh.w_mass[warp] = mine;
    __syncthreads();
    u64 cta = 0, warp_before = 0, cta_before;
    for (int w = 0; w < kSmWarps; ++w) {
        if (w < warp) warp_before += sh.w_mass[w];
        cta += sh.w_mass[w];
    }
    cluster_sync_all();  // x_mass may still be read
    const u64 all = s.cluster_total(cta, cta_before);
    // the first token whose running mass passes u * all
    u64 goal = (u64)((double)fmaxf(u, 0.f) * (double)all);
    if (goal > all - 1) goal = all - 1;
    const u64 start = cta_before + warp_before;
    if (goal >= start && goal < start + mine) {
        u64 run = start;
        eq = eq_before;
        for (int st = s0; st < s1; ++st) {
            const int i = st * 32 + lane;
            const u64 w = kept(i, eq);
            u64 incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const u64 v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, run + incl > goal);
            if (past) {
                if (lane == __ffs(past) - 1) {
                    p.token[r] = (int32_t)(lo + i - mis);
                    if (p.prob) p.prob[r] = (float)((double)w / (double)all);
                }
                break;
            }
            run += __shfl_sync(0xffffffffu, incl, 31);
        }
    }
    (void)dummy;
}

template <bool BF16>
static cudaError_t launch_sample_t(const SampleParams &p, cudaStream_t st) {
    constexpr int esz = BF16 ? 2 : 4;
    const void *kfn = reinterpret_cast<const void *>(sample_kernel<BF16>);
    constexpr size_t head = ((sizeof(SmShared) + 15) / 16) * 16;
    int cl = 1;
    while (cl < kSmMaxCluster && (p.V + cl - 1) / cl * esz > kSmSliceBytes) cl *= 2;
    while (cl < kSmMaxCluster && p.rows * cl * 2 <= num_sms() && p.V / (2 * cl) >= 2048) cl *= 2;
    const size_t smem = head + ((size_t)((p.V + cl - 1) / cl) * esz + 48) / 16 * 16;
    cudaError_t e = allow_smem(kfn, (int)(head + kSmSliceBytes + 48));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(kfn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kfn, (unsigned)(p.rows * cl), (unsigned)cl, kSmThreads, smem, st, p, cl);
}

cudaError_t launch_sample(const SampleParams &p, bool bf16, cudaStream_t st) {
    return bf16 ? launch_sample_t<true>(p, st) : launch_sample_t<false>(p, st);
}

}  // namespace gwa
