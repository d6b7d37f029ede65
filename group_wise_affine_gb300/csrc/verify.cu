// Drafted tokens against the target model's probabilities: which of them
// stand, and the token behind them, by given random numbers (the step that
// takes sampling's place where a draft model, or a look-up, proposes tokens
// ahead; the pages' server has such a mode and prints no rule, so the rule is
// this library's reading, stated in gwa.h).
//
// With p and q the target's and the draft's shares of what the row's filters
// keep, draft d stands if u q(d) < p(d); behind the last that stands a token is
// drawn from max(p - q, 0) in the row of the first that falls, from p where none
// fell.  So the tokens are distributed as the target's own would be.
//
// Drafts are settled in whole numbers, as sampling's tokens are (sample.cuh):
// p(d) = P / SP with 41-bit masses and 60-bit sums, compared as products of 128
// bits.  A token's mass in max(p - q, 0) is the whole number of 2^-40 in
//   t_p - (SP / SQ) t_q,   t = exp2f(y) the parts that the masses are floors of,
// formed in fp32 with the quotient as two of them, so that each token's mass
// has a rounding of its own and none is common to the whole row.  (Exact
// products of 64-bit masses took 120 instructions a token, 78 us for 64 rows
// of 151669 with 4 drafts each; so it takes 25.)  Sums are integer sums: the
// result depends on no split and no order.
//
// Two kernels.  The first is sampling's own (sample_kernel, PLAN), over the
// target rows and the draft rows at once: it leaves what each row's filters
// keep, as a cut and a sum.  This one then has one row a sequence to go over
// (two where a draft fell): a cluster of CTAs a sequence, each a slice of the
// row in pieces of 256 tokens, a warp to a piece.  The pieces' sums are
// scanned, and one warp looks for the token in the piece that holds the drawn
// mass.
//
// Measured, both kernels: 54 sequences with up to 4 drafts, 151669 bf16 tokens,
// filters of all kinds, 134 us: sampling's 112 alone (318 rows, 96.6 MB read, 14.4
// us of HBM bandwidth; see there what a row takes), then this one: issue 44% at
// four CTAs an SM, 25 instructions a token of two rows, scans and cluster barriers.
// 16 sequences with 7 looked-up drafts, 50021 tokens, top-p, 47 us; one
// sequence with 4 drafts, 131072 fp32 tokens, 26.8 us, two launches of a dozen
// barriers each.
#include <algorithm>
#include <type_traits>

#include "sample.cuh"

namespace gwa {

constexpr int kVfThreads = 256, kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 16;
constexpr int kVfPiece = 256;                           // tokens
constexpr int kVfPieces = 524288 / kVfPiece;            // of a CTA, at most
constexpr int kVfScan = kVfPieces / kVfThreads;         // of a thread

template <bool BF16>
struct VfRow {
    using Raw = typename std::conditional<BF16, uint16_t, uint32_t>::type;
    const Raw *x;
    __device__ __forceinline__ float at(int64_t i) const {
        return __uint_as_float(BF16 ? (uint32_t)x[i] << 16 : (uint32_t)x[i]);
    }
};

// What the row's token is drawn from: the kept of p (kind 0), without token
// `drop` (1), or max(p - q, 0) (2).
struct VfMass {
    SmPlan p, q;
    float least_p, least_q;  // times 2^-40
    float hi, lo;            // SP / SQ = hi + lo
    int kind, drop;
    __device__ __forceinline__ void prepare() {
        least_p = (float)p.least * 0x1p-40f;
        least_q = (float)q.least * 0x1p-40f;
        // hi the rounded quotient m 2^e (of sums from 2^40 to 2^59, so e < 0),
        // lo from its exact remainder, SP - m 2^e SQ
        hi = share(p.total, q.total);
        const int e = f32_exp_field(hi) - 150;
        const uint32_t m = (__float_as_uint(hi) & 0x7fffffu) | 0x800000u;
        const __int128 left = ((__int128)p.total << -e) - (__int128)q.total * m;
        lo = __fdiv_rn(__ll2float_rn((long long)left), __ull2float_rn(q.total)) *
             __uint_as_float((uint32_t)(127 + e) << 23);
    }
    template <int KIND>
    __device__ __forceinline__ float of(float xp, float xq, int token) const {
        const float a = p.part(xp, (uint32_t)token, least_p);
        if (KIND == 0) return a;
        if (KIND == 1) return token == drop ? 0.f : a;
        const float b = q.part(xq, (uint32_t)token, least_q);
        return fmaxf(a - fmaf(b, hi, b * lo), 0.f);
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kVfThreads, 4) verify_kernel(VerifyParams p, int cl) {
    constexpr unsigned FULL = 0xffffffffu;
    using Row = VfRow<BF16>;
    using Raw = typename Row::Raw;
    __shared__ u64 s_piece[kVfPieces], s_warp[kVfWarps], s_cta[kVfMaxCluster], s_left;
    __shared__ int s_fell, s_at;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int rank = cl > 1 ? (int)cluster_rank() : 0, b = blockIdx.x / cl;
    if (tid == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int rows = (int)p.rows;
    const int first = min(max(p.q_start[b], 0), rows), next = min(max(p.q_start[b + 1], first), rows);
    const int n = next - first;
    if (rank == 0) {  // rows of no sequence
        for (int i = tid; i < (b == 0 ? first : 0); i += kVfThreads) {
            p.token[i] = -1;
            if (p.prob) p.prob[i] = 0.f;
        }
        for (int i = next + tid; i < (b == p.batch - 1 ? rows : 0); i += kVfThreads) {
            p.token[i] = -1;
            if (p.prob) p.prob[i] = 0.f;
        }
        if (n == 0 && tid == 0) p.accepted[b] = 0;
    }
    if (n == 0) return;  // (the whole cluster)

    // ---- the drafts, 32 at a time
    auto row_of = [&](int i) { return Row{static_cast<const Raw *>(p.logits) + (int64_t)i * p.stride}; };
    auto draft_of = [&](int i) { return Row{static_cast<const Raw *>(p.draft) + (int64_t)i * p.draft_stride}; };
    if (warp == 0) {
        int fell = n - 1;
        for (int j0 = 0; j0 < n - 1; j0 += 32) {
            const int i = first + j0 + lane;
            bool stands = true;
            if (j0 + lane < n - 1) {
                const SmPlan t = p.plan[i];
                const int d = p.ids[i + 1];
                const bool in = d >= 0 && d < p.V;
                const u64 P = in ? t.kept(row_of(i).at(d), (uint32_t)d) : 0;
                u64 Q = 1, SQ = 1;
                if (p.draft) {
                    const SmPlan q = p.plan[rows + i];
                    Q = in ? q.kept(draft_of(i).at(d), (uint32_t)d) : 0;
                    SQ = max(q.total, 1ull);
                }
                const float u = p.u[i];
                const u64 m = u >= 1.f ? 0xffffffull : (u64)(fmaxf(u, 0.f) * 0x1p24f);
                const unsigned __int128 lhs = (unsigned __int128)(m * Q) * t.total;
                const unsigned __int128 rhs = ((unsigned __int128)P * SQ) << 24;
                stands = lhs < rhs;
                if (p.prob && rank == 0) {
                    const float a = P ? share(P, t.total) : 0.f;
                    p.prob[i] = Q ? fminf(1.f, __fdiv_rn(a, share(Q, SQ))) : P ? 1.f : 0.f;
                }
            }
            const unsigned down = __ballot_sync(FULL, !stands);
            if (down && fell == n - 1) fell = j0 + __ffs(down) - 1;
        }
        if (lane == 0) s_fell = fell;
    }
    __syncthreads();
    const int fell = s_fell, at = first + fell;
    if (rank == 0) {
        for (int j = tid; j < n; j += kVfThreads)
            if (j != fell) p.token[first + j] = j < fell ? p.ids[first + j + 1] : -1;
        if (tid == 0) {
            p.accepted[b] = fell;
            if (p.prob) p.prob[next - 1] = 0.f;
        }
    }

    // ---- the token behind them
    VfMass w;
    w.p = p.plan[at];
    if (w.p.total == 0) {  // nothing to draw
        if (rank == 0 && tid == 0) p.token[at] = -1;
        return;
    }
    w.kind = 0;
    w.q = w.p;
    w.drop = -1;
    if (fell < n - 1) {
        if (!p.draft) {
            w.kind = 1;
            w.drop = p.ids[at + 1];
        } else {
            w.q = p.plan[rows + at];
            if (w.q.total) w.kind = 2;
        }
    }
    w.prepare();
    const Row rp = row_of(at), rq = w.kind == 2 ? draft_of(at) : rp;
    const int V = (int)p.V, per_cta = (V + cl - 1) / cl;
    const int lo = min(V, rank * per_cta), hi = min(V, lo + per_cta);
    const int pieces = (hi - lo + kVfPiece - 1) / kVfPiece;
    constexpr int PER = kVfPiece / 32;  // tokens of a lane and piece
    auto fetch = [&](float (&x)[PER], const Row &row, int i0) {
        const Row from{row.x + i0};
#pragma unroll
        for (int j = 0; j < PER; ++j) x[j] = i0 + 32 * j < hi ? from.at(32 * j) : -INFINITY;
    };
    auto each_kind = [&](auto body) {
        if (w.kind == 2)
            body(std::integral_constant<int, 2>{});
        else if (w.kind == 1)
            body(std::integral_constant<int, 1>{});
        else
            body(std::integral_constant<int, 0>{});
    };
    const float u = p.u_draw[b];
    while (true) {
        each_kind([&](auto kind_t) {
            constexpr int kind = decltype(kind_t)::value;
            for (int c = warp; c < pieces; c += kVfWarps) {
                const int i0 = lo + c * kVfPiece + lane;
                float xp[PER], xq[PER] = {};
                fetch(xp, rp, i0);
                if (kind == 2) fetch(xq, rq, i0);
                MassSum sum;
#pragma unroll
                for (int j = 0; j < PER; ++j) sum.add(w.template of<kind>(xp[j], xq[j], i0 + 32 * j));
                // (the constants that the words carry come off once a lane,
                // before the lanes' sums, which then have room)
                const u64 mine = sum.total(PER);
                const uint32_t low = __reduce_add_sync(FULL, (uint32_t)mine & 0xfffffu);
                const uint32_t high = __reduce_add_sync(FULL, (uint32_t)(mine >> 20));
                if (lane == 0) s_piece[c] = ((u64)high << 20) + low;
            }
        });
        __syncthreads();
        // ---- the pieces' sums in order, those of the CTA and of the cluster
        u64 own[kVfScan], mine = 0;
#pragma unroll
        for (int j = 0; j < kVfScan; ++j) {
            const int c = tid * kVfScan + j;
            own[j] = c < pieces ? s_piece[c] : 0;
            mine += own[j];
        }
        const u64 incl = warp_scan(mine);
        if (lane == 31) s_warp[warp] = incl;
        __syncthreads();
        u64 before = incl - mine, cta = 0, all = 0;
        for (int k = 0; k < kVfWarps; ++k) {
            if (k < warp) before += s_warp[k];
            cta += s_warp[k];
        }
        if (cl > 1) {
            cluster_sync_all();  // (all of the cluster run, and have read the last round's)
            if (tid < cl) *cluster_ptr(&s_cta[rank], tid) = cta;
            cluster_sync_all();
            for (int k = 0; k < cl; ++k) {
                if (k < rank) before += s_cta[k];
                all += s_cta[k];
            }
        } else {
            all = cta;
            __syncthreads();
        }
        if (all == 0) {
            // p and q are the same but for roundings (or p is the draft alone):
            // the target's own
            if (w.kind == 0) return;
            w.kind = 0;
            continue;
        }
        const u64 goal = drawn_at(all, u);
        if (tid == 0) s_at = -1;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kVfScan; ++j) {
            if (goal >= before && goal < before + own[j]) {
                s_at = tid * kVfScan + j;
                s_left = goal - before;
            }
            before += own[j];
        }
        __syncthreads();
        if (s_at < 0 || warp > 0) return;
        each_kind([&](auto kind_t) {
            constexpr int kind = decltype(kind_t)::value;
            const int i0 = lo + s_at * kVfPiece + lane;
            float xp[PER], xq[PER] = {};
            fetch(xp, rp, i0);
            if (kind == 2) fetch(xq, rq, i0);
            u64 sum = 0;
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const u64 up = sum + warp_scan(SmRow::whole(w.template of<kind>(xp[j], xq[j], i0 + 32 * j)));
                const unsigned past = __ballot_sync(FULL, up > s_left);
                if (past) {
                    if (lane == __ffs(past) - 1) p.token[at] = i0 + 32 * j;
                    return;
                }
                sum = __shfl_sync(FULL, up, 31);
            }
        });
        return;
    }
}

size_t verify_workspace_bytes(int64_t rows) { return (size_t)rows * 2 * sizeof(SmPlan); }

template <bool BF16>
static cudaError_t launch_verify_t(const VerifyParams &v, cudaStream_t st) {
    const void *kfn = reinterpret_cast<const void *>(verify_kernel<BF16>);
    const cudaError_t e = allow_wide_clusters(kfn);
    if (e != cudaSuccess) return e;
    // Four CTAs an SM.  64 sequences of 151669 tokens, both kernels: clusters of
    // 4 CTAs 162 us, 8 144, 16 148; half as many CTAs of twice the threads 148.
    int cl = 1;
    while (cl < kVfMaxCluster && (int64_t)v.batch * cl * 2 <= 4 * num_sms() && v.V / (2 * cl) >= 4096) cl *= 2;
    return launch_pdl_cluster(kfn, (unsigned)(v.batch * cl), (unsigned)cl, kVfThreads, 0, st, v, cl);
}

cudaError_t launch_verify(const SampleParams &s, const VerifyParams &v, bool bf16, cudaStream_t st) {
    if (s.rows > 0) {  // (sequences without rows accept nothing)
        const cudaError_t e = launch_sample_plan(s, bf16, st);
        if (e != cudaSuccess) return e;
    }
    return bf16 ? launch_verify_t<true>(v, st) : launch_verify_t<false>(v, st);
}

}  // namespace gwa
