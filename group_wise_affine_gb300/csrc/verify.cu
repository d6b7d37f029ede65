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
// Everything is decided in whole numbers, as in sampling (sample.cuh): p(d) =
// P / SP with 41-bit masses and 60-bit sums, compared as products of 128 bits;
// max(p - q, 0) as P SQ - Q SP, both products cut to 64 bits at one common
// scale, so that their sum over the row fits.  The result depends on no split
// and no order.
//
// Two kernels.  The first is sampling's own (sample_kernel, PLAN), over the
// target rows and the draft rows at once: it leaves what each row's filters
// keep, as a cut and a sum.  This one then has one row a sequence to go over
// (two where a draft fell): a cluster of CTAs a sequence, each a slice of the
// row, each warp a run of it; the runs' sums are joined and the warp that
// holds the drawn mass looks for the token.
#include <algorithm>

#include "sample.cuh"

namespace gwa {

constexpr int kVfThreads = 512, kVfWarps = kVfThreads / 32;
constexpr int kVfMaxCluster = 8;

// The logits of a 16-byte chunk, or one.
template <bool BF16>
struct VfRow {
    using Raw = typename std::conditional<BF16, uint16_t, uint32_t>::type;
    const Raw *x;
    __device__ __forceinline__ float at(int64_t i) const {
        return __uint_as_float(BF16 ? (uint32_t)x[i] << 16 : (uint32_t)x[i]);
    }
};

// Masses of max(p - q, 0), or of p alone, at a common scale.
struct VfMass {
    SmPlan p, q;
    int shift_p, shift_q;  // of the products' upper 64 bits
    u64 norm_p, norm_q;    // the other row's sum, its top bit set
    int kind;              // 0: p; 1: p without token `drop`; 2: p - q
    int64_t drop;
    __device__ __forceinline__ void scales() {
        const int lp = __clzll(p.total), lq = __clzll(q.total), e = min(lp, lq);
        // P SQ 2^(lq - 41): of a sum below 2^63 after z more
        const int z = max(0, 24 - max(lp, lq));
        shift_p = lq - e + z;
        shift_q = lp - e + z;
        norm_p = q.total << lq;
        norm_q = p.total << lp;
    }
    __device__ __forceinline__ u64 of(float xp, float xq, int64_t token) const {
        const u64 a = p.kept(xp, (uint32_t)token);
        if (kind == 0 || a == 0) return a;
        if (kind == 1) return token == drop ? 0 : a;
        const u64 b = q.kept(xq, (uint32_t)token);
        const u64 l = __umul64hi(a << 23, norm_p) >> shift_p, r = __umul64hi(b << 23, norm_q) >> shift_q;
        return l > r ? l - r : 0;
    }
};

template <bool BF16>
__global__ void __launch_bounds__(kVfThreads) verify_kernel(VerifyParams p, int cl) {
    constexpr unsigned FULL = 0xffffffffu;
    using Row = VfRow<BF16>;
    using Raw = typename Row::Raw;
    __shared__ u64 s_warp[kVfWarps], s_cta[kVfMaxCluster];
    __shared__ int s_fell;
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
    w.scales();
    const Row rp = row_of(at), rq = w.kind == 2 ? draft_of(at) : rp;
    const int64_t per_cta = (p.V + cl - 1) / cl;
    const int64_t lo = min(p.V, rank * per_cta), hi = min(p.V, lo + per_cta);
    const int64_t run = ((hi - lo + kVfWarps - 1) / kVfWarps + 31) & ~31ll;
    const int64_t a = min(hi, lo + warp * run), e = min(hi, a + run);
    const float u = p.u_draw[b];
    while (true) {
        u64 mine = 0;
        for (int64_t i = a + lane; i < e; i += 32) mine += w.of(rp.at(i), rq.at(i), i);
        mine = warp_sum64(mine);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        u64 before = 0, cta = 0, all = 0;
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
        if (goal < before || goal >= before + mine) return;
        u64 sum = before;
        for (int64_t i0 = a; i0 < e; i0 += 32) {
            const int64_t i = i0 + lane;
            const u64 v = i < e ? w.of(rp.at(i), rq.at(i), i) : 0;
            const u64 incl = warp_scan(v);
            const unsigned past = __ballot_sync(FULL, sum + incl > goal);
            if (past) {
                if (lane == __ffs(past) - 1) p.token[at] = (int32_t)i;
                return;
            }
            sum += __shfl_sync(FULL, incl, 31);
        }
        return;
    }
}

size_t verify_workspace_bytes(int64_t rows) { return (size_t)rows * 2 * sizeof(SmPlan); }

template <bool BF16>
static cudaError_t launch_verify_t(const VerifyParams &v, cudaStream_t st) {
    int cl = 1;
    while (cl < kVfMaxCluster && (int64_t)v.batch * cl * 2 <= 2 * num_sms() && v.V / (2 * cl) >= 4096) cl *= 2;
    return launch_pdl_cluster(reinterpret_cast<const void *>(verify_kernel<BF16>), (unsigned)(v.batch * cl),
                              (unsigned)cl, kVfThreads, 0, st, v, cl);
}

cudaError_t launch_verify(const SampleParams &s, const VerifyParams &v, bool bf16, cudaStream_t st) {
    const cudaError_t e = launch_sample_plan(s, bf16, st);
    if (e != cudaSuccess) return e;
    return bf16 ? launch_verify_t<true>(v, st) : launch_verify_t<false>(v, st);
}

}  // namespace gwa
