// Softmax attention over the paged 4-bit (or 8-bit) KV cache, for tokens by
// the few: one new token a sequence, drafted tokens, short tails.
// "Sanctum-MLX", six-changes table row 5 and the paragraph after it (online
// softmax in fp32, causal mask, GQA without copies), here with the keys
// quantized too and both in pages.
//
//   out[i,h,:] = sum_t p_t (sv_t cv_t + bv_t),
//   p = softmax_t(scale * q[i,h,:] . (sk_t ck_t + bk_t)),
//
// with codes c, and scale s and bias b per token, head and 64 dimensions.
// Codes enter the tensor cores as they are, fp16 subnormals c 2^-24 (masked
// out of the words, nothing else), and the affine map folds into what is
// already there:
//   scores  S^T = C_k Q^T    per 64 dimensions, fp32; then
//           x = sum_g s_g S_g + b_g sum(Q_g);
//   values  O^T += (C_v - c0)^T P'^T  with P' = p * s in fp16, plus
//           sum_t p_t b'_t in fp32, b' = b + c0 s, c0 = 8 (u4) or 128 (u8).
// The centre c0 comes off by an MMA with a constant operand just before each
// tile's codes: with it left in, an output that averages thousands of values
// would be the small difference of two large sums (scores are summed afresh
// for each tile and need none).  fp16 holds P' to 2^-11, bf16 only to 2^-8.
// Its range is met by powers of two: a query row is scaled so that its
// largest element lies in [2^12, 2^13), and the value scales and biases so
// that the largest scale, or bias / (2 c0), met so far lies in [2^5, 2^6) (the
// accumulators are rescaled when a larger one comes, as they are for the
// running maximum).  A product of weight and scale is thus rounded to 2^-11 of
// itself, or to 2^-30 of the largest weight times the largest scale met where
// that is more; in steps that the causal mask hides from some rows to 2^-39.
//
// Work split.  The unit is a step of some keys (STEP) of one sequence, KV head and
// block of up to 8 NN query rows (GQA heads x new tokens); the units of the
// whole batch are laid end to end and cut into equal runs, one per CTA, so
// ragged batches and single long sequences both fill the GPU.  A CTA that
// holds a whole (sequence, head, row block) writes the output itself; the
// pieces of one that was cut go to the workspace, each as its keys' mean value
// and the logarithm of their weights' sum, and a second kernel joins them.
// Lengths are read from the device; nothing of the split depends on host values
// but the grid.
//
// A warp takes a quarter of the step (U MMA tiles of 16 keys), copies its
// codes and parameters with cp.async into its own ring a step ahead, and
// keeps its own softmax state; the four warps merge in shared memory at the
// end of a piece.  (Bulk copies ran slower: pages of 16 tokens make them 1 KB
// and 64 to 128 bytes long, about 22 cycles of an SM each whatever their size.)
//
// Warp-level MMAs (m16n8k16) serve here: with 1 to 32 query rows the work is
// bound by the bytes of the cache and by unpacking codes, and their operands
// live in registers beside the unpacking; a tcgen05 MMA has at least 64 rows.
//
// Measured (u4, both kernels): one token over 4096 keys of 8 heads of 128 10.6
// us, over 131071 42.8 us (3.5 TB/s of cache); 64 sequences of up to 8192, 32
// heads, 70.6 us (3.7 TB/s).  No unit is at its limit: a warp spends 370
// instructions on 16 keys of a head, 24 of them MMAs (of 8 cycles each, 29% of
// the tensor pipe's), the rest unpacking, addresses and softmax; they are
// issued at 2.2 a cycle and SM (55%), and the top stall is the fixed latency
// from one to the next, with 16 warps an SM to hide it.  The bytes alone would
// take half the time.  Short caches are two launches and their dependent reads
// (lengths, pages, codes).
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "mma.cuh"
#include "paged.cuh"

namespace gwa {

constexpr int kPgWarps = 4;

// Shared memory of one warp's ring stage (U tiles of 16 keys).  A
// tile's codes are laid out [group][row][GB bytes], so that the fragment
// reads hit every bank once: key rows in the order of the scores' rows, value
// rows in key order (8-bit rows with their two halves swapped in every other
// pair of rows).
template <int BITS, int D, int NN>
struct PgLayout {
    static constexpr int G = D / 64;
    static constexpr int GB = 8 * BITS;          // code bytes of a group
    static constexpr int U = 2;                  // tiles of a warp's step
    static constexpr int KEYS = 16 * U;          // keys of a warp's step
    static constexpr int STEP = kPgWarps * KEYS; // keys of a CTA's step
    static_assert(STEP == 128, "sdpa_paged_units");
    static constexpr int TILE = 16 * G * GB;     // codes of a tile
    static constexpr int PB = 16 * G * 4;        // parameters of a tile
    static constexpr int K_OFF = 0;
    static constexpr int V_OFF = U * TILE;
    static constexpr int KP_OFF = 2 * U * TILE;
    static constexpr int VP_OFF = KP_OFF + U * PB;
    static constexpr int STAGE = VP_OFF + U * PB;
    static constexpr int S = 2;
    static constexpr int NQ = 8 * NN;
    static constexpr int MERGE = NQ * D * 4;     // a warp's output rows
    static constexpr int WARP_BYTES = S * STAGE > MERGE ? S * STAGE : MERGE;
    static constexpr int BYTES = kPgWarps * WARP_BYTES;
    static constexpr int BY_SMEM = (228 * 1024) / (BYTES + 1024 + kPgWarps * NQ * (12 + 4 * G) + 4 * NQ + NQ * D * 2);
    // resident CTAs by registers: accumulators (4 per 8 rows and 16
    // dimensions) and about 96 more
    static constexpr int BY_REGS = NN * D <= 128 ? 4 : NN * D <= 256 ? 3 : 2;
    static constexpr int CTAS = BY_SMEM < BY_REGS ? (BY_SMEM < 1 ? 1 : BY_SMEM) : BY_REGS;
    // key of score row j (0..7; row j + 8: 8 more); the value product's k
    // positions 2t, 2t + 1, 2t + 8, 2t + 9 are then keys t, t + 4, t + 8, t + 12
    static __device__ __forceinline__ int key_of_row(int j) { return (j >> 1) + 4 * (j & 1); }
};

// Keys that some row of the sequence sees, in steps; row blocks; segments
// (KV head and row block) with keys.
struct PgSeq {
    int first, base, len, rows, nrg, nt, segs;  // base: position of the first new token
};
// Steps that a segment's start and end (queries, merging the warps, the
// output) count for, where there are more steps than CTAs; else a CTA has a
// step.  With it against without it, sequences of many lengths, u4, 32 over 8
// heads of 128: 32 of about 400 keys 15.4 : 17.6 us, 1000 20.4 : 22.4, 4000
// 44.2 : 45.8, 200 of about 1000 77.9 : 90.1; 64 of 2048 each 49.3 : 49.5.
constexpr int kPgHead = 2;
template <int NQ, int STEP>
__device__ __forceinline__ PgSeq pg_seq(const PagedParams &p, int b) {
    const KvSeq s = kv_seq(p.kv, b);
    PgSeq r;
    r.first = s.first;
    r.base = s.end - s.count;
    r.len = s.len;
    r.rows = p.rep * min(s.count, p.kv.max_q);
    if (r.rows > p.split) r.rows = 0;  // the prompt kernel's
    r.nrg = (r.rows + NQ - 1) / NQ;
    r.nt = (s.len + STEP - 1) / STEP;
    r.segs = r.nt > 0 ? p.kv.heads * r.nrg : 0;  // (times nt: the entry point keeps the total below 2^31)
    return r;
}

// Sixteen codes of one key row as the fp16 pairs the MMA takes.  A code left
// in the low mantissa bits of a zero exponent is the fp16 subnormal c 2^-24,
// exact and linear, so unpacking is masking alone.  u4 fields at bits 4-7
// are 16 c 2^-24: the queries they meet are divided by 16 (k_sixteenth).
template <int BITS>
__device__ __forceinline__ void k_fragments(const unsigned char *src, uint32_t (&f)[8]) {
    if constexpr (BITS == 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(src);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t u = j ? w.y : w.x, u8 = u >> 8;
            f[4 * j + 0] = u & 0x000f000fu;
            f[4 * j + 1] = u & 0x00f000f0u;
            f[4 * j + 2] = u8 & 0x000f000fu;
            f[4 * j + 3] = u8 & 0x00f000f0u;
        }
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(src);
        const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = ws[j] & 0x00ff00ffu;
            f[2 * j + 1] = (ws[j] >> 8) & 0x00ff00ffu;
        }
    }
}
template <int BITS>
__device__ __forceinline__ constexpr bool k_sixteenth(int i) {
    return BITS == 4 && i % 2 == 1;
}

// Dimension, within its lane's sixteen, of element e of pair i as
// k_fragments orders them.
template <int BITS>
__device__ __forceinline__ constexpr int k_dim(int i, int e) {
    return BITS == 4 ? 8 * (i / 4) + (i % 4) + 4 * e
                     : 4 * (i / 2) + (i % 2) + 2 * e;
}

// 2^e with the largest of a row in [2^12, 2^13), and 2^-e.
__device__ __forceinline__ void row_scale(float t, float &up, float &down) {
    int p = 0;
    if (t > 0.f && t < 3.0e38f) p = 139 - f32_exp_field(t);
    p = p < -125 ? -125 : p > 125 ? 125 : p;
    up = __uint_as_float((uint32_t)(127 + p) << 23);
    down = __uint_as_float((uint32_t)(127 - p) << 23);
}

template <int BITS, int D, int NN>
__global__ void __launch_bounds__(kPgWarps * kWarp, PgLayout<BITS, D, NN>::CTAS)
    paged_decode_kernel(PagedParams p) {
    using L = PgLayout<BITS, D, NN>;
    constexpr int G = L::G, GB = L::GB, S = L::S, NQ = L::NQ;
    constexpr int U = L::U, KEYS = L::KEYS, STEP = L::STEP;
    constexpr int NT = D / 16;                  // value m-tiles
    constexpr int NCP = L::TILE / 16 / kWarp;   // 16-byte copies per lane, tile
    constexpr int RCH = G * GB / 16;            // 16-byte chunks of a key row
    static_assert(NCP >= 1, "tile copies");
    constexpr float KC = BITS == 4 ? 8.f : 128.f;
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ __align__(16) unsigned char pg_smem[];
    __shared__ float s_m[kPgWarps][NQ], s_l[kPgWarps][NQ], s_f[kPgWarps][NQ];
    __shared__ float s_b[kPgWarps][NQ][G];
    __shared__ float s_den[NQ];
    __shared__ uint4 s_q[NN][G][2][kWarp];

    const int lane = threadIdx.x & (kWarp - 1), warp = threadIdx.x / kWarp;
    const int g = lane >> 2, t = lane & 3;
    const int kv_g = L::key_of_row(g);
    unsigned char *wsm = pg_smem + warp * L::WARP_BYTES;
    // the lane's 16-byte copies of a tile: where they go
    int kdst[NCP], vdst[NCP];
#pragma unroll
    for (int i = 0; i < NCP; ++i) {
        const int ci = lane + 32 * i, r = ci / RCH, rem = ci % RCH;
        const int gg = rem / (GB / 16), ch = rem % (GB / 16);
        const int kr = (r & 8) | ((r & 3) << 1) | ((r >> 2) & 1);
        const int vch = BITS == 8 ? ch ^ (((r >> 1) & 1) << 1) : ch;
        kdst[i] = L::K_OFF + (gg * 16 + kr) * GB + ch * 16;
        vdst[i] = L::V_OFF + (gg * 16 + r) * GB + vch * 16;
    }
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();

    // ---- this CTA's run of units, found by every warp for itself
    const int B = p.kv.batch;
    const int cta = blockIdx.x;
    int total = 0, segs = 0;
    for (int b0 = 0; b0 < B; b0 += kWarp) {
        PgSeq s{};
        if (b0 + lane < B) s = pg_seq<NQ, STEP>(p, b0 + lane);
        total += __reduce_add_sync(FULL, s.segs * s.nt);
        segs += __reduce_add_sync(FULL, s.segs);
    }
    const int head = total > (int)gridDim.x ? kPgHead : 0;
    total += segs * head;
    // sequences without keys: their rows are zero
    for (int i = cta; i < B; i += gridDim.x) {
        const PgSeq s = pg_seq<NQ, STEP>(p, i);
        if (p.status && threadIdx.x == 0 && kv_past(kv_seq(p.kv, i)))
            atomicOr(p.status, (int)kKvBadPage);
        if (p.by_seg)
            for (int k = s.segs + threadIdx.x; k < p.segs; k += blockDim.x)
                p.cuts[i * p.segs + k].slot = -1;
        if (s.nt > 0) continue;
        uint32_t *o = reinterpret_cast<uint32_t *>(p.out + (int64_t)s.first * p.Hq * D);
        for (int64_t k = threadIdx.x; k < (int64_t)(s.rows / p.rep) * p.Hq * (D / 2); k += blockDim.x)
            o[k] = 0u;
    }
    const int ctas = min((int)gridDim.x, total);
    if (!p.by_seg && threadIdx.x == 0) p.cuts[cta].slot = -1;
    if (cta >= ctas) return;
    const int quot = total / ctas, rest = total % ctas;
    const int begin = pg_start(quot, rest, cta), end = pg_start(quot, rest, cta + 1);

    int b = 0, at = 0;  // the sequence of the run's first unit, units before it
    for (int b0 = 0; b0 < B; b0 += kWarp) {
        PgSeq s{};
        if (b0 + lane < B) s = pg_seq<NQ, STEP>(p, b0 + lane);
        const int u = s.segs * (s.nt + head);
        int incl = u;
#pragma unroll
        for (int o = 1; o < kWarp; o <<= 1) {
            const int v = __shfl_up_sync(FULL, incl, o);
            if (lane >= o) incl += v;
        }
        const unsigned past = __ballot_sync(FULL, at + incl > begin);
        if (past) {
            const int l = __ffs(past) - 1;
            b = b0 + l;
            at += __shfl_sync(FULL, incl - u, l);
            break;
        }
        at += __shfl_sync(FULL, incl, kWarp - 1);
    }
    PgSeq sq = pg_seq<NQ, STEP>(p, b);
    int cur = begin;
    int piece = 0;
    const float sl2 = p.scale * 1.4426950408889634f;  // scores in base 2
    // The running maximum moves only when a weight passes 2^8 (weights and
    // their sums stay far inside fp32 and fp16), or from nothing: kNone makes
    // the first weight infinite.
    constexpr float kLazy = 256.f, kNone = -3e38f;
    const int pmask = (1 << p.kv.page_shift) - 1;

    while (cur < end) {
        const int cost = sq.nt + head;  // of a segment
        if (cur >= at + sq.segs * cost) {
            // (never past the batch, unless the lengths change meanwhile)
            if (b + 1 >= B) break;
            at += sq.segs * cost;
            sq = pg_seq<NQ, STEP>(p, ++b);
            continue;
        }
        const int seg = (cur - at) / cost;  // hk * nrg + rg
        const int from = cur - at - seg * cost, to = min(cost, from + (end - cur));
        cur += to - from;
        if (to <= head) continue;  // none of its steps
        const int hk = seg / sq.nrg, rg = seg % sq.nrg;
        const int ta = max(from - head, 0), tb = to - head;
        const int nlive = min(NQ, sq.rows - rg * NQ);
        const int32_t *table = p.kv.page_table + (int64_t)b * p.kv.max_pages;

        // queries: row 8 nn + g, dimensions 64 gg + 16 t .. + 15, as the
        // fragments that every warp reads back for each step
        float fac[NN][2], qs[NN][G][2];
        int lim[NN][2];
#pragma unroll
        for (int nn = 0; nn < NN; ++nn) {
            const int r = rg * NQ + 8 * nn + g;
            float mx = 0.f, down = 1.f, up = 1.f, sum[G];
            uint4 raw[G][2];
#pragma unroll
            for (int gg = 0; gg < G; ++gg) raw[gg][0] = raw[gg][1] = make_uint4(0u, 0u, 0u, 0u);
            if (8 * nn + g < nlive) {
                const uint16_t *src = p.q + (sq.first + r / p.rep) * p.q_stride +
                                      (int64_t)(hk * p.rep + r % p.rep) * D + 16 * t;
#pragma unroll
                for (int gg = 0; gg < G; ++gg) {
                    raw[gg][0] = reinterpret_cast<const uint4 *>(src + 64 * gg)[0];
                    raw[gg][1] = reinterpret_cast<const uint4 *>(src + 64 * gg)[1];
                }
            }
            auto elem = [&](int gg, int d) {
                const uint4 &u = raw[gg][d / 8];
                const int w = (d % 8) / 2;
                const uint32_t v = w == 0 ? u.x : w == 1 ? u.y : w == 2 ? u.z : u.w;
                return d & 1 ? bf16_hi(v) : bf16_lo(v);
            };
#pragma unroll
            for (int gg = 0; gg < G; ++gg)
#pragma unroll
                for (int d = 0; d < 16; ++d) mx = fmaxf(mx, fabsf(elem(gg, d)));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
            row_scale(mx, up, down);
#pragma unroll
            for (int gg = 0; gg < G; ++gg) {
                sum[gg] = 0.f;
                uint32_t qf[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float a = elem(gg, k_dim<BITS>(i, 0)) * up;
                    const float c = elem(gg, k_dim<BITS>(i, 1)) * up;
                    constexpr float r16 = 0.0625f;
                    qf[i] = k_sixteenth<BITS>(i) ? pack_f16(a * r16, c * r16) : pack_f16(a, c);
                    sum[gg] += a + c;
                }
                if ((nn * G + gg) % kPgWarps == warp) {
                    s_q[nn][gg][0][lane] = make_uint4(qf[0], qf[1], qf[2], qf[3]);
                    s_q[nn][gg][1][lane] = make_uint4(qf[4], qf[5], qf[6], qf[7]);
                }
                sum[gg] += __shfl_xor_sync(FULL, sum[gg], 1);
                sum[gg] += __shfl_xor_sync(FULL, sum[gg], 2);
            }
            // the scores' columns 2t, 2t + 1 are rows 8 nn + 2t (+ 1)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int from = (2 * t + h) * 4;
                // scores stay times 2^-24, as the codes are
                fac[nn][h] = __shfl_sync(FULL, down, from) * sl2 * 0x1p24f;
#pragma unroll
                for (int gg = 0; gg < G; ++gg)
                    qs[nn][gg][h] = __shfl_sync(FULL, sum[gg], from) * 0x1p-24f;
                const int i = 8 * nn + 2 * t + h, rr = rg * NQ + i;
                lim[nn][h] = i >= nlive ? 0
                             : p.causal ? min(sq.len, sq.base + rr / p.rep + 1)
                                        : sq.len;
            }
        }
        __syncthreads();
        // every row of the block sees the keys below `all`, none those from
        // `seen` on
        int all = 0x7fffffff;
        const int seen =
            p.causal ? min(sq.len, sq.base + (rg * NQ + nlive - 1) / p.rep + 1) : sq.len;
#pragma unroll
        for (int nn = 0; nn < NN; ++nn)
#pragma unroll
            for (int h = 0; h < 2; ++h) all = min(all, lim[nn][h]);
        if (nlive < NQ) {  // padding rows: masked or not, they are never written
            all = p.causal ? max(0, min(sq.len, sq.base + rg * NQ / p.rep + 1)) : sq.len;
        } else {
            all = __reduce_min_sync(FULL, all);
        }

        float o[NN][NT][4], m[NN][2], l[NN][2], bs[NN][G][2];
#pragma unroll
        for (int nn = 0; nn < NN; ++nn) {
#pragma unroll
            for (int j = 0; j < NT; ++j)
                o[nn][j][0] = o[nn][j][1] = o[nn][j][2] = o[nn][j][3] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                m[nn][h] = kNone;
                l[nn][h] = 0.f;
#pragma unroll
                for (int gg = 0; gg < G; ++gg) bs[nn][gg][h] = 0.f;
            }
        }
        // value scales and biases: times vinv, met up to vlim and 2 KC vlim
        float vinv = 1.f, vlim = -1.f;

        // Page numbers of the tiles of 32 / U steps: lane U j + u holds those of
        // step j's tile u.
        int pages = 0, pages_at = ta - 32;
        auto issue = [&](int step, int to) {
            if (step - pages_at >= 32 / U) {
                pages_at = step;
                const int key = (step + lane / U) * STEP + warp * KEYS + lane % U * 16;
                pages = 0;
                if (step + lane / U < tb && key < sq.len) {
                    pages = table[key >> p.kv.page_shift];
                    if ((unsigned)pages >= (unsigned)p.kv.num_pages) {
                        if (p.status) atomicOr(p.status, (int)kKvBadPage);
                        pages = 0;
                    }
                }
            }
            unsigned char *st = wsm + to * L::STAGE;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int page = __shfl_sync(FULL, pages, U * (step - pages_at) + u);
                const int key = step * STEP + warp * KEYS + u * 16;
                if (key >= sq.len) break;  // warp-uniform
                const int64_t row = (((int64_t)page * p.kv.heads + hk) << p.kv.page_shift) +
                                    (key & pmask);
                const uint4 *ks = reinterpret_cast<const uint4 *>(p.kv.kq) + row * RCH + lane;
                const uint4 *vs = reinterpret_cast<const uint4 *>(p.kv.vq) + row * RCH + lane;
#pragma unroll
                for (int i = 0; i < NCP; ++i) {
                    cp_async<16>(st + kdst[i] + u * L::TILE, ks + 32 * i);
                    cp_async<16>(st + vdst[i] + u * L::TILE, vs + 32 * i);
                }
                // parameters: lanes below 4 G the keys', the next 4 G the values'
                if (lane < 8 * G) {
                    const bool is_k = lane < 4 * G;
                    const int i = is_k ? lane : lane - 4 * G;
                    cp_async<16>(st + (is_k ? L::KP_OFF : L::VP_OFF) + u * L::PB + i * 16,
                                 (is_k ? p.kv.kp : p.kv.vp) + row * G + 4 * i);
                }
            }
        };
        auto scale_rows = [&](int nn, float c0, float c1) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                o[nn][j][0] *= c0;
                o[nn][j][1] *= c1;
                o[nn][j][2] *= c0;
                o[nn][j][3] *= c1;
            }
        };
        // One step of 32 keys.  EDGE: some row does not see all of them.  The
        // largest value scale may then be of a key that this row does not see:
        // weights stay at 1 there instead of 2^8, and scales go up to 2^15
        // instead of 2^6, so that keys of 2^24 times smaller scales keep their
        // place in fp16.  (Such steps are the segment's last ones.)
        auto compute = [&](const unsigned char *stg, const int key0, auto edge_t) {
            constexpr bool EDGE = decltype(edge_t)::value;
            // ---- scores: x[u][kk][nn][h] of key key0 + 16 u + HALF kk + kv_g,
            // less the factor fac of the column
            float x[U][2][NN][2];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int nn = 0; nn < NN; ++nn) x[u][kk][nn][0] = x[u][kk][nn][1] = 0.f;
#pragma unroll
            for (int gg = 0; gg < G; ++gg) {
                uint4 qa[NN], qb[NN];
#pragma unroll
                for (int nn = 0; nn < NN; ++nn) {
                    qa[nn] = s_q[nn][gg][0][lane];
                    qb[nn] = s_q[nn][gg][1][lane];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const unsigned char *kt = stg + L::K_OFF + u * L::TILE + g * GB + t * 2 * BITS;
                    const unsigned char *kp = stg + L::KP_OFF + u * L::PB + kv_g * G * 4;
                    uint32_t f0[8], f1[8];
                    k_fragments<BITS>(kt + gg * 16 * GB, f0);
                    k_fragments<BITS>(kt + gg * 16 * GB + 8 * GB, f1);
                    const uint32_t p0 = *reinterpret_cast<const uint32_t *>(kp + gg * 4);
                    const uint32_t p1 = *reinterpret_cast<const uint32_t *>(kp + (8 * G + gg) * 4);
                    const float s0 = bf16_lo(p0), s1 = bf16_lo(p1);
                    const float b0 = bf16_hi(p0), b1 = bf16_hi(p1);
#pragma unroll
                    for (int nn = 0; nn < NN; ++nn) {
                        float c[4] = {0.f, 0.f, 0.f, 0.f};
                        mma_f16(c, f0[0], f1[0], f0[1], f1[1], qa[nn].x, qa[nn].y);
                        mma_f16(c, f0[2], f1[2], f0[3], f1[3], qa[nn].z, qa[nn].w);
                        mma_f16(c, f0[4], f1[4], f0[5], f1[5], qb[nn].x, qb[nn].y);
                        mma_f16(c, f0[6], f1[6], f0[7], f1[7], qb[nn].z, qb[nn].w);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            x[u][0][nn][h] = fmaf(s0, c[h], fmaf(b0, qs[nn][gg][h], x[u][0][nn][h]));
                            x[u][1][nn][h] = fmaf(s1, c[2 + h], fmaf(b1, qs[nn][gg][h], x[u][1][nn][h]));
                        }
                    }
                }
            }
            // ---- weights, against the maximum so far
            float e[U][2][NN][2], emax = 0.f;
            auto weigh = [&] {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                        for (int nn = 0; nn < NN; ++nn)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                e[u][kk][nn][h] = ex2(fmaf(x[u][kk][nn][h], fac[nn][h], -m[nn][h]));
                                if (EDGE && key0 + 16 * u + 8 * kk + kv_g >= lim[nn][h])
                                    e[u][kk][nn][h] = 0.f;
                            }
            };
            weigh();
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int nn = 0; nn < NN; ++nn)
                        emax = fmaxf(emax, fmaxf(e[u][kk][nn][0], e[u][kk][nn][1]));
            if (__any_sync(FULL, emax > (EDGE ? 1.f : kLazy))) {
                // a new maximum
#pragma unroll
                for (int nn = 0; nn < NN; ++nn) {
                    float cr[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float mt = -INFINITY;
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int kk = 0; kk < 2; ++kk)
                                if (!EDGE || key0 + 16 * u + 8 * kk + kv_g < lim[nn][h])
                                    mt = fmaxf(mt, x[u][kk][nn][h] * fac[nn][h]);
#pragma unroll
                        for (int off = 4; off < kWarp; off <<= 1)
                            mt = fmaxf(mt, __shfl_xor_sync(FULL, mt, off));
                        const float mn = fmaxf(m[nn][h], mt);
                        cr[h] = ex2(m[nn][h] - mn);
                        m[nn][h] = mn;
                        l[nn][h] *= cr[h];
#pragma unroll
                        for (int gg = 0; gg < G; ++gg) bs[nn][gg][h] *= cr[h];
                    }
                    scale_rows(nn, cr[0], cr[1]);
                }
                weigh();
            }
#pragma unroll
            for (int nn = 0; nn < NN; ++nn)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < U; ++u) l[nn][h] += e[u][0][nn][h] + e[u][1][nn][h];
            // ---- values: their parameters, and a larger one than any so far
            uint32_t vw[U][2][G];
            float smax = 0.f, bmax = 0.f;
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                    for (int gg = 0; gg < G; ++gg) {
                        uint32_t &w = vw[u][kk][gg];
                        w = *reinterpret_cast<const uint32_t *>(stg + L::VP_OFF + u * L::PB +
                                                                ((kv_g + 8 * kk) * G + gg) * 4);
                        // past the end lie no parameters (but anything)
                        if (EDGE && key0 + 16 * u + 8 * kk + kv_g >= seen) w = 0u;
                        smax = fmaxf(smax, fabsf(bf16_lo(w)));
                        // (the bias, and the scale's bits below its last place)
                        bmax = fmaxf(bmax, fabsf(__uint_as_float(w)));
                    }
            if (__any_sync(FULL, smax > vlim || bmax > 2.f * KC * vlim)) {
                if (fmaxf(smax, bmax) == INFINITY) {
                    // a key whose parameters are not finite makes its own
                    // readers' rows so, and must not take the others' range
                    smax = bmax = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                            for (int gg = 0; gg < G; ++gg) {
                                const float sv = fabsf(bf16_lo(vw[u][kk][gg])), bv = fabsf(bf16_hi(vw[u][kk][gg]));
                                if (!(fmaxf(sv, bv) < INFINITY)) continue;
                                smax = fmaxf(smax, sv);
                                bmax = fmaxf(bmax, bv);
                            }
                }
                const float top = __uint_as_float(
                    __reduce_max_sync(FULL, __float_as_uint(fmaxf(smax, bmax * (0.5f / KC)))));
                if (top > vlim) {
                    // 2^ex <= top < 2^(ex+1): times 2^(kRange-ex)
                    constexpr int kRange = EDGE ? 14 : 5;
                    const int ex = min(max(f32_exp_field(top), 6), 253);
                    const float ninv = __uint_as_float((uint32_t)min(254 + kRange - ex, 254) << 23);
                    const float vf = vlim < 0.f ? 1.f : ninv / vinv;
#pragma unroll
                    for (int nn = 0; nn < NN; ++nn) {
                        scale_rows(nn, vf, vf);
#pragma unroll
                        for (int gg = 0; gg < G; ++gg) {
                            bs[nn][gg][0] *= vf;
                            bs[nn][gg][1] *= vf;
                        }
                    }
                    vinv = ninv;
                    vlim = __uint_as_float((uint32_t)(ex + 1) << 23);
                }
            }
#pragma unroll
            for (int gg = 0; gg < G; ++gg) {
                uint32_t pb[U][NN][2];
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        const float s = bf16_lo(vw[u][kk][gg]) * vinv;
                        const float bb = fmaf(KC, s, bf16_hi(vw[u][kk][gg]) * vinv);
#pragma unroll
                        for (int nn = 0; nn < NN; ++nn) {
                            const float e0 = e[u][kk][nn][0], e1 = e[u][kk][nn][1];
                            float a0 = e0 * s, a1 = e1 * s;
                            if constexpr (EDGE) {  // a weight of zero takes nothing, whatever s and b
                                a0 = e0 == 0.f ? 0.f : a0;
                                a1 = e1 == 0.f ? 0.f : a1;
                                bs[nn][gg][0] += e0 == 0.f ? 0.f : e0 * bb;
                                bs[nn][gg][1] += e1 == 0.f ? 0.f : e1 * bb;
                            } else {
                                bs[nn][gg][0] = fmaf(e0, bb, bs[nn][gg][0]);
                                bs[nn][gg][1] = fmaf(e1, bb, bs[nn][gg][1]);
                            }
                            pb[u][nn][kk] = movmatrix_t(pack_f16(a0, a1));
                        }
                    }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int half = BITS == 8 ? (g ^ ((t >> 1) << 2)) * 8 : g * 4;
                    const unsigned char *vs = stg + L::V_OFF + u * L::TILE + (gg * 16 + t) * GB + half;
                    // words of the keys at k = 2t, 2t + 1, 2t + 8, 2t + 9
                    uint32_t w[4][BITS / 4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const unsigned char *src = vs + 4 * i * GB;
                        if constexpr (BITS == 4) {
                            w[i][0] = *reinterpret_cast<const uint32_t *>(src);
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2 *>(src);
                            w[i][0] = v.x;
                            w[i][1] = v.y;
                        }
                    }
                    // codes as subnormals again, c 2^-24 in rows g and (u4)
                    // 16 c 2^-24 in rows g + 8; a constant operand takes the
                    // centre off first, on the same scales
                    constexpr uint32_t C0 = BITS == 4 ? 0x80088008u : 0x80808080u;
                    constexpr uint32_t C1 = BITS == 4 ? 0x80808080u : 0x80808080u;
#pragma unroll
                    for (int jj = 0; jj < 4; ++jj) {
                        uint32_t a[4];
                        if constexpr (BITS == 4) {
                            // byte jj: dimensions 8g + 2jj (m-row g), + 1 (g + 8)
                            const uint32_t sel = jj | (jj << 4) | ((4 + jj) << 8) | ((4 + jj) << 12);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t r = __byte_perm(w[2 * k][0], w[2 * k + 1][0], sel);
                                a[2 * k] = r & 0x000f000fu;
                                a[2 * k + 1] = r & 0x00f000f0u;
                            }
                        } else {
                            const int e2 = 2 * (jj & 1);
                            const uint32_t sel = e2 | ((e2 + 1) << 4) | ((4 + e2) << 8) | ((5 + e2) << 12);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t r = __byte_perm(w[2 * k][jj / 2], w[2 * k + 1][jj / 2], sel);
                                a[2 * k] = r & 0x00ff00ffu;
                                a[2 * k + 1] = (r >> 8) & 0x00ff00ffu;
                            }
                        }
#pragma unroll
                        for (int nn = 0; nn < NN; ++nn) {
                            mma_f16(o[nn][4 * gg + jj], C0, C1, C0, C1, pb[u][nn][0], pb[u][nn][1]);
                            mma_f16(o[nn][4 * gg + jj], a[0], a[1], a[2], a[3], pb[u][nn][0],
                                    pb[u][nn][1]);
                        }
                    }
                }
            }
        };
#pragma unroll
        for (int i = 0; i < S - 1; ++i) {
            if (ta + i < tb) issue(ta + i, i);
            cp_async_commit();
        }
        int stage = 0;
        for (int step = ta; step < tb; ++step) {
            if (step + S - 1 < tb) issue(step + S - 1, stage == 0 ? S - 1 : stage - 1);
            cp_async_commit();
            cp_async_wait<S - 1>();
            __syncwarp();
            const int key0 = step * STEP + warp * KEYS;
            if (key0 < sq.len) {  // warp-uniform
                const unsigned char *stg = wsm + stage * L::STAGE;
                if (key0 + KEYS > all)
                    compute(stg, key0, std::true_type{});
                else
                    compute(stg, key0, std::false_type{});
            }
            __syncwarp();  // the stage is free for the next copies
            stage = stage == S - 1 ? 0 : stage + 1;
        }

        // ---- the four warps' states to shared memory, and out
#pragma unroll
        for (int nn = 0; nn < NN; ++nn)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int off = 4; off < kWarp; off <<= 1) {
                    l[nn][h] += __shfl_xor_sync(FULL, l[nn][h], off);
#pragma unroll
                    for (int gg = 0; gg < G; ++gg)
                        bs[nn][gg][h] += __shfl_xor_sync(FULL, bs[nn][gg][h], off);
                }
        __syncwarp();
        float *so = reinterpret_cast<float *>(wsm);
        // the codes' powers of two (rows g and g + 8); vinv's stays in
        constexpr float back = 0x1p24f, back1 = BITS == 4 ? back * 0.0625f : back;
#pragma unroll
        for (int nn = 0; nn < NN; ++nn) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const int d = 64 * (j / 4) + 8 * g + 2 * (j % 4);
                const int r = 8 * nn + 2 * t;
                *reinterpret_cast<float2 *>(so + r * D + d) =
                    make_float2(o[nn][j][0] * back, o[nn][j][2] * back1);
                *reinterpret_cast<float2 *>(so + (r + 1) * D + d) =
                    make_float2(o[nn][j][1] * back, o[nn][j][3] * back1);
            }
            if (g == 0)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = 8 * nn + 2 * t + h;
                    s_m[warp][r] = m[nn][h];
                    s_l[warp][r] = l[nn][h];
                    s_f[warp][r] = vlim < 0.f ? 0x1p127f : vinv;
#pragma unroll
                    for (int gg = 0; gg < G; ++gg) s_b[warp][r][gg] = bs[nn][gg][h];
                }
        }
        __syncthreads();
        const bool whole = ta == 0 && tb == sq.nt;
        float *part = p.part + (int64_t)(2 * cta + piece) * NQ * (D + 4);
        if (threadIdx.x < NQ) {
            const int i = threadIdx.x;
            // the merged rows are times the smallest of the warps' vinv
            float mx = kNone, den = 0.f, v_all = 0x1p127f;
#pragma unroll
            for (int w = 0; w < kPgWarps; ++w) {
                mx = fmaxf(mx, s_m[w][i]);
                v_all = fminf(v_all, s_f[w][i]);
            }
#pragma unroll
            for (int w = 0; w < kPgWarps; ++w) {
                const float f = s_l[w][i] == 0.f ? 0.f : ex2(s_m[w][i] - mx);
                s_f[w][i] = f * (v_all / s_f[w][i]);
                den += f * s_l[w][i];
            }
            s_den[i] = den == 0.f ? 0.f : 1.f / den;
            s_m[0][i] = 1.f / v_all;
            if (!whole) part[i * (D + 4) + D] = den == 0.f ? -INFINITY : mx + __log2f(den);
        }
        __syncthreads();
        constexpr int C4 = D / 4;
        for (int e = threadIdx.x; e < nlive * C4; e += blockDim.x) {
            const int i = e / C4, c4 = e % C4;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kPgWarps; ++w) {
                const float f = s_f[w][i], bw = s_b[w][i][c4 / 16];
                if (f == 0.f) continue;
                const float4 v =
                    reinterpret_cast<const float4 *>(pg_smem + w * L::WARP_BYTES)[i * C4 + c4];
                a.x = fmaf(f, v.x + bw, a.x);
                a.y = fmaf(f, v.y + bw, a.y);
                a.z = fmaf(f, v.z + bw, a.z);
                a.w = fmaf(f, v.w + bw, a.w);
            }
            // (the sum first, the power second: both stay in range)
            const float r = s_den[i], v_back = s_m[0][i];
            a = make_float4(a.x * r * v_back, a.y * r * v_back, a.z * r * v_back, a.w * r * v_back);
            if (whole) {
                const int rr = rg * NQ + i;
                uint2 *dst = reinterpret_cast<uint2 *>(
                    p.out + ((int64_t)(sq.first + rr / p.rep) * p.Hq + hk * p.rep + rr % p.rep) * D);
                dst[c4] = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
            } else {
                reinterpret_cast<float4 *>(part + i * (D + 4))[c4] = a;
            }
        }
        if (threadIdx.x == 0) {
            PgCut *cut = p.by_seg ? p.cuts + b * p.segs + seg : p.cuts + cta;
            if (ta == 0 && !whole) {
                // starts here and goes on: up to the CTA of its last unit
                const int last = pg_owner(quot, rest, at + (seg + 1) * cost - 1);
                *cut = PgCut{2 * cta + piece, cta, last - cta + 1, sq.first, hk * p.rep,
                             rg * NQ, nlive, 0};
            } else if (whole && p.by_seg) {
                cut->slot = -1;
            }
        }
        piece = 1;
        __syncthreads();  // the ring is free again
    }
}

// Joins the pieces of a (sequence, KV head, row block) that the cut spread
// over several CTAs: piece i's mean value o_i and the base-2 logarithm c_i of
// its weights' sum give out = sum_i 2^(c_i - M) o_i / sum_i 2^(c_i - M).
// (Sums of weights times values would leave fp32's range where the values are
// near its end.)  Block (x, y): row y of cut x.  Threads take four dimensions
// each and every NG-th piece, eight pieces' loads in flight, against a maximum
// of their own; the NG groups meet in shared memory.
template <int D, int NQ>
__global__ void __launch_bounds__(256) paged_join_kernel(PagedParams p) {
    constexpr int C4 = D / 4, NG = 256 / C4, AHEAD = 8;
    __shared__ float s_m[NG], s_l[NG];
    __shared__ float4 s_o[NG][C4];
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const PgCut d = p.cuts[blockIdx.x];
    const int i = blockIdx.y;
    if (d.slot < 0 || i >= d.nlive) return;
    const int c4 = threadIdx.x % C4, grp = threadIdx.x / C4;
    float m = -INFINITY, l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = grp; k0 < d.n; k0 += NG * AHEAD) {
        float4 v[AHEAD];
        float c[AHEAD];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int k = k0 + j * NG;
            c[j] = -INFINITY;
            v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k >= d.n) continue;
            const float *src = p.part + ((int64_t)(k == 0 ? d.slot : 2 * (d.cta + k)) * NQ + i) * (D + 4);
            v[j] = reinterpret_cast<const float4 *>(src)[c4];
            c[j] = src[D];
        }
        float mx = m;
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) mx = fmaxf(mx, c[j]);
        // (where no piece of the group has a key that the row sees, m stays
        // below every other's)
        const float sub = mx == -INFINITY ? 0.f : mx;
        const float f0 = ex2(m - sub);
        l *= f0;
        a = make_float4(a.x * f0, a.y * f0, a.z * f0, a.w * f0);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const float f = ex2(c[j] - sub - kPgJoin);
            l += f;
            a.x = fmaf(f, v[j].x, a.x);
            a.y = fmaf(f, v[j].y, a.y);
            a.z = fmaf(f, v[j].z, a.z);
            a.w = fmaf(f, v[j].w, a.w);
        }
        m = mx;
    }
    if (c4 == 0) {
        s_m[grp] = m;
        s_l[grp] = l;
    }
    s_o[grp][c4] = a;
    __syncthreads();
    if (grp) return;
    float mx = -INFINITY, den = 0.f;
#pragma unroll
    for (int k = 0; k < NG; ++k) mx = fmaxf(mx, s_m[k]);
    if (mx == -INFINITY) mx = 0.f;
    a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NG; ++k) {
        const float f = ex2(s_m[k] - mx);
        const float4 v = s_o[k][c4];
        den = fmaf(f, s_l[k], den);
        a.x = fmaf(f, v.x, a.x);
        a.y = fmaf(f, v.y, a.y);
        a.z = fmaf(f, v.z, a.z);
        a.w = fmaf(f, v.w, a.w);
    }
    const float r = den == 0.f ? 0.f : 1.f / den;
    const int rr = d.r0 + i;
    reinterpret_cast<uint2 *>(
        p.out + ((int64_t)(d.first + rr / p.rep) * p.Hq + d.head + rr % p.rep) * D)[c4] =
        make_uint2(pack_bf16(a.x * r, a.y * r), pack_bf16(a.z * r, a.w * r));
}

// ---------------------------------------------------------------- host side
// Row block: the smallest of 8, 16, 32 rows that holds a sequence's rows (16
// at 256 dimensions, whose accumulators take twice the registers).
static int pg_nn(int64_t rows, int D) {
    return rows <= 8 ? 1 : rows <= 16 || D == 256 ? 2 : 4;
}

template <int BITS, int D, int NN>
static int pg_grid(const KvView &kv, int64_t rows) {
    using L = PgLayout<BITS, D, NN>;
    const double units = (double)kv.batch * kv.heads * ((rows + L::NQ - 1) / L::NQ) *
                         (((int64_t)kv.max_kv + L::STEP - 1) / L::STEP);
    const int full = std::min(num_sms() * L::CTAS, kPgMaxCtas);
    return units < full ? std::max((int)units, 1) : full;
}

template <int BITS, int D, int NN>
static cudaError_t launch_pg_t(PagedParams p, void *workspace, cudaStream_t st) {
    using L = PgLayout<BITS, D, NN>;
    const void *kfn = reinterpret_cast<const void *>(paged_decode_kernel<BITS, D, NN>);
    cudaError_t e = allow_smem(kfn, L::BYTES);
    if (e == cudaSuccess) e = prefer_max_shared(kfn);
    if (e != cudaSuccess) return e;
    const int64_t rows = std::min<int64_t>((int64_t)p.rep * p.kv.max_q, p.split);
    const int grid = pg_grid<BITS, D, NN>(p.kv, rows);
    p.cuts = static_cast<PgCut *>(workspace);
    p.part = reinterpret_cast<float *>(p.cuts + kPgMaxCtas);
    const int64_t nrg = (rows + L::NQ - 1) / L::NQ;
    const int64_t segs = nrg * p.kv.heads, all_segs = segs * p.kv.batch;
    // no more joins than segments, and none without a cut: the smaller index
    p.by_seg = all_segs <= grid;
    p.segs = (int)std::min<int64_t>(segs, 0x7fffffff);
    e = launch_pdl(kfn, (unsigned)grid, kPgWarps * kWarp, L::BYTES, st, p);
    if (e != cudaSuccess) return e;
    if (grid == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.by_seg ? all_segs : grid), (unsigned)std::min<int64_t>(L::NQ, rows));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, L::NQ>, p);
}

#define GWA_PG_ALL(X)                                                     \
    X(4, 64, 1) X(4, 64, 2) X(4, 64, 4) X(4, 128, 1) X(4, 128, 2)         \
    X(4, 128, 4) X(4, 256, 1) X(4, 256, 2) X(8, 64, 1) X(8, 64, 2)        \
    X(8, 64, 4) X(8, 128, 1) X(8, 128, 2) X(8, 128, 4) X(8, 256, 1) X(8, 256, 2)

// Rows (new tokens x query heads of a KV head) up to which a sequence goes to
// the few-row kernel.  That kernel against the prompt kernel, u4, eight KV
// heads, us: heads of 128, one sequence of 4096 keys, 32 rows 20.0 : 25.7, 64
// rows 24.0 : 25.6; one of 32768, 32 rows 49.5 : 55.2, 64 rows 73.3 : 55.5;
// 16 of 4096, 16 rows 45 : 86, 32 rows 91 : 86, 64 rows 155 : 87.  Heads of
// 256 (two KV heads), where the prompt kernel has one row tile: one sequence
// of 4096, 64 rows 18 : 49; one of 32768, 48 : 77; 16 of 4096, 32 rows 51 :
// 60, 64 rows 78 : 61.
static int pg_split_rows(int dim) { return dim == 256 ? 64 : 32; }

// Whether a batch can have sequences on either side.
static int pg_split(const KvView &kv, int rep) {
    const int64_t rows = (int64_t)rep * kv.max_q;
    const int most = pg_split_rows(kv.dim);
    if (rows <= most) return (int)rows;  // no prompts
    return kv.batch == 1 ? 0 : most;     // a prompt alone, or both
}

double sdpa_paged_units(int Hq, const KvView &kv) {
    const int rep = Hq / kv.heads, split = pg_split(kv, rep);
    const int rows = (int)std::min<int64_t>((int64_t)rep * kv.max_q, split);
    const int nq = 8 * pg_nn(rows, kv.dim);
    // every layout's step is 128 keys
    const double steps = (double)kv.max_pages * (1 << kv.page_shift) / 128 + 1 + kPgHead;
    const double few = (double)kv.batch * kv.heads * ((rows + nq - 1) / nq) * steps;
    return std::max(few, paged_prefill_units(kv, rep, split));
}

size_t sdpa_paged_workspace_bytes(int Hq, const KvView &kv) {
    const int rep = Hq / kv.heads, split = pg_split(kv, rep);
    const int64_t rows = std::min<int64_t>((int64_t)rep * kv.max_q, split);
    const int nn = pg_nn(rows, kv.dim);
    size_t few = 0;
#define GWA_PG(BB, DD, N)                                                              \
    if (kv.bits == BB && kv.dim == DD && nn == N)                                      \
        few = (size_t)pg_grid<BB, DD, N>(kv, rows) * 2 * 8 * nn * (kv.dim + 4) * sizeof(float);
    GWA_PG_ALL(GWA_PG)
#undef GWA_PG
    const size_t many =
        (int64_t)rep * kv.max_q > split ? paged_prefill_workspace_bytes(kv, rep) : 0;
    return kPgMaxCtas * sizeof(PgCut) + std::max(few, many);
}

cudaError_t launch_sdpa_paged(const uint16_t *q, int64_t q_stride, int Hq,
                              const KvView &kv, float scale, int causal,
                              uint16_t *out, void *workspace, int32_t *status,
                              cudaStream_t st) {
    PagedParams p{};
    p.q = q;
    p.q_stride = q_stride;
    p.Hq = Hq;
    p.rep = Hq / kv.heads;
    p.kv = kv;
    p.scale = scale;
    p.causal = causal;
    p.out = out;
    p.status = status;
    p.split = pg_split(kv, p.rep);
    const int64_t all = (int64_t)p.rep * kv.max_q;
    cudaError_t e = cudaSuccess;
    if (p.split > 0) {
        const int nn = pg_nn(std::min<int64_t>(all, p.split), kv.dim);
        e = cudaErrorInvalidValue;
#define GWA_PG(BB, DD, N) \
    if (kv.bits == BB && kv.dim == DD && nn == N) e = launch_pg_t<BB, DD, N>(p, workspace, st);
        GWA_PG_ALL(GWA_PG)
#undef GWA_PG
    }
    if (e == cudaSuccess && all > p.split) e = launch_paged_prefill(p, workspace, st);
    return e;
}

}  // namespace gwa
