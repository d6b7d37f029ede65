// Softmax attention over the paged 4-bit (or 8-bit) KV cache for prompts and
// chunks of them, on the 5th-generation tensor cores (tcgen05).  The same
// operation as paged_attention.cu, for the sequences with many query rows
// (new tokens x query heads of a KV head), where the work is a pair of dense
// products and the bytes of the cache are few.
//
// A CTA holds a block of MT * 128 rows of one (sequence, KV head) and goes
// over the keys in steps of 64:
//   S = Q K'^T   (M = 128 rows, N = 64 keys; Q and K' in shared memory)
//   P = 2^(S f - m), written to tensor memory over S as fp16
//   O += P V'    (M = 128 rows, N = head_dim; P from tensor memory, V'
//                transposed in shared memory)
// with the running maximum m and sum per row in fp32, one thread to a row; m
// moves only when a step's maximum passes it by 8 (weights up to 2^8, held
// times 2^7), and then O is rescaled in tensor memory.  Each row tile has two score buffers,
// and its scores run two steps ahead of its values, so the tensor cores and
// the softmax of one row tile overlap.
//
// Operands.  u4 keys enter exactly, as the prefill projections' weights do:
// scale * (code - 8) has at most 11 significant bits and is exact in fp16, and
// the rest of the affine map, b' = b + 8 s per group, goes into 16 further
// columns as fp16 hi and lo parts against those of the queries' group sums.
// (u8: scale * (code - 128) has up to 15 bits and is rounded to 11, relative
// 2^-11; two exact parts would double the products.)  Values enter as fp16
// s c + b, rounded once, 2^-11 of a value, and weights as fp16.  A
// query row is scaled by a power of two, and each tile's keys and values by
// one each.  The keys' comes back in the row's factor f; the values' puts the
// largest that the block has met so far into [2^14, 2^15), and where it falls,
// O is rescaled as for the maximum.  Values down to 2^-28 of that largest keep
// their 11 bits, whether a row sees the largest or not; smaller ones are
// rounded to 2^-39 of it.
//
// Warps: 0 and 1 issue the MMAs (a thread each); 2 and 3 turn the keys' and
// the values' parameters into fp16 on the tile's power of two; 4-7 and
// 8-11 are the softmax of row tiles 0 and 1 (with one row tile of 256
// dimensions 4-7 alone), they also load and convert the queries and write the
// output; 12-19 unpack keys and values from global memory into the operand
// tiles, the next tile's codes already in registers.  With two row tiles the
// tensor cores work on one while the softmax of the other runs; with one, the
// scores of the next tile are computed ahead into a second buffer.
//
// The work of the batch, counted in (row block, key tile) units with the
// causal mask's empty tiles left out, is cut into equal runs, one per CTA and
// one CTA per SM, as in the few-row kernel; cut blocks are joined by a second
// kernel.  Every wait is bounded (2 s): a wait that runs out is counted and
// the kernel unwinds without hanging.
//
// Measured: 2048 tokens of 40 heads of 128 over 8192 keys (8 KV heads, u4, 301
// GFLOP) 354 us, 850 TFLOP/s; ragged prompts of up to 1100 tokens, 16 heads of
// 256 over 1733 keys, 128.5 us.  Bound: instructions and the latency from one
// role to the next.  A step of 64 keys and 256 rows takes 2750 cycles; its
// MMAs take 1400 (those of 64 keys run at the rate of shared memory, 49
// cycles each, the values' at the tensor cores', 64), its exponentials 1024
// on the special-function units, and issue slots are used to 64% (41% with one
// row tile).  The
// roles' loops also displace one another in the instruction caches: rolling
// the softmax's two passes over halves of the scores, which reads the scores
// twice, took 395 us to 346.  A block of 256 dimensions has one row tile, so
// nothing hides its start and end (19 thousand cycles of loading queries and
// writing rows beside 13 steps of 4500).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "mma.cuh"
#include "paged.cuh"
#include "tcgen05.cuh"

namespace gwa {

constexpr int kPfThreads = 640;
constexpr int kPfDeqWarps = 8;
constexpr int kPfDeq0 = 12;    // first unpacking warp
constexpr int kPfSlots = 4;    // tiles whose range factors are kept

static __device__ unsigned int g_prefill_timeouts;

// D[tmem] (+)= A[smem] . B[smem]^T, fp16 inputs, fp32 accumulate.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of a K-major tile of `rows` rows and 16 columns without swizzle:
// 8-row, 16-byte core matrices, the two of a row 16 * rows bytes apart.
__device__ __forceinline__ uint64_t smem_desc_ext(uint32_t saddr, int rows) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3fffu);
    d |= (uint64_t)rows << 16;  // leading: next 8 columns
    d |= (uint64_t)(128 >> 4) << 32;   // stride: next 8 rows
    d |= (uint64_t)1 << 46;
    return d;
}

// fp16 inputs, fp32 accumulators, both operands K-major, M = 128.
__device__ __forceinline__ constexpr uint32_t pf_idesc(int n) {
    return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

template <int BITS, int D>
struct PfLayout {
    static constexpr int G = D / 64;
    static constexpr int MT = D <= 128 ? 2 : 1;      // row tiles
    static constexpr int RB = 128 * MT;              // rows of a block
    static constexpr int KT = D <= 128 ? 128 : 64;   // keys of a tile
    static constexpr int NH = KT / 64;               // score steps of a tile
    static constexpr int ST = 2;                     // key and value stages
    static constexpr int RCH = D * BITS / 128;       // 16-byte chunks of a key's codes
    static constexpr int QTILE = 128 * D * 2;        // a row tile's queries
    static constexpr int TILE = KT * D * 2;          // a tile's keys, or values
    static constexpr int QEXT = 128 * 32, KEXT = KT * 32;  // their further columns
    static constexpr size_t Q_OFF = 0;
    static constexpr size_t QX_OFF = Q_OFF + (size_t)MT * QTILE;
    static constexpr size_t KX_OFF = QX_OFF + (size_t)MT * QEXT;
    static constexpr size_t K_OFF = KX_OFF + (size_t)ST * KEXT;
    static constexpr size_t V_OFF = K_OFF + (size_t)ST * TILE;
    // per slot: key scales, value scales and biases, fp16 [G][KT] each
    static constexpr int PROW = KT * 2, PAR = 3 * G * PROW;
    static constexpr size_t P_OFF = V_OFF + (size_t)ST * TILE;
    static constexpr size_t BYTES = P_OFF + (size_t)kPfSlots * PAR;
    static constexpr size_t SMEM = BYTES + 1024;     // alignment slack
    // tensor memory: two score buffers of 64 columns a row tile, then the
    // outputs
    static constexpr int O_COL = 256;
    // unpacking units of a warp: keys KB x CB chunks; values 64 keys x 32
    // dimensions
    static constexpr int KB = RCH >= 4 ? 8 : 16, CB = RCH >= 4 ? 4 : 2;
    static constexpr int KU = KT / KB * (RCH / CB) / kPfDeqWarps;
    static constexpr int VUNITS = NH * 2 * G;        // of a tile
    static constexpr int VU = (VUNITS + kPfDeqWarps - 1) / kPfDeqWarps;
    static constexpr int VW = BITS / 4;              // words of 8 dimensions
    static_assert(KU >= 1 && K_OFF % 1024 == 0 && TILE % 1024 == 0, "tiles");
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

// A row's weights are 2^(kUp + x - m), where a score x passes the running
// maximum m by up to kLazy: at most 2^15.
constexpr float kLazy = 8.f, kUp = 7.f;

// One tile's powers of two, and its keys whose value parameters are not finite.
struct PfTile {
    float k_down, v_up, v_down;
    uint32_t bad[4];  // bit l of word j: key 4 l + j
};

// What is left of a CTA's run: the block and the unit of it where it stands,
// and that unit counted over the whole batch.
struct PfCursor {
    int b, hk, rb, unit, left, at;
    KvSeq s;
    int rows, nrb;
};

// Keys that rows [rb * RB, ...) of a sequence see, in tiles of KT.
template <int RB, int KT>
__device__ __forceinline__ int pf_tiles(const PagedParams &p, const KvSeq &s, int rows, int rb) {
    const int seen = kv_seen(s, (min(rows, (rb + 1) * RB) - 1) / p.rep, p.causal);
    return seen > 0 ? (seen + KT - 1) / KT : 0;
}
template <int RB>
__device__ __forceinline__ int pf_rows(const PagedParams &p, const KvSeq &s) {
    const int rows = p.rep * min(s.count, p.kv.max_q);
    return rows > p.split ? rows : 0;
}
// Units of work.  A block's start and end (queries in, rows out) count as
// pf_head tiles in front of its own: 13 thousand cycles where a tile of 128
// keys takes 7, with one row tile 19 where a tile of 64 keys takes 4.5.  With
// tiles alone as units, CTAs that hold many short blocks were the last to
// finish (ragged prompts of 256 dimensions: 158 us, 126 with).
__host__ __device__ constexpr int pf_head(int kt) { return kt == 64 ? 4 : 2; }
template <int KT>
__device__ __forceinline__ int pf_cost(int tiles) {
    return tiles > 0 ? tiles + pf_head(KT) : 0;
}
template <int RB, int KT>
__device__ __forceinline__ int pf_units(const PagedParams &p, int b) {
    const KvSeq s = kv_seq(p.kv, b);
    const int rows = pf_rows<RB>(p, s);
    const int nrb = (rows + RB - 1) / RB;
    if (!p.causal) return p.kv.heads * nrb * pf_cost<KT>((s.len + KT - 1) / KT);
    int n = 0;
    for (int rb = 0; rb < nrb; ++rb) n += pf_cost<KT>(pf_tiles<RB, KT>(p, s, rows, rb));
    return p.kv.heads * n;
}

// A block's piece of the run: tiles [ta, tb) of nt; the block's last unit.
struct PfPiece {
    int b, hk, rb, ta, tb, nt, rows, last;
    KvSeq s;
};
template <int RB, int KT>
__device__ __noinline__ bool pf_step(const PagedParams &p, PfCursor &c, PfPiece &w) {
    while (c.left > 0) {
        int nt = pf_tiles<RB, KT>(p, c.s, c.rows, c.rb);
        while (c.unit >= pf_cost<KT>(nt)) {  // the next block that sees a key
            c.unit = 0;
            if (++c.rb >= c.nrb) {
                c.rb = 0;
                if (++c.hk >= p.kv.heads || c.nrb == 0) {
                    c.hk = 0;
                    do {
                        // (never past the batch, unless the lengths change meanwhile)
                        if (++c.b >= p.kv.batch) return false;
                        c.s = kv_seq(p.kv, c.b);
                        c.rows = pf_rows<RB>(p, c.s);
                        c.nrb = (c.rows + RB - 1) / RB;
                    } while (c.nrb == 0);
                }
            }
            nt = pf_tiles<RB, KT>(p, c.s, c.rows, c.rb);
        }
        const int cost = pf_cost<KT>(nt), head = cost - nt;
        const int from = c.unit, to = min(cost, from + c.left);
        w.last = c.at - from + cost - 1;
        c.left -= to - from;
        c.at += to - from;
        c.unit = to;
        if (to <= head) continue;  // none of its tiles
        w.b = c.b;
        w.hk = c.hk;
        w.rb = c.rb;
        w.ta = max(from - head, 0);
        w.tb = to - head;
        w.nt = nt;
        w.rows = c.rows;
        w.s = c.s;
        return true;
    }
    return false;
}

// Rows (of one head) of a tile's 16-key blocks, on the first lanes.
template <int KT>
struct PfPages {
    const PagedParams &p;
    int len, tb, hk, b;
    __device__ __forceinline__ int64_t look(int tile, int lane) const {
        const int key = tile * KT + lane * 16;
        int pg = 0;
        if (tile < tb && lane < KT / 16 && key < len) {
            pg = p.kv.page_table[(int64_t)b * p.kv.max_pages + (key >> p.kv.page_shift)];
            if ((unsigned)pg >= (unsigned)p.kv.num_pages) {
                if (p.status) atomicOr(p.status, (int)kKvBadPage);
                pg = 0;
            }
        }
        return (((int64_t)pg * p.kv.heads + hk) << p.kv.page_shift) +
               (key & ((1 << p.kv.page_shift) - 1));
    }
};

// The next piece of a warp's own walk through the run, in shared memory (the
// walk is the same for every warp; registers are short).
template <int RB, int KT>
__device__ __forceinline__ bool pf_next(const PagedParams &p, PfCursor *c, PfPiece *w, int lane) {
    __syncwarp();
    int more = 0;
    if (lane == 0) more = pf_step<RB, KT>(p, *c, *w);
    more = __shfl_sync(0xffffffffu, more, 0);
    __syncwarp();
    return more != 0;
}

// The bounded wait, out of line: the roles' loops are short of instruction
// cache.
__device__ __noinline__ bool pf_wait(uint64_t *bar, uint32_t parity, int *fail) {
    if (mbar_wait_sleep(bar, parity)) return true;
    atomicAdd(&g_prefill_timeouts, 1u);
    *fail = 1;
    return false;
}

template <int BITS, int D>
__global__ void __launch_bounds__(kPfThreads, 1) paged_prefill_kernel(PagedParams p) {
    using L = PfLayout<BITS, D>;
    constexpr int G = L::G, MT = L::MT, RB = L::RB, ST = L::ST, KT = L::KT, NH = L::NH;
    constexpr float KC = BITS == 4 ? 8.f : 128.f;
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ __align__(1024) unsigned char pf_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(pf_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ uint64_t kfull[ST], vfull[ST];
    __shared__ uint64_t sfull[MT][2], pfull[MT][2], odone[MT][2], ofree[MT], qfull[MT];
    __shared__ PfTile s_tile[kPfSlots];
    __shared__ PfCursor s_cur[kPfThreads / 32];
    __shared__ PfPiece s_piece[kPfThreads / 32], s_soft[8][2];
    __shared__ uint64_t rfull[kPfSlots], rempty[kPfSlots];
    __shared__ int s_quot, s_rest;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail;

    const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&kfull[i], kPfDeqWarps + 1);
            mbar_init(&vfull[i], kPfDeqWarps);
        }
        for (int i = 0; i < 2 * MT; ++i) {
            mbar_init(&sfull[i / 2][i % 2], 1);
            mbar_init(&odone[i / 2][i % 2], 1);
            mbar_init(&pfull[i / 2][i % 2], 4);
        }
        for (int i = 0; i < MT; ++i) {
            mbar_init(&ofree[i], 4);
            mbar_init(&qfull[i], 4);
        }
        for (int i = 0; i < kPfSlots; ++i) {
            mbar_init(&rfull[i], 2);
            mbar_init(&rempty[i], MT);
        }
        fence_mbar_init();
        s_fail = 0;
        pdl_launch_dependents();
    }
    if (warp == 0) tmem_alloc(&s_tmem, 512);
    pdl_wait_primary();
    const int cta = blockIdx.x, B = p.kv.batch;
    // ---- this CTA's run
    if (warp == 1) {
        int64_t units = 0;
        for (int b0 = 0; b0 < B; b0 += 32)
            units += b0 + lane < B ? pf_units<RB, KT>(p, b0 + lane) : 0;
        const int total = pg_total(units);
        const int ctas = min((int)gridDim.x, total);
        const int quot = ctas ? total / ctas : 0, rest = ctas ? total % ctas : 0;
        const int begin = pg_start(quot, rest, cta), end = pg_start(quot, rest, cta + 1);
        int at = 0, b = 0;
        for (int b0 = 0; b0 < B; b0 += 32) {
            const int u = b0 + lane < B ? pf_units<RB, KT>(p, b0 + lane) : 0;
            int incl = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
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
            at += __shfl_sync(FULL, incl, 31);
        }
        PfCursor c{};
        {
            c.left = cta < ctas ? end - begin : 0;
            if (c.left > 0) {
                c.b = b;
                c.s = kv_seq(p.kv, b);
                c.rows = pf_rows<RB>(p, c.s);
                c.nrb = (c.rows + RB - 1) / RB;
                const int head = pf_units<RB, KT>(p, b) / p.kv.heads;
                c.hk = (begin - at) / head;
                int in = (begin - at) - c.hk * head;
                for (int n; in >= (n = pf_cost<KT>(pf_tiles<RB, KT>(p, c.s, c.rows, c.rb))); ++c.rb) in -= n;
                c.unit = in;
                c.at = begin;
            }
        }
        if (lane < kPfThreads / 32) s_cur[lane] = c;
        if (lane == 0) {
            s_quot = quot;
            s_rest = rest;
            p.cuts[cta].slot = -1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    PfCursor *const cur = &s_cur[warp];
    const PfPiece &w = s_piece[warp];

    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_try_wait(bar, parity) || pf_wait(bar, parity, &s_fail);
    };

    if (warp < 2) {
        // ------------------------------------------------ MMA issuers
        // Two row tiles: a warp each issues a tile's scores and values.  One:
        // warp 0 issues the scores, warp 1 the values.  (A thread spends 50 to
        // 100 cycles on an MMA or a commit, so one for all of them was the
        // last to finish.)
        if (lane == 0) {
            constexpr uint32_t id_s = pf_idesc(64), id_o = pf_idesc(D);
            const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + L::Q_OFF));
            const uint64_t k_desc = smem_desc_sw128(smem_u32(smem + L::K_OFF));
            const uint64_t v_desc = smem_desc_sw128(smem_u32(smem + L::V_OFF));
            const uint64_t qx_desc = smem_desc_ext(smem_u32(smem + L::QX_OFF), 128);
            const uint64_t kx_desc = smem_desc_ext(smem_u32(smem + L::KX_OFF), KT);
            const int r = MT == 2 ? warp : 0;
            uint32_t n = 0;       // tiles so far
            uint32_t nr = 0;      // score steps of this row tile
            uint32_t pieces = 0;  // blocks of this row tile
            bool ok = true;
            // step j of a piece: scores against 64 keys into buffer s
            auto scores = [&](int j) {
                const uint32_t tile = n + j / NH;
                const int st = tile % ST, h = j % NH, s = (nr + j) & 1;
                if (h == 0 && !wait(&kfull[st], (tile / ST) & 1)) return false;
                // issued by another thread than the values: the buffer's last
                // weights are used
                if (MT == 1 && nr + j >= 2 && !wait(&odone[0][s], (((nr + j) >> 1) - 1) & 1))
                    return false;
                tc_fence_after();
                const uint32_t d = tmem + r * 128 + s * 64;
                const uint64_t a = q_desc + (uint64_t)((r * L::QTILE) >> 4);
                const uint64_t b = k_desc + (uint64_t)((st * L::TILE + h * 8192) >> 4);
                tc_mma_ss(d, qx_desc + (uint64_t)((r * L::QEXT) >> 4),
                          kx_desc + (uint64_t)((st * L::KEXT + h * 1024) >> 4), id_s, 0u);
#pragma unroll
                for (int k = 0; k < 4 * G; ++k)
                    tc_mma_ss(d, a + (k / 4) * 1024 + 2 * (k % 4), b + (k / 4) * (KT * 8) + 2 * (k % 4),
                              id_s, 1u);
                tc_commit(&sfull[r][s]);
                return true;
            };
            // step j: weights in buffer s times the values of its 64 keys
            auto values = [&](int j, int steps) {
                const uint32_t tile = n + j / NH;
                const int st = tile % ST, h = j % NH, s = (nr + j) & 1;
                if (h == 0 && !wait(&vfull[st], (tile / ST) & 1)) return false;
                if (!wait(&pfull[r][s], ((nr + j) >> 1) & 1)) return false;
                if (j == 0 && pieces > 0 && !wait(&ofree[r], (pieces - 1) & 1)) return false;
                tc_fence_after();
                const uint32_t d = tmem + L::O_COL + r * D, a = tmem + r * 128 + s * 64;
                const uint64_t b = v_desc + (uint64_t)((st * L::TILE + h * D * 128) >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_ts(d, a + k * 8, b + 2 * k, id_o, j == 0 && k == 0 ? 0u : 1u);
                // two row tiles: scores of step j + 2, issued after these, tell
                // of them as well, but at the end
                if (MT == 1)
                    tc_commit(&odone[0][s]);
                else if (j + 2 >= steps)
                    tc_commit(&odone[r][steps - 1 - j]);
                if (h == NH - 1) tc_commit(&rempty[tile % kPfSlots]);
                return true;
            };
            while (ok && pf_step<RB, KT>(p, *cur, s_piece[warp])) {
                const int nlive = min(RB, w.rows - w.rb * RB);
                const int tiles = w.tb - w.ta, steps = tiles * NH;
                if (MT == 2 && warp * 128 >= nlive) {
                    // no rows here: the stages are free as soon as they are full
                    for (int i = 0; ok && i < tiles; ++i, ++n) {
                        ok = wait(&kfull[n % ST], (n / ST) & 1);
                        ok = ok && wait(&vfull[n % ST], (n / ST) & 1);
                        if (ok) mbar_arrive(&rempty[n % kPfSlots]);
                    }
                    continue;
                }
                if (MT == 2 || warp == 0) ok = wait(&qfull[r], pieces & 1);
                // scores run two steps ahead of the values
                for (int j = -2; ok && j < steps; ++j) {
                    if (j >= 0 && (MT == 2 || warp == 1)) ok = values(j, steps);
                    if (ok && j + 2 < steps && (MT == 2 || warp == 0)) ok = scores(j + 2);
                }
                n += tiles;
                nr += steps;
                ++pieces;
            }
        }
    } else if (warp >= 4 && warp < 4 + 4 * MT) {
        // ------------------------------------------------ softmax of a row tile
        const int r = (warp - 4) / 4;              // row tile
        const int q4 = warp & 3;                   // tensor-memory lane quarter
        const int row = q4 * 32 + lane;            // of the tile
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint32_t t_o = tmem + L::O_COL + r * D + lane_off;
        uint32_t n = 0, nr = 0;  // tiles so far: of the CTA, of this row tile
        int pieces = 0, piece = 0;
        int longer = 0;          // of the pieces, those of two steps and more
        bool ok = true;
        int turn = 0;
        bool more = pf_next<RB, KT>(p, cur, &s_soft[warp - 4][0], lane);
        for (; ok && more; turn ^= 1) {
            const PfPiece &w = s_soft[warp - 4][turn];
            more = false;
            const int nlive = min(RB, w.rows - w.rb * RB);
            const int tiles = w.tb - w.ta;
            if (r * 128 >= nlive) {
                more = pf_next<RB, KT>(p, cur, &s_soft[warp - 4][turn ^ 1], lane);
            } else {
                // ---- the row's queries: fp16 at a power of two, the group
                // sums in the further columns.  The warp copies its 32 rows
                // into the tile as they are, whole rows at a time; then each
                // thread converts its own row in place.
                const int i_blk = r * 128 + row;
                const bool live = i_blk < nlive;
                const int rr = w.rb * RB + (live ? i_blk : 0);
                const int tok = rr / p.rep, head = w.hk * p.rep + rr % p.rep;
                const uint16_t *src = p.q + (int64_t)(w.s.first + tok) * p.q_stride + (int64_t)head * D;
                unsigned char *const qt = smem + L::Q_OFF + (size_t)r * L::QTILE;
                // chunk c (16 bytes) of a row of the tile
                auto q_at = [&](int row_, int c) {
                    return qt + (c >> 3) * 16384 + row_ * 128 + (((c & 7) ^ (row_ & 7)) * 16);
                };
                constexpr int CR = D / 8, RPI = 32 / CR;  // chunks of a row, rows at a time
#pragma unroll 4
                for (int it = 0; it < 32 / RPI; ++it) {
                    const int from = it * RPI + lane / CR, c = lane % CR;
                    const uint16_t *ptr = reinterpret_cast<const uint16_t *>(
                        __shfl_sync(FULL, reinterpret_cast<unsigned long long>(src), from));
                    unsigned char *dst = q_at(q4 * 32 + from, c);
                    if (r * 128 + q4 * 32 + from < nlive)
                        cp_async<16>(dst, ptr + c * 8);
                    else
                        *reinterpret_cast<uint4 *>(dst) = make_uint4(0u, 0u, 0u, 0u);
                }
                cp_async_commit();
                cp_async_wait<0>();
                __syncwarp();
                float mx = 0.f, sum[G];
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    sum[g] = 0.f;
#pragma unroll 2
                    for (int c = 0; c < 8; ++c) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(q_at(row, g * 8 + c));
                        const uint32_t uw[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = bf16_lo(uw[k]), b = bf16_hi(uw[k]);
                            mx = fmaxf(mx, fmaxf(fabsf(a), fabsf(b)));
                            sum[g] += a + b;
                        }
                    }
                    mx = fmaxf(mx, fabsf(sum[g]));
                }
                float up, down;
                range_scale(mx, up, down);
                if (p.scale < 0.f) up = -up;  // factors are kept non-negative
#pragma unroll 2
                for (int c = 0; c < CR; ++c) {
                    uint4 *at = reinterpret_cast<uint4 *>(q_at(row, c));
                    const uint4 u = *at;
                    float v[8];
                    v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x);
                    v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
                    v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z);
                    v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] *= up;
                    // the order in which the keys' codes unpack
                    if constexpr (BITS == 4)
                        *at = make_uint4(pack_f16(v[0], v[4]), pack_f16(v[1], v[5]),
                                         pack_f16(v[2], v[6]), pack_f16(v[3], v[7]));
                    else
                        *at = make_uint4(pack_f16(v[0], v[2]), pack_f16(v[1], v[3]),
                                         pack_f16(v[4], v[6]), pack_f16(v[5], v[7]));
                }
                {
                    // per group (hi, lo, hi) against the keys' (hi, hi, lo)
                    float e[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) e[k] = 0.f;
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        const float x = sum[g] * up, hi = __half2float(__float2half_rn(x));
                        e[3 * g] = e[3 * g + 2] = hi;
                        e[3 * g + 1] = x - hi;
                    }
                    unsigned char *qx = smem + L::QX_OFF + (size_t)r * L::QEXT + (row >> 3) * 128 + (row & 7) * 16;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<uint4 *>(qx + k * 2048) =
                            make_uint4(pack_f16(e[8 * k], e[8 * k + 1]), pack_f16(e[8 * k + 2], e[8 * k + 3]),
                                       pack_f16(e[8 * k + 4], e[8 * k + 5]), pack_f16(e[8 * k + 6], e[8 * k + 7]));
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&qfull[r]);
                // the next piece, while this one's scores start
                more = pf_next<RB, KT>(p, cur, &s_soft[warp - 4][turn ^ 1], lane);

                const float fac = down * fabsf(p.scale) * 1.4426950408889634f;
                const int lim = live ? kv_seen(w.s, tok, p.causal) : w.s.len;
                const int least = __reduce_min_sync(FULL, lim);
                float m = -INFINITY, l = 0.f, v_up = 0.f, v_down = 1.f;
                const int steps = tiles * NH;
                for (int i = 0; ok && i < steps; ++i) {
                    const uint32_t at = nr + i;  // step of this row tile
                    const int s = at & 1;
                    const uint32_t t_s = tmem + r * 128 + s * 64 + lane_off;
                    ok = __all_sync(FULL, wait(&sfull[r][s], (at >> 1) & 1));
                    if (!ok) break;
                    tc_fence_after();
                    const PfTile &pt = s_tile[(n + i / NH) % kPfSlots];
                    // (never zero, so that a masked score stays -inf: a factor
                    // below leaves every score at zero either way)
                    const float f = fmaxf(fac * pt.k_down, 1e-37f);
                    const int key0 = w.ta * KT + i * 64;
                    const int n_in = key0 + 64 > least ? lim - key0 : 64;
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int c = 0; c < 64; c += 32) {
                        float v[32];
                        tc_ld32_async(t_s + c, v);
                        tc_ld_wait(v);
                        if (key0 + c + 32 > least) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (k + c >= n_in) v[k] = -INFINITY;
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 2) mx = fmaxf(mx, fmaxf(v[k], v[k + 1]));
                    }
                    mx *= f;
                    // ---- rescale
                    float corr = 1.f;
                    if (mx > m + kLazy) {
                        corr = m == -INFINITY ? 0.f : ex2(m - mx);
                        m = mx;
                        l *= corr;
                    }
                    if (i == 0) {
                        v_up = pt.v_up;
                        v_down = pt.v_down;
                        corr = 1.f;
                    } else {
                        if (pt.v_up != v_up) {
                            corr *= pt.v_up * v_down;
                            v_up = pt.v_up;
                            v_down = pt.v_down;
                        }
                        if (__any_sync(FULL, corr != 1.f)) {
                            // the previous step's values are in
                            if (MT == 1)
                                ok = wait(&odone[0][s ^ 1], ((at - 1) >> 1) & 1);
                            else if (i + 1 < steps)
                                ok = wait(&sfull[r][s ^ 1], ((at + 1) >> 1) & 1);
                            else
                                ok = wait(&odone[r][1], longer & 1);
                            ok = __all_sync(FULL, ok);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D; c += 16) {
                                float x[16];
                                uint32_t o[16];
                                tc_ld16(t_o + c, x);
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(x[k] * corr);
                                tc_st16(t_o + c, o);
                            }
                            tc_wait_st();
                        }
                    }
                    // ---- weights
                    // (times 2^7, as their sum: up to 2^15, so that weights
                    // down to 2^-32 of the largest are not lost in fp16)
                    const float sub = m == -INFINITY ? 0.f : m - kUp;
                    const float2 f2 = make_float2(f, f), s2 = make_float2(-sub, -sub);
                    float2 acc = make_float2(0.f, 0.f);
#pragma unroll 1
                    for (int c = 0; c < 64; c += 32) {
                        float v[32];
                        uint32_t o[16];
                        tc_ld32_async(t_s + c, v);
                        tc_ld_wait(v);
                        if (key0 + c + 32 > least) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (k + c >= n_in) v[k] = -INFINITY;
                        }
#pragma unroll
                        for (int k = 0; k < 32; k += 2) {
                            float2 x = fma2(make_float2(v[k], v[k + 1]), f2, s2);
                            x = make_float2(ex2(x.x), ex2(x.y));
                            acc = add2(acc, x);
                            o[k / 2] = pack_f16(x.x, x.y);
                        }
                        tc_st16(t_s + c / 2, o);
                    }
                    l += acc.x + acc.y;
                    if (pt.bad[0] | pt.bad[1] | pt.bad[2] | pt.bad[3]) {
                        // a value that is not finite leaves the products; the
                        // rows that see it are not finite either
                        for (int k = 0; k < 64; ++k) {
                            const int x = (i % NH) * 64 + k;
                            if ((pt.bad[x & 3] >> (x >> 2)) & 1 && key0 + k < lim) l = NAN;
                        }
                    }
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&pfull[r][s]);
                }
                nr += steps;
                // ---- out
                if (ok)
                    ok = __all_sync(FULL, MT == 1 ? wait(&odone[0][(nr - 1) & 1], ((nr - 1) >> 1) & 1)
                                                  : wait(&odone[r][0], pieces & 1));
                if (steps > 1) ++longer;
                if (ok) {
                    tc_fence_after();
                    const bool whole = w.ta == 0 && w.tb == w.nt;
                    // (l first, the values' power second: both stay in range)
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    // the rows leave through the (free) query tile, whole rows at
                    // a time: bf16 at once, fp32 pieces in two halves
                    float *part = p.part + ((int64_t)(2 * cta + piece) * RB + i_blk) * (D + 4);
                    uint16_t *o_row = p.out + ((int64_t)(w.s.first + tok) * p.Hq + head) * D;
                    auto flush = [&](void *mine) {
                        __syncwarp();
#pragma unroll 4
                        for (int it = 0; it < 32 / RPI; ++it) {
                            const int from = it * RPI + lane / CR, c = lane % CR;
                            uint4 *dst = reinterpret_cast<uint4 *>(
                                __shfl_sync(FULL, reinterpret_cast<unsigned long long>(mine), from));
                            const uint4 u = *reinterpret_cast<const uint4 *>(q_at(q4 * 32 + from, c));
                            if (r * 128 + q4 * 32 + from < nlive) dst[c] = u;
                        }
                        __syncwarp();
                    };
                    if (whole) {
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            float x[16];
                            tc_ld16(t_o + c * 16, x);
#pragma unroll
                            for (int k = 0; k < 16; ++k) x[k] = x[k] * inv * v_down;
                            *reinterpret_cast<uint4 *>(q_at(row, 2 * c)) =
                                make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                           pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
                            *reinterpret_cast<uint4 *>(q_at(row, 2 * c + 1)) =
                                make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]),
                                           pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
                        }
                        flush(o_row);
                    } else {
#pragma unroll 1
                        for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                float x[16];
                                tc_ld16(t_o + h * (D / 2) + c * 16, x);
#pragma unroll
                                for (int k = 0; k < 16; k += 4)
                                    *reinterpret_cast<float4 *>(q_at(row, 4 * c + k / 4)) =
                                        make_float4(x[k] * inv * v_down, x[k + 1] * inv * v_down,
                                                    x[k + 2] * inv * v_down, x[k + 3] * inv * v_down);
                            }
                            flush(part + h * (D / 2));
                        }
                        if (live) part[D] = l == 0.f ? -INFINITY : m + __log2f(l);
                    }
                    if (r == 0 && row == 0 && w.ta == 0 && !whole) {
                        const int last = pg_owner(s_quot, s_rest, w.last);
                        p.cuts[cta] = PgCut{2 * cta + piece, cta, last - cta + 1, w.s.first,
                                            w.hk * p.rep, w.rb * RB, nlive, 0};
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ofree[r]);
                ++pieces;
            }
            n += tiles;
            piece = 1;
        }
    } else if (warp == 2 || warp == 3) {
        // ------------------------------------------------ parameters
        // Warp 2 the keys', warp 3 the values': a tile's power of two, then
        // its parameters on that scale as fp16; the keys' further columns.
        const bool is_k = warp == 2;
        const uint32_t *src = is_k ? p.kv.kp : p.kv.vp;
        uint32_t n = 0;
        bool ok = true;
        while (ok && pf_next<RB, KT>(p, cur, &s_piece[warp], lane)) {
            const PfPages<KT> pages{p, w.s.len, w.tb, w.hk, w.b};
            float v_lim = -1.f, up = 1.f, down = 1.f;
            uint32_t x[4][G];  // keys 4 lane + j
            auto load = [&](int64_t base, int tile) {
                const int64_t row = __shfl_sync(FULL, base, lane >> 2) + (lane & 3) * 4;
                const int left = min(KT, w.s.len - tile * KT);
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int g = 0; g < G; ++g)
                        x[j][g] = 4 * lane + j < left ? src[(row + j) * G + g] : 0u;
            };
            int64_t base = pages.look(w.ta, lane);
            load(base, w.ta);
            base = pages.look(w.ta + 1, lane);
            for (int tile = w.ta; ok && tile < w.tb; ++tile, ++n) {
                const uint32_t slot = n % kPfSlots;
                float t = 0.f;
                uint32_t bad = 0u;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int g = 0; g < G; ++g) {
                        // a quarter of KC |scale| + |b'|: below 2^127 where the
                        // group's values are finite
                        const float s = 0.25f * KC * bf16_lo(x[j][g]);
                        const float e = fabsf(s) + fabsf(fmaf(0.25f, bf16_hi(x[j][g]), s));
                        if (e < 0x1p127f) {
                            t = fmaxf(t, e);
                        } else {
                            bad |= 1u << j;
                            // a value that is not finite does not enter the
                            // products (the rows that see it are told)
                            if (!is_k) x[j][g] = 0u;
                        }
                    }
                t = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(t)));
                if (is_k || t > v_lim) {
                    // into [2^14, 2^15).  The values' power only falls within
                    // a block (were it to rise by as much as the values may
                    // shrink, the outputs so far could leave fp32's range).
                    range_scale(t, up, down);
                    up *= 0.25f;
                    down *= 4.f;
                    v_lim = t > 0.f ? 8192.f * down : -1.f;
                }
                if (n >= kPfSlots) {
                    ok = __all_sync(FULL, wait(&rempty[slot], ((n / kPfSlots) & 1) ^ 1));
                    if (!ok) break;
                }
                unsigned char *par = smem + L::P_OFF + slot * L::PAR + lane * 8;
                const bool mine = lane < KT / 4;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    if (!mine) break;
                    float s[4], b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // (value codes enter as code / KC)
                        s[j] = bf16_lo(x[j][g]) * (is_k ? 1.f : KC) * up;
                        b[j] = bf16_hi(x[j][g]) * up;
                    }
                    if (is_k) {
                        *reinterpret_cast<uint2 *>(par + g * L::PROW) =
                            make_uint2(pack_f16(s[0], s[1]), pack_f16(s[2], s[3]));
                    } else {
                        *reinterpret_cast<uint2 *>(par + (G + g) * L::PROW) =
                            make_uint2(pack_f16(s[0], s[1]), pack_f16(s[2], s[3]));
                        *reinterpret_cast<uint2 *>(par + (2 * G + g) * L::PROW) =
                            make_uint2(pack_f16(b[0], b[1]), pack_f16(b[2], b[3]));
                    }
                }
                if (is_k) {
                    if (lane == 0) s_tile[slot].k_down = down;
                } else {
                    uint32_t m[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) m[j] = __ballot_sync(FULL, (bad >> j) & 1u);
                    if (lane == 0) {
                        s_tile[slot].v_up = up;
                        s_tile[slot].v_down = down;
#pragma unroll
                        for (int j = 0; j < 4; ++j) s_tile[slot].bad[j] = m[j];
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&rfull[slot]);
                if (is_k) {
                    // b' as (hi, hi, lo) per group
                    if (n >= ST) {
                        ok = __all_sync(FULL, wait(&rempty[(n - ST) % kPfSlots], ((n - ST) / kPfSlots) & 1));
                        if (!ok) break;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (!mine) break;
                        float e[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) e[k] = 0.f;
#pragma unroll
                        for (int g = 0; g < G; ++g) {
                            const float b = fmaf(KC, bf16_lo(x[j][g]), bf16_hi(x[j][g])) * up;
                            const float hi = __half2float(__float2half_rn(b));
                            e[3 * g] = e[3 * g + 1] = hi;
                            e[3 * g + 2] = b - hi;
                        }
                        const int k = 4 * lane + j;
                        unsigned char *kx = smem + L::KX_OFF + (size_t)(n % ST) * L::KEXT + (k >> 3) * 128 + (k & 7) * 16;
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            *reinterpret_cast<uint4 *>(kx + h * (KT * 16)) =
                                make_uint4(pack_f16(e[8 * h], e[8 * h + 1]), pack_f16(e[8 * h + 2], e[8 * h + 3]),
                                           pack_f16(e[8 * h + 4], e[8 * h + 5]), pack_f16(e[8 * h + 6], e[8 * h + 7]));
                    }
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&kfull[n % ST]);
                }
                if (tile + 1 < w.tb) load(base, tile + 1);
                base = pages.look(tile + 2, lane);
            }
        }
    } else if (warp >= kPfDeq0) {
        // ------------------------------------------------ keys and values
        const int dw = warp - kPfDeq0;
        constexpr int KU = L::KU, VU = L::VU, RCH = L::RCH, VW = L::VW;
        constexpr int KBS = KT / L::KB;  // key blocks of a tile
        const int kl = RCH >= 4 ? lane & 7 : (lane & 7) + 8 * (lane >> 4);  // key of a key unit
        const int kc = RCH >= 4 ? lane >> 3 : (lane >> 3) & 1;              // chunk of it
        const int vc = lane & 7, vd = lane >> 3;  // 8 keys and 8 dimensions of a value unit
        uint32_t n = 0;
        bool ok = true;
        while (ok && pf_next<RB, KT>(p, cur, &s_piece[warp], lane)) {
            const PfPages<KT> pages{p, w.s.len, w.tb, w.hk, w.b};
            uint4 kreg[KU];
            uint32_t vreg[VU][8][VW];
            auto load_k = [&](int64_t base, int tile) {
                const int left = min(KT, w.s.len - tile * KT);  // keys of the tile
#pragma unroll
                for (int u = 0; u < KU; ++u) {
                    const int id = dw + u * kPfDeqWarps;
                    const int k = id % KBS * L::KB + kl, c = id / KBS * L::CB + kc;
                    const int64_t row = __shfl_sync(FULL, base, k >> 4) + (k & 15);
                    kreg[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (k < left) kreg[u] = reinterpret_cast<const uint4 *>(p.kv.kq)[row * RCH + c];
                }
            };
            auto load_v = [&](int64_t base, int tile) {
                const int left = min(KT, w.s.len - tile * KT);
#pragma unroll
                for (int u = 0; u < VU; ++u) {
                    const int id = dw + u * kPfDeqWarps;  // half, then 32 dimensions
                    const int k0 = id % NH * 64 + vc * 8, d32 = id / NH;
                    const int64_t row = __shfl_sync(FULL, base, k0 >> 4) + (k0 & 15);
                    const uint32_t *src = p.kv.vq + row * (D * BITS / 32) + d32 * BITS + vd * VW;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
#pragma unroll
                        for (int x = 0; x < VW; ++x) vreg[u][j][x] = 0u;
                        if (id < L::VUNITS && k0 + j < left) {
                            if constexpr (VW == 1) {
                                vreg[u][j][0] = src[j * (D * BITS / 32)];
                            } else {
                                const uint2 t = *reinterpret_cast<const uint2 *>(src + j * (D * BITS / 32));
                                vreg[u][j][0] = t.x;
                                vreg[u][j][1] = t.y;
                            }
                        }
                    }
                }
            };
            int64_t base = pages.look(w.ta, lane);
            load_k(base, w.ta);
            load_v(base, w.ta);
            base = pages.look(w.ta + 1, lane);
            for (int tile = w.ta; ok && tile < w.tb; ++tile, ++n) {
                const int st = n % ST;
                const uint32_t slot = n % kPfSlots;
                const unsigned char *par = smem + L::P_OFF + slot * L::PAR;
                ok = __all_sync(FULL, wait(&rfull[slot], (n / kPfSlots) & 1));
                // ---- keys: scale (code - centre), exact
                if (ok && n >= ST)
                    ok = __all_sync(FULL, wait(&rempty[(n - ST) % kPfSlots], ((n - ST) / kPfSlots) & 1));
                if (!ok) break;
                unsigned char *kt = smem + L::K_OFF + (size_t)st * L::TILE;
                {
                    __half2 s2[KU];
                    unsigned char *dst[KU];
                    int sw[KU];  // chunk of the row's 128 bytes, swizzled
                    constexpr int OUT = BITS == 4 ? 4 : 2;  // 16-byte chunks out of one in
#pragma unroll
                    for (int u = 0; u < KU; ++u) {
                        const int id = dw + u * kPfDeqWarps;
                        const int k = id % KBS * L::KB + kl, c = id / KBS * L::CB + kc;
                        constexpr int CG = RCH / G;  // chunks of a group
                        s2[u] = __half2half2(
                            *reinterpret_cast<const __half *>(par + c / CG * L::PROW + k * 2));
                        dst[u] = kt + c / CG * (KT * 128) + k * 128;
                        sw[u] = (c % CG * OUT) ^ (k & 7);
                    }
                    // (rolled over a chunk's words, the unpacked one always in x)
#pragma unroll 1
                    for (int j = 0; j < OUT; ++j) {
#pragma unroll
                        for (int u = 0; u < KU; ++u) {
                            uint4 o;
                            if constexpr (BITS == 4) {
                                const __half2 off = __floats2half2_rn(1032.f, 1032.f);
                                const __half2 r16 = __floats2half2_rn(0.0625f, 0.0625f);
                                const __half2 m72 = __floats2half2_rn(-72.f, -72.f);
                                const uint32_t a = kreg[u].x, b = a >> 8;
                                kreg[u].x = kreg[u].y;
                                kreg[u].y = kreg[u].z;
                                kreg[u].z = kreg[u].w;
                                o.x = h2_bits(__hmul2(__hsub2(bits_h2((a & 0x000f000fu) | 0x64006400u), off), s2[u]));
                                o.y = h2_bits(__hmul2(__hfma2(bits_h2((a & 0x00f000f0u) | 0x64006400u), r16, m72), s2[u]));
                                o.z = h2_bits(__hmul2(__hsub2(bits_h2((b & 0x000f000fu) | 0x64006400u), off), s2[u]));
                                o.w = h2_bits(__hmul2(__hfma2(bits_h2((b & 0x00f000f0u) | 0x64006400u), r16, m72), s2[u]));
                            } else {
                                const __half2 off = __floats2half2_rn(1152.f, 1152.f);
                                const uint32_t a = kreg[u].x, b = kreg[u].y;
                                kreg[u].x = kreg[u].z;
                                kreg[u].y = kreg[u].w;
                                o.x = h2_bits(__hmul2(__hsub2(bits_h2((a & 0x00ff00ffu) | 0x64006400u), off), s2[u]));
                                o.y = h2_bits(__hmul2(__hsub2(bits_h2(((a >> 8) & 0x00ff00ffu) | 0x64006400u), off), s2[u]));
                                o.z = h2_bits(__hmul2(__hsub2(bits_h2((b & 0x00ff00ffu) | 0x64006400u), off), s2[u]));
                                o.w = h2_bits(__hmul2(__hsub2(bits_h2(((b >> 8) & 0x00ff00ffu) | 0x64006400u), off), s2[u]));
                            }
                            *reinterpret_cast<uint4 *>(dst[u] + ((sw[u] ^ j) * 16)) = o;
                        }
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&kfull[st]);
                if (tile + 1 < w.tb) load_k(base, tile + 1);

                // ---- values, transposed: code / KC, exact from 1024 + code,
                // times KC scale plus bias.  (Codes left as the subnormals
                // code 2^-24 save an operation, but want scales 2^24 times
                // larger and so leave fp16 only 2^8 of range below the tile's
                // largest value: 2048 tokens over 8192 keys 346 us, 351 so.)
#pragma unroll
                for (int u = 0; u < VU; ++u) {
                    const int id = dw + u * kPfDeqWarps;
                    if (id >= L::VUNITS) break;
                    unsigned char *vt = smem + L::V_OFF + (size_t)st * L::TILE + (id % NH) * (D * 128);
                    const int d0 = id / NH * 32 + vd * 8;
                    const unsigned char *vp = par + (G + id / (2 * NH)) * L::PROW + (id % NH * 64 + vc * 8) * 2;
                    const uint4 sw = *reinterpret_cast<const uint4 *>(vp);
                    const uint4 bw = *reinterpret_cast<const uint4 *>(vp + G * L::PROW);
                    const __half2 s2[4] = {bits_h2(sw.x), bits_h2(sw.y), bits_h2(sw.z), bits_h2(sw.w)};
                    const __half2 b2[4] = {bits_h2(bw.x), bits_h2(bw.y), bits_h2(bw.z), bits_h2(bw.w)};
                    // the fp16 pair 1024 + c as c / by
                    auto over = [](uint32_t c, float by) {
                        return __hfma2(bits_h2(c | 0x64006400u), __floats2half2_rn(1.f / by, 1.f / by),
                                       __floats2half2_rn(-1024.f / by, -1024.f / by));
                    };
#pragma unroll 1
                    for (int jj = 0; jj < 4; ++jj) {
                        uint32_t lo[4], hi[4];  // dimensions 2 jj, 2 jj + 1 of the 8
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            if constexpr (BITS == 4) {
                                const uint32_t sel = 0x4400u + 0x1111u * jj;
                                const uint32_t t = __byte_perm(vreg[u][2 * j][0], vreg[u][2 * j + 1][0], sel);
                                // (codes at bits 4-7 are 16 times their own)
                                lo[j] = h2_bits(__hfma2(over(t & 0x000f000fu, KC), s2[j], b2[j]));
                                hi[j] = h2_bits(__hfma2(over(t & 0x00f000f0u, 16.f * KC), s2[j], b2[j]));
                            } else {
                                const uint32_t sel = 0x5410u + 0x2222u * (jj & 1);
                                const uint32_t t =
                                    __byte_perm(jj < 2 ? vreg[u][2 * j][0] : vreg[u][2 * j][VW - 1],
                                                jj < 2 ? vreg[u][2 * j + 1][0] : vreg[u][2 * j + 1][VW - 1], sel);
                                lo[j] = h2_bits(__hfma2(over(t & 0x00ff00ffu, KC), s2[j], b2[j]));
                                hi[j] = h2_bits(__hfma2(over((t >> 8) & 0x00ff00ffu, KC), s2[j], b2[j]));
                            }
                        }
                        unsigned char *row = vt + (d0 + 2 * jj) * 128;
                        *reinterpret_cast<uint4 *>(row + ((vc ^ ((2 * jj) & 7)) * 16)) =
                            make_uint4(lo[0], lo[1], lo[2], lo[3]);
                        *reinterpret_cast<uint4 *>(row + 128 + ((vc ^ ((2 * jj + 1) & 7)) * 16)) =
                            make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    }
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(&vfull[st]);
                if (tile + 1 < w.tb) load_v(base, tile + 1);
                base = pages.look(tile + 2, lane);
            }
        }
    }
    // ---- rows that see no key are zero: sequences, and blocks of them
    // (written here, beside the products, by the spare warps)
    if (warp >= 2 && warp < 4) {
        const int tid = threadIdx.x - 64;
        for (int b = cta; b < B; b += gridDim.x) {
            const KvSeq s = kv_seq(p.kv, b);
            if (p.status && tid == 0 && kv_past(s)) atomicOr(p.status, (int)kKvBadPage);
            const int rows = pf_rows<RB>(p, s);
            for (int rb = 0; rb * RB < rows; ++rb) {
                if (pf_tiles<RB, KT>(p, s, rows, rb) > 0) continue;
                const int n = min(RB, rows - rb * RB);
                for (int i = tid; i < n * p.kv.heads * (D / 8); i += 64) {
                    const int c = i % (D / 8), h = i / (D / 8) % p.kv.heads, rr = rb * RB + i / (D / 8) / p.kv.heads;
                    reinterpret_cast<uint4 *>(p.out + ((int64_t)(s.first + rr / p.rep) * p.Hq + h * p.rep +
                                                       rr % p.rep) * D)[c] = make_uint4(0u, 0u, 0u, 0u);
                }
            }
        }
    }
    // ---- teardown: without a wait that ran out, every MMA was waited for
    tc_fence_before();
    __syncthreads();
    if (warp < 2 && lane == 0 && s_fail) {
        tc_commit(&sfull[0][warp]);  // completes after every MMA this thread issued
        mbar_wait(&sfull[0][warp], 0, 1000000ull);
        mbar_wait(&sfull[0][warp], 1, 1000000ull);
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// Joins cut blocks: a warp to a row, lanes over the dimensions, the pieces
// (two mostly) one after the other.  A piece is its keys' mean value o_i and
// the base-2 logarithm c_i of its weights' sum: out = sum_i 2^(c_i - M) o_i /
// sum_i 2^(c_i - M).
template <int D>
__global__ void __launch_bounds__(256) paged_prefill_join_kernel(PagedParams p, int rb) {
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const PgCut d = p.cuts[blockIdx.x];
    const int i = blockIdx.y * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (d.slot < 0 || i >= d.nlive) return;
    constexpr int V = D / 32;  // dimensions of a lane
    float m = -INFINITY, l = 0.f, a[V];
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = 0.f;
#pragma unroll 2
    for (int k = 0; k < d.n; ++k) {
        const float *src = p.part + ((int64_t)(k == 0 ? d.slot : 2 * (d.cta + k)) * rb + i) * (D + 4);
        float v[V];
#pragma unroll
        for (int x = 0; x < V; x += 2) {
            const float2 t = *reinterpret_cast<const float2 *>(src + 64 * (x / 2) + 2 * lane);
            v[x] = t.x;
            v[x + 1] = t.y;
        }
        const float mk = src[D];
        const float mx = fmaxf(m, mk), sub = mx == -INFINITY ? 0.f : mx;
        const float f0 = ex2(m - sub), f1 = ex2(mk - sub - kPgJoin);
        m = mx;
        l = fmaf(l, f0, f1);
#pragma unroll
        for (int x = 0; x < V; ++x) a[x] = fmaf(a[x], f0, v[x] * f1);
    }
    const float r = l == 0.f ? 0.f : 1.f / l;
    const int rr = d.r0 + i;
    uint32_t *dst = reinterpret_cast<uint32_t *>(
        p.out + ((int64_t)(d.first + rr / p.rep) * p.Hq + d.head + rr % p.rep) * D);
#pragma unroll
    for (int x = 0; x < V; x += 2) dst[32 * (x / 2) + lane] = pack_bf16(a[x] * r, a[x + 1] * r);
}

// One CTA per SM, no more than there can be units of work.  (No fewer than
// there are, so that the cut, and with it the roundings, is the same for every
// max_kv from the longest length on.)
static int pf_grid(const KvView &kv, int rep) {
    const int rb = kv.dim <= 128 ? 256 : 128, kt = kv.dim <= 128 ? 128 : 64;
    const double units = (double)kv.batch * kv.heads * (((int64_t)rep * kv.max_q + rb - 1) / rb) *
                         (((int64_t)kv.max_kv + kt - 1) / kt + pf_head(kt));
    return units < num_sms() ? std::max((int)units, 1) : num_sms();
}

// The sequences' rows are at most those of all tokens together, and a sequence
// with more than `split` of them has one block that may not be full.
double paged_prefill_units(const KvView &kv, int rep, int split) {
    if ((int64_t)rep * kv.max_q <= split) return 0.;
    const int rb = kv.dim <= 128 ? 256 : 128, kt = kv.dim <= 128 ? 128 : 64;
    const double rows = (double)rep * std::min((double)kv.tokens, (double)kv.batch * kv.max_q);
    const double part = std::min((double)kv.batch, rows / (split + 1));
    const double tiles = (double)kv.max_pages * (1 << kv.page_shift) / kt + 1 + pf_head(kt);
    return kv.heads * (rows / rb + part) * tiles;
}

template <int BITS, int D>
static cudaError_t launch_pf_t(PagedParams p, void *workspace, cudaStream_t st) {
    using L = PfLayout<BITS, D>;
    const void *kfn = reinterpret_cast<const void *>(paged_prefill_kernel<BITS, D>);
    cudaError_t e = allow_smem(kfn, (int)L::SMEM);
    if (e != cudaSuccess) return e;
    const int grid = pf_grid(p.kv, p.rep);
    p.cuts = static_cast<PgCut *>(workspace);
    p.part = reinterpret_cast<float *>(p.cuts + kPgMaxCtas);
    e = launch_pdl(kfn, (unsigned)grid, kPfThreads, L::SMEM, st, p);
    if (e != cudaSuccess || grid == 1) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, (unsigned)(L::RB / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_prefill_join_kernel<D>, p, L::RB);
}

cudaError_t launch_paged_prefill(PagedParams p, void *workspace, cudaStream_t st) {
#define GWA_PF(BB, DD) \
    if (p.kv.bits == BB && p.kv.dim == DD) return launch_pf_t<BB, DD>(p, workspace, st);
    GWA_PF(4, 64) GWA_PF(4, 128) GWA_PF(4, 256)
    GWA_PF(8, 64) GWA_PF(8, 128) GWA_PF(8, 256)
#undef GWA_PF
    return cudaErrorInvalidValue;
}

size_t paged_prefill_workspace_bytes(const KvView &kv, int rep) {
    const int rb = kv.dim <= 128 ? 256 : 128;
    return (size_t)pf_grid(kv, rep) * 2 * rb * (kv.dim + 4) * sizeof(float);
}

unsigned int prefill_timeouts(bool reset) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_prefill_timeouts, sizeof v);
    if (reset) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_prefill_timeouts, &z, sizeof z);
    }
    return v;
}

}  // namespace gwa
