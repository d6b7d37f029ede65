// Low-rank adapters of many requests at once, added to a shared projection's
// output ("Sanctum-MLX", "File map": lora.rs merges one adapter into the
// weights at load; here each token brings its own and nothing is merged):
//
//   t[m,s,:] = scale_a (A_a[s] x_m),       a = ids[m], rank_a rows of A_a[s]
//   y_s[m,n] = base_s[m,n] + B_a[s][n,:] . t[m,s,:]
//
// and for the gated projection SiLU(y_0) y_1.  Two products: x against the A's
// (shrink), whose few results a token go through the workspace, and those
// against the B's (expand).  Products are exact, sums fp32; t enters its
// product as two bf16 parts (together 2^-17 of it), so the output's rounding
// is the only one to count.
//
// Tokens of one adapter are taken together, in tiles, so that an adapter is
// read once for them.  Two ways, by the number of tokens:
//   up to kLoSort: every CTA of both kernels puts the tokens in the order of
//     their adapters itself (1.5 us; a kernel for it would cost a launch).
//     Warp-level MMAs (m16n8k16, an adapter's rows the 16): a tile has few
//     tokens, and the bytes of A and B bound the work.
//   more: runs of neighbours as they come (a prompt's tokens are neighbours),
//     x against A on tcgen05, a kernel that adds up the shares of K once, and
//     the outputs on tcgen05 too, or by warp-level MMAs (see lora_out_tc).
// Each kernel starts while the one in front of it ends, and does what does not
// depend on it (tiles, the first loads of B and base) before it waits.
//
// Bound by bytes: A and B of the adapters at hand, x, base and out.  Measured
// (bf16, replayed with the adapters in L2 where they fit; of the 6.68 TB/s of a
// copy): one token, rank 16, 5120 to 7168, 8.3 us, 0.1 of them bytes: two
// launches that depend on each other, tiles, a round of loads each.  54 tokens
// of 24 adapters of ranks 8 to 64 there, 45 MB, 17.6 us (2.6 TB/s, 0.39): lines
// of L1, as a fragment load of 8 rows touches 8, and two rounds of units.  14
// sequences of up to 5 tokens, gate and up of 13824, rank 32, 19 MB, 12.4 us
// (1.5 TB/s).  Prompts of 5560 tokens, 13824 to 5120, rank 64, 272 MB, 74 us
// (3.7 TB/s): shrink 38 (x at 4 TB/s), join 5, outputs some 27 (the rest is
// launches).
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "mma.cuh"
#include "tcgen05.cuh"
#include "tma.cuh"

namespace gwa {

constexpr int kLoThreads = 256, kLoWarps = kLoThreads / 32;
constexpr int kLoTile = 16;      // tokens of a tile
constexpr int kLoSort = 256;     // tokens that are sorted, a thread each
constexpr int kLoPer = 32;       // tokens of a thread where they are not
constexpr int kLoChunk = kLoThreads * kLoPer;  // tokens of a launch

// The tiles of a launch: tile i is the tokens at places [start[i], start[i +
// 1]), all of one adapter; place i is token order[i] (sorted) or i.
template <bool FEW>
struct LoTiles {
    uint16_t start[(FEW ? kLoSort : kLoChunk) + 1];
    uint16_t order[FEW ? kLoSort : 1];
    __align__(16) int key[FEW ? kLoSort : 1];  // of the places: adapter
    int rank[FEW ? kLoSort : 1];               // and its rank
    int base[FEW ? kLoSort + 1 : 1];           // of the tiles: 16-row blocks of A before it
    int w_max[FEW ? kLoWarps : 16], w_sum[FEW ? kLoWarps : 16];
    __device__ __forceinline__ int token(int place) const { return FEW ? order[place] : place; }
};

// A token's adapter, -1 for none.
__device__ __forceinline__ int lo_id(const LoraParams &p, int tok) {
    const int id = __ldcg(p.ids + tok);
    return (unsigned)id < (unsigned)p.adapters ? id : -1;
}
__device__ __forceinline__ int lo_rank(const LoraParams &p, int id) {
    return id < 0 ? 0 : p.ranks ? min(max(__ldcg(p.ranks + id), 0), p.rank) : p.rank;
}

// Cuts the tokens into tiles of up to TM (all threads of the CTA); returns their
// number.  Up to kLoSort tokens: in the order of their adapters, a thread each.
template <int TM>
__device__ int lo_tiles(const LoraParams &p, LoTiles<true> &sh) {
    constexpr unsigned FULL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int mine = tid < p.M ? lo_id(p, tid) : 0x7fffffff;
    if (tid < p.M && blockIdx.x == 0 && p.status && __ldcg(p.ids + tid) >= p.adapters) atomicOr(p.status, 1);
    const int rank = tid < p.M ? lo_rank(p, mine) : 0;  // (there by the end of the sort)
    sh.key[tid] = mine;
    __syncthreads();
    int at = 0;
    for (int j = 0; j < p.M; j += 4) {
        const int4 k = *reinterpret_cast<const int4 *>(sh.key + j);
        at += (k.x < mine || (k.x == mine && j < tid)) + (k.y < mine || (k.y == mine && j + 1 < tid)) +
              (k.z < mine || (k.z == mine && j + 2 < tid)) + (k.w < mine || (k.w == mine && j + 3 < tid));
    }
    __syncthreads();
    if (tid < p.M) {
        sh.order[at] = (uint16_t)tid;
        sh.key[at] = mine;
        sh.rank[at] = rank;
    }
    __syncthreads();
    // where the run of this place starts: the last place that differs from the
    // one in front of it
    int run = tid == 0 || sh.key[tid] != sh.key[tid - 1] ? tid : -1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, run, o);
        if (lane >= o) run = max(run, v);
    }
    if (lane == 31) sh.w_max[warp] = run;
    __syncthreads();
    for (int w = 0; w < warp; ++w) run = max(run, sh.w_max[w]);
    const bool starts = tid < p.M && (tid - run) % TM == 0;
    const unsigned all = __ballot_sync(FULL, starts);
    if (lane == 0) sh.w_sum[warp] = __popc(all);
    __syncthreads();
    int before = __popc(all & ((1u << lane) - 1u)), total = 0;
    for (int w = 0; w < kLoWarps; ++w) {
        if (w < warp) before += sh.w_sum[w];
        total += sh.w_sum[w];
    }
    if (starts) sh.start[before] = (uint16_t)tid;
    if (tid == 0) sh.start[total] = (uint16_t)p.M;
    __syncthreads();
    return total;
}
// More: runs of neighbours.  A warp reads a share of the tokens, 32 at a time,
// and marks where the adapter changes; then each lane takes one such group.
// (Warps past the kLoWarps have no share.)
template <int TM>
__device__ int lo_tiles(const LoraParams &p, LoTiles<false> &sh) {
    constexpr unsigned FULL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int chunk = (p.M + kLoThreads - 1) / kLoThreads * 32, first = warp * chunk;  // tokens of a warp
    int id[kLoPer];
    int before = first > 0 && first <= p.M && lane == 0 ? lo_id(p, first - 1) : 0x7fffffff;
#pragma unroll
    for (int j = 0; j < kLoPer; ++j) {
        const int tok = first + 32 * j + lane;
        id[j] = 32 * j < chunk && tok < p.M ? __ldcg(p.ids + tok) : -1;
    }
    unsigned mask = 0;  // of the lane's group: where runs start
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kLoPer; ++j) {
        if (32 * j >= chunk) break;
        bad |= id[j] >= p.adapters;
        const int v = (unsigned)id[j] < (unsigned)p.adapters ? id[j] : -1;
        int prev = __shfl_up_sync(FULL, v, 1);
        if (lane == 0) prev = before;
        const unsigned m = __ballot_sync(FULL, first + 32 * j + lane < p.M && v != prev);
        if (lane == j) mask = m;
        before = __shfl_sync(FULL, v, 31);
    }
    if (bad && blockIdx.x == 0 && p.status) atomicOr(p.status, 1);
    const int base = first + 32 * lane;
    int last = mask ? base + 31 - __clz(mask) : -1;  // up to and with the lane's group
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, last, o);
        if (lane >= o) last = max(last, v);
    }
    if (lane == 31) sh.w_max[warp] = last;
    __syncthreads();
    int run = __shfl_up_sync(FULL, last, 1);
    if (lane == 0) run = -1;
    for (int w = 0; w < warp; ++w) run = max(run, sh.w_max[w]);
    unsigned starts = 0;
    const int n = 32 * lane < chunk ? min(32, p.M - base) : 0;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
        if ((mask >> i) & 1u) run = base + i;
        if (i < n && (base + i - run) % TM == 0) starts |= 1u << i;
    }
    int sum = __popc(starts);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sh.w_sum[warp] = sum;
    __syncthreads();
    int at = sum - __popc(starts), total = 0;
    for (int w = 0; w < kLoWarps; ++w) {
        if (w < warp) at += sh.w_sum[w];
        total += sh.w_sum[w];
    }
    for (; starts; starts &= starts - 1) sh.start[at++] = (uint16_t)(base + __ffs(starts) - 1);
    if (tid == 0) sh.start[total] = (uint16_t)p.M;
    __syncthreads();
    return total;
}

__device__ __forceinline__ uint4 lo_load(const uint16_t *p, bool ok) {
    return ok ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// 32 bytes, at once where they begin on 32: a fragment's 8 rows are 8 lines of
// L1, whatever each gives.
__device__ __forceinline__ void lo_load32(const uint16_t *p, bool ok, bool at_once, uint4 &a, uint4 &b) {
    if (at_once) {
        a = b = make_uint4(0u, 0u, 0u, 0u);
        if (ok)
            asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                         : "l"(p));
    } else {
        a = lo_load(p, ok);
        b = lo_load(p + 8, ok);
    }
}

// g / (1 + e^-g).  e^-g passes fp32's range at -88.7 (and 2^126, past which a
// fast quotient gives zero, at -87.3), and the other half may be as large again:
// so 2^-24 / (2^-24 + 2^-24 e^-g), which reaches the least that fp32 can hold.
// The exponent's rounding next to -24 is 2^-21 of the result.  (An infinite g
// below zero gives NaN.)
__device__ __forceinline__ float lo_silu(float g) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(fmaf(g, -1.4426950408889634f, -24.f)) + 0x1p-24f));
    return g * (r * 0x1p-24f);
}

// ------------------------------------------------------------ few tokens
// part[k][m][s][r]: share k's sum of A x.  A CTA's unit is 16 rows of an
// adapter's A and a share of K for a tile; its warps take 256 inputs at a time
// (a warp's loads all at once, straight from global memory as MMA fragments: a
// lane's 32 bytes are the k positions of four MMAs, in the same order on both
// sides).  The shares depend on K alone, and so does the order of a token's
// sums.  WIDE: x and A begin on 32 bytes (see lo_load32).
template <bool WIDE>
__global__ void __launch_bounds__(kLoThreads, 2) lora_few_shrink_kernel(LoraParams p) {
    constexpr int LANE = 16;  // inputs of a lane side by side
    __shared__ LoTiles<true> sh;
    __shared__ float s_acc[kLoWarps][16 * kLoTile];
    __shared__ int s_sum[kLoWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    pdl_wait_primary();
    // (behind the wait: what the next kernel reads before its own wait was
    // written before this one's)
    if (tid == 0) pdl_launch_dependents();
    const int tiles = lo_tiles<kLoTile>(p, sh);
    // ---- units: blocks of the tiles in order, each in ks shares
    const int mine = tid < tiles ? p.nsec * ((sh.rank[sh.start[tid]] + 15) / 16) : 0;
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += s_sum[w];
    if (tid < tiles) sh.base[tid + 1] = incl;
    if (tid == 0) sh.base[0] = 0;
    __syncthreads();
    const int units = sh.base[tiles] * p.ks;
    for (int u = blockIdx.x; u < units; u += gridDim.x) {
        const int blk = u / p.ks, k = u - blk * p.ks;
        int tile = 0;  // the last whose base is not past blk
        for (int o = 128; o; o >>= 1)
            if (tile + o < tiles && sh.base[tile + o] <= blk) tile += o;
        const int at = sh.start[tile], n = sh.start[tile + 1] - at, id = sh.key[at], rank = sh.rank[at];
        const int nb = (rank + 15) / 16, in = blk - sh.base[tile], sec = in / nb, r0 = (in - sec * nb) * 16;
        const uint16_t *a = p.a + (((int64_t)id * p.nsec + sec) * p.rank + r0 + g) * p.K + LANE * t;
        const bool in0 = r0 + g < rank, in1 = r0 + g + 8 < rank, tok0 = g < n, tok1 = g + 8 < n;
        const uint16_t *x0 = p.x + (int64_t)sh.token(at + (tok0 ? g : 0)) * p.K + LANE * t;
        const uint16_t *x1 = p.x + (int64_t)sh.token(at + (tok1 ? g + 8 : 0)) * p.K + LANE * t;
        float acc[2][4] = {};
        const int end = min(p.K, (k + 1) * p.share);
        for (int i0 = k * p.share + warp * 256; i0 < end; i0 += kLoWarps * 256) {
            uint4 va[8], vb[8];
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                const bool ok = i0 + 32 * c + LANE * t < end;
                lo_load32(a + i0 + 32 * c, ok && in0, WIDE, va[c], va[c + 1]);
                lo_load32(a + i0 + 32 * c + (int64_t)8 * p.K, ok && in1, WIDE, vb[c], vb[c + 1]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && n <= 8) break;
                uint4 x[8];
#pragma unroll
                for (int c = 0; c < 8; c += 2)
                    lo_load32((h ? x1 : x0) + i0 + 32 * c, i0 + 32 * c + LANE * t < end && (h ? tok1 : tok0), WIDE, x[c],
                              x[c + 1]);
#pragma unroll
                for (int c = 0; c < 8; ++c) {
                    mma_bf16(acc[h], va[c].x, vb[c].x, va[c].y, vb[c].y, x[c].x, x[c].y);
                    mma_bf16(acc[h], va[c].z, vb[c].z, va[c].w, vb[c].w, x[c].z, x[c].w);
                }
            }
        }
        // [token][row]
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s_acc[warp][(8 * h + 2 * t + (i & 1)) * 16 + g + 8 * (i >> 1)] = acc[h][i];
        __syncthreads();
        const int m = tid / 16, r = tid % 16;
        if (m < n && r0 + r < p.rank) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kLoWarps; ++w) v += s_acc[w][tid];
            p.part[(((int64_t)k * p.M + sh.token(at + m)) * p.nsec + sec) * p.rank + r0 + r] = v;
        }
        __syncthreads();
    }
}

// out = base + scale B t.  A CTA's unit is a tile and some octets of steps of
// 32 outputs of one section, a warp a step; t, summed over the shares, lies in
// shared memory as fragments of the MMA's 16 rows, hi and lo bf16 parts.  B's
// rows and the base come straight from global memory, the first of them before
// the wait for t.  Lane t's outputs of a step are eight neighbours (column c of
// the step's MMA j is output 8 (c / 2) + 2 j + c % 2).
//
// Fragments: of a section's k step, each lane's words 0 and 2 of the hi and of
// the lo part, then its words 1 and 3.  Of a pair of k steps, lane t's ranks are
// 8 t .. 8 t + 7.
constexpr int kLoFrag = 64;  // 16-byte units of a k step

template <int KS, bool SILU, bool VEC, bool WIDE>
__global__ void __launch_bounds__(kLoThreads, KS * (SILU ? 2 : 1) <= 4 ? 2 : 1) lora_few_expand_kernel(LoraParams p) {
    constexpr int S = SILU ? 2 : 1, Q = KS == 1 ? 1 : KS / 2;  // Q: 16-byte units of a lane and row of B
    constexpr int SPAN = WIDE ? 64 : KS == 1 ? 16 : 32;        // ranks whose k steps share lanes
    // first rank of unit q of lane t
    auto rank_of = [](int q, int t) { return WIDE ? 64 * (q / 2) + 16 * t + 8 * (q & 1) : KS == 1 ? 4 * t : 32 * q + 8 * t; };
    __shared__ LoTiles<true> sh;
    __shared__ uint4 frag[S * KS * kLoFrag];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    if (tid == 0) pdl_launch_dependents();
    const int tiles = lo_tiles<kLoTile>(p, sh);
    // ---- units of `run` octets
    int octets = 0;
    for (int s = 0; s < (SILU ? 1 : p.nsec); ++s) octets += p.sec_blocks[s];
    const int run = max(1, (int)(((int64_t)tiles * octets + gridDim.x - 1) / gridDim.x));
    int per = 0;  // of a tile
    for (int s = 0; s < (SILU ? 1 : p.nsec); ++s) per += (p.sec_blocks[s] + run - 1) / run;
    bool waited = false;
    for (int64_t u = blockIdx.x; u < (int64_t)tiles * per; u += gridDim.x) {
        const int tile = (int)(u / per);
        int in = (int)(u - (int64_t)tile * per), sec = 0;
        if constexpr (!SILU)
            for (int c; in >= (c = (p.sec_blocks[sec] + run - 1) / run); ++sec) in -= c;
        const int at = sh.start[tile], n = sh.start[tile + 1] - at, id = sh.key[at], rank = sh.rank[at];
        if (rank == 0 && p.in_place) continue;
        const bool live[2] = {g < n, g + 8 < n};
        const int tok[2] = {sh.token(at + (live[0] ? g : 0)), sh.token(at + (live[1] ? g + 8 : 0))};
        const int64_t N = p.sec_n[sec];
        const int last = min(p.sec_blocks[sec], (in + 1) * run);
        for (int oct = in * run; oct < last; ++oct) {
            const int64_t n0 = ((int64_t)oct * kLoWarps + warp) * 32, col = n0 + 8 * t;
            uint4 base[S][2], b[S][4][Q];
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const int64_t c0 = n0 + 8 * (g >> 1) + (g & 1);  // of MMA j: c0 + 2 j
                const uint16_t *brow = p.b + ((int64_t)max(id, 0) * p.N + p.sec_start[sec + s] + c0) * p.rank;
#pragma unroll
                for (int j = 0; j < 4; ++j, brow += 2 * p.rank)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int r = rank_of(q, t);
                        const bool ok = c0 + 2 * j < N && r < rank;
                        if constexpr (WIDE) {
                            if (q % 2 == 0) lo_load32(brow + r, ok, p.b32, b[s][j][q], b[s][j][q + 1]);
                            continue;
                        }
                        b[s][j][q] = make_uint4(0u, 0u, 0u, 0u);
                        if constexpr (KS == 1) {
                            if (ok) {
                                const uint2 w = __ldcg(reinterpret_cast<const uint2 *>(brow + r));
                                b[s][j][q].x = w.x;
                                b[s][j][q].y = w.y;
                            }
                        } else {
                            if (ok) b[s][j][q] = __ldcg(reinterpret_cast<const uint4 *>(brow + r));
                        }
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint16_t *src = p.base[sec + s] + tok[h] * N + col;
                    base[s][h] = make_uint4(0u, 0u, 0u, 0u);
                    if constexpr (VEC) {
                        if (live[h] && col < N) base[s][h] = __ldcg(reinterpret_cast<const uint4 *>(src));
                    } else {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t x = live[h] && col + 2 * i < N ? __ldcg(src + 2 * i) : 0u;
                            const uint32_t y = live[h] && col + 2 * i + 1 < N ? __ldcg(src + 2 * i + 1) : 0u;
                            w[i] = x | (y << 16);
                        }
                        base[s][h] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (oct == in * run && rank > 0) {
                // ---- t of this unit
                if (!waited) pdl_wait_primary();
                waited = true;
                __syncthreads();  // (the last unit's is read)
                const float scale = p.scale ? p.scale[id] : 1.f;
                const int nk = (rank + SPAN - 1) / SPAN * (SPAN / 16);
                for (int i = tid; i < S * nk * 64; i += kLoThreads) {
                    // four ranks of a token
                    const int s = i / (nk * 64), j = i - s * nk * 64, m = j / (4 * nk), r = (j - m * 4 * nk) * 4;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (m < n && r < rank) {
                        const float *src = p.part + ((int64_t)sh.token(at + m) * p.nsec + sec + s) * p.rank + r;
#pragma unroll 4
                        for (int k = 0; k < p.ks; ++k) {
                            const float4 e = __ldcg(reinterpret_cast<const float4 *>(src + (int64_t)k * p.M * p.nsec * p.rank));
                            v = make_float4(v.x + e.x, v.y + e.y, v.z + e.z, v.w + e.w);
                        }
                    }
                    v.x = v.x * scale;
                    v.y = r + 1 < rank ? v.y * scale : 0.f;
                    v.z = r + 2 < rank ? v.z * scale : 0.f;
                    v.w = r + 3 < rank ? v.w * scale : 0.f;
                    const int ks = KS == 1 ? 0 : WIDE ? r / 64 * 4 + r / 4 % 4 : r / 32 * 2 + (r / 4) % 2;
                    const int ln = (m % 8) * 4 + (KS == 1 ? r / 4 : r % SPAN / (SPAN / 4));
                    const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
                    frag[(s * KS + ks) * kLoFrag + m / 8 * 32 + ln] =
                        make_uint4(h0, h1, pack_bf16(v.x - bf16_lo(h0), v.y - bf16_hi(h0)),
                                   pack_bf16(v.z - bf16_lo(h1), v.w - bf16_hi(h1)));
                }
                __syncthreads();
            }
            if (rank % (WIDE ? 16 : 8)) {
                // entries past the adapter's rank, whatever they hold, are zero
                auto mask = [&](uint32_t &w, int k) { w = k + 1 < rank ? w : k < rank ? w & 0xffffu : 0u; };
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            const int k = rank_of(q, t);
                            mask(b[s][j][q].x, k);
                            mask(b[s][j][q].y, k + 2);
                            if constexpr (KS > 1) {
                                mask(b[s][j][q].z, k + 4);
                                mask(b[s][j][q].w, k + 6);
                            }
                        }
            }
            float acc[S][4][4];
#pragma unroll
            for (int s = 0; s < S; ++s) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t w[4] = {base[s][h].x, base[s][h].y, base[s][h].z, base[s][h].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        acc[s][j][2 * h] = bf16_lo(w[j]);
                        acc[s][j][2 * h + 1] = bf16_hi(w[j]);
                    }
                }
                const uint4 *fr = frag + s * KS * kLoFrag + lane;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if (16 * (k & ~(SPAN / 16 - 1)) >= rank) break;
                    const uint4 even = fr[k * kLoFrag], odd = fr[k * kLoFrag + 32];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 &w = b[s][j][KS == 1 ? 0 : k / 2];
                        const uint32_t b0 = k & 1 ? w.z : w.x, b1 = k & 1 ? w.w : w.y;
                        mma_bf16(acc[s][j], even.x, odd.x, even.y, odd.y, b0, b1);
                        mma_bf16(acc[s][j], even.z, odd.z, even.w, odd.w, b0, b1);
                    }
                }
            }
            if constexpr (SILU) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[0][j][i] = lo_silu(acc[0][j][i]) * acc[1][j][i];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (!live[h]) continue;
                uint16_t *dst = p.out[sec] + tok[h] * N + col;
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = pack_bf16(acc[0][j][2 * h], acc[0][j][2 * h + 1]);
                if constexpr (VEC) {
                    if (col < N) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (col + i < N) dst[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
                }
            }
        }
    }
    // (what runs next waits for this kernel alone)
    pdl_wait_primary();
}

// ------------------------------------------------------------ many tokens
// x against A on the 5th-generation tensor cores: D (128 tokens x C rows of A)
// = x A^T, x and A by TMA in steps of 64 inputs, all sections' rows (up to 256)
// at once, so that x is read once.  Tiles are runs of neighbours of one adapter;
// of a short one only its rows, by sixteens, are copied, and what the MMA makes
// of the others is not stored.  The bytes of x bound it; K is shared out over
// so many CTAs that the last round is nearly full (lo_shares).  fp32 sums go to
// part[k][m][s][r] (see the few tokens' kernel).
//
// Warps: 0 issues the copies, 1 the MMAs (a thread each), 4 to 7 bring the
// results out, two accumulators in turn.  Every wait is bounded (2 s); one that
// runs out is counted and the kernel unwinds.
constexpr int kLtTile = 128, kLtStages = 5;  // (fewer where they do not fit)
constexpr int kLtSmem = 200 * 1024;

static __device__ unsigned int g_lora_timeouts;

__device__ __noinline__ bool lt_wait_slow(uint64_t *bar, uint32_t parity, int *fail) {
    if (mbar_wait_sleep(bar, parity)) return true;
    atomicAdd(&g_lora_timeouts, 1u);
    *fail = 1;
    return false;
}
__device__ __forceinline__ bool lt_wait(uint64_t *bar, uint32_t parity, int *fail) {
    return mbar_try_wait(bar, parity) || lt_wait_slow(bar, parity, fail);
}
__device__ __forceinline__ void lt_mma(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Shares of K for so many units: the fewest steps of 64 inputs in a CTA's row,
// where a unit's start and end count as eight.
__device__ __forceinline__ int lo_shares(int units, int ctas, int steps, int most) {
    int best = 1, least = 0x7fffffff;
    for (int k = 1; k <= most && k <= steps; ++k) {
        const int cost = (units * k + ctas - 1) / ctas * ((steps + k - 1) / k + 8);
        if (cost < least) {
            least = cost;
            best = k;
        }
    }
    return best;
}

__global__ void __launch_bounds__(kLoThreads, 1)
    lora_many_shrink_kernel(const __grid_constant__ CUtensorMap xmap, const __grid_constant__ CUtensorMap xmap16,
                            const __grid_constant__ CUtensorMap amap, LoraParams p, int cols, int half, int stages) {
    extern __shared__ __align__(1024) unsigned char lo_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(lo_raw) + 1023) & ~(uintptr_t)1023);
    __shared__ LoTiles<false> sh;
    __shared__ uint64_t full[kLtStages], empty[kLtStages], accfull[2], accfree[2];
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail, s_issued;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    if (tid == 0) {
        for (int i = 0; i < kLtStages; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accfree[i], 4);
        }
        fence_mbar_init();
        s_fail = s_issued = 0;
    }
    if (tid == 0)
        for (const CUtensorMap *m : {&xmap, &xmap16, &amap})
            asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
    if (warp == 1) tmem_alloc(&s_tmem, 2 * half);
    pdl_wait_primary();
    if (tid == 0) pdl_launch_dependents();  // (see the few tokens' kernel)
    tc_fence_before();
    const int tiles = lo_tiles<kLtTile>(p, sh);  // (synchronizes)
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const int rows = p.nsec * p.rank, passes = (rows + cols - 1) / cols, steps = (p.K + 63) / 64;
    const int ks = lo_shares(tiles * passes, gridDim.x, steps, p.ks);
    if (blockIdx.x == 0 && tid == 0) *p.shares = ks;
    const int units = tiles * passes * ks;
    const int stage_bytes = kLtTile * 128 + cols * 128;

    struct Unit {
        int at, n, id, row, k, c0, c1;
    };
    auto unit = [&](int u, Unit &w) {  // false: nothing to do
        const int tile = u / (passes * ks), in = u - tile * passes * ks, pass = in / ks;
        w.at = sh.start[tile];
        w.n = sh.start[tile + 1] - w.at;
        w.id = lo_id(p, w.at);
        w.row = pass * cols;
        w.k = in - pass * ks;
        w.c0 = steps * w.k / ks;
        w.c1 = steps * (w.k + 1) / ks;
        return lo_rank(p, w.id) > 0;
    };
    Unit w;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
                if (!unit(u, w)) continue;
                const int arow = w.id * rows + w.row;
                // (eight boxes a step are slow to issue: most of a tile is copied
                // whole, its neighbours' rows with it)
                const bool whole = w.n > 48;
                const int boxes = (w.n + 15) / 16;
                for (int c = w.c0; c < w.c1; ++c, ++it) {
                    const uint32_t s = it % stages;
                    if (it >= stages && !(ok = lt_wait(&empty[s], ((it / stages) & 1) ^ 1, &s_fail))) break;
                    unsigned char *xs = smem + s * stage_bytes, *as = xs + kLtTile * 128;
                    mbar_expect_tx(&full[s], (whole ? kLtTile : boxes * 16) * 128 + cols * 128);
                    if (whole)
                        tma_load_2d(xs, &xmap, c * 64, w.at, &full[s]);
                    else
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(xs + b * 2048, &xmap16, c * 64, w.at + 16 * b, &full[s]);
                    tma_load_2d(as, &amap, c * 64, arow, &full[s]);
                    s_issued = it + 1;
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // bf16 inputs, fp32 accumulators, both K-major, M = 128
            const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) |
                                   ((uint32_t)(kLtTile >> 4) << 24);
            uint32_t it = 0, j = 0;
            for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
                if (!unit(u, w)) continue;
                const uint32_t buf = j & 1;
                if (j >= 2 && !(ok = lt_wait(&accfree[buf], ((j >> 1) - 1) & 1, &s_fail))) break;
                for (int c = w.c0; c < w.c1; ++c, ++it) {
                    const uint32_t s = it % stages;
                    if (!(ok = lt_wait(&full[s], (it / stages) & 1, &s_fail))) break;
                    tc_fence_after();
                    const uint64_t a = smem_desc_sw128(smem_u32(smem + s * stage_bytes));
                    const uint64_t b = smem_desc_sw128(smem_u32(smem + s * stage_bytes + kLtTile * 128));
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        lt_mma(tmem + buf * half, a + 2 * k, b + 2 * k, idesc, c > w.c0 || k > 0 ? 1u : 0u);
                    tc_commit(&empty[s]);
                }
                if (!ok) break;
                tc_commit(&accfull[buf]);
                ++j;
            }
        }
    } else if (warp >= 4) {
        const int q = warp & 3, row = q * 32 + lane;
        uint32_t j = 0;
        for (int u = blockIdx.x; ok && u < units; u += gridDim.x) {
            if (!unit(u, w)) continue;
            const uint32_t buf = j & 1;
            ok = __all_sync(0xffffffffu, lt_wait(&accfull[buf], (j >> 1) & 1, &s_fail));
            if (!ok) break;
            tc_fence_after();
            const int valid = min(cols, rows - w.row);
            float *dst = p.part + ((int64_t)w.k * p.M + w.at + row) * rows + w.row;
            for (int c = 0; c < valid && q * 32 < w.n; c += 16) {
                float v[16];
                tc_ld16(tmem + buf * half + c + ((uint32_t)(q * 32) << 16), v);
                if (row < w.n)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        if (c + i < valid)
                            *reinterpret_cast<float4 *>(dst + c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&accfree[buf]);
            ++j;
        }
    }
    // ---- teardown: without a wait that ran out, every copy and MMA was waited for
    tc_fence_before();
    __syncthreads();
    if (s_fail) {
        if (tid == 0)
            for (int k = max(0, s_issued - stages); k < s_issued; ++k)
                if (!mbar_wait(&full[k % stages], (k / stages) & 1)) break;
        if (tid == 32) {
            tc_commit(&accfull[0]);  // completes after every MMA this thread issued
            mbar_wait(&accfull[0], 0, 1000000ull);
            mbar_wait(&accfull[0], 1, 1000000ull);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 2 * half);
}

// low[m][s][r / 4]: t of many tokens, the shares' sums times the scale, as hi and
// lo bf16 parts; zero past the adapter's rank.  (Made once here; each of a
// dozen expanding CTAs summing its tokens' up again took 10 us.)  PLANES: two
// rows of `pitch` bf16 a section instead, the hi and the lo parts, as TMA brings
// them to the tensor cores.
template <bool PLANES>
__global__ void __launch_bounds__(kLoThreads) lora_many_join_kernel(LoraParams p, int pitch) {
    // (before the wait: this kernel starts behind the first one's wait already)
    if (threadIdx.x == 0) pdl_launch_dependents();
    constexpr int AT = 4;  // units of a thread at a time
    const int quads = (PLANES ? pitch : p.rank) / 4, of_token = p.nsec * quads, stride = gridDim.x * kLoThreads;
    const int all = p.M * of_token;  // (8192 tokens x 8 sections x 32 at most)
    const int of_share = p.M * p.nsec * (p.rank / 4);
    int ks = 0;
    for (int i0 = blockIdx.x * kLoThreads + threadIdx.x; i0 < all; i0 += AT * stride) {
        int rank[AT];
        float scale[AT];
#pragma unroll
        for (int x = 0; x < AT; ++x) {
            const int i = i0 + x * stride, id = i < all ? lo_id(p, i / of_token) : -1;
            rank[x] = lo_rank(p, id);
            scale[x] = id >= 0 && p.scale ? __ldcg(p.scale + id) : 1.f;
        }
        if (ks == 0) {
            pdl_wait_primary();
            ks = __ldcg(p.shares);
        }
        float4 v[AT];
#pragma unroll
        for (int x = 0; x < AT; ++x) v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
        for (int k = 0; k < ks; ++k) {
            const float4 *src = reinterpret_cast<const float4 *>(p.part) + (int64_t)k * of_share;
#pragma unroll
            for (int x = 0; x < AT; ++x) {
                const int i = i0 + x * stride, q = i % quads;
                if (q * 4 >= rank[x]) continue;
                const float4 e = __ldcg(src + (PLANES ? i / quads * (p.rank / 4) + q : i));
                v[x] = make_float4(v[x].x + e.x, v[x].y + e.y, v[x].z + e.z, v[x].w + e.w);
            }
        }
#pragma unroll
        for (int x = 0; x < AT; ++x) {
            const int i = i0 + x * stride, r = i % quads * 4;
            if (i >= all) break;
            const float a = v[x].x * scale[x], b = r + 1 < rank[x] ? v[x].y * scale[x] : 0.f;
            const float c = r + 2 < rank[x] ? v[x].z * scale[x] : 0.f, d = r + 3 < rank[x] ? v[x].w * scale[x] : 0.f;
            const uint32_t h0 = pack_bf16(a, b), h1 = pack_bf16(c, d);
            const uint32_t l0 = pack_bf16(a - bf16_lo(h0), b - bf16_hi(h0));
            const uint32_t l1 = pack_bf16(c - bf16_lo(h1), d - bf16_hi(h1));
            if constexpr (PLANES) {
                uint16_t *dst = reinterpret_cast<uint16_t *>(p.low) + (int64_t)(i / quads) * 2 * pitch + r;
                *reinterpret_cast<uint2 *>(dst) = make_uint2(h0, h1);
                *reinterpret_cast<uint2 *>(dst + pitch) = make_uint2(l0, l1);
            } else {
                p.low[i] = make_uint4(h0, h1, l0, l1);
            }
        }
    }
    pdl_wait_primary();
}

// out = base + scale B t.  A warp's unit is a tile of 16 MT tokens and some
// steps of 32 outputs of one section; the eight warps of a CTA take
// neighbouring tiles of the same outputs, so that B comes out of the L1 cache.
// t's fragments are each warp's own copy in shared memory; the next step's base
// is on its way during the products, its B during the stores.
// For what lora_many_out_kernel, below, does not take: rows that are no 16-byte
// units, ranks above 64, fewer tokens or short runs, where a tile of 16 or 32
// tokens leaves less of a product unused than one of 128.  Long runs are slower
// here: 5560 tokens of rank 64, 13824 to 5120, 52 us for 30 there.
template <int KS, bool SILU>
struct LoMany {
    static constexpr int S = SILU ? 2 : 1, MT = KS * S <= 4 && !SILU ? 2 : 1, TM = 16 * MT;
    static constexpr int FRAGS = MT * S * KS * kLoFrag;   // of a warp, 16 bytes each
    static constexpr int SMEM = kLoWarps * FRAGS * 16;
    static constexpr int CTAS = KS * S <= 4 ? 2 : 1;
};
template <int KS, bool SILU, bool VEC>
__global__ void __launch_bounds__(kLoThreads, LoMany<KS, SILU>::CTAS) lora_many_expand_kernel(LoraParams p) {
    using L = LoMany<KS, SILU>;
    constexpr int S = L::S, MT = L::MT, Q = KS == 1 ? 1 : KS / 2;
    extern __shared__ __align__(1024) unsigned char lo_raw[];
    __shared__ LoTiles<false> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    uint4 *const frag = reinterpret_cast<uint4 *>(lo_raw) + warp * L::FRAGS;
    if (tid == 0) pdl_launch_dependents();
    const int tiles = lo_tiles<L::TM>(p, sh), groups = (tiles + kLoWarps - 1) / kLoWarps;
    // ---- units: a group of tiles and a run of a section's steps, as long as
    // leaves the last round of CTAs fullest
    auto units_of = [&](int run) {
        int n = 0;
        for (int s = 0; s < (SILU ? 1 : p.nsec); ++s) n += (p.sec_blocks[s] + run - 1) / run;
        return n;
    };
    int run = 1;
    {
        int steps = 0;
        for (int s = 0; s < (SILU ? 1 : p.nsec); ++s) steps += p.sec_blocks[s];
        const unsigned all = (unsigned)min(steps, 1 << 20) * groups, ctas = gridDim.x;
        unsigned least = 0xffffffffu;
        for (unsigned i = 1; i <= 3; ++i) {
            // for i rounds (a run's start counts as two steps)
            const int c = (int)((all + ctas * i - 1) / (ctas * i)) + (i < 3);
            const unsigned rounds = (groups * min(units_of(c), 1 << 20) + ctas - 1) / ctas, cost = rounds * (c + 2);
            if (cost < least) {
                least = cost;
                run = c;
            }
        }
    }
    const int per = units_of(run);
    bool waited = false;
    for (int64_t u = blockIdx.x; u < (int64_t)groups * per; u += gridDim.x) {
        const int tile = (int)(u / per) * kLoWarps + warp;
        if (tile >= tiles) break;
        int in = (int)(u % per), sec = 0;
        if constexpr (!SILU)
            for (int c; in >= (c = (p.sec_blocks[sec] + run - 1) / run); ++sec) in -= c;
        const int at = sh.start[tile], n = sh.start[tile + 1] - at;
        const int id = lo_id(p, at), rank = lo_rank(p, id);
        if (rank == 0 && p.in_place) continue;
        const int64_t N = p.sec_n[sec];
        const int last = min(p.sec_blocks[sec], (in + 1) * run);
        uint4 base[S][MT][2], b[S][4][Q];
        auto load_base = [&](int step) {
            const int64_t col = (int64_t)step * 32 + 8 * t;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int i = 16 * m + 8 * h + g;
                        const uint16_t *src = p.base[sec + s] + (at + i) * N + col;
                        base[s][m][h] = make_uint4(0u, 0u, 0u, 0u);
                        if constexpr (VEC) {
                            if (i < n && col < N) base[s][m][h] = __ldcg(reinterpret_cast<const uint4 *>(src));
                        } else {
                            uint32_t w[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t x = i < n && col + 2 * k < N ? __ldcg(src + 2 * k) : 0u;
                                const uint32_t y = i < n && col + 2 * k + 1 < N ? __ldcg(src + 2 * k + 1) : 0u;
                                w[k] = x | (y << 16);
                            }
                            base[s][m][h] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
        };
        auto load_b = [&](int step) {
            const int64_t c0 = (int64_t)step * 32 + 8 * (g >> 1) + (g & 1);  // of MMA j: c0 + 2 j
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const uint16_t *brow = p.b + ((int64_t)max(id, 0) * p.N + p.sec_start[sec + s] + c0) * p.rank;
#pragma unroll
                for (int j = 0; j < 4; ++j, brow += 2 * p.rank)
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        const int r = KS == 1 ? 4 * t : 32 * q + 8 * t;
                        const bool in = c0 + 2 * j < N && r < rank;
                        b[s][j][q] = make_uint4(0u, 0u, 0u, 0u);
                        if constexpr (KS == 1) {
                            if (in) {
                                const uint2 w = *reinterpret_cast<const uint2 *>(brow + r);
                                b[s][j][q].x = w.x;
                                b[s][j][q].y = w.y;
                            }
                        } else {
                            if (in) b[s][j][q] = *reinterpret_cast<const uint4 *>(brow + r);
                        }
                    }
            }
            if (rank % 8) {
                // entries past the adapter's rank, whatever they hold, are zero
                auto mask = [&](uint32_t &w, int k) { w = k + 1 < rank ? w : k < rank ? w & 0xffffu : 0u; };
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int q = 0; q < Q; ++q) {
                            const int k = KS == 1 ? 4 * t : 32 * q + 8 * t;
                            mask(b[s][j][q].x, k);
                            mask(b[s][j][q].y, k + 2);
                            if constexpr (KS > 1) {
                                mask(b[s][j][q].z, k + 4);
                                mask(b[s][j][q].w, k + 6);
                            }
                        }
            }
        };
        load_base(in * run);
        load_b(in * run);
        if (!waited) pdl_wait_primary();
        waited = true;
        __syncwarp();  // (the last unit's t is read)
        const int nk = KS == 1 ? 1 : ((rank + 31) / 32) * 2;
        if (rank > 0) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        if (k >= nk) break;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = 16 * m + 8 * h + g, q = KS == 1 ? t : 8 * (k / 2) + 2 * t + k % 2;
                            uint4 *dst = frag + ((m * S + s) * KS + k) * kLoFrag + 32 * h + lane;
                            if (i < n && 4 * q < p.rank)
                                cp_async<16>(dst, p.low + ((int64_t)(at + i) * p.nsec + sec + s) * (p.rank / 4) + q);
                            else
                                *dst = make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
            cp_async_commit();
            cp_async_wait<0>();
        }
        __syncwarp();
        for (int step = in * run; step < last; ++step) {
            const int64_t col = (int64_t)step * 32 + 8 * t;
            float acc[MT][S][4][4];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 &v = base[s][m][h];
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[m][s][j][2 * h] = bf16_lo(w[j]);
                            acc[m][s][j][2 * h + 1] = bf16_hi(w[j]);
                        }
                    }
            if (step + 1 < last) load_base(step + 1);
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if (16 * (KS == 1 ? k : k & ~1) >= rank) break;
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const uint4 *fr = frag + ((m * S + s) * KS + k) * kLoFrag + lane;
                        const uint4 even = fr[0], odd = fr[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint4 &w = b[s][j][KS == 1 ? 0 : k / 2];
                            const uint32_t b0 = k & 1 ? w.z : w.x, b1 = k & 1 ? w.w : w.y;
                            mma_bf16(acc[m][s][j], even.x, odd.x, even.y, odd.y, b0, b1);
                            mma_bf16(acc[m][s][j], even.z, odd.z, even.w, odd.w, b0, b1);
                        }
                    }
                }
            if (step + 1 < last) load_b(step + 1);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if constexpr (SILU) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            acc[m][0][j][i] = lo_silu(acc[m][0][j][i]) * acc[m][1][j][i];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = 16 * m + 8 * h + g;
                    if (i >= n) continue;
                    uint16_t *dst = p.out[sec] + (at + i) * N + col;
                    uint32_t w[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) w[j] = pack_bf16(acc[m][0][j][2 * h], acc[m][0][j][2 * h + 1]);
                    if constexpr (VEC) {
                        if (col < N) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (col + k < N) dst[k] = (uint16_t)(k & 1 ? w[k / 2] >> 16 : w[k / 2] & 0xffffu);
                    }
                }
            }
        }
    }
    // (what runs next waits for this kernel alone)
    pdl_wait_primary();
}

// The same on tcgen05, where TMA can bring base and out (rows of 16-byte units)
// and ranks are up to 64: D (128 tokens x 64 outputs, two such chunks a block) =
// t_hi B^T + t_lo B^T, with the parts of t as rows of 128 bytes, and B's rows as
// they lie.  Work is the bytes of base and out; a CTA takes an equal run of the
// blocks of all tiles, one section of a tile after the other, so that t stays.
// Gate and up are the two chunks of a block.  A block of 128 tokens takes some
// 2500 to 3000 cycles: the three stages' turn is loads 2500, MMAs 1000 (110 each
// at N = 64 and 128 alike, so both chunks of a section go at once), adding 1500,
// out 1000; the bytes would take 2750 at HBM's rate.
//
// Warps: 0 issues the copies of base, B and t, 1 the MMAs (a thread each; with
// a rank inside a k step it first clears what B holds past it), 4 to 11 add D to
// the base where it lies, a thread to a token and half a block, 2 sends the
// results out, 128 or 16 tokens a copy; the rest of a tile below 16 is stored by
// the adding threads, as its neighbours' rows are others'.
constexpr int kLeThreads = 384;
constexpr int kLeStage = 48 * 1024, kLeB = 32 * 1024;  // base's two chunks, then B's
struct LoMaps {
    CUtensorMap t, b, base[kMaxSections], out[kMaxSections];  // 16 tokens
    CUtensorMap base_all[kMaxSections], out_all[kMaxSections];  // a tile's 128
};
template <bool SILU>
struct LoOut {
    static constexpr int COLS = SILU ? 64 : 128;      // outputs of a block
    static constexpr int PARTS = SILU ? 4 : 2;        // operand tiles of t
    static constexpr int STAGES = 3;
    static constexpr int SMEM = 1024 + PARTS * 16384 + STAGES * kLeStage;
};
__device__ __forceinline__ void lt_store(const CUtensorMap *map, const void *src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(smem_u32(src))
                 : "memory");
}

template <bool SILU>
__global__ void __launch_bounds__(kLeThreads, 1)
    lora_many_out_kernel(const __grid_constant__ LoMaps maps, const __grid_constant__ LoraParams p, int pitch) {
    using L = LoOut<SILU>;
    constexpr int ST = L::STAGES;
    constexpr unsigned FULL = 0xffffffffu;
    extern __shared__ __align__(1024) unsigned char lo_raw[];
    unsigned char *const parts = reinterpret_cast<unsigned char *>(
        (reinterpret_cast<uintptr_t>(lo_raw) + 1023) & ~(uintptr_t)1023);
    unsigned char *const stages = parts + L::PARTS * 16384;
    __shared__ LoTiles<false> sh;
    __shared__ uint16_t list[SILU ? 1 : kLoChunk];  // tiles with something to do (SILU: all)
    __shared__ uint64_t full[ST], empty[ST], ready[ST], accfull[2], accfree[2], tfull, tfree;
    __shared__ uint32_t s_tmem;
    __shared__ int s_fail, s_issued, s_parts, s_count[kLeThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    if (tid == 0) {
        pdl_launch_dependents();
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&ready[i], 8);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accfull[i], 1);
            mbar_init(&accfree[i], 8);
        }
        mbar_init(&tfull, 1);
        mbar_init(&tfree, 1);
        fence_mbar_init();
        s_fail = s_issued = s_parts = 0;
    }
    if (warp == 1) tmem_alloc(&s_tmem, 256);
    tc_fence_before();
    const int tiles = lo_tiles<kLtTile>(p, sh);  // (synchronizes)
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    int active = SILU ? tiles : 0;
    for (int t0 = 0; !SILU && t0 < tiles; t0 += kLeThreads) {
        const int i = t0 + tid;
        const bool on = i < tiles && (!p.in_place || lo_rank(p, lo_id(p, sh.start[i])) > 0);
        const unsigned all = __ballot_sync(FULL, on);
        if (lane == 0) s_count[warp] = __popc(all);
        __syncthreads();
        int at = active + __popc(all & ((1u << lane) - 1u));
        for (int w = 0; w < kLeThreads / 32; ++w) {
            if (w < warp) at += s_count[w];
            active += s_count[w];
        }
        if (on) list[at] = (uint16_t)i;
        __syncthreads();
    }

    // ---- the CTA's blocks
    struct Block {
        int64_t left;
        int tile, sec, blk;
        int at, n, id, rank;
        bool fresh;  // t is another than the last block's
    };
    int per = 0;
    for (int s = 0; s < (SILU ? 1 : p.nsec); ++s) per += p.sec_blocks[s];
    auto open = [&](Block &c) {
        const int i = SILU ? c.tile : list[c.tile];
        c.at = sh.start[i];
        c.n = sh.start[i + 1] - c.at;
        c.id = lo_id(p, c.at);
        c.rank = lo_rank(p, c.id);
    };
    auto first = [&] {
        Block c;
        const int64_t all = (int64_t)active * per, from = all * blockIdx.x / gridDim.x;
        c.left = all * (blockIdx.x + 1) / gridDim.x - from;
        c.sec = 0;
        c.fresh = true;
        if (c.left > 0) {
            c.tile = (int)(from / per);
            c.blk = (int)(from - (int64_t)c.tile * per);
            while (c.blk >= p.sec_blocks[c.sec]) c.blk -= p.sec_blocks[c.sec++];
            open(c);
        }
        return c;
    };
    auto next = [&](Block &c) {
        c.fresh = false;
        if (--c.left <= 0) return;
        ++c.blk;
        while (c.blk >= p.sec_blocks[c.sec]) {
            c.blk = 0;
            c.fresh = true;
            if (++c.sec == (SILU ? 1 : p.nsec)) {
                c.sec = 0;
                ++c.tile;
                open(c);
            }
        }
    };
    bool ok = true;
    uint32_t it = 0, t = 0;
    if (warp == 0) {
        if (lane == 0) {
            for (Block c = first(); c.left > 0; next(c), ++it) {
                const uint32_t s = it % ST;
                if (it >= ST && !(ok = lt_wait(&empty[s], ((it / ST) & 1) ^ 1, &s_fail))) break;
                unsigned char *st = stages + s * kLeStage;
                const int col = c.blk * L::COLS;
                const bool all = c.n > 32;  // (a copy takes 100 cycles to issue)
                const int boxes = all ? 8 : (c.n + 15) / 16;
                const int chunks = SILU || col + 64 < p.sec_n[c.sec] ? 2 : 1;
                mbar_expect_tx(&full[s], chunks * boxes * 2048 + 2 * 8192);
                for (int x = 0; x < chunks; ++x) {
                    const int sec = SILU ? x : c.sec, at = SILU ? col : col + 64 * x;
                    if (all)
                        tma_load_2d(st + x * 16384, &maps.base_all[sec], at, c.at, &full[s]);
                    else
                        for (int b = 0; b < boxes; ++b)
                            tma_load_2d(st + x * 16384 + b * 2048, &maps.base[sec], at, c.at + 16 * b, &full[s]);
                }
                for (int x = 0; x < 2; ++x)
                    tma_load_2d(st + kLeB + x * 8192, &maps.b, 0,
                                (int)(max(c.id, 0) * p.N + p.sec_start[SILU ? x : c.sec]) +
                                    (SILU ? col : col + 64 * x),
                                &full[s]);
                s_issued = it + 1;
                if (!c.fresh) continue;
                if (t == 0) {
                    pdl_wait_primary();
                    asm volatile("fence.proxy.async;" ::: "memory");
                } else if (!(ok = lt_wait(&tfree, (t - 1) & 1, &s_fail))) {
                    break;
                }
                mbar_expect_tx(&tfull, L::PARTS * 16384);
                for (int x = 0; x < L::PARTS; ++x)
                    tma_load_2d(parts + x * 16384, &maps.t, ((SILU ? 0 : 2 * c.sec) + x) * pitch, c.at, &tfull);
                s_parts = ++t;
            }
        }
    } else if (warp == 1) {
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(L::COLS >> 3) << 17) |
                               ((uint32_t)(kLtTile >> 4) << 24);
        for (Block c = first(); c.left > 0; ++it) {
            const uint32_t s = it % ST, buf = it & 1;
            unsigned char *bs = stages + s * kLeStage + kLeB;
            if (c.fresh && !__all_sync(FULL, lt_wait(&tfull, t++ & 1, &s_fail))) break;
            if (!__all_sync(FULL, lt_wait(&full[s], (it / ST) & 1, &s_fail))) break;
            if (it >= 2 && !__all_sync(FULL, lt_wait(&accfree[buf], ((it >> 1) - 1) & 1, &s_fail))) break;
            if (c.rank % 16) {
                for (int r = lane; r < 128; r += 32)
                    for (int k = c.rank; k % 16; ++k)
                        *reinterpret_cast<uint16_t *>(bs + r * 128 + (((k >> 3) ^ (r & 7)) << 4) + (k & 7) * 2) = 0;
                fence_proxy_async();
                __syncwarp();
            }
            tc_fence_after();
            const int nk = (c.rank + 15) / 16;
            Block then = c;
            next(then);
            if (lane == 0) {
                // (both chunks of a section at once, 128 outputs, half the MMAs)
                for (int x = 0; x < (SILU ? 2 : 1); ++x) {
                    const uint64_t b = smem_desc_sw128(smem_u32(bs + x * 8192));
                    for (int h = 0; h < 2; ++h) {
                        const uint64_t a = smem_desc_sw128(smem_u32(parts + (2 * x + h) * 16384));
                        for (int k = 0; k < nk; ++k)
                            lt_mma(tmem + buf * 128 + x * 64, a + 2 * k, b + 2 * k, idesc, h + k > 0 ? 1u : 0u);
                    }
                }
                tc_commit(&accfull[buf]);
                if (then.left > 0 && then.fresh) tc_commit(&tfree);
            }
            __syncwarp();
            c = then;
        }
    } else if (warp == 2) {
        if (lane == 0) {
            for (Block c = first(); c.left > 0; next(c), ++it) {
                const uint32_t s = it % ST;
                if (!(ok = lt_wait(&ready[s], (it / ST) & 1, &s_fail))) break;
                const int col = c.blk * L::COLS;
                for (int x = 0; x < (SILU ? 1 : 2); ++x)
                    if (col + 64 * x < p.sec_n[c.sec]) {
                        unsigned char *src = stages + s * kLeStage + x * 16384;
                        if (c.n == kLtTile)
                            lt_store(&maps.out_all[c.sec], src, col + 64 * x, c.at);
                        else
                            for (int b = 0; b < c.n / 16; ++b)
                                lt_store(&maps.out[c.sec], src + b * 2048, col + 64 * x, c.at + 16 * b);
                    }
                asm volatile("cp.async.bulk.commit_group;\n cp.async.bulk.wait_group.read 0;" ::: "memory");
                mbar_arrive(&empty[s]);
            }
            asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        }
    } else if (warp >= 4) {
        const int q = warp & 3, row = q * 32 + lane, half = (warp - 4) / 4;
        for (Block c = first(); c.left > 0; next(c), ++it) {
            const uint32_t s = it % ST, buf = it & 1;
            ok = lt_wait(&full[s], (it / ST) & 1, &s_fail) && lt_wait(&accfull[buf], (it >> 1) & 1, &s_fail);
            if (!__all_sync(FULL, ok)) break;
            tc_fence_after();
            const int64_t N = p.sec_n[c.sec];
            // 64 outputs of a chunk, or 32 of both
            const int in = SILU ? 32 * half : 0, chunk = SILU ? 0 : half;
            const int64_t col = (int64_t)c.blk * L::COLS + 64 * chunk + in;
            unsigned char *src = stages + s * kLeStage + chunk * 16384 + row * 128;
            if (q * 32 < c.n && col < N) {
                float v[2][32];
                if (c.rank > 0) {
                    const uint32_t d = tmem + buf * 128 + chunk * 64 + in + ((uint32_t)(q * 32) << 16);
                    tc_ld32_async(d, v[0]);
                    tc_ld32_async(d + (SILU ? 64 : 32), v[1]);
                    tc_ld_wait(v[0]);
                    tc_ld_tie(v[1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 64; ++i) v[i / 32][i % 32] = -0.f;  // (a base of -0 stays)
                }
                const bool sent = row < (c.n & ~15);
                uint16_t *dst = p.out[c.sec] + (int64_t)(c.at + row) * N + col;
#pragma unroll
                for (int j = 0; j < (SILU ? 4 : 8); ++j) {  // 8 outputs
                    unsigned char *place = src + (((in / 8 + j) ^ (row & 7)) << 4);
                    const uint4 b = *reinterpret_cast<const uint4 *>(place);
                    const uint4 e = SILU ? *reinterpret_cast<const uint4 *>(place + 16384) : b;
                    const uint32_t bw[4] = {b.x, b.y, b.z, b.w}, ew[4] = {e.x, e.y, e.z, e.w};
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = 8 * j + 2 * i;
                        float lo = bf16_lo(bw[i]) + v[SILU ? 0 : at / 32][at % 32];
                        float hi = bf16_hi(bw[i]) + v[SILU ? 0 : at / 32][at % 32 + 1];
                        if constexpr (SILU) {
                            lo = lo_silu(lo) * (bf16_lo(ew[i]) + v[1][at]);
                            hi = lo_silu(hi) * (bf16_hi(ew[i]) + v[1][at + 1]);
                        }
                        w[i] = pack_bf16(lo, hi);
                    }
                    if (sent)
                        *reinterpret_cast<uint4 *>(place) = make_uint4(w[0], w[1], w[2], w[3]);
                    else if (row < c.n && col + 8 * j < N)
                        *reinterpret_cast<uint4 *>(dst + 8 * j) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            tc_fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&accfree[buf]);
                mbar_arrive(&ready[s]);
            }
        }
    }
    // ---- teardown: without a wait that ran out, every copy and MMA was waited for
    tc_fence_before();
    __syncthreads();
    if (s_fail) {
        if (tid == 0) {
            for (int k = max(0, s_issued - ST); k < s_issued; ++k)
                if (!mbar_wait(&full[k % ST], (k / ST) & 1)) break;
            if (s_parts > 0) mbar_wait(&tfull, (s_parts - 1) & 1);
        }
        if (tid == 32) {
            tc_commit(&accfull[0]);  // completes after every MMA this thread issued
            mbar_wait(&accfull[0], 0, 1000000ull);
            mbar_wait(&accfull[0], 1, 1000000ull);
        }
    }
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 256);
    // (what runs next waits for this kernel alone)
    pdl_wait_primary();
}

// ---------------------------------------------------------------- host side
template <int KS, bool SILU, bool VEC>
static cudaError_t launch_few(const LoraParams &p, int grid, cudaStream_t st) {
    // Rows of B in 32-byte units, where adapters do not have smaller ranks of their
    // own (whose lanes then have less to do together): 250 single tokens over 32
    // adapters of rank 64, 5120 to 7168, 33.4 us against 34.8, gate and up of 13824
    // 57.4 against 59.5; ranks 8 to 64, 54 tokens, 18.6 against 17.6.  Where B begins does not count: ranks go to
    // the same k steps wherever it does, so that the sums are the same.
    const bool wide = KS >= 4 && !p.ranks && p.rank % 16 == 0;
    return launch_pdl(wide ? reinterpret_cast<const void *>(lora_few_expand_kernel<KS, SILU, VEC, (KS >= 4)>)
                           : reinterpret_cast<const void *>(lora_few_expand_kernel<KS, SILU, VEC, false>),
                      dim3(grid), kLoThreads, 0, st, p);
}
template <int KS>
static cudaError_t pick_few(const LoraParams &p, int grid, cudaStream_t st) {
    if (p.silu)
        return p.vec ? launch_few<KS, true, true>(p, grid, st) : launch_few<KS, true, false>(p, grid, st);
    return p.vec ? launch_few<KS, false, true>(p, grid, st) : launch_few<KS, false, false>(p, grid, st);
}

// A share of K: 2048 inputs (a CTA's loads at once), more where there would be
// more than eight.
static int lora_share(int K) { return std::max(2048, ((K + 7) / 8 + 255) / 256 * 256); }

static cudaError_t launch_lora_few(LoraParams p, cudaStream_t st) {
    // (no more tiles than these)
    const int64_t tiles = std::min<int64_t>(p.M, std::min<int64_t>(p.M, (int64_t)p.adapters + 1) + p.M / kLoTile);
    const int full = 2 * num_sms();
    p.share = lora_share(p.K);
    p.b32 = (reinterpret_cast<uintptr_t>(p.b) & 31) == 0;
    const int64_t down = tiles * p.nsec * ((p.rank + 15) / 16) * p.ks;
    // (54 tokens of ranks 8 to 64 17.6 us, in 16-byte loads 18.6)
    const bool wide = ((reinterpret_cast<uintptr_t>(p.x) | reinterpret_cast<uintptr_t>(p.a)) & 31) == 0;
    cudaError_t e = launch_pdl(wide ? reinterpret_cast<const void *>(lora_few_shrink_kernel<true>)
                                    : reinterpret_cast<const void *>(lora_few_shrink_kernel<false>),
                               dim3((unsigned)std::min<int64_t>(full, down)), kLoThreads, 0, st, p);
    if (e != cudaSuccess) return e;
    int64_t octets = 0;
    for (int s = 0; s < (p.silu ? 1 : p.nsec); ++s) {
        p.sec_blocks[s] = (int)((p.sec_n[s] + 32 * kLoWarps - 1) / (32 * kLoWarps));
        octets += p.sec_blocks[s];
    }
    const int grid = (int)std::min<int64_t>(full, tiles * octets);
    return p.rank <= 16   ? pick_few<1>(p, grid, st)
           : p.rank <= 32 ? pick_few<2>(p, grid, st)
           : p.rank <= 64 ? pick_few<4>(p, grid, st)
                          : pick_few<8>(p, grid, st);
}

template <int KS, bool SILU, bool VEC>
static cudaError_t launch_many(const LoraParams &p, cudaStream_t st) {
    using L = LoMany<KS, SILU>;
    const void *kfn = reinterpret_cast<const void *>(lora_many_expand_kernel<KS, SILU, VEC>);
    cudaError_t e = allow_smem(kfn, L::SMEM);
    if (e == cudaSuccess) e = prefer_max_shared(kfn);
    if (e != cudaSuccess) return e;
    const dim3 grid(L::CTAS * num_sms());
    if (p.adapters > 0) return launch_pdl(kfn, grid, kLoThreads, L::SMEM, st, p);
    // (alone: what it reads ahead of its wait is another kernel's)
    LoraParams args = p;
    void *argv[] = {&args};
    return cudaLaunchKernel(kfn, grid, dim3(kLoThreads), argv, L::SMEM, st);
}
template <int KS>
static cudaError_t pick_many(const LoraParams &p, cudaStream_t st) {
    if (p.silu) return p.vec ? launch_many<KS, true, true>(p, st) : launch_many<KS, true, false>(p, st);
    return p.vec ? launch_many<KS, false, true>(p, st) : launch_many<KS, false, false>(p, st);
}

template <bool SILU>
static int launch_out(LoraParams p, int pitch, cudaStream_t st) {
    using L = LoOut<SILU>;
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    LoMaps maps{};
    int rc = encode_2d(&maps.t, bf, 2, p.low, (int64_t)p.nsec * 2 * pitch, p.M, 64, kLtTile, sw, "low-rank sums");
    if (!rc) rc = encode_2d(&maps.b, bf, 2, p.b, p.rank, p.adapters * p.N, 64, 64, sw, "adapters");
    for (int s = 0; s < p.nsec && !rc; ++s) {
        p.sec_blocks[s] = (int)((p.sec_n[s] + L::COLS - 1) / L::COLS);
        if (p.sec_n[s] == 0) continue;
        rc = encode_2d(&maps.base[s], bf, 2, p.base[s], p.sec_n[s], p.M, 64, 16, sw, "base");
        if (!rc) rc = encode_2d(&maps.base_all[s], bf, 2, p.base[s], p.sec_n[s], p.M, 64, kLtTile, sw, "base");
        if (rc || (SILU && s)) continue;
        rc = encode_2d(&maps.out[s], bf, 2, p.out[s], p.sec_n[s], p.M, 64, 16, sw, "outputs");
        if (!rc) rc = encode_2d(&maps.out_all[s], bf, 2, p.out[s], p.sec_n[s], p.M, 64, kLtTile, sw, "outputs");
    }
    if (rc) return rc;
    const void *kfn = reinterpret_cast<const void *>(lora_many_out_kernel<SILU>);
    cudaError_t e = allow_smem(kfn, L::SMEM);
    if (e == cudaSuccess) e = launch_pdl(kfn, dim3(num_sms()), kLeThreads, L::SMEM, st, maps, p, pitch);
    return e == cudaSuccess ? GWA_OK : set_error(GWA_ERR_CUDA, "lora: %s", cudaGetErrorString(e));
}

// (rows of t's parts in the tensor cores' k steps)
static int lora_pitch(int rank) { return (rank + 15) / 16 * 16; }

// Outputs on tcgen05 where TMA can bring them (and a row of B has an int's
// coordinate), for long runs: a block takes some 2400 cycles whatever its tokens.
// The whole call there against warp-level MMAs, us: rank 16, 5120 to 7168, one
// run of 512 tokens 24.7 / 20.6, 1024 26.8 / 24.8, 2048 31.0 / 30.9, 4096 48.5 /
// 57.1; rank 64 512 29.5 / 33.4, 1024 34.9 / 38.7; 5560 tokens, 13824 to 5120, 74.8
// / 94.3; gate and up of 13824, rank 32, 2048 64.2 / 75.9, 4096 104.5 / 132.7, rank
// 64, 512 35.5 / 41.2.  54 runs of 30 to 60 tokens 64 / 53.
constexpr int kLoOutTokens = 2048, kLoOutWide = 512, kLoOutRun = 64;
static bool lora_out_tc(const LoraParams &p) {
    return p.vec && p.adapters > 0 && p.rank <= 64 && p.adapters * p.N <= 0x7ffffe00LL &&
           p.M >= (p.rank > 32 ? kLoOutWide : kLoOutTokens);
}

static int launch_lora_many(LoraParams p, bool out_tc, cudaStream_t st) {
    const int pitch = lora_pitch(p.rank);
    const int rows = p.nsec * p.rank, cols = std::min(256, (rows + 15) / 16 * 16);
    if (p.adapters > 0) {
        CUtensorMap xmap, xmap16, amap;
        const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
        const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
        int rc = encode_2d(&xmap, bf, 2, p.x, p.K, p.M, 64, kLtTile, sw, "activations");
        if (!rc) rc = encode_2d(&xmap16, bf, 2, p.x, p.K, p.M, 64, 16, sw, "activations");
        if (!rc) rc = encode_2d(&amap, bf, 2, p.a, p.K, (int64_t)p.adapters * rows, 64, cols, sw, "adapters");
        if (rc) return rc;
        int half = 16;  // columns of an accumulator: a power of two, both at least 32
        while (half < cols) half *= 2;
        const int stages = std::min(kLtStages, kLtSmem / ((kLtTile + cols) * 128));
        const size_t smem = 1024 + (size_t)stages * (kLtTile + cols) * 128;
        const void *kfn = reinterpret_cast<const void *>(lora_many_shrink_kernel);
        cudaError_t e = allow_smem(kfn, 1024 + kLtSmem);
        if (e == cudaSuccess) e = prefer_max_shared(kfn);
        if (e == cudaSuccess)
            e = launch_pdl(kfn, dim3(num_sms()), kLoThreads, smem, st, xmap, xmap16, amap, p, cols, half, stages);
        if (e == cudaSuccess) {
            const int64_t units = (int64_t)p.M * p.nsec * (out_tc ? pitch : p.rank) / 4;
            e = launch_pdl(out_tc ? reinterpret_cast<const void *>(lora_many_join_kernel<true>)
                                  : reinterpret_cast<const void *>(lora_many_join_kernel<false>),
                           dim3((unsigned)std::min<int64_t>(num_sms(), (units + kLoThreads - 1) / kLoThreads)),
                           kLoThreads, 0, st, p, pitch);
        }
        if (e != cudaSuccess) return set_error(GWA_ERR_CUDA, "lora: %s", cudaGetErrorString(e));
    }
    if (out_tc) return p.silu ? launch_out<true>(p, pitch, st) : launch_out<false>(p, pitch, st);
    for (int s = 0; s < (p.silu ? 1 : p.nsec); ++s) p.sec_blocks[s] = (int)((p.sec_n[s] + 31) / 32);
    const cudaError_t e = p.rank <= 16   ? pick_many<1>(p, st)
                          : p.rank <= 32 ? pick_many<2>(p, st)
                          : p.rank <= 64 ? pick_many<4>(p, st)
                                         : pick_many<8>(p, st);
    return e == cudaSuccess ? GWA_OK : set_error(GWA_ERR_CUDA, "lora: %s", cudaGetErrorString(e));
}

// The most shares of K: a few tokens' exactly so many, many tokens' up to so
// many (their kernel chooses).
constexpr int kLoShares = 8, kLoSums = 3 * kLoChunk;  // (of all tokens together)
static int lora_shares(int64_t M, int K) {
    if (M <= kLoSort) return (K + lora_share(K) - 1) / lora_share(K);
    return (int)std::min<int64_t>(kLoShares, kLoSums / M);
}

// 256 bytes (the shares of K that were chosen), the partial sums, and of many
// tokens what they add up to (see lora_many_join_kernel); enough for either way
// of taking more than kLoSort tokens (see launch_lora), and for fewer tokens
// (the whole shares times M go up and down): up to kLoSort tokens have kLoShares
// shares at most, and more have no more sums than both factors allow.
static int64_t lora_sums(int64_t M, int K) { return (int64_t)lora_shares(M, K) * M; }
size_t lora_workspace_bytes(int64_t M, int64_t K, int nsec, int rank) {
    const int64_t m = std::min<int64_t>(M, kLoChunk);
    const int64_t rows = m <= kLoSort ? lora_sums(m, (int)K) : std::min<int64_t>(kLoShares * m, kLoSums);
    return 256 + (size_t)(rows * rank + (m > kLoSort ? m * lora_pitch(rank) : 0)) * nsec * sizeof(float);
}

// Runs shorter than this on the whole go kLoSort tokens at a time through the
// kernels that put them in order.  520 tokens of 32 adapters in runs of 1, 3, 5
// and 8, in order against as they come, us: rank 16, 5120 to 7168, 45 / 158, 46 /
// 70, 45 / 43, 43 / 34; gate and up of 13824, rank 32, 75 / 295, 74 / 115, 72 / 76,
// 64 / 55; rank 16, 13824 to 5120, 43 / 314, 45 / 117, 43 / 72, 42 / 57; 1024 to
// 1024, 25 / 43, 27 / 27, 27 / 21, 23 / 19.  The sides meet at runs of 3 (small
// projections) to more than 8 (many inputs).
constexpr int kLoShortRun = 8;

int launch_lora(LoraParams p, int64_t M, int64_t runs, void *workspace, cudaStream_t st) {
    // (both rules are of the call's mean run: a launch's own runs are not known)
    const int64_t chunk = runs > M / kLoShortRun ? kLoSort : kLoChunk;
    const bool long_runs = runs <= M / kLoOutRun;
    p.shares = static_cast<int32_t *>(workspace);
    p.part = reinterpret_cast<float *>(static_cast<unsigned char *>(workspace) + 256);
    for (int64_t m = 0; m < M; m += chunk) {
        p.M = (int)std::min<int64_t>(chunk, M - m);
        p.ks = lora_shares(p.M, p.K);
        p.low = reinterpret_cast<uint4 *>(p.part + lora_sums(p.M, p.K) * p.nsec * p.rank);
        int rc = GWA_OK;
        if (p.M <= kLoSort) {
            const cudaError_t e = launch_lora_few(p, st);
            if (e != cudaSuccess) rc = set_error(GWA_ERR_CUDA, "lora: %s", cudaGetErrorString(e));
        } else {
            rc = launch_lora_many(p, long_runs && lora_out_tc(p), st);
        }
        if (rc) return rc;
        p.x += (int64_t)p.M * p.K;
        p.ids += p.M;
        for (int s = 0; s < p.nsec; ++s) p.base[s] += p.M * p.sec_n[s];
        for (int s = 0; s < (p.silu ? 1 : p.nsec); ++s) p.out[s] += p.M * p.sec_n[s];
    }
    return GWA_OK;
}

unsigned int lora_timeouts(bool reset) {
    unsigned int v = 0;
    cudaMemcpyFromSymbol(&v, g_lora_timeouts, sizeof v);
    if (reset) {
        const unsigned int z = 0;
        cudaMemcpyToSymbol(g_lora_timeouts, &z, sizeof z);
    }
    return v;
}

}  // namespace gwa
