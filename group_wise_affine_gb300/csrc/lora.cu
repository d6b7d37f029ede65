// Low-rank adapters of many requests at once, added to a shared projection's
// output ("Sanctum-MLX", "File map": lora.rs merges one adapter into the
// weights at load; here each token brings its own and nothing is merged):
//
//   t[m,s,:] = scale_a (A_a[s] x_m),       a = ids[m], rank_a rows of A_a[s]
//   y_s[m,n] = base_s[m,n] + B_a[s][n,:] . t[m,s,:]
//
// and for the gated projection SiLU(y_0) y_1.  Two kernels: x against the A's
// (shrink), whose few results a token go through the workspace, and those
// against the B's (expand).  Products are exact, sums fp32; t enters its
// product as two bf16 parts (together 2^-17 of it), so the output's rounding
// is the only one to count.
//
// Tokens of one adapter are taken together, 16 to a tile, so that an adapter
// is read once for them: up to kLoSort tokens every CTA puts them in the order
// of their adapters itself, beyond that runs of neighbours are taken as they
// come (a prompt's tokens are neighbours).
#include <algorithm>

#include "cluster.cuh"
#include "common.cuh"
#include "internal.h"
#include "mma.cuh"

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
    int key[FEW ? kLoSort : 1];
    int w_max[kLoWarps], w_sum[kLoWarps];
    __device__ __forceinline__ int token(int place) const { return FEW ? order[place] : place; }
};

// A token's adapter, -1 for none.
__device__ __forceinline__ int lo_id(const LoraParams &p, int tok) {
    const int id = p.ids[tok];
    return (unsigned)id < (unsigned)p.adapters ? id : -1;
}
__device__ __forceinline__ int lo_rank(const LoraParams &p, int id) {
    return id < 0 ? 0 : p.ranks ? min(max(p.ranks[id], 0), p.rank) : p.rank;
}

// Cuts the tokens into tiles (all threads of the CTA); returns their number.
template <bool FEW, int TM>
__device__ int lo_tiles(const LoraParams &p, LoTiles<FEW> &sh) {
    constexpr int PER = FEW ? 1 : kLoPer;
    constexpr unsigned FULL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    int id[PER], before;  // the places of this thread, and the one in front
    if constexpr (FEW) {
        const int mine = tid < p.M ? lo_id(p, tid) : 0x7fffffff;
        if (tid < p.M && blockIdx.x == 0 && p.status && p.ids[tid] >= p.adapters) atomicOr(p.status, 1);
        sh.key[tid] = mine;
        __syncthreads();
        int at = 0;
        for (int j = 0; j < p.M; ++j) {
            const int k = sh.key[j];
            at += k < mine || (k == mine && j < tid);
        }
        __syncthreads();
        if (tid < p.M) {
            sh.order[at] = (uint16_t)tid;
            sh.key[at] = mine;
        }
        __syncthreads();
        id[0] = sh.key[tid];
        before = tid ? sh.key[tid - 1] : 0x7ffffffe;
    } else {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int tok = tid * PER + j;
            id[j] = tok < p.M ? lo_id(p, tok) : 0x7fffffff;
            if (tok < p.M && blockIdx.x == 0 && p.status && p.ids[tok] >= p.adapters) atomicOr(p.status, 1);
        }
        before = tid == 0 ? 0x7ffffffe : tid * PER <= p.M ? lo_id(p, tid * PER - 1) : 0x7fffffff;
    }
    // where the run of this thread's first place starts
    int last = -1, prev = before;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        if (id[j] != prev) last = tid * PER + j;
        prev = id[j];
    }
    int incl = last;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, incl, o);
        if (lane >= o) incl = max(incl, v);
    }
    if (lane == 31) sh.w_max[warp] = incl;
    __syncthreads();
    int run = __shfl_up_sync(FULL, incl, 1);
    if (lane == 0) run = -1;
    for (int w = 0; w < warp; ++w) run = max(run, sh.w_max[w]);
    // places where a tile starts
    int n = 0, r = run;
    prev = before;
    uint32_t starts = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        const int at = tid * PER + j;
        if (id[j] != prev) r = at;
        prev = id[j];
        if (at < p.M && (at - r) % TM == 0) {
            starts |= 1u << j;
            ++n;
        }
    }
    int sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(FULL, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sh.w_sum[warp] = sum;
    __syncthreads();
    int at = sum - n, total = 0;
    for (int w = 0; w < kLoWarps; ++w) {
        if (w < warp) at += sh.w_sum[w];
        total += sh.w_sum[w];
    }
    for (; starts; starts &= starts - 1) sh.start[at++] = (uint16_t)(tid * PER + __ffs(starts) - 1);
    if (tid == 0) sh.start[total] = (uint16_t)p.M;
    __syncthreads();
    return total;
}

__device__ __forceinline__ uint4 lo_load(const uint16_t *p, bool ok) {
    return ok ? *reinterpret_cast<const uint4 *>(p) : make_uint4(0u, 0u, 0u, 0u);
}

// part[k][m][s][r]: split k's share of scale A x.  A unit is a tile, 16 rows
// of one section's A and a share of K; a warp takes 128 inputs at a time, 16
// rows of A against 8 or 16 tokens, both straight from global memory as MMA
// fragments (a lane's 16 bytes are the k positions of two MMAs, in the same
// order on both sides).
template <bool FEW>
__global__ void __launch_bounds__(kLoThreads, 2) lora_shrink_kernel(LoraParams p) {
    __shared__ LoTiles<FEW> sh;
    __shared__ float s_acc[kLoWarps][16 * kLoTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    if (tid == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int tiles = lo_tiles<FEW, kLoTile>(p, sh);
    const int blocks = p.nsec * ((p.rank + 15) / 16), per = blocks * p.ks;
    const int chunks = p.K / 32;
    for (int64_t u = blockIdx.x; u < (int64_t)tiles * per; u += gridDim.x) {
        const int tile = (int)(u / per), rem = (int)(u % per);
        const int k = rem % p.ks, sec = rem / p.ks % p.nsec, r0 = rem / p.ks / p.nsec * 16;
        const int at = sh.start[tile], n = sh.start[tile + 1] - at;
        const int id = lo_id(p, sh.token(at)), rank = lo_rank(p, id);
        if (r0 >= rank) continue;
        const uint16_t *a0 = p.a + (((int64_t)id * p.nsec + sec) * p.rank + r0 + g) * p.K + 8 * t;
        const uint16_t *a1 = a0 + (int64_t)8 * p.K;
        const bool in0 = r0 + g < rank, in1 = r0 + g + 8 < rank;
        const bool tok0 = g < n, tok1 = g + 8 < n;
        const uint16_t *x0 = p.x + (int64_t)sh.token(at + (tok0 ? g : 0)) * p.K + 8 * t;
        const uint16_t *x1 = p.x + (int64_t)sh.token(at + (tok1 ? g + 8 : 0)) * p.K + 8 * t;
        const bool wide = n > 8;
        float acc[2][4] = {};
        for (int c0 = (k * kLoWarps + warp) * 4; c0 < chunks; c0 += p.ks * kLoWarps * 4) {
            uint4 va[4], vb[4], xa[4], xb[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const bool ok = c0 + c < chunks;
                const int64_t o = (int64_t)(c0 + c) * 32;
                va[c] = lo_load(a0 + o, ok && in0);
                vb[c] = lo_load(a1 + o, ok && in1);
                xa[c] = lo_load(x0 + o, ok && tok0);
                xb[c] = lo_load(x1 + o, ok && tok1);
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                mma_bf16(acc[0], va[c].x, vb[c].x, va[c].y, vb[c].y, xa[c].x, xa[c].y);
                mma_bf16(acc[0], va[c].z, vb[c].z, va[c].w, vb[c].w, xa[c].z, xa[c].w);
                if (wide) {
                    mma_bf16(acc[1], va[c].x, vb[c].x, va[c].y, vb[c].y, xb[c].x, xb[c].y);
                    mma_bf16(acc[1], va[c].z, vb[c].z, va[c].w, vb[c].w, xb[c].z, xb[c].w);
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
        const int tok = tid / 16, r = tid % 16;
        if (tok < n && r0 + r < p.rank) {
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kLoWarps; ++w) v += s_acc[w][tid];
            if (p.scale) v *= p.scale[id];
            p.part[(((int64_t)k * p.M + sh.token(at + tok)) * p.nsec + sec) * p.rank + r0 + r] = v;
        }
        __syncthreads();
    }
}

// out = base + B t.  A warp takes a tile and some steps of 32 outputs of one
// section; t as fragments of the MMA's 16 rows, hi and lo bf16 parts, B's rows
// straight from global memory.  Lane t's outputs of a step are eight
// neighbours (column c of the step's MMA j is output 8 (c / 2) + 2 j + c % 2).
template <bool FEW, int KS, bool SILU, bool VEC>
__global__ void __launch_bounds__(kLoThreads) lora_expand_kernel(LoraParams p) {
    constexpr int S = SILU ? 2 : 1;
    __shared__ LoTiles<FEW> sh;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    if (tid == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int tiles = lo_tiles<FEW, kLoTile>(p, sh);
    const int64_t units = (int64_t)tiles * p.blocks;
    for (int64_t u = (int64_t)blockIdx.x * kLoWarps + tid / 32; u < units; u += (int64_t)gridDim.x * kLoWarps) {
        // few tokens: a CTA's warps side by side along one tile's outputs;
        // many: a tile each, over the same outputs
        const int tile = FEW ? (int)(u / p.blocks) : (int)(u % tiles);
        int blk = FEW ? (int)(u % p.blocks) : (int)(u / tiles), sec = 0;
        if constexpr (!SILU)
            while (blk >= p.sec_blocks[sec]) blk -= p.sec_blocks[sec++];
        const int at = sh.start[tile], n = sh.start[tile + 1] - at;
        const int id = lo_id(p, sh.token(at)), rank = lo_rank(p, id);
        if (rank == 0 && p.in_place) continue;
        const int64_t N = p.sec_n[sec];
        const bool live[2] = {g < n, g + 8 < n};
        const int64_t tok[2] = {sh.token(at + (live[0] ? g : 0)), sh.token(at + (live[1] ? g + 8 : 0))};
        // ---- t: of a pair of k steps, lane t's ranks are 8 t .. 8 t + 7
        uint32_t hi[S][KS][4], lo[S][KS][4];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = KS == 1 ? 4 * t : 32 * (j / 2) + 8 * t + 4 * (j & 1);
                    float v[4] = {0.f, 0.f, 0.f, 0.f};
                    if (live[h] && r < rank) {
                        const float *src = p.part + (tok[h] * p.nsec + sec + s) * p.rank + r;
                        for (int k = 0; k < p.ks; ++k) {
                            const float4 f = *reinterpret_cast<const float4 *>(src + (int64_t)k * p.M * p.nsec * p.rank);
                            v[0] += f.x;
                            v[1] += f.y;
                            v[2] += f.z;
                            v[3] += f.w;
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (r + i >= rank) v[i] = 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t w = pack_bf16(v[2 * i], v[2 * i + 1]);
                        hi[s][j][h + 2 * i] = w;
                        lo[s][j][h + 2 * i] = pack_bf16(v[2 * i] - bf16_lo(w), v[2 * i + 1] - bf16_hi(w));
                    }
                }
        const uint16_t *brow = p.b + ((int64_t)max(id, 0) * p.N + p.sec_start[sec]) * p.rank;
        for (int step = 0; step < p.steps; ++step) {
            const int64_t n0 = ((int64_t)blk * p.steps + step) * 32;
            if (n0 >= N) break;
            const int64_t col = n0 + 8 * t;
            float acc[S][4][4];
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint16_t *src = p.base[sec + s] + tok[h] * N + col;
                    if constexpr (VEC) {
                        const uint4 v = lo_load(src, live[h] && col < N);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            acc[s][j][2 * h] = bf16_lo(w[j]);
                            acc[s][j][2 * h + 1] = bf16_hi(w[j]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            acc[s][i / 2][2 * h + (i & 1)] =
                                live[h] && col + i < N ? __uint_as_float((uint32_t)src[i] << 16) : 0.f;
                    }
                }
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t c = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
                    const uint16_t *b = brow + (s * N + c) * p.rank;
                    // entries past the adapter's rank, whatever they hold, are zero
                    auto mask = [&](uint32_t w, int r) {
                        return r + 1 < rank ? w : r < rank ? w & 0xffffu : 0u;
                    };
                    if constexpr (KS == 1) {
                        uint2 w = make_uint2(0u, 0u);
                        if (c < N && 4 * t < rank) w = *reinterpret_cast<const uint2 *>(b + 4 * t);
                        w.x = mask(w.x, 4 * t);
                        w.y = mask(w.y, 4 * t + 2);
                        mma_bf16(acc[s][j], hi[s][0][0], hi[s][0][1], hi[s][0][2], hi[s][0][3], w.x, w.y);
                        mma_bf16(acc[s][j], lo[s][0][0], lo[s][0][1], lo[s][0][2], lo[s][0][3], w.x, w.y);
                    } else {
#pragma unroll
                        for (int q = 0; q < KS / 2; ++q) {
                            if (32 * q >= rank) break;
                            const int r = 32 * q + 8 * t;
                            uint4 w = lo_load(b + r, c < N && r < rank);
                            if (rank % 8) {
                                w.x = mask(w.x, r);
                                w.y = mask(w.y, r + 2);
                                w.z = mask(w.z, r + 4);
                                w.w = mask(w.w, r + 6);
                            }
                            uint32_t(&h0)[4] = hi[s][2 * q], (&l0)[4] = lo[s][2 * q];
                            uint32_t(&h1)[4] = hi[s][2 * q + 1], (&l1)[4] = lo[s][2 * q + 1];
                            mma_bf16(acc[s][j], h0[0], h0[1], h0[2], h0[3], w.x, w.y);
                            mma_bf16(acc[s][j], h1[0], h1[1], h1[2], h1[3], w.z, w.w);
                            mma_bf16(acc[s][j], l0[0], l0[1], l0[2], l0[3], w.x, w.y);
                            mma_bf16(acc[s][j], l1[0], l1[1], l1[2], l1[3], w.z, w.w);
                        }
                    }
                }
            if constexpr (SILU) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[0][j][i] = acc[0][j][i] / (1.f + __expf(-acc[0][j][i])) * acc[1][j][i];
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
}

// ------------------------------------------------------------ few tokens
// Both products in one launch: a cluster of CTAs a tile.  Each CTA takes a
// share of K for all of the adapter's rows; the shares' sums go round through
// distributed shared memory, each CTA adding up a part and handing it to all as
// MMA fragments (hi and lo bf16 parts); then each takes a share of the outputs.
// The outputs' first loads (base and B) are on their way before the sums are.
//
// Fragments in shared memory: of a section's k step 32 lanes' hi words, then
// their lo words.
struct LoFragments {
    uint4 hi[32], lo[32];
};

template <int KS, bool SILU, bool VEC>
__global__ void __launch_bounds__(kLoThreads, KS * (SILU ? 2 : 1) <= 4 ? 2 : 1) lora_few_kernel(LoraParams p, int cl) {
    constexpr int S = SILU ? 2 : 1, Q = KS == 1 ? 1 : KS / 2;  // Q: B's loads of a row
    extern __shared__ __align__(16) unsigned char lo_raw[];
    __shared__ LoTiles<true> sh;
    __shared__ float s_acc[kLoWarps][16 * kLoTile];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    const int share = cl > 1 ? (int)cluster_rank() : 0;
    if (tid == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int tiles = lo_tiles<true, kLoTile>(p, sh), tile = blockIdx.x / cl;
    if (tile >= tiles) return;  // (the whole cluster)
    const int at = sh.start[tile], n = sh.start[tile + 1] - at;
    const int id = lo_id(p, sh.token(at)), rank = lo_rank(p, id);
    if (rank == 0 && p.in_place) return;
    const int nb = (rank + 15) / 16, blocks = p.nsec * nb;   // 16-row blocks of A
    const int nk = KS == 1 ? 1 : (nb + 1) & ~1;              // k steps of a section
    float *const red = reinterpret_cast<float *>(lo_raw);
    LoFragments *const frag = reinterpret_cast<LoFragments *>(
        lo_raw + (size_t)p.nsec * ((p.rank + 15) / 16) * 256 * sizeof(float));

    // ---- this CTA's outputs: steps of 32, a warp every eighth
    const int steps = p.blocks, s0 = (int)((int64_t)steps * share / cl), s1 = (int)((int64_t)steps * (share + 1) / cl);
    const bool live[2] = {g < n, g + 8 < n};
    const int64_t tok[2] = {sh.token(at + (live[0] ? g : 0)), sh.token(at + (live[1] ? g + 8 : 0))};
    struct Step {
        int sec;
        int64_t n0, N;
    };
    struct Loads {
        uint4 base[S][2], b[S][4][Q];  // (KS 1: half of b)
    };
    auto place = [&](int step) {
        Step r;
        r.sec = 0;
        if constexpr (!SILU)
            while (step >= p.sec_blocks[r.sec]) step -= p.sec_blocks[r.sec++];
        r.n0 = (int64_t)step * 32;
        r.N = p.sec_n[r.sec];
        return r;
    };
    auto load = [&](Loads &l, int step) {
        const Step r = place(step);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const uint16_t *brow = p.b + ((int64_t)max(id, 0) * p.N + p.sec_start[r.sec + s]) * p.rank;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t c = r.n0 + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    if constexpr (KS == 1) {
                        uint2 w = make_uint2(0u, 0u);
                        if (c < r.N && 4 * t < rank) w = *reinterpret_cast<const uint2 *>(brow + c * p.rank + 4 * t);
                        l.b[s][j][q].x = w.x;
                        l.b[s][j][q].y = w.y;
                    } else {
                        const int rr = 32 * q + 8 * t;
                        l.b[s][j][q] = lo_load(brow + c * p.rank + rr, c < r.N && rr < rank);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t col = r.n0 + 8 * t;
                const uint16_t *src = p.base[r.sec + s] + tok[h] * r.N + col;
                if constexpr (VEC) {
                    l.base[s][h] = lo_load(src, live[h] && col < r.N);
                } else {
                    uint32_t w[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t x = live[h] && col + 2 * i < r.N ? src[2 * i] : 0u;
                        const uint32_t y = live[h] && col + 2 * i + 1 < r.N ? src[2 * i + 1] : 0u;
                        w[i] = x | (y << 16);
                    }
                    l.base[s][h] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    };
    auto use = [&](Loads &l, int step) {
        const Step r = place(step);
        float acc[S][4][4];
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t w[4] = {l.base[s][h].x, l.base[s][h].y, l.base[s][h].z, l.base[s][h].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    acc[s][j][2 * h] = bf16_lo(w[j]);
                    acc[s][j][2 * h + 1] = bf16_hi(w[j]);
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
                        mask(l.b[s][j][q].x, k);
                        mask(l.b[s][j][q].y, k + 2);
                        if constexpr (KS > 1) {
                            mask(l.b[s][j][q].z, k + 4);
                            mask(l.b[s][j][q].w, k + 6);
                        }
                    }
        }
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const LoFragments *f = frag + (r.sec + s) * nk;
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                if (32 * q >= rank) break;
#pragma unroll
                for (int b = 0; b < (KS == 1 ? 1 : 2); ++b) {
                    const uint4 hi = f[(KS == 1 ? 0 : 2 * q) + b].hi[lane], lo = f[(KS == 1 ? 0 : 2 * q) + b].lo[lane];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4 &w = l.b[s][j][q];
                        const uint32_t b0 = b ? w.z : w.x, b1 = b ? w.w : w.y;
                        mma_bf16(acc[s][j], hi.x, hi.y, hi.z, hi.w, b0, b1);
                        mma_bf16(acc[s][j], lo.x, lo.y, lo.z, lo.w, b0, b1);
                    }
                }
            }
        }
        if constexpr (SILU) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    acc[0][j][i] = acc[0][j][i] / (1.f + __expf(-acc[0][j][i])) * acc[1][j][i];
        }
        const int64_t col = r.n0 + 8 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!live[h]) continue;
            uint16_t *dst = p.out[r.sec] + tok[h] * r.N + col;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack_bf16(acc[0][j][2 * h], acc[0][j][2 * h + 1]);
            if constexpr (VEC) {
                if (col < r.N) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (col + i < r.N) dst[i] = (uint16_t)(i & 1 ? w[i / 2] >> 16 : w[i / 2] & 0xffffu);
            }
        }
    };

    // ---- x against A: `side` blocks of A at a time, 8 / side warps each
    int side = 1;
    while (side < 8 && side < blocks) side *= 2;
    const int deep = kLoWarps / side, groups = (p.K / 32 + 3) / 4;
    const int g0 = (int)((int64_t)groups * share / cl), g1 = (int)((int64_t)groups * (share + 1) / cl);
    const bool wide = n > 8;
    for (int b0 = 0; b0 < blocks; b0 += side) {
        const int blk = b0 + warp / deep, sec = blk / max(nb, 1), r0 = blk % max(nb, 1) * 16;
        float acc[2][4] = {};
        if (blk < blocks) {
            const uint16_t *a0 = p.a + (((int64_t)id * p.nsec + sec) * p.rank + r0 + g) * p.K + 8 * t;
            const uint16_t *a1 = a0 + (int64_t)8 * p.K;
            const bool in0 = r0 + g < rank, in1 = r0 + g + 8 < rank;
            const uint16_t *x0 = p.x + tok[0] * p.K + 8 * t, *x1 = p.x + tok[1] * p.K + 8 * t;
            for (int gr = g0 + warp % deep; gr < g1; gr += deep) {
                uint4 va[4], vb[4], xa[4], xb[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const bool ok = gr * 4 + c < p.K / 32;
                    const int o = (gr * 4 + c) * 32;
                    va[c] = lo_load(a0 + o, ok && in0);
                    vb[c] = lo_load(a1 + o, ok && in1);
                    xa[c] = lo_load(x0 + o, ok && live[0]);
                    xb[c] = lo_load(x1 + o, ok && live[1]);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    mma_bf16(acc[0], va[c].x, vb[c].x, va[c].y, vb[c].y, xa[c].x, xa[c].y);
                    mma_bf16(acc[0], va[c].z, vb[c].z, va[c].w, vb[c].w, xa[c].z, xa[c].w);
                    if (wide) {
                        mma_bf16(acc[1], va[c].x, vb[c].x, va[c].y, vb[c].y, xb[c].x, xb[c].y);
                        mma_bf16(acc[1], va[c].z, vb[c].z, va[c].w, vb[c].w, xb[c].z, xb[c].w);
                    }
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
        for (int j = 0; j < side && b0 + j < blocks; ++j) {
            float v = 0.f;
            for (int w = 0; w < deep; ++w) v += s_acc[j * deep + w][tid];
            red[(b0 + j) * 256 + tid] = v;
        }
        __syncthreads();
    }
    Loads first, second;
    if (s0 + warp < s1) load(first, s0 + warp);

    // ---- the CTAs' sums: units of a token's four rows
    if (rank > 0) {
        if (cl > 1) cluster_sync_all();
        const float scale = p.scale ? p.scale[id] : 1.f;
        const int units = p.nsec * nk * 64;
        for (int u = (int)((int64_t)units * share / cl) + tid; u < (int)((int64_t)units * (share + 1) / cl); u += kLoThreads) {
            const int sec = u / (nk * 64), blk = u / 64 % nk, m = u / 4 % 16, r4 = u % 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (blk < nb) {
                const float *src = red + (sec * nb + blk) * 256 + m * 16 + 4 * r4;
                if (cl == 1) {
                    v = *reinterpret_cast<const float4 *>(src);
                } else {
                    for (int c = 0; c < cl; ++c) {
                        const float4 f = ld_cluster_f32x4(src, c);
                        v = make_float4(v.x + f.x, v.y + f.y, v.z + f.z, v.w + f.w);
                    }
                }
            }
            v = make_float4(v.x * scale, v.y * scale, v.z * scale, v.w * scale);
            // where the expansion's fragments have it
            const int r = 16 * blk + 4 * r4;
            const int ks = KS == 1 ? 0 : r / 32 * 2 + (r / 4) % 2, ln = (m % 8) * 4 + (KS == 1 ? r / 4 : r % 32 / 8), h = m / 8;
            const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
            const uint32_t l0 = pack_bf16(v.x - bf16_lo(h0), v.y - bf16_hi(h0));
            const uint32_t l1 = pack_bf16(v.z - bf16_lo(h1), v.w - bf16_hi(h1));
            uint32_t *dh = reinterpret_cast<uint32_t *>(&frag[sec * nk + ks].hi[ln]) + h;
            uint32_t *dl = reinterpret_cast<uint32_t *>(&frag[sec * nk + ks].lo[ln]) + h;
            for (int c = 0; c < cl; ++c) {
                uint32_t *rh = cl > 1 ? cluster_ptr(dh, c) : dh, *rl = cl > 1 ? cluster_ptr(dl, c) : dl;
                rh[0] = h0;
                rh[2] = h1;
                rl[0] = l0;
                rl[2] = l1;
            }
        }
        if (cl > 1)
            cluster_sync_all();
        else
            __syncthreads();
    }

    // ---- the outputs, two steps' loads in turn
    for (int step = s0 + warp; step < s1; step += 2 * kLoWarps) {
        const bool more = step + kLoWarps < s1;
        if (more) load(second, step + kLoWarps);
        use(first, step);
        if (!more) break;
        if (step + 2 * kLoWarps < s1) load(first, step + 2 * kLoWarps);
        use(second, step + kLoWarps);
    }
}

// ---------------------------------------------------------------- host side
static int lora_split(int64_t M, int K, int nsec, int rank, int adapters) {
    const int64_t tiles = std::min<int64_t>(M, adapters) + M / kLoTile;
    const int64_t units = std::max<int64_t>(1, tiles * nsec * ((rank + 15) / 16));
    int ks = 1;
    while (ks < 8 && units * ks * 2 <= 2 * num_sms() && K / (2 * ks) >= 512) ks *= 2;
    return ks;
}

size_t lora_workspace_bytes(int64_t M, int64_t K, int nsec, int rank, int adapters) {
    if (M <= kLoSort) return 0;
    const int64_t m = std::min<int64_t>(M, kLoChunk);
    return (size_t)lora_split(m, (int)K, nsec, rank, adapters) * m * nsec * rank * sizeof(float);
}

template <bool FEW, int KS, bool SILU, bool VEC>
static cudaError_t launch_expand(const LoraParams &p, int grid, cudaStream_t st) {
    return launch_pdl(reinterpret_cast<const void *>(lora_expand_kernel<FEW, KS, SILU, VEC>), dim3(grid),
                      kLoThreads, 0, st, p);
}
template <bool FEW, int KS>
static cudaError_t pick_expand(const LoraParams &p, int grid, cudaStream_t st) {
    if (p.silu)
        return p.vec ? launch_expand<FEW, KS, true, true>(p, grid, st)
                     : launch_expand<FEW, KS, true, false>(p, grid, st);
    return p.vec ? launch_expand<FEW, KS, false, true>(p, grid, st)
                 : launch_expand<FEW, KS, false, false>(p, grid, st);
}

template <int KS, bool SILU, bool VEC>
static cudaError_t launch_few(const LoraParams &p, int tiles, cudaStream_t st) {
    const void *kfn = reinterpret_cast<const void *>(lora_few_kernel<KS, SILU, VEC>);
    const int nb = (p.rank + 15) / 16, nk = KS == 1 ? 1 : (nb + 1) & ~1;
    const int smem = p.nsec * (nb * 256 * (int)sizeof(float) + nk * (int)sizeof(LoFragments));
    cudaError_t e = allow_smem(kfn, kMaxSections * (8 * 1024 + 8 * (int)sizeof(LoFragments)));
    if (e == cudaSuccess) e = allow_wide_clusters(kfn);
    if (e != cudaSuccess) return e;
    int cl = 1;
    while (cl < 16 && tiles * cl * 2 <= 2 * num_sms()) cl *= 2;
    return launch_pdl_cluster(kfn, (unsigned)(tiles * cl), (unsigned)cl, kLoThreads, (size_t)smem, st, p, cl);
}
template <int KS>
static cudaError_t pick_few(const LoraParams &p, int tiles, cudaStream_t st) {
    if (p.silu)
        return p.vec ? launch_few<KS, true, true>(p, tiles, st) : launch_few<KS, true, false>(p, tiles, st);
    return p.vec ? launch_few<KS, false, true>(p, tiles, st) : launch_few<KS, false, false>(p, tiles, st);
}

static cudaError_t launch_lora_few(LoraParams p, cudaStream_t st) {
    const int tiles = std::min<int64_t>(p.M, std::min<int64_t>(p.M, (int64_t)p.adapters + 1) + p.M / kLoTile);
    p.blocks = 0;
    for (int s = 0; s < (p.silu ? 1 : p.nsec); ++s) {
        p.sec_blocks[s] = (int)((p.sec_n[s] + 31) / 32);
        p.blocks += p.sec_blocks[s];
    }
    return p.rank <= 16   ? pick_few<1>(p, tiles, st)
           : p.rank <= 32 ? pick_few<2>(p, tiles, st)
           : p.rank <= 64 ? pick_few<4>(p, tiles, st)
                          : pick_few<8>(p, tiles, st);
}

template <bool FEW>
static cudaError_t launch_lora_t(LoraParams p, cudaStream_t st) {
    const int64_t tiles = std::min<int64_t>(p.M, std::min<int64_t>(p.M, p.adapters + 1) + p.M / kLoTile);
    const int64_t units = (FEW ? tiles : (int64_t)p.M) * p.nsec * ((p.rank + 15) / 16) * p.ks;
    const int full = 2 * num_sms();
    cudaError_t e = launch_pdl(reinterpret_cast<const void *>(lora_shrink_kernel<FEW>),
                               dim3((unsigned)std::min<int64_t>(full, units)), kLoThreads, 0, st, p);
    if (e != cudaSuccess) return e;
    // steps of a warp: as many as leave every warp of the GPU one
    const int64_t all = p.silu ? p.sec_n[0] : p.N;
    int64_t steps = tiles * ((all + 31) / 32) / ((int64_t)full * kLoWarps);
    p.steps = (int)std::min<int64_t>(std::max<int64_t>(steps, 1), 16);
    p.blocks = 0;
    for (int s = 0; s < (p.silu ? 1 : p.nsec); ++s) {
        p.sec_blocks[s] = (int)((p.sec_n[s] + 32 * p.steps - 1) / (32 * p.steps));
        p.blocks += p.sec_blocks[s];
    }
    const int64_t want = ((FEW ? tiles : (int64_t)p.M) * p.blocks + kLoWarps - 1) / kLoWarps;
    const int grid = (int)std::min<int64_t>(full, want);
    return p.rank <= 16   ? pick_expand<FEW, 1>(p, grid, st)
           : p.rank <= 32 ? pick_expand<FEW, 2>(p, grid, st)
           : p.rank <= 64 ? pick_expand<FEW, 4>(p, grid, st)
                          : pick_expand<FEW, 8>(p, grid, st);
}

cudaError_t launch_lora(LoraParams p, int64_t M, cudaStream_t st) {
    p.ks = lora_split(std::min<int64_t>(M, kLoChunk), p.K, p.nsec, p.rank, p.adapters);
    for (int64_t m = 0; m < M; m += kLoChunk) {
        p.M = (int)std::min<int64_t>(kLoChunk, M - m);
        const cudaError_t e = p.M <= kLoSort ? launch_lora_few(p, st) : launch_lora_t<false>(p, st);
        if (e != cudaSuccess) return e;
        p.x += (int64_t)p.M * p.K;
        p.ids += p.M;
        for (int s = 0; s < p.nsec; ++s) p.base[s] += p.M * p.sec_n[s];
        for (int s = 0; s < (p.silu ? 1 : p.nsec); ++s) p.out[s] += p.M * p.sec_n[s];
    }
    return cudaSuccess;
}

}  // namespace gwa
