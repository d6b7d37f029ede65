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
    __align__(16) int key[FEW ? kLoSort : 1];  // of the places: adapter
    int rank[FEW ? kLoSort : 1];               // and its rank
    int base[FEW ? kLoSort + 1 : 1];           // of the tiles: 16-row blocks of A before it
    int w_max[kLoWarps], w_sum[kLoWarps];
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
// part[k][m][s][r]: share k's sum of A x.  A CTA's unit is 16 rows of an
// adapter's A and a share of K for a tile; its warps take 256 inputs at a time
// (a warp's loads all at once, straight from global memory as MMA fragments: a
// lane's 16 bytes are the k positions of two MMAs, in the same order on both
// sides).  The shares depend on K alone, and so does the order of a token's sums.
__global__ void __launch_bounds__(kLoThreads, 2) lora_few_shrink_kernel(LoraParams p) {
    __shared__ LoTiles<true> sh;
    __shared__ float s_acc[kLoWarps][16 * kLoTile];
    __shared__ int s_sum[kLoWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    pdl_wait_primary();
    // (behind the wait: what the next kernel reads before its own wait was
    // written before this one's)
    if (tid == 0) pdl_launch_dependents();
    const int tiles = lo_tiles<true, kLoTile>(p, sh);
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
        const uint16_t *a = p.a + (((int64_t)id * p.nsec + sec) * p.rank + r0 + g) * p.K + 8 * t;
        const bool in0 = r0 + g < rank, in1 = r0 + g + 8 < rank, tok0 = g < n, tok1 = g + 8 < n;
        const uint16_t *x0 = p.x + (int64_t)sh.token(at + (tok0 ? g : 0)) * p.K + 8 * t;
        const uint16_t *x1 = p.x + (int64_t)sh.token(at + (tok1 ? g + 8 : 0)) * p.K + 8 * t;
        float acc[2][4] = {};
        const int end = min(p.K, (k + 1) * p.share);
        for (int i0 = k * p.share + warp * 256; i0 < end; i0 += kLoWarps * 256) {
            uint4 va[8], vb[8];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const bool ok = i0 + 32 * c < end;
                va[c] = lo_load(a + i0 + 32 * c, ok && in0);
                vb[c] = lo_load(a + i0 + 32 * c + (int64_t)8 * p.K, ok && in1);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && n <= 8) break;
                uint4 x[8];
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    x[c] = lo_load((h ? x1 : x0) + i0 + 32 * c, i0 + 32 * c < end && (h ? tok1 : tok0));
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

template <int KS, bool SILU, bool VEC>
__global__ void __launch_bounds__(kLoThreads, KS * (SILU ? 2 : 1) <= 4 ? 2 : 1) lora_few_expand_kernel(LoraParams p) {
    constexpr int S = SILU ? 2 : 1, Q = KS == 1 ? 1 : KS / 2;  // Q: B's loads of a row
    __shared__ LoTiles<true> sh;
    __shared__ uint4 frag[S * KS * kLoFrag];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32, g = lane >> 2, t = lane & 3;
    if (tid == 0) pdl_launch_dependents();
    const int tiles = lo_tiles<true, kLoTile>(p, sh);
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
                        const int r = KS == 1 ? 4 * t : 32 * q + 8 * t;
                        const bool ok = c0 + 2 * j < N && r < rank;
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
                const int nk = KS == 1 ? 1 : ((rank + 31) / 32) * 2;
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
                    const int ks = KS == 1 ? 0 : r / 32 * 2 + (r / 4) % 2;
                    const int ln = (m % 8) * 4 + (KS == 1 ? r / 4 : r % 32 / 8);
                    const uint32_t h0 = pack_bf16(v.x, v.y), h1 = pack_bf16(v.z, v.w);
                    frag[(s * KS + ks) * kLoFrag + m / 8 * 32 + ln] =
                        make_uint4(h0, h1, pack_bf16(v.x - bf16_lo(h0), v.y - bf16_hi(h0)),
                                   pack_bf16(v.z - bf16_lo(h1), v.w - bf16_hi(h1)));
                }
                __syncthreads();
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
                    if (16 * (KS == 1 ? k : k & ~1) >= rank) break;
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
                        acc[0][j][i] = __fdividef(acc[0][j][i], 1.f + __expf(-acc[0][j][i])) * acc[1][j][i];
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

// ---------------------------------------------------------------- host side
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
static cudaError_t launch_few(const LoraParams &p, int grid, cudaStream_t st) {
    return launch_pdl(reinterpret_cast<const void *>(lora_few_expand_kernel<KS, SILU, VEC>), dim3(grid),
                      kLoThreads, 0, st, p);
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
    const int64_t down = tiles * p.nsec * ((p.rank + 15) / 16) * p.ks;
    cudaError_t e = launch_pdl(reinterpret_cast<const void *>(lora_few_shrink_kernel),
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

static int lora_split(int64_t M, int K, int nsec, int rank, int adapters) {
    if (M <= kLoSort) return (K + lora_share(K) - 1) / lora_share(K);
    const int64_t tiles = std::min<int64_t>(M, adapters) + M / kLoTile;
    const int64_t units = std::max<int64_t>(1, tiles * nsec * ((rank + 15) / 16));
    int ks = 1;
    while (ks < 8 && units * ks * 2 <= 2 * num_sms() && K / (2 * ks) >= 512) ks *= 2;
    return ks;
}

size_t lora_workspace_bytes(int64_t M, int64_t K, int nsec, int rank, int adapters) {
    const int64_t m = std::min<int64_t>(M, kLoChunk);
    const int64_t tail = M > m && M % kLoChunk <= kLoSort ? M % kLoChunk : 0;
    auto bytes = [&](int64_t n) {
        return (size_t)lora_split(n, (int)K, nsec, rank, adapters) * n * nsec * rank * sizeof(float);
    };
    return std::max(bytes(m), bytes(tail));
}

cudaError_t launch_lora(LoraParams p, int64_t M, cudaStream_t st) {
    for (int64_t m = 0; m < M; m += kLoChunk) {
        p.M = (int)std::min<int64_t>(kLoChunk, M - m);
        p.ks = lora_split(p.M, p.K, p.nsec, p.rank, p.adapters);
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
