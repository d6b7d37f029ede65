// Paged KV cache in the library's affine format: append (with the rotary
// embedding and the quantization on the way), read back, and the rotary
// table.  "Sanctum-MLX", six-changes table row 5 and "File map"
// (`turboquant/`, the 4-bit cache) and "The Cathedral Doubled Itself", "The
// trap that ate three hours" (RoPE per head at the cache offset); the pages
// give no paging and quantize values only.
//
// One token's key head of D dimensions: the rotary embedding of its first
// rot_dim dimensions (pairs i, i + rot_dim/2; cos and sin from the table, in
// fp32, each product and the sum rounded once), rounded to bf16, then per 64
// dimensions the affine rule of the weight quantizer:
//   scale = bf16_rn((max - min) / (2^b - 1)), bias = min,
//   code = clamp(rint((x - bias) / scale), 0, 2^b - 1).
// The rounding to bf16 before the rule is a choice: the bias is then exactly
// the minimum, and the cache holds bit for bit what rotating into a bf16
// buffer and quantizing that would give.
//
// Bound: bytes.  A token moves (2 Hq + 2 Hkv) D 2 bytes of bf16 (q in and
// out, k and v in) and writes 2 Hkv (D b/8 + D/16) of cache, so 8192 tokens
// of 40 + 2 x 8 heads of 128 are 211 MB, 31 us of HBM bandwidth; one token is
// a launch.  Measured: 46 us for those (the append alone; 4.6 TB/s), 5 us for
// one token with its read-back.  A warp takes one token's heads in steps of 32
// lanes x 16 dimensions (two 16-byte loads a lane, two steps in flight).
// Queries and keys are loaded so that a lane holds both pieces of a rotated
// pair; its cos and sin stay in registers for all the token's heads (reading
// them per head would be four times the head's own bytes).  A rotated key
// then goes through shared memory into the order of its groups, four lanes
// each.  No unit is at its limit (issue 55%, HBM 46%): with 31% of the warps
// resident a load's latency shows behind the quantization's instructions
// (about 350 of a step's 450).  With 32 query heads 42 us, where lanes that
// divide when a quotient is near a half-integer made it 78, and eight values a
// lane with the pairs exchanged by shuffles 50.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"
#include "mma.cuh"
#include "quantize.cuh"

namespace gwa {

struct AppendParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out;
    int64_t q_stride, k_stride, v_stride;
    int Hq;
    KvView kv;
    const float2 *rope;
    int64_t rope_rows;
    int rot;    // rotated dimensions
    int qsteps, ksteps, steps;  // a token's warp steps: queries', keys', and all
    int per;    // steps of a warp task
    int nblk;   // warp tasks per token
    int32_t *status;
};

// A rotated pair's pieces of eight dimensions, a of the first half and b of
// the second: a cos - b sin and b cos + a sin, each product and each sum
// rounded once.
__device__ __forceinline__ void kv_turn(uint4 &a, uint4 &b, const float2 (&cs)[8]) {
    uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 e = cs[2 * i], f = cs[2 * i + 1];
        const float x0 = bf16_lo(x[i]), x1 = bf16_hi(x[i]);
        const float y0 = bf16_lo(y[i]), y1 = bf16_hi(y[i]);
        x[i] = pack_bf16(__fsub_rn(__fmul_rn(x0, e.x), __fmul_rn(y0, e.y)),
                         __fsub_rn(__fmul_rn(x1, f.x), __fmul_rn(y1, f.y)));
        y[i] = pack_bf16(__fadd_rn(__fmul_rn(y0, e.x), __fmul_rn(x0, e.y)),
                         __fadd_rn(__fmul_rn(y1, f.x), __fmul_rn(x1, f.y)));
    }
    a = make_uint4(x[0], x[1], x[2], x[3]);
    b = make_uint4(y[0], y[1], y[2], y[3]);
}

template <int BITS, int D>
__global__ void __launch_bounds__(256, 3) kv_append_kernel(AppendParams p) {
    constexpr int CH = D / 8;      // 16-byte pieces of a head
    constexpr int LPH = CH / 2;    // lanes per head, two pieces each
    constexpr int HPW = 32 / LPH;  // heads of a step
    constexpr int UNROLL = 2;      // steps with their loads in flight
    __shared__ uint4 stage[8][64];  // a warp's step, from one order of pieces to the other
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int l = lane % LPH, hsub = lane / LPH;
    uint4 *const own = &stage[threadIdx.x / 32][hsub * CH];
    const int Hkv = p.kv.heads;
    const int half8 = p.rot / 16;   // pieces of a rotated half
    // queries and keys: a lane's two pieces are those of a rotated pair,
    // where there is one, so nothing passes between lanes
    const int c0 = l < half8 ? l : 2 * l, c1 = l < half8 ? l + half8 : 2 * l + 1;
    const int s_begin = blockIdx.y * p.per, s_end = min(p.steps, s_begin + p.per);
    for (int64_t tok = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; tok < p.kv.tokens;
         tok += (int64_t)gridDim.x * 8) {
        const KvToken at = kv_locate(p.kv, tok, lane);
        // a token of no sequence has no keys and values to write, and its
        // queries are zero; so are those past the rotary table
        bool drop = at.seq < 0;
        const int t_end = drop ? min(s_end, p.qsteps) : s_end;
        // where the token's keys and values go (-1: nowhere)
        int64_t row = -1;
        unsigned bad = 0u;
        bool turn = p.rot > 0 && at.pos >= 0;
        if (at.pos >= 0) {
            row = kv_row(p.kv, at.seq, at.pos);
            if (row < 0) bad |= kKvBadPage;
            if (p.rot > 0 && at.pos >= p.rope_rows) {
                bad |= kKvBadRope;
                row = -1;
                turn = false;
                drop = true;
            }
        }
        if (bad && lane == 0 && p.status) atomicOr(p.status, (int)bad);
        turn = turn && l < half8;
        float2 cs[8];
        if (turn && s_begin < p.qsteps + p.ksteps) {
            const float4 *const src = reinterpret_cast<const float4 *>(
                p.rope + (int64_t)at.pos * (p.rot / 2) + l * 8);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 t = src[i];
                cs[2 * i] = make_float2(t.x, t.y);
                cs[2 * i + 1] = make_float2(t.z, t.w);
            }
        }
        for (int s0 = s_begin; s0 < t_end; s0 += UNROLL) {
            uint4 a[UNROLL], b[UNROLL];
            // a step: its kind (queries, keys, values), first head and heads
            auto step = [&](int s, int &kind, int &h, int &n) {
                kind = s < p.qsteps ? 0 : s < p.qsteps + p.ksteps ? 1 : 2;
                h = (kind == 0 ? s : kind == 1 ? s - p.qsteps : s - p.qsteps - p.ksteps) * HPW + hsub;
                n = kind == 0 ? p.Hq : Hkv;
            };
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                int kind, h, n;
                step(s0 + j, kind, h, n);
                a[j] = b[j] = make_uint4(0u, 0u, 0u, 0u);
                if (s0 + j < t_end && h < n && !(kind == 0 && drop)) {
                    const uint4 *src = reinterpret_cast<const uint4 *>(
                        kind == 0   ? p.q + tok * p.q_stride
                        : kind == 1 ? p.k + tok * p.k_stride
                                    : p.v + tok * p.v_stride) + h * CH;
                    a[j] = src[kind < 2 ? c0 : 2 * l];
                    b[j] = src[kind < 2 ? c1 : 2 * l + 1];
                }
            }
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                if (s0 + j >= t_end) break;
                int kind, h, n;
                step(s0 + j, kind, h, n);
                if (kind < 2 && turn) kv_turn(a[j], b[j], cs);
                if (kind == 0) {
                    if (h < n) {
                        uint4 *const dst = reinterpret_cast<uint4 *>(p.q_out + (tok * p.Hq + h) * D);
                        dst[c0] = a[j];
                        dst[c1] = b[j];
                    }
                    continue;
                }
                if (row < 0) continue;
                if (kind == 1) {
                    // neighbouring pieces from here on: four lanes a group
                    __syncwarp();
                    own[c0] = a[j];
                    own[c1] = b[j];
                    __syncwarp();
                    a[j] = own[2 * l];
                    b[j] = own[2 * l + 1];
                }
                const uint32_t x[8] = {a[j].x, a[j].y, a[j].z, a[j].w,
                                       b[j].x, b[j].y, b[j].z, b[j].w};
                uint32_t word[BITS / 2];
                uint16_t sb, bb;
                quantize_group16<BITS>(x, word, sb, bb);
                if (h >= n) continue;
                const int64_t at_h = kv_head_row(p.kv, row, h);
                uint32_t *const dst = (kind == 2 ? p.kv.vq : p.kv.kq) + at_h * (D * BITS / 32);
                if constexpr (BITS == 4)
                    reinterpret_cast<uint2 *>(dst)[l] = make_uint2(word[0], word[1]);
                else
                    reinterpret_cast<uint4 *>(dst)[l] =
                        make_uint4(word[0], word[1], word[2], word[3]);
                if ((l & 3) == 0)
                    ((kind == 2 ? p.kv.vp : p.kv.kp) + at_h * (D / 64))[l >> 2] =
                        (uint32_t)sb | ((uint32_t)bb << 16);
            }
        }
    }
}

// The values that the cache holds for the batch's tokens, as bf16 (scale *
// code + bias, rounded once to fp32 and once to bf16); zeros for a token that
// has no place in the cache.  Bound by bytes: 2 D bytes written per head
// against D b/8 + D/16 read.
template <int BITS, int D>
__global__ void __launch_bounds__(256)
    kv_read_kernel(KvView kv, int per, uint16_t *__restrict__ k,
                   uint16_t *__restrict__ v, int32_t *status) {
    constexpr int CH = D / 8, HPW = 32 / CH;
    constexpr int UNROLL = 4;  // steps with their loads in flight
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int c = lane % CH, hsub = lane / CH;
    const int heads = 2 * kv.heads, steps = (heads + HPW - 1) / HPW;
    const int blk = blockIdx.y;
    for (int64_t tok = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; tok < kv.tokens;
         tok += (int64_t)gridDim.x * 8) {
        const KvToken at = kv_locate(kv, tok, lane);
        const int64_t row =
            at.seq >= 0 && at.pos >= 0 ? kv_row(kv, at.seq, at.pos) : -1;
        if (row < 0 && at.seq >= 0 && at.pos >= 0 && lane == 0 && status)
            atomicOr(status, (int)kKvBadPage);
        const int s1 = min(steps, (blk + 1) * per);
        for (int s0 = blk * per; s0 < s1; s0 += UNROLL) {
            uint2 u[UNROLL];
            uint32_t par[UNROLL];
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                const int h = (s0 + j) * HPW + hsub;
                u[j] = make_uint2(0u, 0u);
                par[j] = 0u;
                if (s0 + j >= s1 || h >= heads || row < 0) continue;
                const bool is_v = h >= kv.heads;
                const int64_t at_h = kv_head_row(kv, row, is_v ? h - kv.heads : h);
                const uint32_t *src = (is_v ? kv.vq : kv.kq) + at_h * (D * BITS / 32);
                par[j] = ((is_v ? kv.vp : kv.kp) + at_h * (D / 64))[c >> 3];
                if constexpr (BITS == 4)
                    u[j].x = src[c];
                else
                    u[j] = reinterpret_cast<const uint2 *>(src)[c];
            }
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                const int h = (s0 + j) * HPW + hsub;
                if (s0 + j >= s1 || h >= heads) continue;
                const bool is_v = h >= kv.heads;
                const float s = bf16_lo(par[j]), b = bf16_hi(par[j]);
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t code = BITS == 4 ? (u[j].x >> (4 * i)) & 15u
                                                    : ((i < 4 ? u[j].x : u[j].y) >> (8 * (i & 3))) & 255u;
                    x[i] = fmaf((float)code, s, b);  // (no place: zeros)
                }
                reinterpret_cast<uint4 *>(
                    (is_v ? v : k) + (tok * kv.heads + (is_v ? h - kv.heads : h)) * D)[c] =
                    make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                               pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            }
        }
    }
}

// Head steps of a warp task and tasks of a token.  Few tokens: two steps to a
// warp, so that a token spreads over many warps; many: as many steps as still
// fill the GPU, so that the rotary entries and the token's place are read for
// more heads.
static void kv_tasks(int64_t tokens, int steps, int &per, int &nblk) {
    per = steps;
    while (per > 2 && tokens * ((steps + per - 1) / per) < (int64_t)num_sms() * 32)
        per = (per + 1) / 2;
    nblk = (steps + per - 1) / per;
}

// Blocks of eight warps, a token each; y: a token's tasks.
static dim3 kv_grid(int64_t tokens, int nblk) {
    return dim3((unsigned)std::min<int64_t>((tokens + 7) / 8, 1 << 20), (unsigned)nblk);
}

cudaError_t launch_kv_append(const uint16_t *q, int64_t q_stride, uint16_t *q_out,
                             int Hq, const uint16_t *k, int64_t k_stride,
                             const uint16_t *v, int64_t v_stride, const KvView &kv,
                             const float *rope, int64_t rope_rows, int rot_dim,
                             int32_t *status, cudaStream_t st) {
    AppendParams p{};
    p.q = q; p.k = k; p.v = v; p.q_out = q_out;
    p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
    p.Hq = Hq;
    p.kv = kv;
    p.rope = reinterpret_cast<const float2 *>(rope);
    p.rope_rows = rope_rows;
    p.rot = rot_dim;
    p.status = status;
    const int hpw = 32 / (kv.dim / 16);
    p.qsteps = (Hq + hpw - 1) / hpw;
    p.ksteps = (kv.heads + hpw - 1) / hpw;
    p.steps = p.qsteps + 2 * p.ksteps;
    kv_tasks(kv.tokens, p.steps, p.per, p.nblk);
    const dim3 grid = kv_grid(kv.tokens, p.nblk);
#define GWA_KV(BB, DD)                                                         \
    if (kv.bits == BB && kv.dim == DD)                                         \
        return launch_pdl(reinterpret_cast<const void *>(kv_append_kernel<BB, DD>), \
                          grid, 256u, 0, st, p);
    GWA_KV(4, 64) GWA_KV(4, 128) GWA_KV(4, 256)
    GWA_KV(8, 64) GWA_KV(8, 128) GWA_KV(8, 256)
#undef GWA_KV
    return cudaErrorInvalidValue;
}

cudaError_t launch_kv_read(const KvView &kv, uint16_t *k, uint16_t *v,
                           int32_t *status, cudaStream_t st) {
    const int hpw = 32 / (kv.dim / 8);
    const int steps = (2 * kv.heads + hpw - 1) / hpw;
    int per, nblk;
    kv_tasks(kv.tokens, steps, per, nblk);
    const dim3 grid = kv_grid(kv.tokens, nblk);
#define GWA_KV(BB, DD)                                                       \
    if (kv.bits == BB && kv.dim == DD)                                       \
        return launch_pdl(reinterpret_cast<const void *>(kv_read_kernel<BB, DD>), \
                          grid, 256u, 0, st, kv, per, k, v, status);
    GWA_KV(4, 64) GWA_KV(4, 128) GWA_KV(4, 256)
    GWA_KV(8, 64) GWA_KV(8, 128) GWA_KV(8, 256)
#undef GWA_KV
    return cudaErrorInvalidValue;
}

}  // namespace gwa
