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
// of 40 + 8 heads of 128 are 249 MB, 37 us of HBM bandwidth; one token is a
// launch.  A lane holds eight dimensions (one 16-byte load), a head takes
// D/8 lanes, eight lanes share a group's minimum and maximum by shuffles,
// and the partner of a rotated pair sits rot_dim/16 lanes away.  A warp
// keeps its lanes' cos and sin in registers over several heads of one token
// (reading them per head would be four times the bytes of the head itself).
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
    int qsteps, steps;  // a token's warp steps: queries', and all
    int per;    // steps of a warp task
    int nblk;   // warp tasks per token
    int32_t *status;
};

// Eight table entries.
__device__ __forceinline__ void load_cs(const float2 *src, float2 (&cs)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float4 t = reinterpret_cast<const float4 *>(src)[i];
        cs[2 * i] = make_float2(t.x, t.y);
        cs[2 * i + 1] = make_float2(t.z, t.w);
    }
}

template <int BITS, int D>
__global__ void __launch_bounds__(256, 4) kv_append_kernel(AppendParams p) {
    constexpr int CH = D / 8;       // 16-byte pieces of a head
    constexpr int HPW = 32 / CH;    // heads of a key or value step
    constexpr int QPW = 2 * HPW;    // heads of a query step
    constexpr int UNROLL = 2;       // steps with their loads in flight
    constexpr unsigned FULL = 0xffffffffu;
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int Hkv = p.kv.heads;
    const int half8 = p.rot / 16;   // pieces of a rotated half
    const int64_t tasks = p.kv.tokens * p.nblk;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32; w < tasks;
         w += (int64_t)gridDim.x * blockDim.x / 32) {
        const int64_t tok = w / p.nblk;
        const int blk = (int)(w % p.nblk);
        const KvToken at = kv_locate(p.kv, tok, lane);
        if (at.seq < 0) continue;  // a token of no sequence: nothing is written
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
            }
        }
        if (bad && lane == 0 && p.status) atomicOr(p.status, (int)bad);
        const float2 *const table = p.rope + (int64_t)at.pos * (p.rot / 2);  // read where turn
        int s0 = blk * p.per;
        const int s1 = min(p.steps, s0 + p.per);

        // ---- queries: a lane holds two pieces, those of a rotated pair
        // where there is one, so nothing passes between lanes
        if (s0 < p.qsteps) {
            const int l = lane % (CH / 2), hsub = lane / (CH / 2);
            const bool rot = turn && l < half8;
            const int c0 = l < half8 ? l : 2 * l, c1 = l < half8 ? l + half8 : 2 * l + 1;
            float2 cs[8];
            if (rot) load_cs(table + l * 8, cs);
            const uint4 *const src = reinterpret_cast<const uint4 *>(p.q + tok * p.q_stride);
            uint4 *const dst = reinterpret_cast<uint4 *>(p.q_out + tok * p.Hq * D);
            for (const int s2 = min(s1, p.qsteps); s0 < s2; s0 += UNROLL) {
                uint4 a[UNROLL], b[UNROLL];
#pragma unroll
                for (int j = 0; j < UNROLL; ++j)
                    if (const int h = (s0 + j) * QPW + hsub; s0 + j < s2 && h < p.Hq) {
                        a[j] = src[h * CH + c0];
                        b[j] = src[h * CH + c1];
                    }
#pragma unroll
                for (int j = 0; j < UNROLL; ++j) {
                    const int h = (s0 + j) * QPW + hsub;
                    if (s0 + j >= s2 || h >= p.Hq) continue;
                    if (rot) {
                        uint32_t x[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
                        uint32_t y[4] = {b[j].x, b[j].y, b[j].z, b[j].w};
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
                        a[j] = make_uint4(x[0], x[1], x[2], x[3]);
                        b[j] = make_uint4(y[0], y[1], y[2], y[3]);
                    }
                    dst[h * CH + c0] = a[j];
                    dst[h * CH + c1] = b[j];
                }
            }
            s0 = p.qsteps;
        }
        if (s0 >= s1 || row < 0) continue;

        // ---- keys and values: a lane holds one piece, a group eight lanes
        const int c = lane % CH, hsub = lane / CH;
        const bool rot = turn && c < 2 * half8, second = c >= half8;
        const int partner = !rot ? lane : second ? lane - half8 : lane + half8;
        float2 cs[8];
        if (rot) {
            load_cs(table + (second ? c - half8 : c) * 8, cs);
            // first half: a cos - b sin; second: b cos + a sin
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i].y = second ? cs[i].y : -cs[i].y;
        }
        for (; s0 < s1; s0 += UNROLL) {
            uint4 u[UNROLL];
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                const int h = (s0 + j - p.qsteps) * HPW + hsub;
                u[j] = make_uint4(0u, 0u, 0u, 0u);
                if (s0 + j < s1 && h < 2 * Hkv) {
                    const uint16_t *src = h < Hkv ? p.k + tok * p.k_stride + h * D
                                                  : p.v + tok * p.v_stride + (h - Hkv) * D;
                    u[j] = reinterpret_cast<const uint4 *>(src)[c];
                }
            }
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                if (s0 + j >= s1) break;
                const int h = (s0 + j - p.qsteps) * HPW + hsub;
                uint4 o = u[j];
                if (turn && (s0 + j - p.qsteps) * HPW < Hkv) {  // a step with keys
                    uint4 other;
                    other.x = __shfl_sync(FULL, o.x, partner);
                    other.y = __shfl_sync(FULL, o.y, partner);
                    other.z = __shfl_sync(FULL, o.z, partner);
                    other.w = __shfl_sync(FULL, o.w, partner);
                    if (rot && h < Hkv) {
                        const uint32_t a[4] = {o.x, o.y, o.z, o.w};
                        const uint32_t b[4] = {other.x, other.y, other.z, other.w};
                        uint32_t r[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float2 e = cs[2 * i], f = cs[2 * i + 1];
                            r[i] = pack_bf16(__fadd_rn(__fmul_rn(bf16_lo(a[i]), e.x),
                                                       __fmul_rn(bf16_lo(b[i]), e.y)),
                                             __fadd_rn(__fmul_rn(bf16_hi(a[i]), f.x),
                                                       __fmul_rn(bf16_hi(b[i]), f.y)));
                        }
                        o = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                }
                float x[8];
                x[0] = bf16_lo(o.x); x[1] = bf16_hi(o.x);
                x[2] = bf16_lo(o.y); x[3] = bf16_hi(o.y);
                x[4] = bf16_lo(o.z); x[5] = bf16_hi(o.z);
                x[6] = bf16_lo(o.w); x[7] = bf16_hi(o.w);
                uint32_t code[8];
                uint16_t sb, bb;
                quantize_group8<BITS>(x, code, sb, bb);
                if (h >= 2 * Hkv) continue;
                const bool is_v = h >= Hkv;
                const int64_t at_h = kv_head_row(p.kv, row, is_v ? h - Hkv : h);
                uint32_t *dst = (is_v ? p.kv.vq : p.kv.kq) + at_h * (D * BITS / 32);
                if constexpr (BITS == 4)
                    dst[c] = pack_u4(code);
                else
                    reinterpret_cast<uint2 *>(dst)[c] = pack_u8(code);
                if ((c & 7) == 0)
                    ((is_v ? p.kv.vp : p.kv.kp) + at_h * (D / 64))[c >> 3] =
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
    kv_read_kernel(KvView kv, int per, int nblk, uint16_t *__restrict__ k,
                   uint16_t *__restrict__ v, int32_t *status) {
    constexpr int CH = D / 8, HPW = 32 / CH;
    constexpr int UNROLL = 4;  // steps with their loads in flight
    if (threadIdx.x == 0) pdl_launch_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31;
    const int c = lane % CH, hsub = lane / CH;
    const int heads = 2 * kv.heads, steps = (heads + HPW - 1) / HPW;
    for (int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
         w < kv.tokens * nblk; w += (int64_t)gridDim.x * blockDim.x / 32) {
        const int64_t tok = w / nblk;
        const int blk = (int)(w % nblk);
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
    while (per > 2 && tokens * ((steps + per - 1) / per) < (int64_t)num_sms() * 64)
        per = (per + 1) / 2;
    nblk = (steps + per - 1) / per;
}

// Warp tasks of 8-warp blocks, at most eight blocks an SM (all its warps).
static unsigned kv_grid(int64_t tasks) {
    const int64_t blocks = (tasks + 7) / 8, cap = (int64_t)num_sms() * 8;
    return (unsigned)(blocks < cap ? blocks : cap);
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
    const int hpw = 32 / (kv.dim / 8);
    p.qsteps = (Hq + 2 * hpw - 1) / (2 * hpw);
    p.steps = p.qsteps + (2 * kv.heads + hpw - 1) / hpw;
    kv_tasks(kv.tokens, p.steps, p.per, p.nblk);
    const unsigned grid = kv_grid(kv.tokens * p.nblk);
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
    const unsigned grid = kv_grid(kv.tokens * nblk);
#define GWA_KV(BB, DD)                                                       \
    if (kv.bits == BB && kv.dim == DD)                                       \
        return launch_pdl(reinterpret_cast<const void *>(kv_read_kernel<BB, DD>), \
                          grid, 256u, 0, st, kv, per, nblk, k, v, status);
    GWA_KV(4, 64) GWA_KV(4, 128) GWA_KV(4, 256)
    GWA_KV(8, 64) GWA_KV(8, 128) GWA_KV(8, 256)
#undef GWA_KV
    return cudaErrorInvalidValue;
}

}  // namespace gwa
