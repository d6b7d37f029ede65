// Affine group quantization of bf16 weights: the requantize step of
// "Sanctum-MLX", "The April 2026 cutover" (LoRA merge at load dequantizes,
// adds the delta and requantizes at group size 64; "File map": lora.rs also
// merges the switch_mlp expert weights).  The pages state no rule; the
// reading used here, per group of 64 consecutive inputs of a row:
//
//   scale = bf16_rn((max - min) / (2^b - 1)),  bias = min (a bf16 already;
//   a zero minimum is stored as +0),
//   code  = clamp(rint((w - bias) / scale), 0, 2^b - 1), or 0 if scale == 0,
//
// in IEEE fp32 (correctly rounded divide, round half to even), codes packed
// lowest bits first.  Finite inputs only.
//
// Eight lanes share a group: each loads 16 bytes (eight inputs), the lanes
// agree on the minimum and maximum with three shuffles, and each packs its
// eight codes into one (u4) or two (u8) words; the group's first lane writes
// the scale and bias.  A warp covers four consecutive groups per step, so
// its loads are 512 contiguous bytes.  The HBM floor is 2 bytes read and
// b/8 + 1/16 written per weight (~54 us for a 27648 x 5120 u4 weight), but
// the exactly rounded codes take ~10 instructions per weight, so the kernel
// runs at about a third of HBM bandwidth, limited by instruction issue
// (issuing four steps' loads ahead changed nothing).
#include "common.cuh"
#include "internal.h"
#include "quantize.cuh"

namespace gwa {

template <int BITS>
__global__ void __launch_bounds__(256)
    quantize_affine_kernel(const uint16_t *__restrict__ w, int64_t groups,
                           uint32_t *__restrict__ wq, uint16_t *__restrict__ sc,
                           uint16_t *__restrict__ bi) {
    const int lane = threadIdx.x & (kWarp - 1);
    const int sub = lane >> 3, l8 = lane & 7;
    const int64_t warp = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / kWarp;
    const int64_t nwarps = (int64_t)gridDim.x * blockDim.x / kWarp;
    // every lane of a warp takes the same trip count (the shuffles need all
    // 32); groups past the end compute on zeros and store nothing
    for (int64_t q4 = warp * 4; q4 < groups; q4 += nwarps * 4) {
        const int64_t g = q4 + sub;
        const bool live = g < groups;
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (live)
            u = reinterpret_cast<const uint4 *>(w)[g * 8 + l8];
        float v[8];
        v[0] = bf16_lo(u.x); v[1] = bf16_hi(u.x);
        v[2] = bf16_lo(u.y); v[3] = bf16_hi(u.y);
        v[4] = bf16_lo(u.z); v[5] = bf16_hi(u.z);
        v[6] = bf16_lo(u.w); v[7] = bf16_hi(u.w);
        uint32_t q[8];
        uint16_t sbits, bbits;
        quantize_group8<BITS>(v, q, sbits, bbits);
        if (!live) continue;
        if constexpr (BITS == 4) {
            wq[g * 8 + l8] = pack_u4(q);
        } else {
            reinterpret_cast<uint2 *>(wq)[g * 8 + l8] = pack_u8(q);
        }
        if (l8 == 0) {
            sc[g] = sbits;
            bi[g] = bbits;
        }
    }
}

cudaError_t launch_quantize(const uint16_t *w, int64_t N, int64_t K, int bits,
                            uint32_t *wq, uint16_t *sc, uint16_t *bi,
                            cudaStream_t st) {
    const int64_t groups = N * (K / kGroup);
    if (groups == 0) return cudaSuccess;
    constexpr int kThreads = 256;  // 8 warps: 32 groups per block and step
    int64_t blocks = (groups + 31) / 32;
    const int64_t cap = (int64_t)num_sms() * 8;  // 2048 threads per SM
    if (blocks > cap) blocks = cap;
    if (bits == 4)
        quantize_affine_kernel<4><<<(unsigned)blocks, kThreads, 0, st>>>(
            w, groups, wq, sc, bi);
    else
        quantize_affine_kernel<8><<<(unsigned)blocks, kThreads, 0, st>>>(
            w, groups, wq, sc, bi);
    return cudaGetLastError();
}

}  // namespace gwa
