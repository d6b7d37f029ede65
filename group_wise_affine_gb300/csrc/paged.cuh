// What the two kernels of the paged attention share: their parameters and how
// a batch's work is cut into equal runs of units, one per CTA.
#pragma once

#include "common.cuh"
#include "internal.h"
#include "kv.cuh"

namespace gwa {

constexpr int kPgMaxCtas = 2048;
// The joins' weights are at most 2^-11: of 2048 pieces they sum up to no more
// than 1, and their sums of means stay in the values' range.
constexpr float kPgJoin = 11.f;

// A (sequence, KV head, row block) that the cut spread over several CTAs: its
// first piece's slot (-1: nothing to join), further pieces in the slots 2 (cta
// + k); rows r0 .. r0 + nlive of the sequence whose first token is `first`,
// query heads from `head`.
struct PgCut {
    int slot, cta, n, first, head, r0, nlive, pad;
};

struct PagedParams {
    const uint16_t *q;
    int64_t q_stride;
    int Hq, rep;
    KvView kv;
    float scale;
    int causal;
    uint16_t *out;    // [tokens, Hq, dim]
    PgCut *cuts;      // what the join has to do
    int segs;         // (KV head, row block) pairs of a sequence, at most
    int by_seg;       // cuts are indexed by sequence and pair, else by CTA
    float *part;      // [2 ctas][rows of a block][dim + 4], see the joins
    int32_t *status;
    // sequences with up to `split` rows (new tokens x query heads of a KV
    // head) go to the few-row kernel, the others to the prompt kernel
    int split;
};

// `total` units over `ctas` CTAs: the first total % ctas take one more.
__device__ __forceinline__ int pg_start(int quot, int rest, int c) {
    return quot * c + min(c, rest);
}
__device__ __forceinline__ int pg_owner(int quot, int rest, int unit) {
    const int big = rest * (quot + 1);
    return unit < big ? unit / (quot + 1) : rest + (unit - big) / quot;
}

// A total over the lanes of values whose own sums fit: as an int, or 0 if it
// does not fit one (starts that decrease can name a token for many sequences;
// of a batch that the entry point let through it always fits).
__device__ __forceinline__ int pg_total(int64_t v) {
    const unsigned lo = __reduce_add_sync(0xffffffffu, (unsigned)v & 0xffffu);
    const unsigned hi = __reduce_add_sync(0xffffffffu, (unsigned)min(v >> 16, (int64_t)0x7ffffff));
    return hi < 0x7fd0u ? (int)((hi << 16) + lo) : 0;
}

// Prompt kernel (paged_prefill.cu): its launch over the sequences with more
// than p.split rows, and the bytes of its partial outputs.
cudaError_t launch_paged_prefill(PagedParams p, void *workspace, cudaStream_t st);
size_t paged_prefill_workspace_bytes(const KvView &kv, int rep);
double paged_prefill_units(const KvView &kv, int rep, int split);

}  // namespace gwa
