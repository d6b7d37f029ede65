// The paged KV cache and a batch over it, as the kernels see them
// (gwa_kv_cache and gwa_kv_batch in include/gwa.h).  Everything read from the
// device arrays is checked here, so a bad length or page never becomes an
// address out of range.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace gwa {

constexpr unsigned kKvBadPage = 1u;  // page outside the cache or the table
constexpr unsigned kKvBadRope = 2u;  // position past the rotary table

// New tokens [first, first + count) of sequence b, cache length len (0 <=
// len <= the pages' capacity).
struct KvSeq {
    int first, count, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvView &kv, int b) {
    const int n = (int)kv.tokens;
    const int a = min(max(kv.q_start[b], 0), n);
    const int e = min(max(kv.q_start[b + 1], a), n);
    const int64_t cap = (int64_t)kv.max_pages << kv.page_shift;
    KvSeq s;
    s.first = a;
    s.count = e - a;
    s.len = (int)min((int64_t)max(kv.kv_len[b], 0), min(cap, (int64_t)0x7fffff00));
    return s;
}

// The sequence of a token and its position there (seq -1: none; a negative
// position: more new tokens than the cache length).  Called by a whole warp:
// the lanes search 32 entries of q_start at a time (non-decreasing).
struct KvToken {
    int seq, pos;
};
__device__ __forceinline__ KvToken kv_locate(const KvView &kv, int64_t tok, int lane) {
    int lo = 0, n = kv.batch + 1;  // the answer's entry lies in [lo, lo + n)
    KvToken r{-1, -1};
    while (true) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const bool le = lane * step < n && kv.q_start[i] <= tok;
        const int c = __popc(__ballot_sync(0xffffffffu, le));
        if (c == 0) return r;
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
        if (step == 1) break;
    }
    if (lo >= kv.batch) return r;
    const KvSeq s = kv_seq(kv, lo);
    const int i = (int)(tok - s.first);
    if (i < 0 || i >= s.count) return r;
    r.seq = lo;
    r.pos = s.len - s.count + i;
    return r;
}

// Row page * heads * page_size + slot of a position (-1: no such page); head
// h's entry is kv_head_row of it.
__device__ __forceinline__ int64_t kv_row(const KvView &kv, int seq, int pos) {
    const int j = pos >> kv.page_shift;
    if (j >= kv.max_pages) return -1;
    const int page = kv.page_table[(int64_t)seq * kv.max_pages + j];
    if (page < 0 || page >= kv.num_pages) return -1;
    return (((int64_t)page * kv.heads) << kv.page_shift) +
           (pos & ((1 << kv.page_shift) - 1));
}
__device__ __forceinline__ int64_t kv_head_row(const KvView &kv, int64_t row, int h) {
    return row + ((int64_t)h << kv.page_shift);
}

}  // namespace gwa
