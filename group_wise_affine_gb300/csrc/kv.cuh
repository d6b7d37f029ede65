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

// New tokens [first, first + count) of sequence b, which end at position end;
// keys in the cache len = end, or the page table's capacity where that is less.
struct KvSeq {
    int first, count, end, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvView &kv, int start, int next, int len) {
    const int n = (int)kv.tokens;
    const int a = min(max(start, 0), n);
    const int e = min(max(next, a), n);
    const int64_t cap = (int64_t)kv.max_pages << kv.page_shift;
    KvSeq s;
    s.first = a;
    s.count = e - a;
    s.end = min(max(len, 0), 0x7fffff00);
    s.len = (int)min((int64_t)s.end, cap);
    return s;
}
__device__ __forceinline__ KvSeq kv_seq(const KvView &kv, int b) {
    return kv_seq(kv, kv.q_start[b], kv.q_start[b + 1], kv.kv_len[b]);
}

// The sequence of a token and its position there (seq -1: none; a negative
// position: more new tokens than the cache length).  Called by a whole warp:
// the lanes search 32 entries of q_start at a time (non-decreasing).
struct KvToken {
    int seq, pos;
};
__device__ __forceinline__ KvToken kv_locate(const KvView &kv, int64_t tok, int lane) {
    constexpr unsigned FULL = 0xffffffffu;
    int lo = 0, n = kv.batch + 1;  // the answer's entry lies in [lo, lo + n)
    KvToken r{-1, -1};
    int start, next, len;  // of the lane's entry in the last round
    while (true) {
        const int step = (n + 31) / 32, i = lo + lane * step;
        const bool in = lane * step < n;
        start = in ? kv.q_start[i] : 0;
        // (read along with the starts: the answer needs no further look)
        next = in && step == 1 && i < kv.batch ? kv.q_start[i + 1] : 0;
        len = in && step == 1 && i < kv.batch ? kv.kv_len[i] : 0;
        const int c = __popc(__ballot_sync(FULL, in && start <= tok));
        if (c == 0) return r;
        lo += (c - 1) * step;
        n = min(step, n - (c - 1) * step);
        if (step == 1) {
            start = __shfl_sync(FULL, start, c - 1);
            next = __shfl_sync(FULL, next, c - 1);
            len = __shfl_sync(FULL, len, c - 1);
            break;
        }
    }
    if (lo >= kv.batch) return r;
    const KvSeq s = kv_seq(kv, start, next, len);
    const int i = (int)(tok - s.first);
    if (i < 0 || i >= s.count) return r;
    r.seq = lo;
    r.pos = s.end - s.count + i;
    return r;
}

// Keys that new token i of a sequence sees.
__device__ __forceinline__ int kv_seen(const KvSeq &s, int i, int causal) {
    return causal ? min(s.len, s.end - s.count + i + 1) : s.len;
}
// Whether new tokens lie past the page table.
__device__ __forceinline__ bool kv_past(const KvSeq &s) { return s.end > s.len && s.count > 0; }

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
