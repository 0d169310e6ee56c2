// Pages and packed rows on the device: where a row of a packed tensor lies in a paged pool.
#pragma once

#include "kvc_internal.h"

namespace kvc {

// The last i of [0, n_seq) with start[i] <= row, or 0: the one sequence that can hold `row`.  Any contents of
// start are safe: only start[0 .. n_seq) is read.
__device__ __forceinline__ int find_seq(const int32_t *start, int n_seq, int row) {
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(start + mid) <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// The same by a whole warp for one row: 32 places are looked at together, so that up to 32 sequences take one
// round of loads and 65,535 four (a thread alone: one dependent load for each halving).
__device__ __forceinline__ int find_seq_warp(const int32_t *start, int n_seq, int row) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = n_seq;   // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const int v = i < n ? __ldcg(start + lo + i) : 0;
        const int below = max(__popc(__ballot_sync(0xffffffffu, i < n && v <= row)), 1);
        lo += (below - 1) * step;
        n = min(step, n - (below - 1) * step);
    }
    return lo;
}

// The pool position of position `pos` of sequence i, or -1 for a hole.
__device__ __forceinline__ int page_slot(const PagedView &p, int i, int pos) {
    const int lp = pos / p.page_size;
    if (pos < 0 || lp >= p.max_pages) return -1;
    const int page = __ldcg(p.table + (int64_t)i * p.max_pages + lp);
    if ((unsigned)page >= (unsigned)p.n_pages) return -1;
    return page * p.page_size + (pos - lp * p.page_size);
}

// The pool position of packed row `row`, which no sequence but i can hold: -1 for a hole or a row before the
// sequence's position 0, -2 for a row that belongs to no sequence.
__device__ __forceinline__ int row_slot(const PagedView &p, const int32_t *row_start, int i, int row) {
    const int s0 = __ldcg(row_start + i), s1 = __ldcg(row_start + i + 1), len = max(__ldcg(p.len + i), 0);
    return s0 <= row && row < s1 ? page_slot(p, i, len - (s1 - row)) : -2;
}

// The pool positions of `rows` packed rows from row0, into shared memory, by the whole CTA.  What counts is the
// chain of dependent loads (the search, the sequence, its page): where there are few rows each is searched by
// a warp, and the rest of the chain is walked for all rows at once.
__device__ __forceinline__ void row_slots(const PagedView &p, const int32_t *row_start, int row0, int rows, int *slots) {
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (p.n_seq > 4 && rows <= 4 * warps) {
        int mine = 0;
        for (int j = 0; warp + j * warps < rows; ++j) {
            const int i = find_seq_warp(row_start, p.n_seq, row0 + warp + j * warps);
            if (lane == j) mine = i;
        }
        const int r = warp + lane * warps;
        if (r < rows) slots[r] = row_slot(p, row_start, mine, row0 + r);
    } else {
        for (int r = threadIdx.x; r < rows; r += blockDim.x)
            slots[r] = row_slot(p, row_start, find_seq(row_start, p.n_seq, row0 + r), row0 + r);
    }
}

}  // namespace kvc
