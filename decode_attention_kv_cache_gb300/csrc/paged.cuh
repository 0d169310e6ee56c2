// Pages and packed rows on the device: where a row of a packed tensor lies in a paged pool.
#pragma once

#include "kvc_internal.h"

namespace kvc {

// The sequence that holds `row`: i with start[i] <= row < start[i + 1], or -1.  Any contents of start are
// safe: only start[0 .. n_seq] is read.
__device__ __forceinline__ int find_seq(const int32_t *start, int n_seq, int row) {
    int lo = 0, hi = n_seq;   // start[lo] <= row (or lo == 0), start[hi] > row (or hi == n_seq)
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldcg(start + mid) <= row) lo = mid; else hi = mid;
    }
    return (__ldcg(start + lo) <= row && row < __ldcg(start + lo + 1)) ? lo : -1;
}

// The pool position of position `pos` of sequence i, or -1 for a hole.
__device__ __forceinline__ int page_slot(const PagedView &p, int i, int pos) {
    const int lp = pos / p.page_size;
    if (pos < 0 || lp >= p.max_pages) return -1;
    const int page = __ldcg(p.table + (int64_t)i * p.max_pages + lp);
    if ((unsigned)page >= (unsigned)p.n_pages) return -1;
    return page * p.page_size + (pos - lp * p.page_size);
}

// The pool position of packed row `row`: -1 for a hole or a row before its sequence's position 0, -2 for a
// row that belongs to no sequence.
__device__ __forceinline__ int row_slot(const PagedView &p, const int32_t *row_start, int row) {
    const int i = find_seq(row_start, p.n_seq, row);
    if (i < 0) return -2;
    const int len = max(__ldcg(p.len + i), 0);
    return page_slot(p, i, len - (__ldcg(row_start + i + 1) - row));
}

}  // namespace kvc
