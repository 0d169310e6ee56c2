// The page table, the lengths and the places of the packed rows, from what each sequence's length changes by.
//
//   lengths: new = clamp(old + rows, 0, 2^31 - 1); a sequence uses P(n) = min(ceil(n / page), max_pages) pages.
//   entries [P(old), P(new)) take pages from the front of the ring of free ones, in the order of sequences and entries (a page
//   that is not there is -1, a hole); entries [P(new), P(old)) give theirs back at the ring's end, in the same order.
//   starts = the running sum of the rows that are added; a row's position and its place in the pool.
//
// One CTA makes the three running sums over the sequences (pages taken, pages given back, rows), 1,024 of them at a time, and
// changes the table and the ring by warps; where there are few rows it places them too, looking them up in shared memory,
// else a second kernel does, by all SMs.  What bounds it is a chain of dependent steps: lengths, sums, ring, table.
// Pages that are given back lie behind those that may be taken, so that no cell is read and written in one call.
#include "kvc_internal.h"
#include "paged.cuh"

namespace kvc {
namespace {

// At most: a thread for each sequence, and for each two rows, 128 at least.  In pairs of calls, back to back: 64 sequences that grow
// and shrink by a token 6.0 us (a call 3.0; with 1,024 threads 6.9), 1,024 of them 10.1, 64 with two ends and two prompts 11.4, 1,024
// with 40 prompts and 60 ends, then as many rewound, 110,000 rows in all, 24.
constexpr int THREADS = 1024;
constexpr int ROW_THREADS = 256;
constexpr int FEW = 4;        // entries of a sequence that one thread changes

__device__ __forceinline__ int pages_of(int n, const AdvanceArgs &a) {
    return (int)min(((unsigned)n + (unsigned)a.page_size - 1u) / (unsigned)a.page_size, (unsigned)a.max_pages);
}
__device__ __forceinline__ int length_after(int old, int rows) {
    return (int)min(max((int64_t)old + rows, (int64_t)0), (int64_t)INT32_MAX);
}

// Cell k of a ring that begins at cell `head`; both below the number of cells.
__device__ __forceinline__ int32_t *cell(const AdvanceArgs &a, int head, int64_t k) {
    const int64_t c = head + k;
    return a.ring + (c < a.n_pages ? c : c - a.n_pages);
}
// Entries [from, to) of sequence i from a ring of `count` pages that begins at `head`: the first-th on.  By `step` lanes, of
// which this is the lane-th; several loads at once, since what counts is their latency (of 512 entries one at a time
// 6 us).
template <int AT_ONCE>
__device__ __forceinline__ void take(const AdvanceArgs &a, int head, int count, int i, int from, int to, int64_t first, int lane,
                                     int step) {
    int32_t *entry = a.table + (int64_t)i * a.max_pages;
    for (int e0 = from + lane; e0 < to; e0 += AT_ONCE * step) {
        int page[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int64_t k = first + (e0 - from) + (int64_t)u * step;
            page[u] = to - e0 > u * step && k < count ? __ldcg(cell(a, head, k)) : -1;
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u)
            if (to - e0 > u * step) entry[e0 + u * step] = page[u];
    }
}
// How many entries [from, to) of sequence i hold pages of the pool; WRITE: these go to the ring, the at-th after its
// last on, as long as there is room, and the entries become holes.  By one lane, or (WARP) by all.
template <bool WRITE, bool WARP>
__device__ __forceinline__ int give(const AdvanceArgs &a, int head, int count, int i, int from, int to, int64_t at) {
    constexpr int STEP = WARP ? 32 : 1, AT_ONCE = WARP ? 8 : FEW;
    const int lane = WARP ? threadIdx.x & 31 : 0;
    int32_t *entry = a.table + (int64_t)i * a.max_pages;
    int n = 0;
    for (int e0 = from; e0 < to; e0 += AT_ONCE * STEP) {
        int page[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) page[u] = to - e0 > u * STEP + lane ? __ldcg(entry + e0 + u * STEP + lane) : -1;
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const bool good = (unsigned)page[u] < (unsigned)a.n_pages;
            const unsigned all = WARP ? __ballot_sync(0xffffffffu, good) : good;
            if (WRITE) {
                const int64_t j = at + n + __popc(all & ((1u << lane) - 1));
                if (good && count + j < a.n_pages) *cell(a, head, count + j) = page[u];
                if (to - e0 > u * STEP + lane) entry[e0 + u * STEP + lane] = -1;
            }
            n += __popc(all);
        }
    }
    return n;
}

// The position and the place of packed row `row`, which no sequence but i can hold.
__device__ __forceinline__ void place(const AdvanceArgs &a, int row, int i, int s0, int s1, int len) {
    int pos = -1, slot = -1;
    if (s0 <= row && row < s1) {
        pos = len - (s1 - row);
        slot = page_slot({a.table, a.len, a.n_seq, a.max_pages, a.page_size, a.n_pages}, i, pos);
    }
    if (a.pos) a.pos[row] = pos;
    if (a.slots) a.slots[row] = slot;
}
// find_seq in shared memory.
__device__ __forceinline__ int find_here(const int *start, int n_seq, int row) {
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= row) lo = mid; else hi = mid;
    }
    return lo;
}

// `rows_too`: places the rows as well (n_seq <= THREADS).
__global__ void __launch_bounds__(THREADS) pages_advance_kernel(const AdvanceArgs a, bool rows_too) {
    __shared__ int64_t sums[3][32];
    __shared__ int new_len[THREADS], starts[THREADS + 1];
    // sequences of which many entries change, for all warps: their threads, entries, and place among those taken or given
    __shared__ int n_drop, n_many, drops[THREADS], many[THREADS], from[THREADS], to[THREADS], held[THREADS];
    __shared__ int64_t first[THREADS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    // any contents of the state are safe
    const int s0 = __ldcg(a.state), head = (unsigned)s0 < (unsigned)a.n_pages ? s0 : 0;
    const int count = min(max(__ldcg(a.state + 1), 0), a.n_pages), missing = max(__ldcg(a.state + 2), 0);
    int64_t before[3] = {0, 0, 0};       // taken, given back, rows of the sequences before these
    for (int i0 = 0; i0 < a.n_seq; i0 += threads) {
        const int i = i0 + tid;
        int old = 0, now = 0, had = 0, has = 0, rows = 0;
        if (i < a.n_seq) {
            old = max(__ldcg(a.len + i), 0);
            rows = __ldcg(a.rows + i);
            now = length_after(old, rows);
            had = pages_of(old, a);
            has = pages_of(now, a);
        }
        // A thread changes the few entries of its sequence; warps take those of which many change.
        const int grow = max(has - had, 0), drop = max(had - has, 0);
        if (tid == 0) n_drop = n_many = 0;
        __syncthreads();
        from[tid] = min(had, has);
        to[tid] = max(had, has);
        if (drop > FEW) drops[atomicAdd(&n_drop, 1)] = tid;
        // which entries hold pages is not known beforehand
        int back = drop > 0 && drop <= FEW ? give<false, false>(a, head, count, i, has, had, 0) : 0;
        __syncthreads();
        if (n_drop > 0) {
            for (int j = warp; j < n_drop; j += warps) {
                const int t = drops[j], n = give<false, true>(a, head, count, i0 + t, from[t], to[t], 0);
                if (lane == 0) held[t] = n;
            }
            __syncthreads();
            if (drop > FEW) back = held[tid];
        }
        int64_t x[3] = {grow, back, max(rows, 0)};
        const int64_t own[3] = {x[0], x[1], x[2]};
#pragma unroll
        for (int d = 1; d < 32; d <<= 1)
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const int64_t up = __shfl_up_sync(0xffffffffu, x[c], d);
                if (lane >= d) x[c] += up;
            }
        if (lane == 31)
            for (int c = 0; c < 3; ++c) sums[c][warp] = x[c];
        __syncthreads();
        int64_t total[3];
#pragma unroll
        for (int c = 0; c < 3; ++c) {
            int64_t s = lane < warps ? sums[c][lane] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, s, d);
                if (lane >= d) s += up;
            }
            x[c] += before[c] + (warp > 0 ? __shfl_sync(0xffffffffu, s, max(warp - 1, 0)) : 0);
            total[c] = __shfl_sync(0xffffffffu, s, 31);
            before[c] += total[c];
        }
        new_len[tid] = now;
        starts[tid + 1] = (int)min(x[2], (int64_t)INT32_MAX);
        if (tid == 0) starts[0] = 0;
        if (i < a.n_seq) {
            a.len[i] = now;
            a.starts[i + 1] = starts[tid + 1];
            if (i == 0) a.starts[0] = 0;
        }
        const int64_t taken = x[0] - own[0], given = x[1] - own[1];   // before this sequence
        if (grow > 0 && grow <= FEW) take<FEW>(a, head, count, i, had, has, taken, 0, 1);
        if (drop > 0 && drop <= FEW) give<true, false>(a, head, count, i, has, had, given);
        if (grow > FEW || drop > FEW) {
            first[tid] = grow > 0 ? taken : given;
            held[tid] = grow;
            many[atomicAdd(&n_many, 1)] = tid;
        }
        __syncthreads();
        for (int j = warp; j < n_many; j += warps) {
            const int t = many[j];
            if (held[t] > 0) take<8>(a, head, count, i0 + t, from[t], to[t], first[t], lane, 32);
            else give<true, true>(a, head, count, i0 + t, from[t], to[t], first[t]);
        }
        __syncthreads();
    }
    if (tid == 0) {
        const int64_t out = min(before[0], (int64_t)count), in = min(before[1], (int64_t)a.n_pages - count);
        a.state[0] = (int)((head + out) % a.n_pages);
        a.state[1] = (int)(count - out + in);
        a.state[2] = (int)min(missing + before[0] - out, (int64_t)INT32_MAX);
    }
    if (!rows_too) return;
    for (int row = tid; row < a.n_rows; row += threads) {
        const int i = find_here(starts, a.n_seq, row);
        place(a, row, i, starts[i], starts[i + 1], new_len[i]);
    }
}

__global__ void __launch_bounds__(ROW_THREADS) pages_rows_kernel(const AdvanceArgs a) {
    __shared__ int starts[THREADS + 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int row = blockIdx.x * ROW_THREADS + threadIdx.x;
    const bool here = a.n_seq <= THREADS;
    if (here) {
        for (int i = threadIdx.x; i <= a.n_seq; i += ROW_THREADS) starts[i] = __ldcg(a.starts + i);
        __syncthreads();
    }
    if (row >= a.n_rows) return;
    const int i = here ? find_here(starts, a.n_seq, row) : find_seq(a.starts, a.n_seq, row);
    place(a, row, i, __ldcg(a.starts + i), __ldcg(a.starts + i + 1), __ldcg(a.len + i));
}

}  // namespace

int launch_pages_advance(const AdvanceArgs &a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    int threads = 128;
    while (threads < THREADS && (threads < a.n_seq || 2 * threads < a.n_rows)) threads *= 2;
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // few rows: no second launch
    const bool rows_too = a.n_seq <= THREADS && a.n_rows <= 8 * threads;
    if (cudaLaunchKernelEx(&cfg, pages_advance_kernel, a, rows_too) != cudaSuccess) return KVC_ECUDA;
    if (!rows_too && a.n_rows > 0 && (a.pos || a.slots)) {
        cfg.gridDim = dim3((unsigned)(((int64_t)a.n_rows + ROW_THREADS - 1) / ROW_THREADS));
        cfg.blockDim = dim3(ROW_THREADS);
        if (cudaLaunchKernelEx(&cfg, pages_rows_kernel, a) != cudaSuccess) return KVC_ECUDA;
    }
    return cudaGetLastError() == cudaSuccess ? KVC_OK : KVC_ECUDA;
}

}  // namespace kvc
