// Even shares of ragged rows: the rows' units of work (chunks of slots, pages), one row after another, form one sequence
// of U units, and W runs of nearly equal length cut it wherever rows begin and end.  A few long rows, many short ones and
// rows of unlike lengths then load the GPU alike, and no launch shape depends on lengths that only the device knows.
#pragma once

#include <cstdint>

namespace kvc {

// per_cta runs for each CTA of the launch (consecutive ones), W in all; every run has at least one unit: the first `more` runs
// have each + 1, the others each.  (One division a share: U w / W for each of a CTA's runs took longer than the search.)
struct Share {
    int64_t U, each;
    int per_cta, W, more;
};

// first unit of run w
__device__ __forceinline__ int64_t run_start(const Share &s, int w) { return s.each * w + min(w, s.more); }

// run of unit x
__device__ __forceinline__ int run_of(const Share &s, int64_t x) {
    const int64_t first = (s.each + 1) * s.more;  // units of the longer runs
    return x < first ? (int)(x / (s.each + 1)) : s.more + (int)((x - first) / s.each);
}

// A run of at least min_run units where there are that many, and at most kRuns runs a CTA
template <int kRuns>
__device__ __forceinline__ Share share_units(int64_t U, int ctas, int min_run) {
    Share s;
    s.U = U;
    const int64_t enough = (int64_t)ctas * min_run * (kRuns - 1);  // beyond this every run of every CTA is used
    s.per_cta = U > enough ? kRuns : max(1, (int)(((unsigned)U + ctas * min_run - 1) / (unsigned)(ctas * min_run)));
    s.W = (int)min(U, (int64_t)ctas * s.per_cta);
    if (s.W == 0) s.each = s.more = 0;
    else if (U <= INT32_MAX) s.each = (unsigned)U / (unsigned)s.W, s.more = (int)((unsigned)U - (unsigned)s.each * (unsigned)s.W);
    else s.each = U / s.W, s.more = (int)(U - s.each * s.W);
    return s;
}

template <int kRuns>
struct RunTable {
    long long scan[32];
    int row[kRuns];     // the run's first row ...
    int off[kRuns];     // ... and its first unit in that row
};

// Share out the rows' units, count(r) of them in row r.  Every CTA sums the counts itself (each thread its share of
// the rows, then a scan over the CTA) and finds where its runs start.  All threads call it; the table is ready on return.
template <int kRuns, typename Count>
__device__ __forceinline__ Share share_rows(int rows, int min_run, RunTable<kRuns> &t, Count count) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int each = (rows + (int)blockDim.x - 1) / (int)blockDim.x;
    const int r0 = min(rows, tid * each), r1 = min(rows, r0 + each);
    long long mine = 0;
    int first = 0;
    for (int r = r0; r < r1; ++r) {
        const int n = count(r);
        if (r == r0) first = n;
        mine += n;
    }
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) t.scan[warp] = x;
    __syncthreads();
    long long before = x - mine;
    int64_t U = 0;
    for (int k = 0; k < nw; ++k) {
        if (k < warp) before += t.scan[k];
        U += t.scan[k];
    }
    const Share s = share_units<kRuns>(U, gridDim.x, min_run);
    if (mine > 0) {
        // the CTA's runs that start in this thread's rows
        const int w0 = blockIdx.x * s.per_cta;
        for (int k = 0; k < s.per_cta && w0 + k < s.W; ++k) {
            const int64_t at = run_start(s, w0 + k);
            if (at < before || at >= before + mine) continue;
            int64_t left = at - before;
            int r = r0, n = first;
            while (left >= n) {
                left -= n;
                n = count(++r);
            }
            t.row[k] = r;
            t.off[k] = (int)left;
        }
    }
    __syncthreads();
    return s;
}

}  // namespace kvc
