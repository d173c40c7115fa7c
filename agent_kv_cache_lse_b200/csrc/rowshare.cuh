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

constexpr int kShareThreads = 256;  // threads of a CTA that shares rows

struct RunTable {
    long long scan[kShareThreads / 32];
    long long before[kShareThreads];  // units before each thread's rows
};

// Share out the rows' units, count(r) of them in row r.  Every CTA sums the counts itself: each thread its share of
// the rows, then a scan over the CTA.  Warp k of a CTA takes the CTA's k-th run, if it has one (`run` below W): it finds the
// run's first row, and its first unit in that row, in the scan.  All threads of the CTA call it, whole warps with the same
// results; row and off are 0 for a warp without a run.
template <int kRuns, typename Count>
__device__ __forceinline__ Share share_rows(int rows, int min_run, RunTable &t, Count count, int &run, int &row, int &off) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int each = (rows + kShareThreads - 1) / kShareThreads;
    const int r0 = min(rows, tid * each), r1 = min(rows, r0 + each);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += count(r);
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
#pragma unroll
    for (int k = 0; k < kShareThreads / 32; ++k) {
        if (k < warp) before += t.scan[k];
        U += t.scan[k];
    }
    t.before[tid] = before;
    __syncthreads();
    const Share s = share_units<kRuns>(U, gridDim.x, min_run);
    run = warp < s.per_cta ? (int)blockIdx.x * s.per_cta + warp : s.W;
    row = off = 0;
    if (run >= s.W) return s;
    // the thread whose rows hold the run's first unit: the last with no more units before it
    const int64_t at = run_start(s, run);
    int who = 0;
#pragma unroll
    for (int step = kShareThreads / 2; step > 0; step /= 2)
        if (t.before[who + step] <= at) who += step;
    int left = (int)(at - t.before[who]);
    row = who * each;
    for (int end = min(rows, row + each); row < end; row += 32) {  // of its rows, 32 at a time
        const int n = row + lane < end ? count(row + lane) : 0;
        int incl = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, incl > left);
        if (past) {
            const int k = __ffs(past) - 1;
            off = left - __shfl_sync(0xffffffffu, incl - n, k);
            row += k;
            return s;
        }
        left -= __shfl_sync(0xffffffffu, incl, 31);
    }
    run = s.W;  // only if the counts changed meanwhile
    row = 0;
    return s;
}

}  // namespace kvc
