// Block tables and slot maps from the lengths of the requests' new tokens (kvc_reserve_slots).
//
// Sequence s brings c_s tokens, T = sum c_s in all, packed: token t = start_s + i.  Row r (sequence, layer, KV head)
// holds n_r slots, so it grows by need_r = ceil((n_r + c_s) / P) - ceil(n_r / P) pages, taken from the top of the
// free-page stack: with `total` pages taken in all and off_r those of lower rows, the row's k-th new page is
// free_pages[depth - total + off_r + k].  Token t of row r then lives in slot n_r + i, whose physical slot is
// page * P + (n_r + i) % P.
//
// The plan (one CTA): a thread takes a run of sequences and a run of rows, one scan over the CTA gives token_start and off_r,
//   and the refusals, the new lengths and the new depth follow.  A thread reads a row's old length before it writes its
//   new one, so row_len_out may be the cache's own row_len; the fill takes the old length as new length - c_s.
// The fill: for every (token, layer, head) its slot.  The thread whose slot opens a page enters that page in the block
//   table: a slot at offset 0 is past the old length only in a page the row did not hold, and nobody in this
//   launch reads that entry (new pages come from the stack).  A CTA takes kTile tokens of 32 rows: slot_pos, labels and crf
//   run along a row, the slot map along the rows of a token, so lanes are tokens of a row while the former are written and
//   the map goes through shared memory and out with lanes as rows (a thread a cell in the map's order, with
//   scattered writes to the rows and a search of the sequence for each cell, took 29 us where this takes 12, both under the profiler).
// The bytes are few; what counts is the chain of dependent loads and the launches.  A decode step's few cells are
// filled by the planning CTA itself; else the fill is a second launch that is resident before the plan ends
// (programmatic dependent launch).  Measured a call: 5.2 us for a decode step of 16 sequences (128 rows), 12.2 us for 28,049 prompt tokens
// of 33 sequences in 1,056 rows (15.8 MB written, 2.4 us of them by bandwidth; the plan's and the fill's load chains, and
// the fill's 5.3 M warp instructions, are the rest).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kBatch = 4;          // rows whose loads a planning thread has side by side
constexpr int kTile = 32;          // tokens a CTA of the fill takes
constexpr int kStarts = 1024;      // sequences whose token_start a CTA searches in shared memory
constexpr int kAloneTiles = 4;     // tiles (kTile tokens of 32 rows) that the planning CTA fills itself

struct ReserveArgs {
    CacheView c;
    const int32_t *new_count, *next_pos;
    uint8_t label;
    float *crf;
    const int32_t *free_pages;
    int64_t free_capacity;
    const int64_t *free_count;
    int32_t max_tokens;
    int32_t *row_len_out;
    int64_t *free_count_out;
    int32_t *token_start, *token_pos;
    int64_t *slot_map;
    int64_t *ws;  // [rows]: first new page's index on the stack, -1 for a refused row; [rows]: 1 when the call is refused
    uint64_t recip;  // ceil(2^37 / page_size)
    int32_t *status;
};

// x / page_size for 0 <= x < 2^25 (page_size <= 2^12: the error x * page_size / 2^37 stays below 1); a division by a
// variable is 30 instructions, and three of them a cell were a quarter of the fill's time
__device__ __forceinline__ int page_of(const ReserveArgs &a, int x) { return (int)(((uint64_t)(uint32_t)x * a.recip) >> 37); }
__device__ __forceinline__ int pages_for(const ReserveArgs &a, int slots) { return page_of(a, slots + a.c.page_size - 1); }

// tokens sequence s brings (a negative count is reported where the scan meets it)
__device__ __forceinline__ int count_of(const ReserveArgs &a, int s) { return max(0, a.new_count[s]); }

// positions next_pos .. next_pos + c - 1 must be token positions (0 .. INT32_MAX - 1)
__device__ __forceinline__ bool bad_positions(const ReserveArgs &a, int s, int cnt) {
    return cnt > 0 && (a.next_pos[s] < 0 || (int64_t)a.next_pos[s] + cnt > INT32_MAX);
}

// the sequence of token t: token_start[s] <= t < token_start[s + 1]
__device__ __forceinline__ int sequence_of(const int32_t *token_start, int S, int t) {
    int s = 0;
    for (int hi = S; hi - s > 1;) {
        const int mid = (s + hi) / 2;
        if (token_start[mid] <= t) s = mid;
        else hi = mid;
    }
    return s;
}

// Fill kTile tokens from t0 on for 32 rows of their sequences from lh0 on (kThreads threads; all of them call it)
template <int kThreads>
__device__ __forceinline__ void fill_tile(const ReserveArgs &a, int t0, int lh0, bool refused, int total) {
    __shared__ int seq_s[kTile], start_s[kTile], cnt_s[kTile], pos_s[kTile], starts_s[kStarts];
    __shared__ int64_t map_s[kTile][33];
    const CacheView &c = a.c;
    const int per = c.num_layers * c.num_kv_heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int here = min(kTile, a.max_tokens - t0), rows = min(32, per - lh0), S = c.num_seqs;
    if (S < kStarts) {
        for (int s = threadIdx.x; s <= S; s += kThreads) starts_s[s] = a.token_start[s];
        __syncthreads();
    }
    const int32_t *starts = S < kStarts ? starts_s : a.token_start;
    if (threadIdx.x < kTile && (int)threadIdx.x < here) {
        const int t = t0 + threadIdx.x;
        int s = -1, start = 0, cnt = 0, pos = -1;
        if (t < total && !refused) {
            s = sequence_of(starts, S, t);
            start = starts[s];
            cnt = starts[s + 1] - start;
            if (!bad_positions(a, s, cnt)) pos = a.next_pos[s] + t - start;
        }
        seq_s[threadIdx.x] = s;
        start_s[threadIdx.x] = start;
        cnt_s[threadIdx.x] = cnt;
        pos_s[threadIdx.x] = pos;
        if (lh0 == 0) a.token_pos[t] = pos;
    }
    __syncthreads();
    // a warp: 32 tokens of one row at a time; the dependent loads of all its rows go side by side
    constexpr int kItems = 32 * (kTile / 32) / (kThreads / 32);
    const int P = c.page_size;
    int row[kItems], slot[kItems], first[kItems];
    int64_t at[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int x = warp + k * (kThreads / 32), j = x % 32, i = x / 32 * 32 + lane;
        row[k] = -1;
        if (j < rows && i < here && seq_s[i] >= 0) {
            row[k] = seq_s[i] * per + lh0 + j;
            at[k] = a.ws[row[k]];
            const int n = a.row_len_out[row[k]] - cnt_s[i];
            slot[k] = n + t0 + i - start_s[i];
            first[k] = pages_for(a, n);
        }
    }
    int32_t page[kItems];
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        if (row[k] < 0 || at[k] < 0) continue;
        const int lp = page_of(a, slot[k]);
        page[k] = lp < first[k] ? c.block_table[(int64_t)row[k] * c.max_pages_per_row + lp] : a.free_pages[at[k] + lp - first[k]];
    }
#pragma unroll
    for (int k = 0; k < kItems; ++k) {
        const int x = warp + k * (kThreads / 32), j = x % 32, i = x / 32 * 32 + lane;
        if (j >= rows || i >= here) continue;
        int64_t value = -1;
        if (row[k] >= 0 && at[k] >= 0) {
            const int lp = page_of(a, slot[k]), o = slot[k] - lp * P;
            const bool ok = page[k] >= 0 && page[k] < c.num_pages;
            if (ok) value = (int64_t)page[k] * P + o;
            else report(a.status, KVC_DEV_BAD_PAGE, row[k]);
            if (lp >= first[k] && o == 0) c.block_table[(int64_t)row[k] * c.max_pages_per_row + lp] = page[k];
            const int64_t ms = (int64_t)row[k] * c.max_slots + slot[k];
            c.slot_pos[ms] = pos_s[i];
            if (c.slot_label) c.slot_label[ms] = a.label;
            if (a.crf) a.crf[ms] = 0.f;
        }
        map_s[i][j] = value;
    }
    __syncthreads();
    // a warp: 32 rows of one token
    for (int i = warp; i < here; i += kThreads / 32)
        if (lane < rows) a.slot_map[(int64_t)(t0 + i) * per + lh0 + lane] = map_s[i][lane];
}

// kAlone: the cells are few and this CTA fills them too
template <bool kAlone>
__global__ void __launch_bounds__(kPlanThreads, 1) reserve_plan_kernel(ReserveArgs a) {
    __shared__ long long red_t[32], red_p[32];
    const CacheView &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5, per = c.num_layers * c.num_kv_heads;
    begin_dependent();
    const long long depth = *a.free_count;
    const int se = (c.num_seqs + kPlanThreads - 1) / kPlanThreads, s0 = min(c.num_seqs, tid * se), s1 = min(c.num_seqs, s0 + se);
    const int re = (c.rows + kPlanThreads - 1) / kPlanThreads, r0 = min(c.rows, tid * re), r1 = min(c.rows, r0 + re);
    long long tokens = 0, pages = 0;  // of this thread's sequences and rows
    for (int s = s0; s < s1; ++s) {
        if (a.new_count[s] < 0) report(a.status, KVC_DEV_BAD_LENGTH, s * per);
        tokens += count_of(a, s);
    }
    // the new pages of each row (-1: it cannot take its tokens), kBatch rows with their loads side by side
    int len[kBatch], cnt[kBatch];
    int64_t off[kBatch];  // the row's first new page among this thread's (-1: refused); one batch is kept to the end, more go through ws
    for (int b0 = r0; b0 < r1; b0 += kBatch) {
        int next[kBatch], code[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = b0 + k, s = r < r1 ? r / per : 0;
            len[k] = r < r1 ? c.row_len[r] : 0;
            cnt[k] = r < r1 ? count_of(a, s) : 0;
            next[k] = r < r1 ? a.next_pos[s] : 0;
        }
        int32_t joined[kBatch];  // the page that a row's first token joins
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            code[k] = KVC_DEV_OK;
            joined[k] = 0;
            if (cnt[k] == 0) continue;
            if (len[k] < 0 || len[k] > c.max_slots || next[k] < 0 || (int64_t)next[k] + cnt[k] > INT32_MAX) {
                code[k] = KVC_DEV_BAD_LENGTH;
            } else if ((int64_t)len[k] + cnt[k] > c.max_slots) {
                code[k] = KVC_DEV_FREED_OVERFLOW;
            } else {
                const int held = pages_for(a, len[k]);
                if (held * c.page_size != len[k]) joined[k] = c.block_table[(int64_t)(b0 + k) * c.max_pages_per_row + held - 1];
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int r = b0 + k;
            if (r >= r1) continue;
            if (code[k] == KVC_DEV_OK && (joined[k] < 0 || joined[k] >= c.num_pages)) code[k] = KVC_DEV_BAD_PAGE;
            if (code[k] != KVC_DEV_OK) report(a.status, code[k], r);
            off[k] = code[k] == KVC_DEV_OK ? pages : -1;
            if (r1 - r0 > kBatch) a.ws[r] = off[k];
            if (code[k] == KVC_DEV_OK && cnt[k]) pages += pages_for(a, len[k] + cnt[k]) - pages_for(a, len[k]);
        }
    }
    long long xt = tokens, xp = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long yt = __shfl_up_sync(0xffffffffu, xt, o), yp = __shfl_up_sync(0xffffffffu, xp, o);
        if (lane >= o) xt += yt, xp += yp;
    }
    if (lane == 31) red_t[w] = xt, red_p[w] = xp;
    __syncthreads();
    // every warp scans the warps' sums for itself
    long long wt = red_t[lane], wp = red_p[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long yt = __shfl_up_sync(0xffffffffu, wt, o), yp = __shfl_up_sync(0xffffffffu, wp, o);
        if (lane >= o) wt += yt, wp += yp;
    }
    const long long all_tokens = __shfl_sync(0xffffffffu, wt, 31), all_pages = __shfl_sync(0xffffffffu, wp, 31);
    const long long before_t = __shfl_sync(0xffffffffu, wt, (w + 31) & 31), before_p = __shfl_sync(0xffffffffu, wp, (w + 31) & 31);
    long long at = (w ? before_t : 0) + xt - tokens;
    for (int s = s0; s < s1; ++s) {
        a.token_start[s] = (int)min(at, (long long)a.max_tokens);
        at += count_of(a, s);
    }
    const bool over = all_tokens > a.max_tokens, shallow = depth < 0 || depth > a.free_capacity || all_pages > depth;
    const bool refuse = over || shallow;
    // the depth was read by everyone before the barrier above, so free_count_out may be free_count
    if (tid == 0) {
        if (refuse) report(a.status, over ? KVC_DEV_BAD_LENGTH : KVC_DEV_FREED_OVERFLOW, -1);
        a.token_start[c.num_seqs] = (int)min(all_tokens, (long long)a.max_tokens);
        a.ws[c.rows] = refuse ? 1 : 0;
        *a.free_count_out = refuse ? depth : depth - all_pages;
    }
    const long long base = depth - all_pages + (w ? before_p : 0) + xp - pages;
    for (int b0 = r0; b0 < r1; b0 += kBatch) {
        if (r1 - r0 > kBatch) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (b0 + k < r1) off[k] = a.ws[b0 + k], len[k] = c.row_len[b0 + k], cnt[k] = count_of(a, (b0 + k) / per);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (b0 + k < r1) {
                const bool take = !refuse && off[k] >= 0;
                a.ws[b0 + k] = take ? base + off[k] : -1;
                a.row_len_out[b0 + k] = take ? len[k] + cnt[k] : len[k];
            }
    }
    if constexpr (kAlone) {
        __syncthreads();  // what the CTA wrote above is read below
        for (int t0 = 0; t0 < a.max_tokens; t0 += kTile)
            for (int lh0 = 0; lh0 < per; lh0 += 32) {
                fill_tile<kPlanThreads>(a, t0, lh0, refuse, (int)min(all_tokens, (long long)a.max_tokens));
                __syncthreads();
            }
    }
}

__global__ void __launch_bounds__(kFillThreads) reserve_fill_kernel(ReserveArgs a) {
    begin_dependent();
    fill_tile<kFillThreads>(a, blockIdx.x * kTile, blockIdx.y * 32, a.ws[a.c.rows] != 0, a.token_start[a.c.num_seqs]);
}

}  // namespace

cudaError_t launch_reserve(const CacheView &c, const int32_t *new_count, const int32_t *next_pos, uint8_t label, float *crf,
                           const int32_t *free_pages, int64_t free_capacity, const int64_t *free_count,
                           int32_t max_tokens, int32_t *row_len_out, int64_t *free_count_out, int32_t *token_start, int32_t *token_pos,
                           int64_t *slot_map, int64_t *ws, int32_t *status, cudaStream_t stream) {
    ReserveArgs a{c, new_count, next_pos, label, crf, free_pages, free_capacity, free_count, max_tokens, row_len_out, free_count_out,
                  token_start, token_pos, slot_map, ws, ((1ull << 37) + c.page_size - 1) / c.page_size, status};
    const int64_t tiles_t = ((int64_t)max_tokens + kTile - 1) / kTile, tiles_r = (c.num_layers * c.num_kv_heads + 31) / 32;
    if (tiles_t * tiles_r <= kAloneTiles) {
        return launch_dependent(reserve_plan_kernel<true>, dim3(1), kPlanThreads, 0, stream, a);
    }
    cudaError_t e = launch_dependent(reserve_plan_kernel<false>, dim3(1), kPlanThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_dependent(reserve_fill_kernel, dim3((unsigned)tiles_t, (unsigned)tiles_r), kFillThreads, 0, stream, a);
}

}  // namespace kvc
