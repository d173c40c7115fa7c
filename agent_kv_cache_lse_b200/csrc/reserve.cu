// Block tables and slot maps from the lengths of the requests' new tokens (kvc_reserve_slots).
//
// Sequence s brings c_s tokens, T = sum c_s in all, packed: token t = start_s + i.  Row r (sequence, layer, KV head)
// holds n_r slots, so it grows by need_r = ceil((n_r + c_s) / P) - ceil(n_r / P) pages, taken from the top of the
// free-page stack: with `total` pages taken in all and off_r those of lower rows, the row's k-th new page is
// free_pages[depth - total + off_r + k].  Token t of row r then lives in slot n_r + i, whose physical slot is
// page * P + (n_r + i) % P.
//
// Launch A (one CTA): exclusive scans of c_s (token_start) and need_r (off_r), the refusals, the new lengths and
//   the new stack depth.  A thread reads a row's old length before it writes its new one, so row_len_out may be the
//   cache's own row_len; launch B takes the old length as new length - c_s.
// Launch B: a thread per (token, layer, head).  The thread whose slot opens a page enters that page in the block
//   table: a slot at offset 0 is past the old length only in a page the row did not hold, and nobody in this
//   launch reads that entry (new pages come from the stack).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kFillThreads = 256;

struct ReserveArgs {
    CacheView c;
    const int32_t *new_count, *next_pos;
    uint8_t label;
    float *crf;
    const int32_t *free_pages;
    const int64_t *free_count;
    int32_t max_tokens;
    int32_t *row_len_out;
    int64_t *free_count_out;
    int32_t *token_start, *token_pos;
    int64_t *slot_map;
    int64_t *ws;  // [rows]: first new page's index on the stack, -1 for a refused row; [rows]: 1 when the call is refused
    int32_t *status;
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

// tokens sequence s brings (a negative count is reported where the scan meets it)
__device__ __forceinline__ int count_of(const ReserveArgs &a, int s) { return max(0, a.new_count[s]); }

// positions next_pos .. next_pos + c - 1 must be token positions (0 .. INT32_MAX - 1)
__device__ __forceinline__ bool bad_positions(const ReserveArgs &a, int s, int cnt) {
    return cnt > 0 && (a.next_pos[s] < 0 || (int64_t)a.next_pos[s] + cnt > INT32_MAX);
}

// new pages of row r, or -1 and the device code when the row cannot take its tokens
__device__ __forceinline__ int row_need(const ReserveArgs &a, int r, int *code) {
    const CacheView &c = a.c;
    const int s = r / (c.num_layers * c.num_kv_heads), n = a.c.row_len[r], cnt = count_of(a, s);
    if (cnt == 0) return 0;
    if (n < 0 || n > c.max_slots || bad_positions(a, s, cnt)) return *code = KVC_DEV_BAD_LENGTH, -1;
    if ((int64_t)n + cnt > c.max_slots) return *code = KVC_DEV_FREED_OVERFLOW, -1;
    if (n % c.page_size != 0) {  // the first token joins the row's last page
        const int32_t pg = c.block_table[(int64_t)r * c.max_pages_per_row + n / c.page_size];
        if (pg < 0 || pg >= c.num_pages) return *code = KVC_DEV_BAD_PAGE, -1;
    }
    return cdiv(n + cnt, c.page_size) - cdiv(n, c.page_size);
}

__global__ void __launch_bounds__(kPlanThreads) reserve_plan_kernel(ReserveArgs a) {
    __shared__ long long red[32];
    const CacheView &c = a.c;
    // block-wide exclusive scan of 64-bit values, carried over tiles of kPlanThreads
    auto scan = [&](long long v, long long &carry) {
        const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
        long long x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();
        if (lane == 31) red[w] = x;
        __syncthreads();
        long long before = 0, total = 0;
        for (int k = 0; k < kPlanThreads / 32; ++k) {
            if (k < w) before += red[k];
            total += red[k];
        }
        const long long ex = carry + before + x - v;
        carry += total;
        return ex;
    };
    long long tokens = 0;
    for (int s0 = 0; s0 < c.num_seqs; s0 += kPlanThreads) {
        const int s = s0 + threadIdx.x;
        if (s < c.num_seqs && a.new_count[s] < 0) report(a.status, KVC_DEV_BAD_LENGTH, s * c.num_layers * c.num_kv_heads);
        const long long ex = scan(s < c.num_seqs ? count_of(a, s) : 0, tokens);
        if (s < c.num_seqs) a.token_start[s] = (int)min(ex, (long long)a.max_tokens);
    }
    long long total = 0;
    for (int r0 = 0; r0 < c.rows; r0 += kPlanThreads) {
        const int r = r0 + threadIdx.x;
        int need = 0, code = 0;
        if (r < c.rows) {
            need = row_need(a, r, &code);
            if (need < 0) report(a.status, code, r);
        }
        const long long ex = scan(max(need, 0), total);
        if (r < c.rows) a.ws[r] = need < 0 ? -1 : ex;
    }
    const long long depth = *a.free_count;
    const bool over = tokens > a.max_tokens, refuse = over || (total > 0 && total > depth);
    __syncthreads();  // the depth is read by everyone before thread 0 may write it (free_count_out may be free_count)
    if (threadIdx.x == 0) {
        if (refuse) report(a.status, over ? KVC_DEV_BAD_LENGTH : KVC_DEV_FREED_OVERFLOW, -1);
        a.token_start[c.num_seqs] = (int)min(tokens, (long long)a.max_tokens);
        a.ws[c.rows] = refuse ? 1 : 0;
        *a.free_count_out = refuse ? depth : depth - total;
    }
    for (int r = threadIdx.x; r < c.rows; r += kPlanThreads) {
        const bool take = !refuse && a.ws[r] >= 0;
        if (take) a.ws[r] += depth - total;
        const int n = c.row_len[r];
        a.row_len_out[r] = take ? n + count_of(a, r / (c.num_layers * c.num_kv_heads)) : n;
    }
}

__global__ void __launch_bounds__(kFillThreads) reserve_fill_kernel(ReserveArgs a) {
    const CacheView &c = a.c;
    const int per = c.num_layers * c.num_kv_heads, P = c.page_size, S = c.num_seqs;
    const int total = a.token_start[S];
    const bool refused = a.ws[c.rows] != 0;
    const int64_t cells = (int64_t)a.max_tokens * per;
    for (int64_t x = (int64_t)blockIdx.x * kFillThreads + threadIdx.x; x < cells; x += (int64_t)gridDim.x * kFillThreads) {
        const int t = (int)(x / per), lh = (int)(x % per);
        if (t >= total || refused) {
            a.slot_map[x] = -1;
            if (lh == 0) a.token_pos[t] = -1;
            continue;
        }
        int s = 0;  // the sequence with token_start[s] <= t < token_start[s + 1]
        for (int hi = S; hi - s > 1;) {
            const int mid = (s + hi) / 2;
            if (a.token_start[mid] <= t) s = mid;
            else hi = mid;
        }
        const int cnt = count_of(a, s), i = t - a.token_start[s], r = s * per + lh;
        if (lh == 0) a.token_pos[t] = bad_positions(a, s, cnt) ? -1 : a.next_pos[s] + i;
        const int64_t at = a.ws[r];
        if (at < 0) {
            a.slot_map[x] = -1;
            continue;
        }
        const int n = a.row_len_out[r] - cnt, slot = n + i, lp = slot / P, first = cdiv(n, P);
        int32_t *entry = c.block_table + (int64_t)r * c.max_pages_per_row + lp;
        const int32_t pg = lp < first ? *entry : a.free_pages[at + lp - first];
        const bool ok = pg >= 0 && pg < c.num_pages;
        if (!ok) report(a.status, KVC_DEV_BAD_PAGE, r);
        a.slot_map[x] = ok ? (int64_t)pg * P + slot % P : -1;
        if (lp >= first && slot % P == 0) *entry = pg;
        const int64_t ms = (int64_t)r * c.max_slots + slot;
        c.slot_pos[ms] = a.next_pos[s] + i;
        if (c.slot_label) c.slot_label[ms] = a.label;
        if (a.crf) a.crf[ms] = 0.f;
    }
}

}  // namespace

cudaError_t launch_reserve(const CacheView &c, const int32_t *new_count, const int32_t *next_pos, uint8_t label, float *crf,
                           const int32_t *free_pages, const int64_t *free_count, int32_t max_tokens,
                           int32_t *row_len_out, int64_t *free_count_out, int32_t *token_start, int32_t *token_pos,
                           int64_t *slot_map, int64_t *ws, int32_t *status, cudaStream_t stream) {
    ReserveArgs a{c, new_count, next_pos, label, crf, free_pages, free_count, max_tokens, row_len_out, free_count_out,
                  token_start, token_pos, slot_map, ws, status};
    reserve_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || max_tokens == 0) return e;
    const int64_t cells = (int64_t)max_tokens * c.num_layers * c.num_kv_heads;
    const int grid = (int)std::min<int64_t>((cells + kFillThreads - 1) / kFillThreads, (int64_t)device_sms() * 8);
    reserve_fill_kernel<<<grid, kFillThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc
