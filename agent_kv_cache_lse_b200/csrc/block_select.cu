// The choice of pages a decode query attends to (kvc_select_blocks).
//
// For a page whose keys lie between lo and hi elementwise, max(q_d lo_d, q_d hi_d) summed over d bounds q . k from
// above for every key of the page.  Summed over the query heads g of the row's group that is
//     score_b = sum_d (sum_g max(q_gd, 0)) hi_bd + (sum_g min(q_gd, 0)) lo_bd = sum_d up_d hi_bd + down_d lo_bd,
// one dot product of 2 D terms a page whatever the group's size.  It is taken in 64 bits: which pages are chosen is a
// whole number, and with 32 bits two orders of summation would choose differently at the border.  A bound that is not
// finite always makes the sum NaN or +inf (0 * inf, or inf - inf, where the factors' signs do not), and NaN ranks as
// +inf.
//
// Launch A: a warp a page; 16 bytes a lane of [lo | hi], the matching up or down in registers as doubles.  The score
//   becomes an order-preserving 64-bit key in the workspace: 0 for a page that is hidden or past the row's length,
//   all ones for the pages that are always taken, and else the key of the score (never 0 or all ones).
// Launch B: a CTA a row; radix search over the keys, eight bits at a time from the top, for the top_k-th largest, then
//   one pass in index order that lists the keys above it and the first of those equal to it.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPickThreads = 512;

struct SelectArgs {
    CacheView c;
    const void *bounds;
    const int32_t *block_pos;
    const void *q;
    const int32_t *q_pos;
    int32_t num_q_heads, top_k, sink, recent;
    int32_t *block_list, *block_count;
    unsigned long long *keys;  // [rows][max_pages_per_row]
    int32_t *status;
};

constexpr unsigned long long kAlways = ~0ull;

// larger score -> larger key; NaN ranks as +inf, -0 as 0
__device__ __forceinline__ unsigned long long score_key(double s) {
    if (isnan(s)) s = __longlong_as_double(0x7ff0000000000000ll);
    const unsigned long long b = (unsigned long long)__double_as_longlong(s + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) block_score_kernel(SelectArgs a) {
    constexpr int N = 16 / sizeof(T);          // elements of a lane's load
    constexpr int LOADS = 2 * D / (32 * N) > 0 ? 2 * D / (32 * N) : 1;
    constexpr int LANES = 2 * D / (N * LOADS); // lanes that hold a page's elements (16 at bf16, D 64; else 32)
    constexpr int PAGES = 32 / LANES;          // pages a warp takes at a time
    __shared__ double w[2 * D];                // [down | up]
    const CacheView &c = a.c;
    const int row = blockIdx.y, lane = threadIdx.x & 31, P = c.page_size, Hkv = c.num_kv_heads;
    const int seq = row / (c.num_layers * Hkv), G = a.num_q_heads / Hkv;
    const int n = c.row_len[row];
    if (n < 0 || n > c.max_slots) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, KVC_DEV_BAD_LENGTH, row);
        return;
    }
    const int nb = (n + P - 1) / P;
    if ((int)(blockIdx.x * kWarps * PAGES) >= nb) return;
    const T *q = static_cast<const T *>(a.q) + ((int64_t)(row / Hkv) * a.num_q_heads + (row % Hkv) * G) * D;
    for (int d = threadIdx.x; d < D; d += kThreads) {
        double up = 0, down = 0;
        for (int g = 0; g < G; ++g) {
            const double x = (double)static_cast<float>(q[g * D + d]);
            up += x > 0 ? x : (x <= 0 ? 0 : x);  // a NaN stays
            down += x < 0 ? x : (x >= 0 ? 0 : x);
        }
        w[d] = down;
        w[D + d] = up;
    }
    __syncthreads();
    const int sub = lane % LANES, half = lane / LANES;
    double wr[LOADS][N];
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) wr[k][i] = w[(k * LANES + sub) * N + i];
    const int qpos = a.q_pos[seq];
    const int64_t base = (int64_t)row * c.max_pages_per_row;
    const T *bounds = static_cast<const T *>(a.bounds) + base * 2 * D;
    const int stride = gridDim.x * kWarps * PAGES;
    for (int b0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * PAGES; b0 < nb; b0 += stride) {
        const int b = b0 + half;
        double s = 0;
        if (b < nb) {
#pragma unroll
            for (int k = 0; k < LOADS; ++k) {
                const uint4 u = *reinterpret_cast<const uint4 *>(bounds + (int64_t)b * 2 * D + (k * LANES + sub) * N);
                const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (N == 8) {
                        s = fma(wr[k][2 * i], (double)__uint_as_float(x[i] << 16), s);
                        s = fma(wr[k][2 * i + 1], (double)__uint_as_float(x[i] & 0xffff0000u), s);
                    } else {
                        s = fma(wr[k][i], (double)__uint_as_float(x[i]), s);
                    }
                }
            }
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (sub == 0 && b < nb) {
            unsigned long long key = 0;
            if (a.block_pos[base + b] <= qpos) key = b < a.sink || b >= nb - a.recent ? kAlways : score_key(s);
            a.keys[base + b] = key;
        }
    }
}

__global__ void __launch_bounds__(kPickThreads) block_pick_kernel(SelectArgs a) {
    __shared__ unsigned hist[256];
    __shared__ int red[32];
    __shared__ unsigned long long prefix_s;
    __shared__ int remaining_s;
    const CacheView &c = a.c;
    const int row = blockIdx.x, tid = threadIdx.x, P = c.page_size;
    int n = c.row_len[row];
    if (n < 0 || n > c.max_slots) n = 0;
    const int nb = (n + P - 1) / P;
    const unsigned long long *keys = a.keys + (int64_t)row * c.max_pages_per_row;
    int32_t *list = a.block_list + (int64_t)row * a.top_k;
    int mine = 0;
    for (int b = tid; b < nb; b += kPickThreads) mine += keys[b] != 0;
    const int visible = block_sum<int>(mine, red), k = min(a.top_k, visible);
    if (tid == 0) {
        prefix_s = 0;
        remaining_s = k;
        a.block_count[row] = k;
    }
    for (int i = k + tid; i < a.top_k; i += kPickThreads) list[i] = -1;
    if (k == 0) return;
    unsigned long long mask = 0;
    for (int shift = 56; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kPickThreads) hist[i] = 0;
        __syncthreads();
        const unsigned long long prefix = prefix_s;
        for (int b = tid; b < nb; b += kPickThreads) {
            const unsigned long long key = keys[b];
            if (key != 0 && (key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1u);
        }
        __syncthreads();
        if (tid < 32) {  // lane covers bins 255 - 8 lane .. 248 - 8 lane
            int sum = 0;
            for (int i = 0; i < 8; ++i) sum += hist[255 - 8 * tid - i];
            const int rem = remaining_s;  // read by every lane before one of them writes it below
            int incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, incl, o);
                if (tid >= o) incl += y;
            }
            __syncwarp();
            if (incl - sum < rem && incl >= rem) {
                int run = incl - sum;
                for (int i = 0; i < 8; ++i) {
                    const int bin = 255 - 8 * tid - i;
                    if (run + (int)hist[bin] >= rem) {
                        prefix_s = prefix | ((unsigned long long)bin << shift);
                        remaining_s = rem - run;
                        break;
                    }
                    run += hist[bin];
                }
            }
        }
        mask |= 255ull << shift;
        __syncthreads();
    }
    // keys above the threshold, and the first `equal` of those at it, in index order
    const unsigned long long T = prefix_s;
    const int equal = remaining_s;
    int out = 0, ties = 0;
    for (int b0 = 0; b0 < nb; b0 += kPickThreads) {
        const int b = b0 + tid;
        const unsigned long long key = b < nb ? keys[b] : 0;
        int tile_ties, tile_out;
        const int tie = ties + block_exclusive_scan(key == T, red, &tile_ties);
        const bool take = key > T || (key == T && tie < equal);
        const int at = out + block_exclusive_scan(take, red, &tile_out);
        if (take) list[at] = b;
        ties += tile_ties;
        out += tile_out;
    }
}

template <typename T>
void score(const SelectArgs &a, dim3 grid, cudaStream_t stream) {
    if (a.c.head_dim == 128) block_score_kernel<T, 128><<<grid, kThreads, 0, stream>>>(a);
    else block_score_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a);
}

}  // namespace

cudaError_t launch_select_blocks(const CacheView &c, const void *bounds, const int32_t *block_pos, const void *q,
                                 const int32_t *q_pos, int32_t num_q_heads, int32_t top_k, int32_t sink, int32_t recent,
                                 int32_t *block_list, int32_t *block_count, void *ws, int32_t *status,
                                 cudaStream_t stream) {
    SelectArgs a{c, bounds, block_pos, q, q_pos, num_q_heads, top_k, sink, recent, block_list, block_count,
                 static_cast<unsigned long long *>(ws), status};
    const int wide = (c.max_pages_per_row + kWarps - 1) / kWarps;
    const dim3 grid(std::max(1, std::min((device_sms() * 8 + c.rows - 1) / c.rows, wide)), c.rows);
    if (c.dtype == KVC_BF16) score<__nv_bfloat16>(a, grid, stream);
    else score<float>(a, grid, stream);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    block_pick_kernel<<<c.rows, kPickThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc
