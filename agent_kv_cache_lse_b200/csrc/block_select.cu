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
// Launch A: a warp takes kPages loads' pages at a time, 16 bytes a lane of [lo | hi], the matching up or down in registers as
// doubles.  Conversion instructions to 64 bits run at a fraction of the rate of 64-bit multiply-adds (with them the kernel
// took three times the time of its bytes), so an element becomes a double by moving its bits: sign, 8-bit exponent
// and mantissa into the places of a double without correcting the exponent's bias, which is the value times 2^-896,
// subnormal values included; up and down carry 2^800 in return, and what is left orders nothing.  A bound that is not finite
// would pass as a large number there; times 0 in its own type it is NaN, which marks the page.  The pages' sums are
// joined together, halving the pages a lane holds with each of the first two shuffles; the tree is the same for all pages,
// so equal bounds have equal scores.  The score becomes an order-preserving 64-bit key in the workspace: 0 for a page that is
// hidden or past the row's length, all ones for the pages that are always taken, and else the key of the score (never
// 0 or all ones).
// Launch B (resident before A ends, by programmatic dependent launch): a CTA a row.  The keys of a row share their leading
// bits; below those, a histogram of the next 11 bits finds the digit in which the last key taken lies, usually with
// a handful of keys, which are ranked by (key, index) directly; while there are more than kFew, the next 11 bits follow.
// One pass in index order then lists the pages at or above the last one.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 8;           // of the scoring launch, a multiprocessor
constexpr int kPages = 4;          // loads a lane has in flight
constexpr int kPickThreads = 512;
constexpr int kBins = 2048, kBits = 11;
constexpr int kFew = 32;           // keys that one warp ranks
constexpr int kCached = 8192;      // keys of a row that stay in shared memory

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

// s += w * x * 2^-896 for the elements x of a 32-bit word (see above), and z NaN where one is not finite
template <typename T>
struct Element;
template <>
struct Element<__nv_bfloat16> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void add(uint32_t u, const double *w, double &s, uint32_t &z) {
        s = fma(w[0], __hiloint2double(((int)(u << 16) >> 3) & (int)0x8fffe000, 0), s);
        s = fma(w[1], __hiloint2double(((int)u >> 3) & (int)0x8fffe000, 0), s);
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(u), "r"(0u));
    }
};
template <>
struct Element<float> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void add(uint32_t u, const double *w, double &s, uint32_t &z) {
        s = fma(w[0], __hiloint2double(((int)u >> 3) & (int)0x8fffffff, (int)(u << 29)), s);
        asm("fma.rn.f32 %0, %1, %2, %0;" : "+r"(z) : "r"(u), "r"(0u));
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtas) block_score_kernel(SelectArgs a) {
    constexpr int N = 16 / sizeof(T);          // elements of a lane's load
    constexpr int LOADS = 2 * D / (32 * N) > 0 ? 2 * D / (32 * N) : 1;  // a page
    constexpr int LANES = 2 * D / (N * LOADS); // lanes that hold a page's elements (16 at bf16, D 64; else 32)
    constexpr int SIDE = 32 / LANES;           // pages side by side
    constexpr int BATCH = kPages / LOADS * SIDE;  // pages a warp takes at a time: 4, 8 or (fp32, D 128) 2
    constexpr int DEEP = BATCH / SIDE;         // of them in the same lanes
    __shared__ double w[2 * D];                // [down | up]
    begin_dependent();
    const CacheView &c = a.c;
    const int row = blockIdx.y, lane = threadIdx.x & 31, P = c.page_size, Hkv = c.num_kv_heads;
    const int seq = row / (c.num_layers * Hkv), G = a.num_q_heads / Hkv;
    const int n = c.row_len[row];
    if (n < 0 || n > c.max_slots) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, KVC_DEV_BAD_LENGTH, row);
        return;
    }
    const int nb = (n + P - 1) / P;
    if ((int)(blockIdx.x * kWarps * BATCH) >= nb) return;
    const int64_t base = (int64_t)row * c.max_pages_per_row;
    const int sub = lane % LANES, side = lane / LANES;
    const T *bounds = static_cast<const T *>(a.bounds) + base * 2 * D + sub * N;
    const int stride = gridDim.x * kWarps * BATCH;
    int b0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * BATCH;
    uint4 u[DEEP][LOADS];
    auto load = [&](int first) {  // lanes past the row's end repeat its last page
#pragma unroll
        for (int i = 0; i < DEEP; ++i)
#pragma unroll
            for (int k = 0; k < LOADS; ++k)
                u[i][k] = *reinterpret_cast<const uint4 *>(bounds + (int64_t)min(first + i * SIDE + side, nb - 1) * 2 * D + k * LANES * N);
    };
    if (b0 < nb) load(b0);
    const T *q = static_cast<const T *>(a.q) + ((int64_t)(row / Hkv) * a.num_q_heads + (row % Hkv) * G) * D;
    for (int d = threadIdx.x; d < D; d += kThreads) {
        double up = 0, down = 0;
        for (int g = 0; g < G; ++g) {
            const double x = (double)static_cast<float>(q[g * D + d]) * 0x1p800;
            up += x > 0 ? x : (x <= 0 ? 0 : x);  // a NaN stays
            down += x < 0 ? x : (x >= 0 ? 0 : x);
        }
        w[d] = down;
        w[D + d] = up;
    }
    __syncthreads();
    double wr[LOADS][N];
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) wr[k][i] = w[(k * LANES + sub) * N + i];
    const int qpos = a.q_pos[seq];
    for (; b0 < nb; b0 += stride) {
        double s[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
            uint32_t z = 0;
#pragma unroll
            for (int k = 0; k < LOADS; ++k) {
                const uint32_t x[4] = {u[i][k].x, u[i][k].y, u[i][k].z, u[i][k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) Element<T>::add(x[j], &wr[k][j * Element<T>::N], s[i], z);
            }
            if (z & 0x7fff7fffu) s[i] = __longlong_as_double(0x7ff8000000000000ll);  // 0 * finite is +-0
        }
        if (b0 + stride < nb) load(b0 + stride);
        // after step 1 (of LANES / 2) a lane holds DEEP / 2 pages, after step 2 one: page `mine` of its DEEP
        int mine = 0, o = LANES / 2;
#pragma unroll
        for (int have = DEEP; have > 1; have /= 2, o /= 2) {
            const bool high = (sub & o) != 0;
#pragma unroll
            for (int i = 0; i < have / 2; ++i) {
                const double keep = high ? s[i + have / 2] : s[i], send = high ? s[i] : s[i + have / 2];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
            mine += high ? have / 2 : 0;
        }
        const int writers = 2 * o;  // lanes that hold the same page
#pragma unroll
        for (; o > 0; o /= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
        const int b = b0 + mine * SIDE + side;
        if (sub % writers == 0 && b < nb) {
            unsigned long long key = 0;
            if (a.block_pos[base + b] <= qpos) key = b < a.sink || b >= nb - a.recent ? kAlways : score_key(s[0]);
            a.keys[base + b] = key;
        }
    }
}

__global__ void __launch_bounds__(kPickThreads, 2) block_pick_kernel(SelectArgs a) {
    __shared__ unsigned hist[kBins];
    __shared__ int red[32];
    __shared__ int counts_s[kPickThreads / 32][2];
    __shared__ unsigned long long range_s[kPickThreads / 32][2];
    __shared__ unsigned long long few_key[kFew];
    __shared__ int few_at[kFew], few_n, digit_s, above_s, cut_at;
    __shared__ unsigned long long cut_key;
    extern __shared__ unsigned long long cache[];
    const CacheView &c = a.c;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = c.page_size;
    begin_dependent();
    int n = c.row_len[row];
    if (n < 0 || n > c.max_slots) n = 0;
    const int nb = (n + P - 1) / P;
    const unsigned long long *keys = a.keys + (int64_t)row * c.max_pages_per_row;
    int32_t *list = a.block_list + (int64_t)row * a.top_k;
    // what there is: pages that can be taken, that always are, and the range of the others' keys
    int visible = 0, always = 0;
    unsigned long long lo = kAlways, hi = 0;
    for (int b = tid; b < nb; b += kPickThreads) {
        const unsigned long long key = keys[b];
        if (nb <= kCached) cache[b] = key;
        visible += key != 0;
        if (key == kAlways) {
            ++always;
        } else if (key != 0) {
            lo = min(lo, key);
            hi = max(hi, key);
        }
    }
    if (nb <= kCached) keys = cache;
    visible = __reduce_add_sync(0xffffffffu, visible);
    always = __reduce_add_sync(0xffffffffu, always);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    if (lane == 0) {
        counts_s[warp][0] = visible;
        counts_s[warp][1] = always;
        range_s[warp][0] = lo;
        range_s[warp][1] = hi;
    }
    for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
    __syncthreads();
    visible = always = 0;
    for (int i = 0; i < kPickThreads / 32; ++i) {
        visible += counts_s[i][0];
        always += counts_s[i][1];
        lo = min(lo, range_s[i][0]);
        hi = max(hi, range_s[i][1]);
    }
    const int k = min(a.top_k, visible);
    if (tid == 0) a.block_count[row] = k;
    for (int i = k + tid; i < a.top_k; i += kPickThreads) list[i] = -1;
    if (k == 0) return;
    // the last page taken: key cut, at index last (or the first `equal` of the pages at key cut, when last is -1)
    int want = k - always, equal = 0, last = INT32_MAX;
    unsigned long long cut = 1;  // all that are visible
    if (want == 0) {
        cut = kAlways;
    } else if (want < visible - always) {
        // keys from lo to hi: they agree above bit `top`
        int top = 63 - __clzll((long long)(lo ^ hi));  // -1: all the same
        unsigned long long prefix = top < 0 ? lo : (top == 63 ? 0 : lo >> (top + 1) << (top + 1)), fixed = top == 63 ? 0 : ~0ull << (top + 1);
        for (;;) {
            if (top < 0) {
                cut = prefix;
                equal = want;
                last = -1;
                break;
            }
            const int shift = max(0, top - kBits + 1);
            for (int b = tid; b < nb; b += kPickThreads) {
                const unsigned long long key = keys[b];
                if (key != 0 && key != kAlways && (key & fixed) == prefix) atomicAdd(&hist[(key >> shift) & (kBins - 1)], 1u);
            }
            __syncthreads();
            // the digit at which the keys from the top down reach `want`: four bins a thread, from the top
            constexpr int PER = kBins / kPickThreads;
            int mine = 0;
            for (int i = 0; i < PER; ++i) mine += hist[kBins - 1 - tid * PER - i];
            int all;
            const int before = block_exclusive_scan(mine, red, &all);
            if (before < want && before + mine >= want) {
                int run = before;
                for (int i = 0;; ++i) {
                    const int d = kBins - 1 - tid * PER - i;
                    if (run + (int)hist[d] >= want) {
                        digit_s = d;
                        above_s = run;
                        few_n = 0;
                        break;
                    }
                    run += hist[d];
                }
            }
            __syncthreads();
            const int digit = digit_s, here = hist[digit];
            want -= above_s;
            prefix |= (unsigned long long)digit << shift;
            fixed |= (unsigned long long)(kBins - 1) << shift;
            top = shift - 1;
            if (want == here) {  // all of the digit's keys
                cut = prefix;
                break;
            }
            if (here <= kFew) {
                for (int b = tid; b < nb; b += kPickThreads) {
                    const unsigned long long key = keys[b];
                    if (key != kAlways && (key & fixed) == prefix && key != 0) {
                        const int i = atomicAdd(&few_n, 1);
                        few_key[i] = key;
                        few_at[i] = b;
                    }
                }
                __syncthreads();
                if (warp == 0 && lane < here) {
                    const unsigned long long key = few_key[lane];
                    const int at = few_at[lane];
                    int rank = 0;
                    for (int i = 0; i < here; ++i) rank += few_key[i] > key || (few_key[i] == key && few_at[i] < at);
                    if (rank == want - 1) cut_key = key, cut_at = at;
                }
                __syncthreads();
                cut = cut_key;
                last = cut_at;
                break;
            }
            __syncthreads();  // the histogram is read
            for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
            __syncthreads();
        }
    }
    // in index order, a run of pages a thread
    const int each = (nb + kPickThreads - 1) / kPickThreads, b1 = min(nb, (tid + 1) * each);
    int ties = 0, all;
    if (last < 0) {
        for (int b = tid * each; b < b1; ++b) ties += keys[b] == cut;
        ties = block_exclusive_scan(ties, red, &all);
    }
    auto taken = [&](int b, unsigned long long key, int &tie) {
        return key > cut || (key == cut && (last < 0 ? tie++ < equal : b <= last));
    };
    int tie = ties, found = 0;
    for (int b = tid * each; b < b1; ++b) found += taken(b, keys[b], tie);
    int at = block_exclusive_scan(found, red, &all);
    tie = ties;
    for (int b = tid * each; b < b1; ++b)
        if (taken(b, keys[b], tie)) list[at++] = b;
}

template <typename T>
cudaError_t score(const SelectArgs &a, dim3 grid, cudaStream_t stream) {
    return launch_dependent(a.c.head_dim == 128 ? block_score_kernel<T, 128> : block_score_kernel<T, 64>, grid, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t launch_select_blocks(const CacheView &c, const void *bounds, const int32_t *block_pos, const void *q,
                                 const int32_t *q_pos, int32_t num_q_heads, int32_t top_k, int32_t sink, int32_t recent,
                                 int32_t *block_list, int32_t *block_count, void *ws, int32_t *status,
                                 cudaStream_t stream) {
    SelectArgs a{c, bounds, block_pos, q, q_pos, num_q_heads, top_k, sink, recent, block_list, block_count,
                 static_cast<unsigned long long *>(ws), status};
    // CTAs a row: the GPU's worth for all rows together, as long as each of their warps has a batch of pages; and so many
    // that none has more than 16 batches, whose CTAs then even out rows of unlike lengths (16 sequences of 8K to 33K tokens,
    // 4 layers: 107 us with the first rule alone, 102 / 92 / 91 us with at most 4 / 8 / 16 batches)
    const int wide = (c.max_pages_per_row + kWarps * kPages - 1) / (kWarps * kPages);
    const dim3 grid(std::max(std::min(device_sms() * kCtas / c.rows, wide), (wide + 15) / 16), c.rows);
    cudaError_t e = c.dtype == KVC_BF16 ? score<__nv_bfloat16>(a, grid, stream) : score<float>(a, grid, stream);
    if (e != cudaSuccess) return e;
    const size_t bytes = (size_t)std::min(c.max_pages_per_row, kCached) * sizeof(unsigned long long);
    static int done[kMaxDevices];
    e = dyn_smem_at_least(reinterpret_cast<const void *>(block_pick_kernel), bytes, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(block_pick_kernel, dim3(c.rows), kPickThreads, bytes, stream, a);
}

}  // namespace kvc
