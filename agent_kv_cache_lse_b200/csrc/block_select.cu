// The choice of pages a decode query attends to (kvc_select_blocks).
//
// For a page whose keys lie between lo and hi elementwise, max(q_d lo_d, q_d hi_d) summed over d bounds q . k from
// above for every key of the page.  Summed over the query heads g of the row's group that is
//     score_b = sum_d (sum_g max(q_gd, 0)) hi_bd + (sum_g min(q_gd, 0)) lo_bd = sum_d up_d hi_bd + down_d lo_bd,
// one dot product of 2 D terms a page whatever the group's size.  Which pages are chosen is a whole number, and with 32
// bits two orders of summation would choose differently at the border, so the choice is that of the scores in 64 bits.
// A page with a bound that is not finite ranks as +inf, like one whose score is NaN, whatever the factors' signs make of it.
//
// 64-bit arithmetic for every page took 80 instructions a page and warp and 1.4 times the time of the bytes.  But only pages
// at the border need it.  With x in 32 bits, of 8 multiply-adds a lane and 5 sums across lanes on factors rounded once (14
// roundings of at most 2^-24 each, of sums of magnitudes), |x - score| <= e = 2^-20 M U, where M bounds |lo| and |hi| over the row and
// U = sum_d up_d - down_d, as long as no sum can leave fp32's range (M U < 2^126; past it every page is ranked in 64 bits).
// If c is the k-th largest x, a page above c + 2 e has a score above those of all but fewer than k pages and is taken, one
// below c - 2 e is not, and the pages between are ranked by their scores in 64 bits: mostly there is one page between, and
// nothing to rank.
//
// Launch A: a warp takes kPages loads' pages at a time, 16 bytes a lane of [lo | hi], the matching up or down in registers.
//   The pages' sums are joined together, halving the pages a lane holds with each of the first two shuffles.  x becomes an
//   order-preserving 32-bit key in the workspace: 0 for a page that is hidden or past the row's length, all ones for the
//   pages that are always taken, else the key of x (never 0 or all ones), of +inf for a page with a bound that is not
//   finite (times 0 in its own type it is NaN, which marks it).  Each CTA leaves its largest finite |bound|, the first U.
// Launch B: a CTA a row.  The keys of a row share their leading bits; below those, a histogram of the next 11 bits finds the
//   digit in which the k-th key lies, usually with a handful of keys, which are ranked directly; while there are more than
//   kFew, the next 11 bits follow.  The 64-bit scores between c - 2 e and c + 2 e, if they have to be ranked, go the same
//   way.  One pass in index order then lists the pages.
// Measured a call: 77 us for 677,000 pages of 512 rows (16 sequences of 8K to 33K tokens, 4 layers; 62 us launch A, 5.6 TB/s), 89 us with
// 64-bit scores throughout; 11 to 12 us for 8 rows of 2,048 pages, of which the bytes are 1.3 (a dozen barriers of launch B the rest).
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
constexpr int kAhead = 4;          // keys a picking thread has in flight beside the row's length
constexpr int kFew = 32;           // keys that one warp ranks
constexpr int kCached = 16384;     // keys of a row that stay in shared memory

struct SelectArgs {
    CacheView c;
    const void *bounds;
    const int32_t *block_pos;
    const void *q;
    const int32_t *q_pos;
    int32_t num_q_heads, top_k, sink, recent;
    int32_t *block_list, *block_count;
    unsigned long long *exact;  // [rows][max_pages_per_row]: keys of the 64-bit scores, where they were needed
    uint32_t *keys;             // [rows][max_pages_per_row]: keys of the 32-bit scores
    float *stats;               // [rows][1 + spread]: U, then the CTAs' largest finite |bound|
    int32_t spread;             // entries of stats for a row's CTAs
    int32_t ctas, pages_a_cta;  // CTAs a row has, and pages each takes in a round
    int32_t *status;
};

constexpr uint32_t kAlways = ~0u;
constexpr uint32_t kInfinite = 0xff800000u;  // float_key(+inf)

// larger score -> larger key; NaN ranks as +inf, -0 as 0
__device__ __forceinline__ unsigned long long score_key(double s) {
    if (isnan(s)) s = __longlong_as_double(0x7ff0000000000000ll);
    const unsigned long long b = (unsigned long long)__double_as_longlong(s + 0.0);
    return (b >> 63) ? ~b : (b | 0x8000000000000000ull);
}

// s += w * x over the elements x of a 32-bit word, m their largest |x| (in their own type; the sign is not kept), and z NaN
// where one is not finite
template <typename T>
struct Element;
template <>
struct Element<__nv_bfloat16> {
    static constexpr int N = 2;
    static __device__ __forceinline__ void add(uint32_t u, const float2 &w, float2 &s, uint32_t &m, uint32_t &z) {
        s = __ffma2_rn(w, make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)), s);
        asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(u));
        asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(z) : "r"(u), "r"(0u));
    }
    static __device__ __forceinline__ float largest(uint32_t m) {
        return fmaxf(fabsf(__uint_as_float(m << 16)), fabsf(__uint_as_float(m & 0xffff0000u)));
    }
};
template <>
struct Element<float> {
    static constexpr int N = 1;
    static __device__ __forceinline__ void add(uint32_t u, const float2 &w, float2 &s, uint32_t &m, uint32_t &z) {
        s.x = fmaf(w.x, __uint_as_float(u), s.x);
        m = __float_as_uint(fmaxf(__uint_as_float(m), fabsf(__uint_as_float(u))));
        asm("fma.rn.f32 %0, %1, %2, %0;" : "+r"(z) : "r"(u), "r"(0u));
    }
    static __device__ __forceinline__ float largest(uint32_t m) { return __uint_as_float(m); }
};

// up and down of the row's group, as doubles: w[d] = down, w[D + d] = up (kThreads threads; not synchronised)
template <typename T, int D>
__device__ __forceinline__ void factors(const SelectArgs &a, int row, double *w) {
    const int Hkv = a.c.num_kv_heads, G = a.num_q_heads / Hkv;
    const T *q = static_cast<const T *>(a.q) + ((int64_t)(row / Hkv) * a.num_q_heads + (row % Hkv) * G) * D;
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        double up = 0, down = 0;
        for (int g = 0; g < G; ++g) {
            const double x = (double)static_cast<float>(q[g * D + d]);
            up += x > 0 ? x : (x <= 0 ? 0 : x);  // a NaN stays
            down += x < 0 ? x : (x >= 0 ? 0 : x);
        }
        w[d] = down;
        w[D + d] = up;
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtas) block_score_kernel(SelectArgs a) {
    constexpr int N = 16 / sizeof(T);          // elements of a lane's load
    constexpr int LOADS = 2 * D / (32 * N) > 0 ? 2 * D / (32 * N) : 1;  // a page
    constexpr int LANES = 2 * D / (N * LOADS); // lanes that hold a page's elements (16 at bf16, D 64; else 32)
    constexpr int SIDE = 32 / LANES;           // pages side by side
    constexpr int BATCH = kPages / LOADS * SIDE;  // pages a warp takes at a time: 4, 8 or (fp32, D 128) 2
    constexpr int DEEP = BATCH / SIDE;         // of them in the same lanes
    __shared__ double w[2 * D];                // [down | up]
    __shared__ float red[kWarps];
    begin_dependent();
    const CacheView &c = a.c;
    const int row = blockIdx.y, lane = threadIdx.x & 31, P = c.page_size, Hkv = c.num_kv_heads;
    const int seq = row / (c.num_layers * Hkv);
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
    factors<T, D>(a, row, w);
    __syncthreads();
    constexpr int E = Element<T>::N;
    float2 wr[LOADS][N / E];  // the factors of a word's elements
#pragma unroll
    for (int k = 0; k < LOADS; ++k)
#pragma unroll
        for (int i = 0; i < N / E; ++i) {
            const double *f = w + (k * LANES + sub) * N + i * E;
            wr[k][i] = make_float2((float)f[0], (float)f[E - 1]);
        }
    const int qpos = a.q_pos[seq];
    float top = 0.f;  // largest finite |bound| this lane has seen
    for (; b0 < nb; b0 += stride) {
        float s[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < DEEP; ++i) {
            uint32_t z = 0, m = 0;
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < LOADS; ++k) {
                const uint32_t x[4] = {u[i][k].x, u[i][k].y, u[i][k].z, u[i][k].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) Element<T>::add(x[j], wr[k][j], sum, m, z);
            }
            s[i] = sum.x + sum.y;
            if (z & 0x7fff7fffu) s[i] = __uint_as_float(0x7fc00000u);  // 0 * finite is +-0
            else top = fmaxf(top, Element<T>::largest(m));
        }
        if (b0 + stride < nb) load(b0 + stride);
        // after step 1 (of LANES / 2) a lane holds DEEP / 2 pages, after step 2 one: page `mine` of its DEEP
        int mine = 0, o = LANES / 2;
#pragma unroll
        for (int have = DEEP; have > 1; have /= 2, o /= 2) {
            const bool high = (sub & o) != 0;
#pragma unroll
            for (int i = 0; i < have / 2; ++i) {
                const float keep = high ? s[i + have / 2] : s[i], send = high ? s[i] : s[i + have / 2];
                s[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
            mine += high ? have / 2 : 0;
        }
        const int writers = 2 * o;  // lanes that hold the same page
#pragma unroll
        for (; o > 0; o /= 2) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
        const int b = b0 + mine * SIDE + side;
        if (sub % writers == 0 && b < nb) {
            uint32_t key = 0;
            if (a.block_pos[base + b] <= qpos)
                key = b < a.sink || b >= nb - a.recent ? kAlways : isnan(s[0]) ? kInfinite : float_key(s[0] + 0.f);
            a.keys[base + b] = key;
        }
    }
    top = warp_max(top);
    __syncthreads();
    if (lane == 0) red[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int i = 1; i < kWarps; ++i) top = fmaxf(top, red[i]);
        a.stats[(int64_t)row * (1 + a.spread) + 1 + blockIdx.x] = top;
    }
    if (blockIdx.x == 0) {  // U, summed in 64 bits and rounded up
        double x = 0;
        for (int d = threadIdx.x; d < D; d += kThreads) x += w[D + d] - w[d];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        __syncthreads();  // red is read
        if (lane == 0) red[threadIdx.x >> 5] = __double2float_ru(x);
        __syncthreads();
        if (threadIdx.x == 0) {
            float all = 0.f;
            for (int i = 0; i < kWarps; ++i) all = __fadd_ru(all, red[i]);
            a.stats[(int64_t)row * (1 + a.spread)] = all;
        }
    }
}

// The last of the `want` largest keys of a row, ties to the lower index: key `cut` at index `last`, or, with last -1, the first
// `equal` pages with key cut.
template <typename K>
struct Cut {
    K cut;
    int equal, last;
};
struct SearchShared {
    unsigned hist[kBins];
    unsigned long long few_key[kFew], cut_key;
    int few_at[kFew], few_n, digit, above, cut_at;
    int red[3][32];  // of the scans: one barrier each, so each place has its own
};

// exclusive scan over the CTA, with one barrier; `red` may be used again after the next one
__device__ __forceinline__ int scan_once(int v, int (&red)[32]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) red[w] = x;
    __syncthreads();
    const int before = __reduce_add_sync(0xffffffffu, lane < w ? red[lane] : 0);
    return before + x - v;
}

// key(b, k): whether page b takes part, and its key.  Keys lie between lo and hi, and there are more than want of them.
// All threads of the CTA call it, with the histogram cleared, and get the result.
template <typename K, typename Key>
__device__ __forceinline__ Cut<K> search(int nb, int want, K lo, K hi, SearchShared &sh, Key key) {
    constexpr int W = sizeof(K) * 8;
    const int tid = threadIdx.x, lane = tid & 31;
    // the keys agree above bit `top`
    int top = W - 1 - (W == 32 ? __clz((int)(lo ^ hi)) : __clzll((long long)(lo ^ hi)));
    K fixed = top == W - 1 ? (K)0 : (K)(~(K)0 << (top + 1)), prefix = lo & fixed;
    for (;;) {
        if (top < 0) return Cut<K>{prefix, want, -1};  // all the same
        const int shift = max(0, top - kBits + 1);
        for (int b = tid; b < nb; b += kPickThreads) {
            K k;
            if (key(b, k) && (k & fixed) == prefix) atomicAdd(&sh.hist[(unsigned)(k >> shift) & (kBins - 1)], 1u);
        }
        __syncthreads();
        // the digit at which the keys from the top down reach `want`: four bins a thread, from the top
        constexpr int PER = kBins / kPickThreads;
        int mine = 0;
        for (int i = 0; i < PER; ++i) mine += sh.hist[kBins - 1 - tid * PER - i];
        const int before = scan_once(mine, sh.red[0]);
        if (before < want && before + mine >= want) {
            int run = before;
            for (int i = 0;; ++i) {
                const int d = kBins - 1 - tid * PER - i;
                if (run + (int)sh.hist[d] >= want) {
                    sh.digit = d;
                    sh.above = run;
                    sh.few_n = 0;
                    break;
                }
                run += sh.hist[d];
            }
        }
        __syncthreads();
        const int digit = sh.digit, here = sh.hist[digit];
        want -= sh.above;
        prefix |= (K)digit << shift;
        fixed |= (K)(kBins - 1) << shift;
        top = shift - 1;
        if (here <= kFew) {
            for (int b = tid; b < nb; b += kPickThreads) {
                K k;
                if (key(b, k) && (k & fixed) == prefix) {
                    const int i = atomicAdd(&sh.few_n, 1);
                    sh.few_key[i] = k;
                    sh.few_at[i] = b;
                }
            }
            __syncthreads();
            if (tid < 32 && lane < here) {
                const unsigned long long k = sh.few_key[lane];
                const int at = sh.few_at[lane];
                int rank = 0;
                for (int i = 0; i < here; ++i) rank += sh.few_key[i] > k || (sh.few_key[i] == k && sh.few_at[i] < at);
                if (rank == want - 1) sh.cut_key = k, sh.cut_at = at;
            }
            __syncthreads();
            return Cut<K>{(K)sh.cut_key, 0, sh.cut_at};
        }
        __syncthreads();  // the histogram is read
        for (int i = tid; i < kBins; i += kPickThreads) sh.hist[i] = 0;
        __syncthreads();
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kPickThreads, 2) block_pick_kernel(SelectArgs a) {
    constexpr int kPickWarps = kPickThreads / 32;
    __shared__ SearchShared sh;
    __shared__ int counts_s[kPickWarps][2];
    __shared__ uint32_t range_s[kPickWarps][2];
    __shared__ float top_s[kPickWarps];
    __shared__ int over_s, between_s;
    extern __shared__ uint32_t cache[];
    begin_dependent();
    const CacheView &c = a.c;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, P = c.page_size;
    const int64_t base = (int64_t)row * c.max_pages_per_row;
    const uint32_t *keys = a.keys + base;
    // the first keys of a thread come with the row's length (past it they are whatever the workspace held, and not used)
    uint32_t ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        const int b = tid + i * kPickThreads;
        ahead[i] = b < c.max_pages_per_row ? keys[b] : 0;
    }
    int n = c.row_len[row];
    if (n < 0 || n > c.max_slots) n = 0;
    const int nb = (n + P - 1) / P;
    const float *stats = a.stats + (int64_t)row * (1 + a.spread);
    int32_t *list = a.block_list + (int64_t)row * a.top_k;
    // what there is: pages that can be taken, that always are, the range of the others' keys, the largest bound
    int visible = 0, always = 0;
    uint32_t lo = kAlways, hi = 0;
    float top = 0.f;
    for (int i = tid; i < min(a.ctas, (nb + a.pages_a_cta - 1) / a.pages_a_cta); i += kPickThreads) top = fmaxf(top, stats[1 + i]);
    const float U = nb > 0 ? stats[0] : 0.f;
    auto count = [&](int b, uint32_t key) {
        if (nb <= kCached) cache[b] = key;
        visible += key != 0;
        if (key == kAlways) {
            ++always;
        } else if (key != 0) {
            lo = min(lo, key);
            hi = max(hi, key);
        }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
        if (tid + i * kPickThreads < nb) count(tid + i * kPickThreads, ahead[i]);
    for (int b = tid + kAhead * kPickThreads; b < nb; b += kPickThreads) count(b, keys[b]);
    if (nb <= kCached) keys = cache;
    visible = __reduce_add_sync(0xffffffffu, visible);
    always = __reduce_add_sync(0xffffffffu, always);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) {
        counts_s[warp][0] = visible;
        counts_s[warp][1] = always;
        range_s[warp][0] = lo;
        range_s[warp][1] = hi;
        top_s[warp] = top;
    }
    for (int i = tid; i < kBins; i += kPickThreads) sh.hist[i] = 0;
    if (tid == 0) over_s = between_s = 0;
    __syncthreads();
    {  // every warp joins the warps' for itself, a lane a warp
        const int i = lane % kPickWarps;
        visible = __reduce_add_sync(0xffffffffu, lane < kPickWarps ? counts_s[i][0] : 0);
        always = __reduce_add_sync(0xffffffffu, lane < kPickWarps ? counts_s[i][1] : 0);
        lo = __reduce_min_sync(0xffffffffu, range_s[i][0]);
        hi = __reduce_max_sync(0xffffffffu, range_s[i][1]);
        top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_s[i])));  // not negative
    }
    const int k = min(a.top_k, visible);
    if (tid == 0) a.block_count[row] = k;
    for (int i = k + tid; i < a.top_k; i += kPickThreads) list[i] = -1;
    if (k == 0) return;
    const int want = k - always;  // of the pages that are not always taken
    uint32_t from = 1, above = 0;  // taken: pages with a key above `above`; to be ranked: the others from `from` on
    unsigned long long *exact = a.exact + base;
    Cut<unsigned long long> cut{0, 0, INT32_MAX};  // of those, all
    if (want == 0) {
        from = kAlways;
        above = kAlways - 1;
    } else if (want < visible - always) {
        const float x = key_float(search<uint32_t>(nb, want, lo, hi, sh, [&](int b, uint32_t &key) {
            key = keys[b];
            return key != 0 && key != kAlways;
        }).cut);
        const float reach = top * U;  // no partial sum of a finite page is larger
        const float e = 2.1f * (0x1p-20f * reach + 0x1p-130f);  // 2 e, with room for the roundings here
        from = 1;
        above = kAlways - 1;
        if (reach < 0x1p126f) {  // else a sum may have left fp32's range (inf, or NaN from two signs), and nothing is known
            from = float_key(x - e);
            above = float_key(x + e);
        }
        int between = 0, over = 0;
        for (int b = tid; b < nb; b += kPickThreads) {
            const uint32_t key = keys[b];
            over += key > above && key != kAlways;
            between += key >= from && key <= above && key != 0;
        }
        over = __reduce_add_sync(0xffffffffu, over);
        between = __reduce_add_sync(0xffffffffu, between);
        if (lane == 0 && over) atomicAdd(&over_s, over);
        if (lane == 0 && between) atomicAdd(&between_s, between);
        __syncthreads();
        between = between_s;
        const int rest = want - over_s;
        if (rest < between) {  // rank them by their scores in 64 bits
            __shared__ double w[2 * D];
            factors<T, D>(a, row, w);
            for (int i = tid; i < kBins; i += kPickThreads) sh.hist[i] = 0;
            __syncthreads();
            for (int b0 = warp * 32; b0 < nb; b0 += kPickThreads) {
                const uint32_t key = b0 + lane < nb ? keys[b0 + lane] : 0;
                for (unsigned todo = __ballot_sync(0xffffffffu, key != 0 && key >= from && key <= above); todo; todo &= todo - 1) {
                    const int b = b0 + __ffs(todo) - 1;
                    const T *v = static_cast<const T *>(a.bounds) + (base + b) * 2 * D;
                    double s = 0;
                    for (int i = lane; i < 2 * D; i += 32) {
                        const float x = static_cast<float>(v[i]);
                        s = isfinite(x) ? fma(w[i], (double)x, s) : __longlong_as_double(0x7ff8000000000000ll);  // NaN stays
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                    if (lane == 0) exact[b] = score_key(s);
                }
            }
            __syncthreads();
            cut = search<unsigned long long>(nb, rest, 0ull, ~0ull, sh, [&](int b, unsigned long long &key) {
                const uint32_t k32 = keys[b];
                const bool in = k32 != 0 && k32 >= from && k32 <= above;
                if (in) key = exact[b];
                return in;
            });
        }
    }
    // in index order, a run of pages a thread
    const int each = (nb + kPickThreads - 1) / kPickThreads, b1 = min(nb, (tid + 1) * each);
    auto ranked = [&](uint32_t key) { return key != 0 && key >= from && key <= above; };
    int ties = 0;
    if (cut.last < 0) {
        for (int b = tid * each; b < b1; ++b) ties += ranked(keys[b]) && exact[b] == cut.cut;
        ties = scan_once(ties, sh.red[1]);
    }
    auto taken = [&](int b, int &tie) {
        const uint32_t key = keys[b];
        if (key == 0 || key < from) return false;
        if (key > above || cut.last == INT32_MAX) return true;
        const unsigned long long x = exact[b];
        return x > cut.cut || (x == cut.cut && (cut.last < 0 ? tie++ < cut.equal : b <= cut.last));
    };
    int tie = ties, found = 0;
    for (int b = tid * each; b < b1; ++b) found += taken(b, tie);
    int at = scan_once(found, sh.red[2]);
    tie = ties;
    for (int b = tid * each; b < b1; ++b)
        if (taken(b, tie)) list[at++] = b;
}

template <typename T, int D>
cudaError_t launch(SelectArgs a, cudaStream_t stream) {
    // CTAs a row: the GPU's worth for all rows together, as long as each of their warps has a batch of pages; and so many
    // that none has more than 16 batches, whose CTAs then even out rows of unlike lengths (16 sequences of 8K to 33K tokens,
    // 4 layers: 107 us with the first rule alone, 102 / 92 / 91 us with at most 4 / 8 / 16 batches)
    const CacheView &c = a.c;
    constexpr int kBatch = kPages * 512 / (2 * D * (int)sizeof(T));  // pages of a warp's loads
    a.pages_a_cta = kWarps * kBatch;
    const int wide = (c.max_pages_per_row + a.pages_a_cta - 1) / a.pages_a_cta;
    a.ctas = std::max(std::min(device_sms() * kCtas / c.rows, wide), (wide + 15) / 16);
    cudaError_t e = launch_dependent(block_score_kernel<T, D>, dim3(a.ctas, c.rows), kThreads, 0, stream, a);
    if (e != cudaSuccess) return e;
    const size_t bytes = (size_t)std::min(c.max_pages_per_row, kCached) * sizeof(uint32_t);
    static int done[kMaxDevices];
    e = dyn_smem_at_least(reinterpret_cast<const void *>(block_pick_kernel<T, D>), bytes, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(block_pick_kernel<T, D>, dim3(c.rows), kPickThreads, bytes, stream, a);
}

// entries of a row's stats beside U: at least the CTAs of a row, whose warps have at least two pages each
int64_t stats_spread(int64_t max_pages) { return (max_pages + 2 * kWarps - 1) / (2 * kWarps); }

}  // namespace

size_t select_blocks_workspace(int64_t rows, int64_t max_pages) {
    return (size_t)((rows * max_pages * 12 + rows * (1 + stats_spread(max_pages)) * 4 + 7) / 8 * 8);
}

cudaError_t launch_select_blocks(const CacheView &c, const void *bounds, const int32_t *block_pos, const void *q,
                                 const int32_t *q_pos, int32_t num_q_heads, int32_t top_k, int32_t sink, int32_t recent,
                                 int32_t *block_list, int32_t *block_count, void *ws, int32_t *status,
                                 cudaStream_t stream) {
    const int64_t pages = (int64_t)c.rows * c.max_pages_per_row;
    unsigned long long *exact = static_cast<unsigned long long *>(ws);
    uint32_t *keys = reinterpret_cast<uint32_t *>(exact + pages);
    SelectArgs a{c, bounds, block_pos, q, q_pos, num_q_heads, top_k, sink, recent, block_list, block_count,
                 exact, keys, reinterpret_cast<float *>(keys + pages), (int32_t)stats_spread(c.max_pages_per_row), 0, 0, status};
    if (c.dtype == KVC_BF16)
        return c.head_dim == 128 ? launch<__nv_bfloat16, 128>(a, stream) : launch<__nv_bfloat16, 64>(a, stream);
    return c.head_dim == 128 ? launch<float, 128>(a, stream) : launch<float, 64>(a, stream);
}

}  // namespace kvc
