// Elementwise minimum and maximum of every page's keys, and the page's lowest position (kvc_block_bounds).
//
// bounds[row][b][0][d] = min k[d], bounds[row][b][1][d] = max k[d] over the row's slots in page b, exact in the cache's
// type (a minimum rounds nothing); a NaN among the keys of an element gives NaN.  Reading K once is all there is to
// it, so a warp takes a page: D * sizeof(T) / 16 lanes cover a key row with 16 bytes each, and the warp's key groups
// join with shuffles at the end.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

struct BoundsArgs {
    CacheView c;
    const int32_t *from_len;
    void *bounds;
    int32_t *block_pos;
    int32_t *status;
};

// lower (kMax false) or upper of the two words' elements; NaN wins
template <typename T, bool kMax>
__device__ __forceinline__ uint32_t pick(uint32_t x, uint32_t y) {
    uint32_t r;
    if constexpr (sizeof(T) == 2) {
        if constexpr (kMax) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
        else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    } else {
        float f;
        if constexpr (kMax) asm("max.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
        else asm("min.NaN.f32 %0, %1, %2;" : "=f"(f) : "f"(__uint_as_float(x)), "f"(__uint_as_float(y)));
        r = __float_as_uint(f);
    }
    return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) bounds_kernel(BoundsArgs a) {
    constexpr int N = 16 / sizeof(T), LK = D / N, ROWS = 32 / LK;
    const CacheView &c = a.c;
    const int row = blockIdx.y, lane = threadIdx.x & 31, sub = lane % LK, grp = lane / LK, P = c.page_size;
    const int n = c.row_len[row];
    if (n < 0 || n > c.max_slots) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, KVC_DEV_BAD_LENGTH, row);
        return;
    }
    const int nb = (n + P - 1) / P, first = a.from_len ? max(0, a.from_len[row]) / P : 0;
    for (int b = first + blockIdx.x * kWarps + (threadIdx.x >> 5); b < nb; b += gridDim.x * kWarps) {
        const int64_t rb = (int64_t)row * c.max_pages_per_row + b;
        const int32_t pg = c.block_table[rb];
        if (pg < 0 || pg >= c.num_pages) {
            if (lane == 0) {
                report(a.status, KVC_DEV_BAD_PAGE, row);
                a.block_pos[rb] = INT32_MAX;
            }
            continue;
        }
        const int cnt = min(P, n - b * P);  // at least 1
        const T *kp = static_cast<const T *>(c.k_pool) + (int64_t)pg * P * D + sub * N;
        uint4 lo, hi;
        lo = hi = *reinterpret_cast<const uint4 *>(kp + min(grp, cnt - 1) * D);  // groups past the end repeat the last key
#pragma unroll 8
        for (int i = grp + ROWS; i < cnt; i += ROWS) {
            const uint4 u = *reinterpret_cast<const uint4 *>(kp + i * D);
            lo.x = pick<T, false>(lo.x, u.x), hi.x = pick<T, true>(hi.x, u.x);
            lo.y = pick<T, false>(lo.y, u.y), hi.y = pick<T, true>(hi.y, u.y);
            lo.z = pick<T, false>(lo.z, u.z), hi.z = pick<T, true>(hi.z, u.z);
            lo.w = pick<T, false>(lo.w, u.w), hi.w = pick<T, true>(hi.w, u.w);
        }
        int pos = INT32_MAX;
        for (int i = lane; i < cnt; i += 32) pos = min(pos, c.slot_pos[(int64_t)row * c.max_slots + b * P + i]);
        __syncwarp();
#pragma unroll
        for (int o = LK; o < 32; o <<= 1) {
            lo.x = pick<T, false>(lo.x, __shfl_xor_sync(0xffffffffu, lo.x, o));
            lo.y = pick<T, false>(lo.y, __shfl_xor_sync(0xffffffffu, lo.y, o));
            lo.z = pick<T, false>(lo.z, __shfl_xor_sync(0xffffffffu, lo.z, o));
            lo.w = pick<T, false>(lo.w, __shfl_xor_sync(0xffffffffu, lo.w, o));
            hi.x = pick<T, true>(hi.x, __shfl_xor_sync(0xffffffffu, hi.x, o));
            hi.y = pick<T, true>(hi.y, __shfl_xor_sync(0xffffffffu, hi.y, o));
            hi.z = pick<T, true>(hi.z, __shfl_xor_sync(0xffffffffu, hi.z, o));
            hi.w = pick<T, true>(hi.w, __shfl_xor_sync(0xffffffffu, hi.w, o));
        }
        pos = __reduce_min_sync(0xffffffffu, pos);
        T *out = static_cast<T *>(a.bounds) + rb * 2 * D + sub * N;
        if (grp == 0) *reinterpret_cast<uint4 *>(out) = lo;
        if (grp == ROWS - 1) *reinterpret_cast<uint4 *>(out + D) = hi;
        if (lane == 0) a.block_pos[rb] = pos;
    }
}

template <typename T>
cudaError_t launch(const BoundsArgs &a, dim3 grid, cudaStream_t stream) {
    if (a.c.head_dim == 128) bounds_kernel<T, 128><<<grid, kThreads, 0, stream>>>(a);
    else bounds_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_bounds(const CacheView &c, const int32_t *from_len, void *bounds, int32_t *block_pos,
                                int32_t *status, cudaStream_t stream) {
    BoundsArgs a{c, from_len, bounds, block_pos, status};
    // a warp a page while that leaves the GPU's resident warps room, else the rows' CTAs walk their pages
    const int wide = (c.max_pages_per_row + kWarps - 1) / kWarps;
    const int xb = std::max(1, std::min((device_sms() * 8 + c.rows - 1) / c.rows, wide));
    const dim3 grid(xb, c.rows);
    return c.dtype == KVC_BF16 ? launch<__nv_bfloat16>(a, grid, stream) : launch<float>(a, grid, stream);
}

}  // namespace kvc
