// A compaction's freed pages pushed onto the free-page stack (kvc_push_pages).
//
// A compaction begins its freed list anew, so a stack that outlives it has to take the list over before the next one:
// free_pages[depth + i] = freed[i], depth += num_freed, num_freed = 0.  Launch A copies, launch B (one thread) moves the counts
// once every CTA of A has read them.  4 bytes read and written a page; the two launches bound it.
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;

struct PushArgs {
    int32_t *free_pages;
    int64_t free_capacity;
    int64_t *free_count;
    const int32_t *freed;
    int64_t freed_capacity;
    int64_t *num_freed;
    int32_t *status;
};

// pages to push: all of the list, or none when a count is out of range or the stack too small
__device__ __forceinline__ int64_t pages_to_push(const PushArgs &a, int64_t depth, int64_t n) {
    return depth < 0 || depth > a.free_capacity || n < 0 || n > a.freed_capacity || n > a.free_capacity - depth ? -1 : n;
}

__global__ void __launch_bounds__(kThreads) push_copy_kernel(PushArgs a) {
    const int64_t depth = *a.free_count, n = pages_to_push(a, depth, *a.num_freed);
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreads)
        a.free_pages[depth + i] = a.freed[i];
}

__global__ void push_count_kernel(PushArgs a) {
    const int64_t depth = *a.free_count, n = pages_to_push(a, depth, *a.num_freed);
    if (n < 0) {
        report(a.status, KVC_DEV_FREED_OVERFLOW, -1);
        return;
    }
    *a.free_count = depth + n;
    *a.num_freed = 0;
}

}  // namespace

cudaError_t launch_push(int32_t *free_pages, int64_t free_capacity, int64_t *free_count, const int32_t *freed,
                        int64_t freed_capacity, int64_t *num_freed, int32_t *status, cudaStream_t stream) {
    const PushArgs a{free_pages, free_capacity, free_count, freed, freed_capacity, num_freed, status};
    const int64_t most = std::min(free_capacity, freed_capacity);
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>((most + kThreads - 1) / kThreads, device_sms()));
    push_copy_kernel<<<grid, kThreads, 0, stream>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    push_count_kernel<<<1, 1, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvc
