// Norms of queries and keys for each head, the position rotation, and the write into the cache, in one pass
// (kvc_norm_rope_write).
//
// For every head vector x of a query or key (head_dim elements):
//     y = x * rsqrt(mean(x^2) + eps) * w          (skipped without a weight)
// and over the first rope_dim elements, with f_j = position * inv_freq[j],
//     (y_a, y_b) <- (y_a cos f_j - y_b sin f_j, y_a sin f_j + y_b cos f_j)
// where (a, b) = (j, j + rope_dim / 2), or (2j, 2j + 1) when interleaved.  Everything between the load and the store is
// fp32 with one rounding at the end; the angle alone is taken in 64 bits, because position * inv_freq of a far
// position has no fraction bits left in 32: it is reduced to turns in [-1/2, 1/2] before it becomes fp32.
//
// Queries go to q_out, keys and values to the cache slots of the slot map.  A token's angles serve all its layers and
// heads, so a CTA takes a token, puts the rope_dim / 2 (cos, sin) pairs into shared memory once, and then groups of
// D * sizeof(T) / 16 lanes (16 bytes a lane) take a head vector each.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxD = 128;

struct NormRopeArgs {
    CacheView c;
    const void *qkv;
    int64_t token_stride;       // elements between tokens of qkv
    int32_t num_tokens;
    const int32_t *token_count; // tokens present, or null for num_tokens
    int32_t num_q_heads;
    const void *q_weight, *k_weight;
    float eps;
    const float *inv_freq;
    int32_t rope_dim, interleaved;
    const int32_t *token_pos;
    const int64_t *slot_map;
    void *q_out;
    int32_t *status;
};

// 16 bytes of T as fp32 and back (round to nearest even)
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 store(const float (&x)[8]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 store(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
};

// cos and sin of position * inv_freq
__device__ __forceinline__ float2 turn(int pos, float inv_freq) {
    constexpr double kInvTwoPi = 0.15915494309189533577;
    const double turns = (double)pos * (double)inv_freq * kInvTwoPi;
    float s, c;
    sincospif(2.f * (float)(turns - rint(turns)), &s, &c);
    return make_float2(c, s);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(NormRopeArgs a) {
    constexpr int N = Vec<T>::N, LK = D / N, GROUPS = kThreads / LK;
    __shared__ float2 cs[kMaxD / 2];
    const CacheView &c = a.c;
    const int sub = threadIdx.x % LK, grp = threadIdx.x / LK, e0 = sub * N;
    const unsigned mask = LK == 32 ? 0xffffffffu : ((1u << LK) - 1) << ((threadIdx.x & 31) / LK * LK);
    const int L = c.num_layers, Hq = a.num_q_heads, Hkv = c.num_kv_heads, H = Hq + 2 * Hkv, R = a.rope_dim, half = R / 2;
    const int tokens = a.token_count ? min(max(*a.token_count, 0), a.num_tokens) : a.num_tokens;
    const int64_t slots = c.num_pages * c.page_size;
    for (int t = blockIdx.x; t < tokens; t += gridDim.x) {
        const int pos = a.token_pos[t];
        __syncthreads();  // the previous token's angles are read
        if ((int)threadIdx.x < half) cs[threadIdx.x] = turn(pos, a.inv_freq[threadIdx.x]);
        __syncthreads();
        const T *src = static_cast<const T *>(a.qkv) + (int64_t)t * a.token_stride;
        for (int v = grp; v < L * H; v += GROUPS) {
            const int l = v / H, h = v % H;
            uint4 u = *reinterpret_cast<const uint4 *>(src + (int64_t)v * D + e0);
            T *dst;
            if (h < Hq) {
                dst = static_cast<T *>(a.q_out) + (((int64_t)t * L + l) * Hq + h) * D;
            } else {
                const int kvh = (h - Hq) % Hkv;
                const int64_t slot = a.slot_map[((int64_t)t * L + l) * Hkv + kvh];
                if (slot < 0 || slot >= slots) {
                    if (slot != -1 && sub == 0) report(a.status, KVC_DEV_BAD_PAGE, -1);
                    continue;
                }
                dst = static_cast<T *>(const_cast<void *>(h < Hq + Hkv ? c.k_pool : c.v_pool)) + slot * D;
            }
            if (h < Hq + Hkv) {
                float x[N];
                Vec<T>::load(u, x);
                const T *w = static_cast<const T *>(h < Hq ? a.q_weight : a.k_weight);
                if (w) {
                    float ss = 0.f;
#pragma unroll
                    for (int i = 0; i < N; ++i) ss += x[i] * x[i];
#pragma unroll
                    for (int o = 1; o < LK; o <<= 1) ss += __shfl_xor_sync(mask, ss, o);
                    const float r = rsqrtf(ss / D + a.eps);
                    float wv[N];
                    Vec<T>::load(*reinterpret_cast<const uint4 *>(w + l * D + e0), wv);
#pragma unroll
                    for (int i = 0; i < N; ++i) x[i] = x[i] * r * wv[i];
                }
                if (a.interleaved) {
                    if (e0 < R)
#pragma unroll
                        for (int i = 0; i < N; i += 2) {
                            const float2 f = cs[(e0 + i) / 2];
                            const float p = x[i] * f.x - x[i + 1] * f.y;
                            x[i + 1] = x[i] * f.y + x[i + 1] * f.x;
                            x[i] = p;
                        }
                } else if (R) {
                    // the partner of element e is e + half or e - half, `half / N` lanes away (half is a multiple of 8)
                    const bool low = e0 < half, in = e0 < R;
                    const int other = in ? (low ? sub + half / N : sub - half / N) : sub;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const float y = __shfl_sync(mask, x[i], other, LK);
                        if (in) {
                            const float2 f = cs[low ? e0 + i : e0 + i - half];
                            x[i] = low ? x[i] * f.x - y * f.y : y * f.y + x[i] * f.x;
                        }
                    }
                }
                u = Vec<T>::store(x);
            }
            *reinterpret_cast<uint4 *>(dst + e0) = u;
        }
    }
}

template <typename T>
cudaError_t launch(const NormRopeArgs &a, cudaStream_t stream) {
    const int grid = std::min(a.num_tokens, device_sms() * 8);
    if (a.c.head_dim == 128) norm_rope_kernel<T, 128><<<grid, kThreads, 0, stream>>>(a);
    else norm_rope_kernel<T, 64><<<grid, kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const CacheView &c, const void *qkv, int64_t token_stride, int32_t num_tokens,
                             const int32_t *token_count, int32_t num_q_heads, const void *q_weight, const void *k_weight,
                             float eps, const float *inv_freq, int32_t rope_dim, bool interleaved, const int32_t *token_pos,
                             const int64_t *slot_map, void *q_out, int32_t *status, cudaStream_t stream) {
    NormRopeArgs a{c, qkv, token_stride, num_tokens, token_count, num_q_heads, q_weight, k_weight, eps, inv_freq,
                   rope_dim, interleaved ? 1 : 0, token_pos, slot_map, q_out, status};
    return c.dtype == KVC_BF16 ? launch<__nv_bfloat16>(a, stream) : launch<float>(a, stream);
}

}  // namespace kvc
