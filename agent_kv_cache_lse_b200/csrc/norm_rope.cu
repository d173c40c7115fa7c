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
// Queries go to q_out, keys and values to the cache slots of the slot map.  The bytes bound it (each is read once and
// written once), with the instructions close behind, so both steps are folded into
//     out_e = rsqrt(mean(x^2) + eps) * (C_e x_e + S_e x_p),    C_e = w_e cos f, S_e = -+ w_p sin f,  p the partner of e
// (C = w, S = 0 past rope_dim): two multiply-adds an element and one product, in pairs (f32x2).
// A lane takes two 16-byte pieces of a head vector, an element and its partner both (pieces p and p + rope_dim / 2; past
// rope_dim, and when interleaved, neighbours), so that no lane needs another's elements (one piece a lane, and
// the partner's loaded and converted beside it, took 28 M warp instructions for 8,192 tokens where this takes 21 M).  A warp takes
// 2 to 8 vectors a step, and a lane always has
// the same elements: its C and S are the same for all query heads, or all key heads, of a token and layer.  The steps of
// all tokens (each token's layers, and in them the queries, then the keys and values) form one sequence that is cut into equal runs, one a
// warp.  A warp takes its run in groups of up to kSteps steps of one kind, streamed through a ring of kRing stages of its
// own with cp.async (a lane's registers then hold no loads in flight: with batches of loads in registers the kernel was
// bound by occupancy or by spills).  When it comes to a new token it makes that token's rope_dim / 2 pairs (cos, sin) in
// shared memory, and at a layer's queries and keys its C and S.  Measured a call: 153 us for 32,768 tokens of 32 + 2 x 8 heads of
// 128 (bf16, 5.3 TB/s read and written, 52% of the issue slots), 3.7 us for 16 tokens, 10.2 us for 1,003 fp32 tokens of two
// layers (37 MB).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtas = 3;                                 // a multiprocessor
constexpr int kSteps = 4;                                // steps a group
constexpr int kRing = 2;                                 // groups a warp has in shared memory
constexpr int kMaxD = 128;
constexpr int kVectors = kSteps * 1024;                  // bytes of a group's vectors
constexpr int kStage = kVectors + 32 * 8 + 16;           // and its slots, and its position
constexpr int kWarpBytes = kRing * kStage + kMaxD / 2 * 8;  // and the token's (cos, sin) pairs

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
    int32_t rope_dim;
    const int32_t *token_pos;
    const int64_t *slot_map;
    void *q_out;
    int32_t *status;
};

// 16 bytes of T as pairs of fp32 and back (round to nearest even)
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const uint4 &u, float2 (&x)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    static __device__ __forceinline__ uint4 store(const float2 (&x)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void load(const uint4 &u, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 store(const float2 (&x)[2]) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
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

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
template <int BYTES>
__device__ __forceinline__ void cp(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(BYTES) : "memory");
}

// A place in the sequence of steps: step `s` of the query heads, or of the key and value heads (`kv`), of a token and
// layer; `left` steps to the run's end.
struct Place {
    int token, layer, kv, s, left;
};

template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kCtas) norm_rope_kernel(NormRopeArgs a) {
    begin_dependent();
    constexpr int N = Vec<T>::N, PV = D / N, LK = PV / 2, VW = 32 / LK;  // elements a piece; pieces, lanes a vector; vectors a step
    extern __shared__ __align__(16) unsigned char smem[];
    const CacheView &c = a.c;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LK, grp = lane / LK;
    unsigned char *ring = smem + warp * kWarpBytes;
    float2 *cs = reinterpret_cast<float2 *>(ring + kRing * kStage);
    const int L = c.num_layers, Hq = a.num_q_heads, Hkv = c.num_kv_heads, H = Hq + 2 * Hkv, R = a.rope_dim, half = R / 2;
    const int sq = (Hq + VW - 1) / VW, skv = (2 * Hkv + VW - 1) / VW;  // steps of a layer's queries, and keys and values
    // this lane's pieces; R is a multiple of 16, so both lie in the rotated part (`in`) or neither does
    const bool apart = !kInter && sub * N < half;
    const int p0 = apart ? sub : 2 * sub, p1 = apart ? sub + half / N : 2 * sub + 1;
    const bool in = p0 * N < R;
    const int64_t pool_slots = c.num_pages * c.page_size;

    // this lane's frequencies, for the pairs it makes of each token
    float freq[kMaxD / 64];
#pragma unroll
    for (int i = 0; i < kMaxD / 64; ++i) freq[i] = lane + 32 * i < half ? a.inv_freq[lane + 32 * i] : 0.f;

    // the run
    const int tokens = a.token_count ? min(max(*a.token_count, 0), a.num_tokens) : a.num_tokens;
    const int64_t all = (int64_t)tokens * L * (sq + skv), W = min((int64_t)gridDim.x * kWarps, all);
    const int64_t w = (int64_t)blockIdx.x * kWarps + warp;
    Place next{0, 0, 0, 0, 0};
    if (w < W) {
        const int64_t lo = all * w / W;
        const int per = sq + skv;
        next.token = (int)(lo / ((int64_t)L * per));
        const int y = (int)(lo - (int64_t)next.token * L * per);
        next.layer = y / per;
        next.s = y - next.layer * per;
        if (next.s >= sq) next.s -= sq, next.kv = 1;
        next.left = (int)(all * (w + 1) / W - lo);
    }
    Place here = next;
    // steps of the group at p, and p past it
    auto group = [&](const Place &p) { return min(min(kSteps, (p.kv ? skv : sq) - p.s), p.left); };
    auto advance = [&](Place &p, int n) {
        p.left -= n;
        p.s += n;
        if (p.s == (p.kv ? skv : sq)) {
            p.s = 0;
            p.kv ^= 1;
            if (!p.kv && ++p.layer == L) p.layer = 0, ++p.token;
        }
    };
    int in_stage = 0;  // the stage that takes the next group
    auto issue = [&]() {
        if (next.left > 0) {
            const int n = group(next);
            const uint32_t dst = smem_u32(ring + in_stage * kStage);
            const int h0 = next.s * VW, there = min(n * VW, (next.kv ? 2 * Hkv : Hq) - h0);  // vectors of the group
            const unsigned char *from = reinterpret_cast<const unsigned char *>(
                static_cast<const T *>(a.qkv) + (int64_t)next.token * a.token_stride +
                (next.layer * H + (next.kv ? Hq : 0) + h0) * D) + lane * 16;
#pragma unroll
            for (int k = 0; k < kVectors / 512; ++k)
                if (k * 32 + lane < there * PV) cp<16>(dst + k * 512 + lane * 16, from + k * 512);
            if (next.kv && lane < there) {  // keys, then values: the slot of head h and of head Hkv + h is the same
                const int h = h0 + lane;
                cp<8>(dst + kVectors + lane * 8,
                      a.slot_map + ((int64_t)next.token * L + next.layer) * Hkv + (h < Hkv ? h : h - Hkv));
            }
            if (lane == 0) cp<4>(dst + kVectors + 256, a.token_pos + next.token);
            advance(next, n);
        }
        in_stage = in_stage + 1 == kRing ? 0 : in_stage + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");  // one a call, empty or not
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) issue();

    float2 C[2][N / 2], S[2][N / 2];
    // the vectors' two pieces, normalised (where there is a weight) and rotated
    auto apply = [&](uint4 &u0, uint4 &u1, bool norm) {
        float2 x[2][N / 2];
        Vec<T>::load(u0, x[0]);
        Vec<T>::load(u1, x[1]);
        float r = 1.f;
        if (norm) {
            float2 s0 = __fmul2_rn(x[0][0], x[0][0]), s1 = __fmul2_rn(x[1][0], x[1][0]);
#pragma unroll
            for (int i = 1; i < N / 2; ++i) s0 = __ffma2_rn(x[0][i], x[0][i], s0), s1 = __ffma2_rn(x[1][i], x[1][i], s1);
            float sum = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
            for (int o = 1; o < LK; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            r = rsqrtf(sum * (1.f / D) + a.eps);
        }
        const float2 rr = make_float2(r, r);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            const float2 y0 = kInter ? make_float2(x[0][i].y, x[0][i].x) : x[1][i];
            const float2 y1 = kInter ? make_float2(x[1][i].y, x[1][i].x) : x[0][i];
            float2 z0 = __fmul2_rn(C[0][i], x[0][i]), z1 = __fmul2_rn(C[1][i], x[1][i]);
            if (in) z0 = __ffma2_rn(S[0][i], y0, z0), z1 = __ffma2_rn(S[1][i], y1, z1);  // else y's bits do not matter
            x[0][i] = __fmul2_rn(z0, rr);
            x[1][i] = __fmul2_rn(z1, rr);
        }
        u0 = Vec<T>::store(x[0]);
        u1 = Vec<T>::store(x[1]);
    };
    int token = -1, made = -1;  // the token that cs is for; the layer and kind of it that C and S are for
    for (int st = 0; here.left > 0; st = st + 1 == kRing ? 0 : st + 1) {
        issue();
        asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
        __syncwarp();
        const unsigned char *stage = ring + st * kStage;
        const int n = group(here), t = here.token, l = here.layer, kv = here.kv, h0 = here.s * VW;
        advance(here, n);
        const T *w_ = static_cast<const T *>(kv ? a.k_weight : a.q_weight);
        const bool norm = w_ != nullptr;
        if ((t != token || made != 2 * l + kv) && !(kv && h0 >= Hkv)) {  // values alone need no factors
            if (t != token && half) {
                const int pos = *reinterpret_cast<const int32_t *>(stage + kVectors + 256);
#pragma unroll
                for (int i = 0; i < kMaxD / 64; ++i)
                    if (lane + 32 * i < half) cs[lane + 32 * i] = turn(pos, freq[i]);
                __syncwarp();
            }
            token = t;
            made = 2 * l + kv;
            float2 w[2][N / 2];
#pragma unroll
            for (int i = 0; i < N / 2; ++i) w[0][i] = w[1][i] = make_float2(1.f, 1.f);
            if (norm) {
                Vec<T>::load(*reinterpret_cast<const uint4 *>(w_ + l * D + p0 * N), w[0]);
                Vec<T>::load(*reinterpret_cast<const uint4 *>(w_ + l * D + p1 * N), w[1]);
            }
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (!in) {
                    C[0][i] = w[0][i], C[1][i] = w[1][i];
                    S[0][i] = S[1][i] = make_float2(0.f, 0.f);
                } else if constexpr (kInter) {
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 f = cs[(k ? p1 : p0) * N / 2 + i];
                        C[k][i] = make_float2(w[k][i].x * f.x, w[k][i].y * f.x);
                        S[k][i] = make_float2(-w[k][i].y * f.y, w[k][i].x * f.y);
                    }
                } else {
                    const float2 f = cs[p0 * N + 2 * i], g = cs[p0 * N + 2 * i + 1];
                    C[0][i] = make_float2(w[0][i].x * f.x, w[0][i].y * g.x);
                    C[1][i] = make_float2(w[1][i].x * f.x, w[1][i].y * g.x);
                    S[0][i] = make_float2(-w[1][i].x * f.y, -w[1][i].y * g.y);
                    S[1][i] = make_float2(w[0][i].x * f.y, w[0][i].y * g.y);
                }
            }
        }
        const uint4 *from = reinterpret_cast<const uint4 *>(stage) + grp * PV;
        if (!kv) {
            uint4 *out = reinterpret_cast<uint4 *>(static_cast<T *>(a.q_out) + (((int64_t)t * L + l) * Hq + h0 + grp) * D);
            for (int k = 0; k < n; ++k, from += VW * PV, out += VW * PV) {
                uint4 u0 = from[p0], u1 = from[p1];
                apply(u0, u1, norm);
                if (h0 + k * VW + grp < Hq) out[p0] = u0, out[p1] = u1;
            }
        } else {
            const int64_t *slots = reinterpret_cast<const int64_t *>(stage + kVectors) + grp;
            for (int k = 0; k < n; ++k, from += VW * PV, slots += VW) {
                const int h = h0 + k * VW + grp;
                uint4 u0 = from[p0], u1 = from[p1];
                if (h - grp < Hkv) {  // keys among the step's vectors
                    uint4 r0 = u0, r1 = u1;
                    apply(r0, r1, norm);
                    if (h < Hkv) u0 = r0, u1 = r1;
                }
                if (h < 2 * Hkv) {
                    const int64_t slot = *slots;
                    if (slot >= 0 && slot < pool_slots) {
                        uint4 *out = static_cast<uint4 *>(const_cast<void *>(h < Hkv ? c.k_pool : c.v_pool)) + slot * PV;
                        out[p0] = u0;
                        out[p1] = u1;
                    } else if (slot != -1 && sub == 0) {
                        report(a.status, KVC_DEV_BAD_PAGE, -1);
                    }
                }
            }
        }
        __syncwarp();  // every lane is done with the stage before the next group refills it
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <typename T, int D, bool kInter>
cudaError_t launch_kind(const NormRopeArgs &a, cudaStream_t stream) {
    constexpr int VW = 64 / (D / Vec<T>::N);
    const int64_t steps = (int64_t)a.num_tokens * a.c.num_layers *
                          ((a.num_q_heads + VW - 1) / VW + (2 * a.c.num_kv_heads + VW - 1) / VW);
    const int grid = (int)std::min<int64_t>((steps + kWarps - 1) / kWarps, (int64_t)device_sms() * kCtas);
    static int done[kMaxDevices];
    const size_t bytes = (size_t)kWarps * kWarpBytes;
    cudaError_t e = dyn_smem_at_least(reinterpret_cast<const void *>(norm_rope_kernel<T, D, kInter>), bytes, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(norm_rope_kernel<T, D, kInter>, dim3(grid), kThreads, bytes, stream, a);
}

template <typename T>
cudaError_t launch(const NormRopeArgs &a, bool interleaved, cudaStream_t stream) {
    if (a.c.head_dim == 128) return interleaved ? launch_kind<T, 128, true>(a, stream) : launch_kind<T, 128, false>(a, stream);
    return interleaved ? launch_kind<T, 64, true>(a, stream) : launch_kind<T, 64, false>(a, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const CacheView &c, const void *qkv, int64_t token_stride, int32_t num_tokens,
                             const int32_t *token_count, int32_t num_q_heads, const void *q_weight, const void *k_weight,
                             float eps, const float *inv_freq, int32_t rope_dim, bool interleaved, const int32_t *token_pos,
                             const int64_t *slot_map, void *q_out, int32_t *status, cudaStream_t stream) {
    NormRopeArgs a{c, qkv, token_stride, num_tokens, token_count, num_q_heads, q_weight, k_weight, eps, inv_freq,
                   rope_dim, token_pos, slot_map, q_out, status};
    return c.dtype == KVC_BF16 ? launch<__nv_bfloat16>(a, interleaved, stream) : launch<float>(a, interleaved, stream);
}

}  // namespace kvc
