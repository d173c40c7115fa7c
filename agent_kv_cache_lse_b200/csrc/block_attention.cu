// Attention of one new token over the pages of a list, or over the whole row, split evenly over the GPU and joined
// (kvc_block_attention).
//
// For each row, the G query heads of its group and the slots i of the listed pages (all pages without a list) that are
// below row_len and at or before the query's position:
//     l[g, i] = q_g . k_i / sqrt(D),  lse[g] = log sum_i exp(l[g, i]),  out[g] = sum_i exp(l[g, i] - lse[g]) v_i.
// K and V are read once and nothing of size [heads][slots] is kept, so a row may have any length.
//
// The split.  A row's slots, in list order, are cut into chunks of CH (16 at bf16, 8 at fp32); the chunks of all rows, one
// row after another, form one sequence of U chunks, and W warps of the launch take equal runs
// [U w / W, U (w + 1) / W) of it, wherever rows begin and end.  So the load is even whether there are a few long rows, many
// short ones or rows of unlike lengths, and no warp waits for another.  Every CTA sums the rows' chunk counts
// (from row_len, or the list's length) to find where its warps start.
//
// A warp streams its chunks' K and V rows through a ring of kRing stages of its own with 16-byte cp.async, kRing - 1
// chunks ahead, keeps a running maximum m, sum s and output o for each head (online softmax), and at the end of its run or of
// a row leaves (m, s, o) as a part in the workspace.  Parts are numbered w + row: along the sequence each new part has a new
// warp or a new row, never both old, so the number is unique and a row's parts are consecutive.  A second launch joins each
// (row, head): M = max m_j, out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) s_j, in the order of the parts, so results
// repeat bit for bit.
//
// bf16: the chunk's two contractions are warp-level tensor-core tiles (m16n8k16, fp32 accumulate), S = K Q^T with the 16 keys
// as rows and the heads (padded to 8) as columns, O^T += V^T P with D as rows.  P is split into three bf16 parts whose sum
// keeps 24 bits, all of fp32's: two parts (16 bits) left the fp32 output 5e-6 off where the plain form is 4e-7 off.
// fp32: a lane owns 8 elements of D of a key and all dot products are fp32 FMAs.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace kvc {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kRing = 3;       // stages a warp
constexpr int kMinRun = 2;     // chunks a run, where there are that many
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kJoinThreads = 512;

struct AttnArgs {
    CacheView c;
    const void *q;         // [S][L][Hq][D], cache dtype
    const int32_t *q_pos;  // [S]
    int32_t num_q_heads, group;
    const int32_t *list;   // [rows][list_stride] or null
    int32_t list_stride;
    const int32_t *list_len;
    float *out, *lse;
    float *parts;          // [W + rows][group * (D + 2)]: o, then m and s of each head
    int64_t *row_start;    // [rows]: first chunk of the row in the sequence (written where the row has chunks)
    int64_t *total;        // U
    float scale_log2;      // log2(e) / sqrt(D)
    int32_t *status;
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
// c += A (16 x 16, row) * B (16 x 8, col), bf16 operands, fp32 accumulate
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movm_t(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 2^(x - ref): zero for x = -inf (a hidden key, an empty part), whatever ref is; ref is finite otherwise
__device__ __forceinline__ float weight(float x, float ref) { return x == -INFINITY ? 0.f : ex2(x - ref); }

// (x, y) as three bf16x2 whose sum is (x, y) to 24 bits
__device__ __forceinline__ void split3(float x, float y, uint32_t (&w)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        x -= __low2float(h);
        y -= __high2float(h);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
}

// slots of row r that take part, in list order (0 for a row whose length or list is not usable; `tell` reports it)
__device__ __forceinline__ int row_slots(const AttnArgs &a, int r, bool tell) {
    const CacheView &c = a.c;
    const int n = c.row_len[r], P = c.page_size;
    if (n < 0 || n > c.max_slots) {
        if (tell) report(a.status, KVC_DEV_BAD_LENGTH, r);
        return 0;
    }
    if (!a.list) return n;
    const int k = a.list_len[r], nb = (n + P - 1) / P;
    if (k == 0) return 0;
    const int last = k > 0 && k <= a.list_stride ? a.list[(int64_t)r * a.list_stride + k - 1] : -1;
    if (k > nb || last < 0 || last >= nb) {
        if (tell) report(a.status, KVC_DEV_BAD_LIST, r);
        return 0;
    }
    return k * P - (last == nb - 1 ? nb * P - n : 0);  // only the row's last page may be partly filled
}

// How U chunks are shared out: `per_cta` warps of each CTA take runs, W in all, every run at least one chunk (kMinRun where
// U allows it, so that a short launch does not spread into parts that cost more to join than to stream).
struct Share {
    int per_cta, W;
};
__device__ __forceinline__ Share share_of(int64_t U, int ctas) {
    const int64_t per = U / ((int64_t)ctas * kMinRun);
    Share s;
    s.per_cta = (int)(per < 1 ? 1 : per > kWarps ? kWarps : per);
    s.W = (int)min(U, (int64_t)ctas * s.per_cta);
    return s;
}
// first chunk of run w
__device__ __forceinline__ int64_t run_start(int64_t U, int w, int W) { return U * w / W; }

template <typename T, int D, int GM, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(AttnArgs a) {
    constexpr bool MM = sizeof(T) == 2;
    constexpr int CH = MM ? 16 : 8;
    constexpr int RB = D * (int)sizeof(T);            // bytes of a key
    constexpr int PC = RB / 16;                       // 16-byte pieces of a key
    constexpr uint32_t kHalf = CH * RB;               // bytes of a chunk's K (or V)
    constexpr uint32_t kStage = 2 * kHalf + CH * 4;   // K rows, V rows, positions
    constexpr int NS = D / 16;
    constexpr int LK = D / 8, KW = 32 / LK, STEPS = CH / KW;  // fp32: lanes a key, keys a step
    constexpr float kSlack = 8.f;                     // bf16: the maximum moves only when a logit passes it by 8 (log2)
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ long long scan_s[kWarps];
    __shared__ int start_row[kWarps];
    __shared__ long long start_off[kWarps];
    const CacheView &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.group, Hkv = c.num_kv_heads, P = c.page_size;

    // where the warps' runs start: each thread sums the chunks of its share of the rows, the CTA scans the sums
    int64_t U = 0;
    {
        const int share = (c.rows + kThreads - 1) / kThreads;
        const int r0 = min(c.rows, tid * share), r1 = min(c.rows, r0 + share);
        long long mine = 0;
        for (int r = r0; r < r1; ++r) mine += (row_slots(a, r, blockIdx.x == 0) + CH - 1) / CH;
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) scan_s[warp] = x;
        if (tid < kWarps) start_row[tid] = c.rows, start_off[tid] = 0;
        __syncthreads();
        long long before = x - mine;
        for (int k = 0; k < kWarps; ++k) {
            if (k < warp) before += scan_s[k];
            U += scan_s[k];
        }
        const Share sh = share_of(U, gridDim.x);
        for (int k = 0; k < sh.per_cta && blockIdx.x * sh.per_cta + k < sh.W; ++k) {
            const int64_t s = run_start(U, blockIdx.x * sh.per_cta + k, sh.W);
            if (s >= before && s < before + mine) {  // the run starts in one of this thread's rows
                int64_t at = before;
                for (int r = r0; r < r1; ++r) {
                    const int nch = (row_slots(a, r, false) + CH - 1) / CH;
                    if (s < at + nch) {
                        start_row[k] = r;
                        start_off[k] = s - at;
                        break;
                    }
                    at += nch;
                }
            }
        }
        if (blockIdx.x == 0) {  // the join looks rows up in the sequence
            int64_t at = before;
            for (int r = r0; r < r1; ++r) {
                a.row_start[r] = at;
                at += (row_slots(a, r, false) + CH - 1) / CH;
            }
            if (tid == 0) *a.total = U;
        }
        __syncthreads();
    }

    unsigned char *ring = smem + (size_t)warp * kRing * kStage;
    const T *kp = static_cast<const T *>(c.k_pool);
    const T *vp = static_cast<const T *>(c.v_pool);
    const Share sh = share_of(U, gridDim.x);
    const int w = blockIdx.x * sh.per_cta + warp;
    if (warp >= sh.per_cta || w >= sh.W) return;
    int64_t left = run_start(U, w + 1, sh.W) - run_start(U, w, sh.W);
    int off = (int)start_off[warp];
    for (int row = start_row[warp]; left > 0; ++row, off = 0) {
        const int slots = row_slots(a, row, false);
        const int nch = (slots + CH - 1) / CH;
        const int cnt = (int)min((int64_t)(nch - off), left);
        if (cnt <= 0) continue;
        left -= cnt;
        const int n = c.row_len[row], nb = (n + P - 1) / P;
        const int seq = row / (c.num_layers * Hkv), qpos = a.q_pos[seq];
        const int64_t hbase = (int64_t)(row / Hkv) * a.num_q_heads + (row % Hkv) * G;
        const int32_t *bt = c.block_table + (int64_t)row * c.max_pages_per_row;
        const int32_t *list = a.list ? a.list + (int64_t)row * a.list_stride : nullptr;
        const int32_t *posr = c.slot_pos + (int64_t)row * c.max_slots;
        bool bad_page = false, bad_list = false;

        // Page lookups.  kWhole (the page size is a multiple of CH): a chunk lies in one page, and lane l looks up
        // chunk 32 j + l of the run, a batch of 32 chunks ahead of its use.  Else every lane looks up the page of its own
        // key, one chunk ahead.  `slot` is the key's (chunk's first) logical slot, -1 where there is none to read.
        auto look = [&](int stream, int &slot, int64_t &src) {
            slot = -1;
            src = 0;
            if (stream < 0 || stream >= slots) return;
            const int j = stream / P, o = stream - j * P;
            int b = j;
            if (list) {
                b = list[j];
                if (b < 0 || b >= nb || (j > 0 && list[j - 1] >= b)) {
                    bad_list = true;
                    return;
                }
            }
            const int32_t pg = bt[b];
            if (pg < 0 || pg >= c.num_pages) {
                bad_page = true;
                return;
            }
            slot = b * P + o;
            src = (int64_t)pg * P + o;
        };
        int sl[2] = {-1, -1};
        int64_t sr[2] = {0, 0};
        if constexpr (kWhole) {
            look(lane < cnt ? (off + lane) * CH : -1, sl[0], sr[0]);
            look(32 + lane < cnt ? (off + 32 + lane) * CH : -1, sl[1], sr[1]);
        } else {
            look((off)*CH + (lane & (CH - 1)), sl[0], sr[0]);
        }
        uint32_t ok[kRing];  // the stages' readable keys, a bit each
#pragma unroll
        for (int i = 0; i < kRing; ++i) ok[i] = 0;
        // stage `st` takes chunk i of the run; returns its readable keys
        auto issue = [&](int i, int st) -> uint32_t {
            uint32_t m = 0;
            if (i < cnt) {
                const uint32_t dst = smem_u32(ring + (size_t)st * kStage);
                if constexpr (kWhole) {
                    const int which = (i >> 5) & 1;
                    const int s0 = __shfl_sync(0xffffffffu, which ? sl[1] : sl[0], i & 31);
                    const int64_t src = __shfl_sync(0xffffffffu, which ? sr[1] : sr[0], i & 31);
                    if (s0 >= 0) {
                        const char *ks = reinterpret_cast<const char *>(kp + src * D);
                        const char *vs = reinterpret_cast<const char *>(vp + src * D);
#pragma unroll
                        for (uint32_t e = 0; e < (uint32_t)(CH * PC / 32); ++e) {
                            // piece p of key r lands at piece p ^ (r & 7): the eight rows of an ldmatrix phase then
                            // fall in distinct banks
                            const uint32_t x = e * 32 + lane, r = x / PC, p = x % PC;
                            const uint32_t db = r * RB + ((MM ? (p ^ (r & 7)) : p) << 4);
                            cp16(dst + db, ks + x * 16);
                            cp16(dst + kHalf + db, vs + x * 16);
                        }
                        if (lane < CH) cp4(dst + 2 * kHalf + lane * 4, posr + s0 + lane);
                        const int here = min(CH, n - s0);
                        m = here >= CH ? (1u << CH) - 1 : (1u << max(here, 0)) - 1;
                    }
                } else {
                    const bool mine = sl[0] >= 0 && sl[0] < n;
                    m = __ballot_sync(0xffffffffu, mine) & ((1u << CH) - 1);
#pragma unroll
                    for (uint32_t e = 0; e < (uint32_t)(CH * PC / 32); ++e) {
                        const uint32_t x = e * 32 + lane, r = x / PC, p = x % PC;
                        const int64_t src = __shfl_sync(0xffffffffu, sr[0], r);
                        const uint32_t db = r * RB + ((MM ? (p ^ (r & 7)) : p) << 4);
                        if ((m >> r) & 1u) {
                            cp16(dst + db, reinterpret_cast<const char *>(kp + src * D) + p * 16);
                            cp16(dst + kHalf + db, reinterpret_cast<const char *>(vp + src * D) + p * 16);
                        }
                    }
                    if (lane < CH && mine) cp4(dst + 2 * kHalf + lane * 4, posr + sl[0]);
                    look(i + 1 < cnt ? (off + i + 1) * CH + (lane & (CH - 1)) : -1, sl[0], sr[0]);
                }
            }
            cp_commit();  // one group a call, empty or not, so that the group count stays in step
            return m;
        };
#pragma unroll
        for (int i = 0; i < kRing - 1; ++i) ok[i] = issue(i, i);

        // bf16: a lane holds heads hm = 2 (lane % 4) and hm + 1; O[d][h] for d = 16 t + lane / 4 (+ 8).  fp32: a lane holds
        // elements d0 .. d0 + 3 and D / 2 + d0 .. + 3 of every head
        float mm[2] = {-INFINITY, -INFINITY}, ms[2] = {0.f, 0.f};
        float oc[MM ? NS : 1][4];
        uint32_t qb[MM ? NS : 1][2];
        float m[MM ? 1 : GM], s[MM ? 1 : GM], o[MM ? 1 : GM][8], qv[MM ? 1 : GM][8];
        const int kslot = lane / LK, d0 = (lane % LK) * 4;
        if constexpr (MM) {
            const int hq = lane >> 2;
            const uint16_t *qg = reinterpret_cast<const uint16_t *>(static_cast<const T *>(a.q) + (hbase + hq) * D);
#pragma unroll
            for (int t = 0; t < NS; ++t) {
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int at = 16 * t + 8 * u + 2 * (lane & 3);
                    qb[t][u] = hq < G ? (uint32_t)qg[at] | ((uint32_t)qg[at + 1] << 16) : 0u;
                }
#pragma unroll
                for (int u = 0; u < 4; ++u) oc[t][u] = 0.f;
            }
        } else {
#pragma unroll
            for (int g = 0; g < GM; ++g) {
                m[g] = -INFINITY;
                s[g] = 0.f;
                const float *qg = static_cast<const float *>(a.q) + (hbase + g) * D + d0;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    o[g][u] = 0.f;
                    qv[g][u] = g < G ? qg[(u & 3) + (u >> 2) * (D / 2)] : 0.f;
                }
            }
        }

        int st = 0;
        for (int i = 0; i < cnt; ++i) {
            {
                const int k = i + kRing - 1, sk = st == 0 ? kRing - 1 : st - 1;
                if constexpr (kWhole) {
                    if ((k & 31) == 0 && k >= 32) {  // batch k / 32 begins; the one before it makes room for the next
                        const int x = k + 32 + lane;
                        if ((k >> 5) & 1) look(x < cnt ? (off + x) * CH : -1, sl[0], sr[0]);
                        else look(x < cnt ? (off + x) * CH : -1, sl[1], sr[1]);
                    }
                }
                const uint32_t mk = issue(k, sk);
#pragma unroll
                for (int x = 0; x < kRing; ++x)
                    if (x == sk) ok[x] = mk;
            }
            cp_wait<kRing - 1>();  // this lane's copies of chunk i have landed
            __syncwarp();          // and so have the other lanes'
            uint32_t vis = 0;
#pragma unroll
            for (int x = 0; x < kRing; ++x)
                if (x == st) vis = ok[x];
            unsigned char *stage = ring + (size_t)st * kStage;
            const int32_t *ps = reinterpret_cast<const int32_t *>(stage + 2 * kHalf);
            vis &= __ballot_sync(0xffffffffu, lane < CH && ps[lane & (CH - 1)] <= qpos);
            if constexpr (MM) {
                const uint32_t kb = smem_u32(stage), vb = kb + kHalf;
                if (vis != (1u << CH) - 1) {  // hidden keys' V rows are zeroed: their P is 0, and 0 * NaN is not
                    for (int e = lane; e < CH * PC; e += 32)
                        if (!((vis >> (e / PC)) & 1u))
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + e * 16), "r"(0u) : "memory");
                    __syncwarp();
                }
                // S[key][head]: ldmatrix phase x reads keys (lane & 7) + 8 (x & 1), piece 2 t + x / 2
                float sc[4] = {0.f, 0.f, 0.f, 0.f};
                {
                    const int key = (lane & 7) + ((lane >> 3) & 1) * 8;
                    const uint32_t rowa = kb + key * RB;
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        uint32_t af[4];
                        ldsm_x4(rowa + ((((uint32_t)(2 * t + (lane >> 4))) ^ (key & 7)) << 4), af);
                        mma16816(sc, af, qb[t][0], qb[t][1]);
                    }
                }
                const int ka = lane >> 2;
                const bool va = (vis >> ka) & 1u, vc = (vis >> (ka + 8)) & 1u;
                const float l00 = va ? sc[0] * a.scale_log2 : -INFINITY, l01 = va ? sc[1] * a.scale_log2 : -INFINITY;
                const float l10 = vc ? sc[2] * a.scale_log2 : -INFINITY, l11 = vc ? sc[3] * a.scale_log2 : -INFINITY;
                float lm0 = fmaxf(l00, l10), lm1 = fmaxf(l01, l11);
                if (__any_sync(0xffffffffu, lm0 > mm[0] + kSlack || lm1 > mm[1] + kSlack)) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        lm0 = fmaxf(lm0, __shfl_xor_sync(0xffffffffu, lm0, x));
                        lm1 = fmaxf(lm1, __shfl_xor_sync(0xffffffffu, lm1, x));
                    }
                    const float n0 = fmaxf(mm[0], lm0), n1 = fmaxf(mm[1], lm1);
                    const float f0 = weight(mm[0], n0), f1 = weight(mm[1], n1);
                    ms[0] *= f0;
                    ms[1] *= f1;
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        oc[t][0] *= f0;
                        oc[t][1] *= f1;
                        oc[t][2] *= f0;
                        oc[t][3] *= f1;
                    }
                    mm[0] = n0;
                    mm[1] = n1;
                }
                const float p00 = weight(l00, mm[0]), p01 = weight(l01, mm[1]);
                const float p10 = weight(l10, mm[0]), p11 = weight(l11, mm[1]);
                ms[0] += p00 + p10;
                ms[1] += p01 + p11;
                // P as the B operand [key][head], transposed from the [key][head] rows this lane holds
                uint32_t pa[3], pb[3];
                split3(p00, p01, pa);
                split3(p10, p11, pb);
#pragma unroll
                for (int x = 0; x < 3; ++x) {
                    pa[x] = movm_t(pa[x]);
                    pb[x] = movm_t(pb[x]);
                }
                // O^T[d][head] += V^T (d x 16 keys) . P: ldmatrix.trans phase x reads keys (lane & 7) + 8 (x / 2), piece
                // 2 t + (x & 1)
                {
                    const int key = (lane & 7) + ((lane >> 4) & 1) * 8;
                    const uint32_t rowa = vb + key * RB;
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        uint32_t af[4];
                        ldsm_x4_t(rowa + ((((uint32_t)(2 * t + ((lane >> 3) & 1))) ^ (key & 7)) << 4), af);
#pragma unroll
                        for (int x = 0; x < 3; ++x) mma16816(oc[t], af, pa[x], pb[x]);
                    }
                }
            } else {
                const float *Ks = reinterpret_cast<const float *>(stage), *Vs = Ks + CH * D;
                float l[STEPS][GM], cm[GM];
#pragma unroll
                for (int g = 0; g < GM; ++g) cm[g] = -INFINITY;
#pragma unroll
                for (int t = 0; t < STEPS; ++t) {
                    const int key = t * KW + kslot;
                    const bool v = (vis >> key) & 1u;
                    const float4 x0 = *reinterpret_cast<const float4 *>(Ks + key * D + d0);
                    const float4 x1 = *reinterpret_cast<const float4 *>(Ks + key * D + D / 2 + d0);
#pragma unroll
                    for (int g = 0; g < GM; ++g) {
                        float d = qv[g][0] * x0.x + qv[g][1] * x0.y + qv[g][2] * x0.z + qv[g][3] * x0.w;
                        d += qv[g][4] * x1.x + qv[g][5] * x1.y + qv[g][6] * x1.z + qv[g][7] * x1.w;
#pragma unroll
                        for (int x = LK / 2; x > 0; x >>= 1) d += __shfl_xor_sync(0xffffffffu, d, x);
                        l[t][g] = v ? d * a.scale_log2 : -INFINITY;
                        cm[g] = fmaxf(cm[g], l[t][g]);
                    }
                }
#pragma unroll
                for (int g = 0; g < GM; ++g) {
#pragma unroll
                    for (int x = LK; x < 32; x <<= 1) cm[g] = fmaxf(cm[g], __shfl_xor_sync(0xffffffffu, cm[g], x));
                    if (cm[g] > m[g]) {  // warp-uniform: a new maximum rescales the running sum and output
                        const float f = weight(m[g], cm[g]);
                        s[g] *= f;
#pragma unroll
                        for (int u = 0; u < 8; ++u) o[g][u] *= f;
                        m[g] = cm[g];
                    }
                }
#pragma unroll
                for (int t = 0; t < STEPS; ++t) {
                    const int key = t * KW + kslot;
                    if ((vis >> key) & 1u) {
                        const float4 x0 = *reinterpret_cast<const float4 *>(Vs + key * D + d0);
                        const float4 x1 = *reinterpret_cast<const float4 *>(Vs + key * D + D / 2 + d0);
                        const float y[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                        for (int g = 0; g < GM; ++g) {
                            const float p = weight(l[t][g], m[g]);
                            s[g] += p;
#pragma unroll
                            for (int u = 0; u < 8; ++u) o[g][u] = fmaf(p, y[u], o[g][u]);
                        }
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage before the next issue refills it
            st = st + 1 == kRing ? 0 : st + 1;
        }
        cp_wait<0>();
        if (bad_page) report(a.status, KVC_DEV_BAD_PAGE, row);
        if (bad_list) report(a.status, KVC_DEV_BAD_LIST, row);

        // the part
        float *part = a.parts + (int64_t)(w + row) * G * (D + 2), *stat = part + G * D;
        if constexpr (MM) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                ms[0] += __shfl_xor_sync(0xffffffffu, ms[0], x);
                ms[1] += __shfl_xor_sync(0xffffffffu, ms[1], x);
            }
            const int hm = 2 * (lane & 3);
#pragma unroll
            for (int u = 0; u < 2; ++u)
                if (hm + u < G) {
                    if (lane < 4) {
                        stat[2 * (hm + u)] = mm[u];
                        stat[2 * (hm + u) + 1] = ms[u];
                    }
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        part[(hm + u) * D + 16 * t + (lane >> 2)] = oc[t][u];
                        part[(hm + u) * D + 16 * t + (lane >> 2) + 8] = oc[t][2 + u];
                    }
                }
        } else {
#pragma unroll
            for (int g = 0; g < GM; ++g) {
                if (g < G) {
#pragma unroll
                    for (int x = LK; x < 32; x <<= 1) {
                        s[g] += __shfl_xor_sync(0xffffffffu, s[g], x);
#pragma unroll
                        for (int u = 0; u < 8; ++u) o[g][u] += __shfl_xor_sync(0xffffffffu, o[g][u], x);
                    }
                    if (lane == 0) stat[2 * g] = m[g], stat[2 * g + 1] = s[g];
                    if (kslot == 0) {
                        *reinterpret_cast<float2 *>(part + g * D + d0) = make_float2(o[g][0], o[g][1]);
                        *reinterpret_cast<float2 *>(part + g * D + d0 + 2) = make_float2(o[g][2], o[g][3]);
                        *reinterpret_cast<float2 *>(part + g * D + D / 2 + d0) = make_float2(o[g][4], o[g][5]);
                        *reinterpret_cast<float2 *>(part + g * D + D / 2 + d0 + 2) = make_float2(o[g][6], o[g][7]);
                    }
                }
            }
        }
        __syncwarp();
    }
}

// One CTA a (row, head): kJoinThreads / D threads an element of the output, each over every such part of the row's
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a, int ctas, int CH) {
    constexpr int SL = kJoinThreads / D;
    __shared__ float red[32];
    __shared__ float acc_s[SL][D];
    const CacheView &c = a.c;
    const int row = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, G = a.group;
    const int64_t head = (int64_t)(row / c.num_kv_heads) * a.num_q_heads + (row % c.num_kv_heads) * G + g;
    const int nch = (row_slots(a, row, false) + CH - 1) / CH;
    float *out = a.out + head * D;
    if (nch == 0) {
        for (int d = tid; d < D; d += kJoinThreads) out[d] = 0.f;
        if (tid == 0) a.lse[head] = -INFINITY;
        return;
    }
    const int64_t U = *a.total, x0 = a.row_start[row], x1 = x0 + nch - 1;
    const int W = share_of(U, ctas).W;
    // run of chunk x: the last w with U w / W <= x
    const int w0 = (int)(((x0 + 1) * W - 1) / U), w1 = (int)(((x1 + 1) * W - 1) / U);
    const int64_t rec = (int64_t)G * (D + 2);
    const float *part = a.parts + (int64_t)(w0 + row) * rec;
    const int np = w1 - w0 + 1;
    float mx = -INFINITY;
    for (int j = tid; j < np; j += kJoinThreads) mx = fmaxf(mx, part[j * rec + G * D + 2 * g]);
    const float M = block_max(mx, red);
    const int d = tid % D, sl = tid / D;
    float acc = 0.f, sum = 0.f;
    for (int j = sl; j < np; j += SL) {
        const float f = weight(part[j * rec + G * D + 2 * g], M);
        sum += f * part[j * rec + G * D + 2 * g + 1];
        acc += f * part[j * rec + g * D + d];
    }
    acc_s[sl][d] = acc;
    __shared__ float sum_s[SL];
    if (d == 0) sum_s[sl] = sum;
    __syncthreads();
    if (sl == 0) {
        acc = 0.f;
        sum = 0.f;
        for (int k = 0; k < SL; ++k) {
            acc += acc_s[k][d];
            sum += sum_s[k];
        }
        out[d] = sum > 0.f ? acc / sum : (sum == 0.f ? 0.f : sum);
        if (d == 0) a.lse[head] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * kLn2;
    }
}

template <typename T, int D, int GM>
cudaError_t launch_main(const AttnArgs &a, int grid, cudaStream_t stream) {
    constexpr int CH = sizeof(T) == 2 ? 16 : 8;
    constexpr size_t kSmem = (size_t)kWarps * kRing * (2 * CH * D * sizeof(T) + CH * 4);
    static_assert(kSmem <= 226 * 1024, "shared memory");
    const bool whole = a.c.page_size % CH == 0;
    auto kernel = whole ? attention_kernel<T, D, GM, true> : attention_kernel<T, D, GM, false>;
    static int done[2][kMaxDevices];
    cudaError_t e = dyn_smem_at_least(reinterpret_cast<const void *>(kernel), kSmem, done[whole]);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kThreads, kSmem, stream>>>(a);
    return cudaGetLastError();
}

template <int D>
cudaError_t launch(const AttnArgs &a, int grid, cudaStream_t stream) {
    const bool bf16 = a.c.dtype == KVC_BF16;
    cudaError_t e;
    if (bf16) e = launch_main<__nv_bfloat16, D, 8>(a, grid, stream);
    else if (a.group == 1) e = launch_main<float, D, 1>(a, grid, stream);
    else if (a.group == 2) e = launch_main<float, D, 2>(a, grid, stream);
    else if (a.group <= 4) e = launch_main<float, D, 4>(a, grid, stream);
    else e = launch_main<float, D, 8>(a, grid, stream);
    if (e != cudaSuccess) return e;
    join_kernel<D><<<dim3(a.c.rows, a.group), kJoinThreads, 0, stream>>>(a, grid, bf16 ? 16 : 8);
    return cudaGetLastError();
}

}  // namespace

size_t block_attention_workspace(int64_t rows, int32_t group, int32_t head_dim) {
    const int64_t warps = (int64_t)device_sms() * kWarps;
    const int64_t head = (rows + 1) * (int64_t)sizeof(int64_t);  // row starts, then the total
    return (size_t)(head + (head & 8) + (warps + rows) * group * (head_dim + 2) * (int64_t)sizeof(float));
}

cudaError_t launch_block_attention(const CacheView &c, const void *q, const int32_t *q_pos, int32_t num_q_heads,
                                   const int32_t *list, int32_t list_stride, const int32_t *list_len, float *out,
                                   float *lse, void *ws, int32_t *status, cudaStream_t stream) {
    AttnArgs a{};
    a.c = c;
    a.q = q;
    a.q_pos = q_pos;
    a.num_q_heads = num_q_heads;
    a.group = num_q_heads / c.num_kv_heads;
    a.list = list;
    a.list_stride = list_stride;
    a.list_len = list_len;
    a.out = out;
    a.lse = lse;
    a.row_start = static_cast<int64_t *>(ws);
    a.total = a.row_start + c.rows;
    a.parts = reinterpret_cast<float *>(a.row_start + (c.rows + 1 + ((c.rows + 1) & 1)));
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.head_dim));
    a.status = status;
    const int grid = device_sms();
    return c.head_dim == 128 ? launch<128>(a, grid, stream) : launch<64>(a, grid, stream);
}

}  // namespace kvc
