// Attention of one new token over the pages of a list, or over the whole row, split evenly over the GPU and joined
// (kvc_block_attention).
//
// For each row, the G query heads of its group and the slots i of the listed pages (all pages without a list) that are
// below row_len and at or before the query's position:
//     l[g, i] = q_g . k_i / sqrt(D),  lse[g] = log sum_i exp(l[g, i]),  out[g] = sum_i exp(l[g, i] - lse[g]) v_i.
// K and V are read once and nothing of size [heads][slots] is kept, so a row may have any length.
//
// The split.  A row's slots, in list order, are cut into chunks of CH (16 at bf16, 8 at fp32), and the chunks of all
// rows are shared out evenly over the launch's warps (rowshare.cuh).  A warp streams its run's K and V rows through a ring of
// stages of its own with 16-byte cp.async, one or more chunks ahead, and keeps a running maximum m, sum s and output o
// for each head (online softmax).  A row that lies inside one run is finished by its warp.  The parts (m, s, o) of one
// that does not are joined within the CTA through shared memory, and if the row goes on in other CTAs, the CTA leaves one
// part in the workspace: slot 1 of the CTA where the row begins, slot 0 of the others.  A second launch, which is
// resident before the first ends (programmatic dependent launch), joins those: M = max m_j,
// out = sum_j 2^(m_j - M) o_j / sum_j 2^(m_j - M) s_j.  All joins are in the order of the sequence, so results repeat
// bit for bit.
//
// bf16: the chunk's two contractions are warp-level tensor-core tiles (m16n8k16, fp32 accumulate), S = K Q^T with the 16 keys
// as rows and the heads (padded to 8) as columns, O^T += V^T P with D as rows.  P is split into three bf16 parts whose sum
// keeps 24 bits, all of fp32's; two would keep 16, and the output is fp32.
// A tensor-core step truncates when it adds to its accumulator, which over a run of hundreds of chunks drifts (7e-6 at 138
// chunks), so each chunk's product starts from zero and is added to the run's output by a rounded fp32 addition.
// fp32: a lane owns 8 elements of D of a key and all dot products are fp32 FMAs.
// Measured a call (bf16, 8 KV heads, 4 query heads each): 219 us for 16 sequences of 8K to 33K slots (1.39 GB, 6.3 TB/s), 95 us for
// one of 131,072, 35 us for 128 chosen pages of 16 sequences (136 MB): a warp's first chunk is there after 6 to 7 us, the SMs' last
// ones lie 12 to 19% apart, and the joins take 5 us.
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "rowshare.cuh"

namespace kvc {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
static_assert(kThreads == kShareThreads, "rows are shared out by the whole CTA");
constexpr int kMinRun = 1;     // chunks a run (2: 11.3 us where 1 takes 10.0 for 8 rows of 512 slots, and no faster at other sizes)
constexpr int kMaxGroup = 8;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kJoinThreads = 256;

struct AttnArgs {
    CacheView c;
    const void *q;         // [S][L][Hq][D], cache dtype
    const int32_t *q_pos;  // [S]
    int32_t num_q_heads, group;
    const int32_t *list;   // [rows][list_stride] or null
    int32_t list_stride;
    const int32_t *list_len;
    float *out, *lse;
    float *parts;          // [CTAs][2][group * (D + 2)]: o, then m and s of each head
    int2 *spans;           // [CTAs]: the row that begins in the CTA and goes on after it (-1: none), and its last CTA
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

// slots of row r that take part, in list order, those of a partly filled last page all counted (0 for a row whose length or
// list is not usable; `tell` reports it)
__device__ __forceinline__ int row_slots(const AttnArgs &a, int r, bool tell) {
    const CacheView &c = a.c;
    const int n = c.row_len[r], k = a.list ? a.list_len[r] : 0, P = c.page_size;  // one round trip for both
    if (n < 0 || n > c.max_slots) {
        if (tell) report(a.status, KVC_DEV_BAD_LENGTH, r);
        return 0;
    }
    if (!a.list) return n;
    if (k < 0 || k > a.list_stride || k > (n + P - 1) / P) {
        if (tell) report(a.status, KVC_DEV_BAD_LIST, r);
        return 0;
    }
    return k * P;
}

// Stages a warp: 16 KB of K and V, 8 KB of them in flight while the other 8 are worked on.  More in flight saturates the
// memory system, and it then serves some SMs 25% faster than others: 3 stages of 8 KB took 229 us where 2 took 223 us
// (16 sequences, 8K to 33K slots, 8 heads; the SMs' ends lay 60 us apart), 99.4 where 2 took 97.5 (one of 131,072 slots).
template <typename T, int D>
constexpr int ring_stages() {
    return 16384 / (2 * (sizeof(T) == 2 ? 16 : 8) * D * (int)sizeof(T));
}

// out and lse of one (row, head) from a sum of weights and the weighted sum of V elements
__device__ __forceinline__ float ratio(float acc, float sum) { return sum == 0.f ? 0.f : acc / sum; }
__device__ __forceinline__ float log_sum(float m, float sum) { return sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2; }

template <typename T, int D, int GM, bool kWhole>
__global__ void __launch_bounds__(kThreads, 1) attention_kernel(AttnArgs a) {
    constexpr bool MM = sizeof(T) == 2;
    constexpr int CH = MM ? 16 : 8;
    constexpr int RB = D * (int)sizeof(T);            // bytes of a key
    constexpr int PC = RB / 16;                       // 16-byte pieces of a key
    constexpr uint32_t kHalf = CH * RB;               // bytes of a chunk's K (or V)
    constexpr uint32_t kStage = 2 * kHalf + CH * 4;   // K rows, V rows, positions
    constexpr int kRing = ring_stages<T, D>();
    constexpr int NS = D / 16;
    constexpr int LK = D / 8, KW = 32 / LK, STEPS = CH / KW;  // fp32: lanes a key, keys a step
    constexpr float kSlack = 8.f;                     // bf16: the maximum moves only when a logit passes it by 8 (log2)
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ RunTable runs;
    __shared__ int4 segs[2 * kWarps];  // parts left in shared memory, in order: row (-1: none), begins here, ends here,
                                       // chunks the row has after the run
    const CacheView &c = a.c;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.group, Hkv = c.num_kv_heads, P = c.page_size, rec = G * (D + 2);
    begin_dependent();
    if (tid < 2 * kWarps) segs[tid] = make_int4(-1, 0, 0, 0);
    if (tid == 0) a.spans[blockIdx.x] = make_int2(-1, 0);
    int w, crow, coff;  // this warp's run; the next chunk to look up
    const Share sh = share_rows<kWarps>(c.rows, kMinRun, runs, [&](int r) {
        return (row_slots(a, r, blockIdx.x == 0) + CH - 1) / CH;
    }, w, crow, coff);
    unsigned char *ring = smem + (size_t)warp * kRing * kStage;
    const T *kp = static_cast<const T *>(c.k_pool);
    const T *vp = static_cast<const T *>(c.v_pool);
    // where a run's first part goes when its row ends in the run but began before it; its last part goes to the warp's
    // own ring, which is free by then
    float *head_part = reinterpret_cast<float *>(smem + (size_t)kWarps * kRing * kStage) + warp * rec;
    int total = w < sh.W ? (int)(run_start(sh, w + 1) - run_start(sh, w)) : 0;  // chunks of the run

    // Lookups.  Lane l of batch j knows chunk 32 j + l of the run: its row, its place in the row's chunks and how many follow
    // it there, and, where a chunk lies in one page (kWhole: the page size is a multiple of CH), its first slot (-1: not
    // readable), where that is in the pool, and its keys.  A batch is filled a batch ahead of its use, so that the run's
    // loads go on across rows.  Else every lane looks up the page of its own key, one chunk ahead.
    int b_row[2], b_off[2], b_left[2], b_slot[2], b_keys[2];
    int64_t b_src[2];
    int cslots = total > 0 ? row_slots(a, crow, false) : 0;
    auto look = [&](int row, int stream, int slots, int &slot, int64_t &src, int &keys) {
        slot = -1;
        src = 0;
        keys = 0;
        if (stream >= slots) return;
        const int j = stream / P, o = stream - j * P, n = c.row_len[row];
        int b = j;
        if (a.list) {
            const int32_t *list = a.list + (int64_t)row * a.list_stride;
            b = list[j];
            if (b < 0 || (int64_t)b * P >= n || (j > 0 && list[j - 1] >= b)) {
                report(a.status, KVC_DEV_BAD_LIST, row);
                return;
            }
        }
        const int32_t pg = c.block_table[(int64_t)row * c.max_pages_per_row + b];
        if (pg < 0 || pg >= c.num_pages) {
            report(a.status, KVC_DEV_BAD_PAGE, row);
            return;
        }
        slot = b * P + o;
        src = (int64_t)pg * P + o;
        keys = max(0, min(CH, n - slot));  // the page may end behind the row's last slot
    };
    auto fill = [&](int base, int &brow, int &boff, int &bleft, int &bslot, int64_t &bsrc, int &bkeys) {
        const int need = min(32, total - base);
        if (need <= 0) return;
        int row = crow, o = coff + lane, slots = cslots;
        if ((cslots + CH - 1) / CH - coff > need) {
            coff += need;
        } else {  // the batch goes on in the rows after crow, 32 of them at a time
            int got = 0;
            for (int r = crow, o0 = coff;; r += 32, o0 = 0) {
                if (r >= c.rows) {  // only if the lengths changed meanwhile
                    total = base + got;
                    break;
                }
                const int sl = r + lane < c.rows ? row_slots(a, r + lane, false) : 0;
                const int have = (sl + CH - 1) / CH - (lane == 0 ? o0 : 0);
                int incl = have;
#pragma unroll
                for (int x = 1; x < 32; x <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, incl, x);
                    if (lane >= x) incl += y;
                }
                const int all = __shfl_sync(0xffffffffu, incl, 31), x = lane - got;
                int k = 0;  // the row of this lane's chunk: the number of rows that end at or before it
#pragma unroll
                for (int half = 16; half > 0; half >>= 1)
                    if (x >= __shfl_sync(0xffffffffu, incl, k + half - 1)) k += half;
                const int before = __shfl_sync(0xffffffffu, incl - have, k), s = __shfl_sync(0xffffffffu, sl, k);
                if (x >= 0 && x < all) {
                    row = r + k;
                    o = x - before + (k == 0 ? o0 : 0);
                    slots = s;
                }
                got += all;
                if (got >= need) break;
            }
            crow = __shfl_sync(0xffffffffu, row, need - 1);
            coff = __shfl_sync(0xffffffffu, o, need - 1) + 1;
            cslots = __shfl_sync(0xffffffffu, slots, need - 1);
        }
        brow = row;
        boff = o;
        bleft = (slots + CH - 1) / CH - 1 - o;
        if constexpr (kWhole) {
            if (lane < need) look(row, o * CH, slots, bslot, bsrc, bkeys);
        } else {
            bslot = slots;
        }
    };
    // x[which] of lane l
    auto pick = [&](const auto (&x)[2], int i) { return __shfl_sync(0xffffffffu, ((i >> 5) & 1) ? x[1] : x[0], i & 31); };
    fill(0, b_row[0], b_off[0], b_left[0], b_slot[0], b_src[0], b_keys[0]);
    fill(32, b_row[1], b_off[1], b_left[1], b_slot[1], b_src[1], b_keys[1]);
    int k_row = 0, k_slot = -1, k_keys = 0;  // this lane's key of the next chunk to load (pages that are no multiple of CH)
    int64_t k_src = 0;
    auto look_key = [&](int i) {
        if (i >= total) return;
        k_row = pick(b_row, i);
        const int o = pick(b_off, i), slots = pick(b_slot, i);
        look(k_row, o * CH + (lane & (CH - 1)), slots, k_slot, k_src, k_keys);
    };
    if constexpr (!kWhole) look_key(0);
    uint32_t ok[kRing];  // the stages' readable keys, a bit each
#pragma unroll
    for (int i = 0; i < kRing; ++i) ok[i] = 0;
    // stage `st` takes chunk i of the run; returns its readable keys
    auto issue = [&](int i, int st) -> uint32_t {
        uint32_t m = 0;
        if (i < total) {
            const uint32_t dst = smem_u32(ring + (size_t)st * kStage);
            if constexpr (kWhole) {
                const int s0 = pick(b_slot, i), row = pick(b_row, i), keys = pick(b_keys, i);
                const int64_t src = pick(b_src, i);
                if (s0 >= 0) {
                    const char *ks = reinterpret_cast<const char *>(kp + src * D);
                    const char *vs = reinterpret_cast<const char *>(vp + src * D);
#pragma unroll
                    for (uint32_t e = 0; e < (uint32_t)(CH * PC / 32); ++e) {
                        // piece p of key r lands at piece p ^ (r & 7): the eight rows of an ldmatrix phase then fall in
                        // distinct banks
                        const uint32_t x = e * 32 + lane, r = x / PC, p = x % PC;
                        const uint32_t db = r * RB + ((MM ? (p ^ (r & 7)) : p) << 4);
                        cp16(dst + db, ks + x * 16);
                        cp16(dst + kHalf + db, vs + x * 16);
                    }
                    if (lane < CH) cp4(dst + 2 * kHalf + lane * 4, c.slot_pos + (int64_t)row * c.max_slots + s0 + lane);
                    m = (1u << keys) - 1;
                }
            } else {
                const bool mine = k_keys > 0;
                m = __ballot_sync(0xffffffffu, mine) & ((1u << CH) - 1);
#pragma unroll
                for (uint32_t e = 0; e < (uint32_t)(CH * PC / 32); ++e) {
                    const uint32_t x = e * 32 + lane, r = x / PC, p = x % PC;
                    const int64_t src = __shfl_sync(0xffffffffu, k_src, r);
                    const uint32_t db = r * RB + ((MM ? (p ^ (r & 7)) : p) << 4);
                    if ((m >> r) & 1u) {
                        cp16(dst + db, reinterpret_cast<const char *>(kp + src * D) + p * 16);
                        cp16(dst + kHalf + db, reinterpret_cast<const char *>(vp + src * D) + p * 16);
                    }
                }
                if (lane < CH && mine) cp4(dst + 2 * kHalf + lane * 4, c.slot_pos + (int64_t)k_row * c.max_slots + k_slot);
                look_key(i + 1);
            }
        }
        cp_commit();  // one group a call, empty or not, so that the group count stays in step
        return m;
    };
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) ok[i] = issue(i, i);

    // while the first chunks come: rows without slots, an even share of the rows a warp, a lane a row to look
    const int rows_each = (c.rows + (int)gridDim.x * kWarps - 1) / ((int)gridDim.x * kWarps);
    const int e0 = (warp * (int)gridDim.x + (int)blockIdx.x) * rows_each, e1 = min(c.rows, e0 + rows_each);
    for (int r0 = e0; r0 < e1; r0 += 32) {
        unsigned empty = __ballot_sync(0xffffffffu, r0 + lane < e1 && row_slots(a, r0 + lane, false) == 0);
        for (; empty; empty &= empty - 1) {
            const int r = r0 + __ffs(empty) - 1;
            const int64_t head = (int64_t)(r / Hkv) * a.num_q_heads + (r % Hkv) * G;
            for (int e = lane; e < G * D; e += 32) a.out[head * D + e] = 0.f;
            if (lane < G) a.lse[head + lane] = -INFINITY;
        }
    }

    // bf16: a lane holds heads hm = 2 (lane % 4) and hm + 1; O[d][h] for d = 16 t + lane / 4 (+ 8).  fp32: a lane holds
    // elements d0 .. d0 + 3 and D / 2 + d0 .. + 3 of every head
    float mm[2], ms[2];
    float oc[MM ? NS : 1][4];
    uint32_t qb[MM ? NS : 1][2];
    float m[MM ? 1 : GM], s[MM ? 1 : GM], o[MM ? 1 : GM][8], qv[MM ? 1 : GM][8];
    const int kslot = lane / LK, d0 = (lane % LK) * 4;
    int row = -1, qpos = 0;  // the row of the chunk at hand, -1 between rows
    int64_t hbase = 0;
    bool begins = false;
    auto begin_row = [&](int i) {
        row = pick(b_row, i);
        begins = pick(b_off, i) == 0;
        qpos = a.q_pos[row / (c.num_layers * Hkv)];
        hbase = (int64_t)(row / Hkv) * a.num_q_heads + (row % Hkv) * G;
        mm[0] = mm[1] = -INFINITY;
        ms[0] = ms[1] = 0.f;
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
    };

    int st = 0;
    for (int i = 0; i < total; ++i) {
        if (row < 0) begin_row(i);
        {
            const int k = i + kRing - 1, sk = st == 0 ? kRing - 1 : st - 1;
            if ((k & 31) == 4 && k > 32) {  // batch k / 32 - 1 is consumed: batch k / 32 + 1 takes its place
                const int base = (k & ~31) + 32;
                if ((k >> 5) & 1) fill(base, b_row[0], b_off[0], b_left[0], b_slot[0], b_src[0], b_keys[0]);
                else fill(base, b_row[1], b_off[1], b_left[1], b_slot[1], b_src[1], b_keys[1]);
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
                    float pv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int x = 0; x < 3; ++x) mma16816(pv, af, pa[x], pb[x]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) oc[t][u] += pv[u];
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

        // the row's result, or its part
        const int after = pick(b_left, i);
        if (after > 0 && i + 1 < total) continue;
        const bool ends = after == 0, whole = begins && ends;
        float *part = whole ? a.out + hbase * D : ends ? head_part : reinterpret_cast<float *>(ring);
        float *stat = part + G * D;
        if (!whole && lane == 0) segs[2 * warp + (ends ? 0 : 1)] = make_int4(row, begins, ends, after);
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
                        if (whole) {
                            a.lse[hbase + hm + u] = log_sum(mm[u], ms[u]);
                        } else {
                            stat[2 * (hm + u)] = mm[u];
                            stat[2 * (hm + u) + 1] = ms[u];
                        }
                    }
                    const float div = whole ? ms[u] : 1.f;
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        part[(hm + u) * D + 16 * t + (lane >> 2)] = ratio(oc[t][u], div);
                        part[(hm + u) * D + 16 * t + (lane >> 2) + 8] = ratio(oc[t][2 + u], div);
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
                    if (lane == 0) {
                        if (whole) a.lse[hbase + g] = log_sum(m[g], s[g]);
                        else stat[2 * g] = m[g], stat[2 * g + 1] = s[g];
                    }
                    const float div = whole ? s[g] : 1.f;
                    if (kslot == 0)
#pragma unroll
                        for (int u = 0; u < 8; ++u) part[g * D + (u >> 2) * (D / 2) + d0 + (u & 3)] = ratio(o[g][u], div);
                }
            }
        }
        __syncwarp();
        row = -1;
    }
    cp_wait<0>();
    __syncthreads();

    // join the parts of each row the CTA shares; a warp's elements are of one head, lane k weighs part k
    auto seg = [&](int k) {
        const size_t at = (k & 1) ? (size_t)(k >> 1) * kRing * kStage : (size_t)kWarps * kRing * kStage + (size_t)(k >> 1) * rec * 4;
        return reinterpret_cast<const float *>(smem + at);
    };
    const int4 mine = segs[lane % (2 * kWarps)];
    unsigned open = __ballot_sync(0xffffffffu, lane < 2 * kWarps && mine.x >= 0);
    while (open) {
        const int first = __ffs(open) - 1, row = __shfl_sync(0xffffffffu, mine.x, first);
        const unsigned group = __ballot_sync(0xffffffffu, mine.x == row) & open;
        open &= ~group;
        const int last = 31 - __clz(group), after = __shfl_sync(0xffffffffu, mine.w, last);
        const bool begins = __shfl_sync(0xffffffffu, mine.y, first), ends = __shfl_sync(0xffffffffu, mine.z, last);
        const bool whole = begins && ends;
        const int64_t hbase = (int64_t)(row / Hkv) * a.num_q_heads + (row % Hkv) * G;
        float *part = whole ? a.out + hbase * D : a.parts + (int64_t)(2 * blockIdx.x + (begins ? 1 : 0)) * rec;
        for (int e = 2 * tid; e < G * D; e += 2 * kThreads) {
            const int g = e / D;
            const bool has = (group >> lane) & 1u;
            const float2 ms = has ? reinterpret_cast<const float2 *>(seg(lane) + G * D)[g] : make_float2(-INFINITY, 0.f);
            const float M = warp_max(ms.x), f = weight(ms.x, M), sum = warp_sum(f * ms.y);
            float2 acc = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int k = first; k <= last; ++k) {
                const float fk = __shfl_sync(0xffffffffu, f, k);
                if ((group >> k) & 1u) {
                    const float2 x = *reinterpret_cast<const float2 *>(seg(k) + e);
                    acc.x += fk * x.x;
                    acc.y += fk * x.y;
                }
            }
            part[e] = whole ? ratio(acc.x, sum) : acc.x;
            part[e + 1] = whole ? ratio(acc.y, sum) : acc.y;
            if (e == g * D) {
                if (whole) a.lse[hbase + g] = log_sum(M, sum);
                else part[G * D + 2 * g] = M, part[G * D + 2 * g + 1] = sum;
            }
        }
        if (begins && !ends && tid == 0) {  // the CTA's last row: where does it end?
            const int64_t next = run_start(sh, min(sh.W, (int)(blockIdx.x + 1) * sh.per_cta));
            a.spans[blockIdx.x] = make_int2(row, min((int)gridDim.x - 1, run_of(sh, next + after - 1) / sh.per_cta));
        }
    }
}

// Joins the parts of a row that lies in several CTAs: a CTA of this launch for each CTA of the first (the one where the
// row begins) and head; four elements a thread, and threads of one element take every SL-th part each.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(AttnArgs a) {
    constexpr int LANES = D / 4, SL = kJoinThreads / LANES;
    __shared__ float4 acc_s[SL][LANES];
    __shared__ float sum_s[SL], max_s[SL];
    const int first = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, G = a.group, rec = G * (D + 2);
    begin_dependent();
    const int2 span = a.spans[first];
    const int row = span.x, np = span.y - first + 1;
    if (row < 0) return;
    const int64_t head = (int64_t)(row / a.c.num_kv_heads) * a.num_q_heads + (row % a.c.num_kv_heads) * G + g;
    auto part = [&](int j) { return a.parts + (int64_t)(2 * (first + j) + (j == 0 ? 1 : 0)) * rec; };
    const int d = tid % LANES, sl = tid / LANES;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.f, m = -INFINITY;  // relative to the largest maximum of this thread's parts so far
#pragma unroll 4
    for (int j = sl; j < np; j += SL) {
        const float *p = part(j);
        const float2 ms = *reinterpret_cast<const float2 *>(p + G * D + 2 * g);
        const float2 x = reinterpret_cast<const float2 *>(p + g * D)[2 * d], y = reinterpret_cast<const float2 *>(p + g * D)[2 * d + 1];
        const float top = fmaxf(m, ms.x), old = weight(m, top), f = weight(ms.x, top);
        m = top;
        sum = sum * old + f * ms.y;
        acc.x = acc.x * old + f * x.x;
        acc.y = acc.y * old + f * x.y;
        acc.z = acc.z * old + f * y.x;
        acc.w = acc.w * old + f * y.y;
    }
    acc_s[sl][d] = acc;
    if (d == 0) sum_s[sl] = sum, max_s[sl] = m;
    __syncthreads();
    if (sl == 0) {
        float M = -INFINITY;
        for (int k = 0; k < SL; ++k) M = fmaxf(M, max_s[k]);
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        sum = 0.f;
        for (int k = 0; k < SL; ++k) {
            const float f = weight(max_s[k], M);
            acc.x += f * acc_s[k][d].x;
            acc.y += f * acc_s[k][d].y;
            acc.z += f * acc_s[k][d].z;
            acc.w += f * acc_s[k][d].w;
            sum += f * sum_s[k];
        }
        float *out = a.out + head * D + 4 * d;
        out[0] = ratio(acc.x, sum);
        out[1] = ratio(acc.y, sum);
        out[2] = ratio(acc.z, sum);
        out[3] = ratio(acc.w, sum);
        if (d == 0) a.lse[head] = log_sum(M, sum);
    }
}

template <typename T, int D, int GM>
cudaError_t launch_main(const AttnArgs &a, int grid, cudaStream_t stream) {
    constexpr int CH = sizeof(T) == 2 ? 16 : 8;
    constexpr size_t kRings = (size_t)kWarps * ring_stages<T, D>() * (2 * CH * D * sizeof(T) + CH * 4);
    static_assert(kRings + kWarps * kMaxGroup * (D + 2) * 4 <= 226 * 1024, "shared memory");
    const size_t bytes = kRings + (size_t)kWarps * a.group * (D + 2) * 4;
    const bool whole = a.c.page_size % CH == 0;
    auto kernel = whole ? attention_kernel<T, D, GM, true> : attention_kernel<T, D, GM, false>;
    static int done[2][kMaxDevices];
    cudaError_t e = dyn_smem_at_least(reinterpret_cast<const void *>(kernel), bytes, done[whole]);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(grid), kThreads, bytes, stream, a);
}

template <int D>
cudaError_t launch(const AttnArgs &a, int grid, cudaStream_t stream) {
    cudaError_t e;
    if (a.c.dtype == KVC_BF16) e = launch_main<__nv_bfloat16, D, 8>(a, grid, stream);
    else if (a.group == 1) e = launch_main<float, D, 1>(a, grid, stream);
    else if (a.group == 2) e = launch_main<float, D, 2>(a, grid, stream);
    else if (a.group <= 4) e = launch_main<float, D, 4>(a, grid, stream);
    else e = launch_main<float, D, 8>(a, grid, stream);
    if (e != cudaSuccess) return e;
    return launch_dependent(join_kernel<D>, dim3(grid, a.group), kJoinThreads, 0, stream, a);
}

}  // namespace

size_t block_attention_workspace(int32_t group, int32_t head_dim) {
    const size_t ctas = (size_t)device_sms();
    return ctas * (sizeof(int2) + 2 * (size_t)group * (head_dim + 2) * sizeof(float));
}

cudaError_t launch_block_attention(const CacheView &c, const void *q, const int32_t *q_pos, int32_t num_q_heads,
                                   const int32_t *list, int32_t list_stride, const int32_t *list_len, float *out,
                                   float *lse, void *ws, int32_t *status, cudaStream_t stream) {
    const int grid = device_sms();
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
    a.spans = static_cast<int2 *>(ws);
    a.parts = reinterpret_cast<float *>(a.spans + grid);
    a.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)c.head_dim));
    a.status = status;
    return c.head_dim == 128 ? launch<128>(a, grid, stream) : launch<64>(a, grid, stream);
}

}  // namespace kvc
