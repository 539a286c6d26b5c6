// kv_attn.cuh -- what attention over either cache shares: the call's parameters, the rows of an item and what
// they see, divisions by numbers that the host knows, and the steps of the tensor cores' products.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace qmd {

// n / d for 0 <= n < 2^31 and a divisor that the host knows, by a product: floor(n m / 2^shift)
// with m = ceil(2^shift / d), shift = 31 + ceil(log2 d) (an integer division is some 40 dependent
// instructions, and there are a dozen before a warp's first load).
struct FastDiv {
    unsigned d, m, shift;
};

static inline FastDiv fast_div(unsigned d)
{
    unsigned l = 0;
    while ((1ull << l) < d)
        ++l;
    return {d, (unsigned)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

__device__ __forceinline__ int operator/(int n, const FastDiv &f)
{
    return (int)((uint64_t)(unsigned)n * f.m >> f.shift);
}

struct AttnArgs {
    KvParams kv;
    const float *q;
    float *out;
    float *part;     // workspace: [CTA][2][R][D] sums, then [CTA][2][R][2] maximum and weight sum
    unsigned *ctr;   // workspace: a counter per CTA
    int64_t q_stride, out_stride, window;
    uint64_t wait_ns;
    int group;  // query heads to a key/value head
    FastDiv by_group, by_blocks, by_heads, by_grid;  // blocks of a page, key/value heads, CTAs
    float scale_log2e;
    float *lse = nullptr;  // [rows][query heads], or nothing
};

constexpr int ATT_MAX_ROWS_FLOATS = 16 * 128;  // the largest R x D of an instance (8 x 256 is the same)
constexpr float ATT_NONE = -3.0e38f;           // the maximum before any score

// tma_load_3d with the default L2 policy: the cache is read again in the next step.
__device__ __forceinline__ void load_tile(uint32_t dst, const void *tmap, int x, int block, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(x), "r"(0), "r"(block), "r"(bar)
        : "memory");
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^n for an integer n, exactly: 0 under 2^-126, infinity from 2^128 on.  (n's lowest byte comes to stand in
// the low bits of 1.5 * 2^23 + 127 + n.)
__device__ __forceinline__ float pow2(float n)
{
    return __uint_as_float(__float_as_uint(fminf(fmaxf(n, -127.0f), 128.0f) + 12583039.0f) << 23);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose_8x8(uint32_t v)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// counters (a CTA each, to a multiple of 16 bytes), then the parts and their maxima and sums
static inline size_t counter_bytes(const DeviceInfo &dev) { return ((size_t)dev.sm_count * 4 + 15) / 16 * 16; }

static inline AttnArgs attn_args(const KvParams &kv, const float *q, int64_t q_stride, int q_heads, float scale,
                                 int64_t window, float *out, int64_t out_stride, void *ws, const DeviceInfo &dev)
{
    return {kv, q, out, reinterpret_cast<float *>(static_cast<char *>(ws) + counter_bytes(dev)),
            static_cast<unsigned *>(ws), q_stride, out_stride, window, wait_limit_ns(), q_heads / kv.heads,
            fast_div((unsigned)(q_heads / kv.heads)), fast_div((unsigned)kv.page_blocks),
            fast_div((unsigned)kv.heads), fast_div((unsigned)dev.sm_count),
            scale * 1.4426950408889634f};
}

struct Group {  // the rows of a row group and what they see
    int lo, hi;  // blocks [lo, hi) that any of them sees
    int rows;    // query rows in the group
};

__device__ __forceinline__ int row_end(const KvSeq &q, int i) { return max(0, q.len - q.n + 1 + i); }
__device__ __forceinline__ int row_begin(const AttnArgs &a, int end)
{
    return a.window > 0 && end > a.window ? (int)(end - a.window) : 0;
}

template <int R>
__device__ __forceinline__ Group group_of(const AttnArgs &a, const KvSeq &q, int cg)
{
    Group g;
    g.rows = min(R, q.n * a.group - cg * R);
    const int last = row_end(q, (cg * R + g.rows - 1) / a.by_group);
    g.lo = row_begin(a, row_end(q, cg * R / a.by_group)) / KV_BLOCK;
    g.hi = (last + KV_BLOCK - 1) / KV_BLOCK;
    return g;
}

// Query row r of a group that starts at query row `first`: its row of the call and its query head.
__device__ __forceinline__ int64_t row_offset(const AttnArgs &a, int row0, int head, int r, int64_t stride, int dim)
{
    const int i = r / a.by_group;
    return (int64_t)(row0 + i) * stride + (head * a.group + r - i * a.group) * dim;
}

struct Job {  // an item cut at the end of a warp's range
    int start, end;    // its units, counted from the CTA's first
    int row0, first;   // the sequence's first row; the group's first query row
    int head, rows;    // rows 0: no job
    int pad[2];
};

// The units of all items in one line, sequence after sequence.  Of up to 32 sequences every lane holds one:
// its units, and those before it; of more, s_pre[s] in shared memory holds those before sequence s.
struct UnitLine {
    bool few, too_many;  // too_many: more units than 31 bits count
    int before, units_of, units;
};

// All threads of the W warps call it; units_of(sequence) is its number of units (64 bits).
template <int W, class UnitsOf>
__device__ __forceinline__ UnitLine unit_line(const KvParams &p, UnitsOf units_of, int64_t *s_warp, int *s_pre)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // up to 32 sequences: every warp for itself, a lane a sequence; else through shared memory
    UnitLine l = {p.seqs <= 32, false, 0, 0, 0};
    if (l.few) {
        int64_t u = lane < p.seqs ? units_of(kv_seq(p, lane)) : 0;
        l.units_of = (int)min(u, (int64_t)INT_MAX);
        const bool big = __any_sync(0xffffffffu, u > INT_MAX / 32);  // the 32-bit sum may run over
        if (big) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                u += __shfl_xor_sync(0xffffffffu, u, o);
            l.too_many = u > INT_MAX;
        }
        unsigned sum = (unsigned)l.units_of;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o)
                sum += x;
        }
        l.before = (int)(sum - (unsigned)l.units_of);
        l.units = (int)__shfl_sync(0xffffffffu, sum, 31);
    } else {
        int64_t total = 0;
        for (int s0 = 0; s0 < p.seqs; s0 += W * 32) {
            const int s = s0 + tid;
            const int64_t u = s < p.seqs ? units_of(kv_seq(p, s)) : 0;
            int64_t sum = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o)
                    sum += x;
            }
            __syncthreads();
            if (lane == 31)
                s_warp[warp] = sum;
            __syncthreads();
            int64_t base = total;
            for (int w = 0; w < W; ++w) {
                if (w < warp)
                    base += s_warp[w];
                total += s_warp[w];
            }
            if (s < p.seqs)
                s_pre[s] = (int)(base + sum - u);
        }
        l.units = (int)total;
        l.too_many = total > INT_MAX;
        if (tid == 0)
            s_pre[p.seqs] = l.units;
        __syncthreads();
    }
    return l;
}

// The sequence that holds unit `at`, its first unit and how many it has.  A whole warp calls it.
__device__ __forceinline__ int line_find(const UnitLine &l, const KvParams &p, int at, const int *s_pre, int *first, int *count)
{
    if (l.few) {
        const int s = 31 - __clz(__ballot_sync(0xffffffffu, l.units_of > 0 && l.before <= at));
        *first = __shfl_sync(0xffffffffu, l.before, s);
        *count = __shfl_sync(0xffffffffu, l.units_of, s);
        return s;
    }
    int lo = 0, hi = p.seqs;  // s_pre[lo] <= at < s_pre[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pre[mid] <= at)
            lo = mid;
        else
            hi = mid;
    }
    *first = s_pre[lo];
    *count = s_pre[lo + 1] - s_pre[lo];
    return lo;
}

// Up to 32 sequences: those that have units.
__device__ __forceinline__ unsigned line_live(const UnitLine &l) { return __ballot_sync(0xffffffffu, l.units_of > 0); }

// The next sequence with units after s (there is one).
__device__ __forceinline__ int line_next(const KvParams &p, unsigned live, int s, const int *s_pre)
{
    if (p.seqs <= 32)
        return __ffs(live & ~((2u << s) - 1)) - 1;
    do
        ++s;
    while (s_pre[s + 1] == s_pre[s]);
    return s;
}

// A row's log-sum-exp from its maximum (log2) and its sum of weights over it.
__device__ __forceinline__ void store_lse(const AttnArgs &a, int row0, int head, int r, float m, float l)
{
    a.lse[row_offset(a, row0, head, r, a.group * a.kv.heads, 1)] =
        l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// The joins of items that were cut: inside the CTA, then between CTAs.  Warp w's first part lies in smem + slots +
// w * slot_bytes, its last in its ring at smem + w * ring; s_ml holds their maxima and sums.  The CTA's range is
// units u0 .. u0 + span - 1, pw to a warp, per to a CTA.  Every thread calls it, after a barrier.
template <int D, int R, int W, bool LSE>
__device__ __forceinline__ void join_parts(const AttnArgs &a, const Job *s_job, const float2 *s_ml, int *s_last,
                                           unsigned char *smem, int ring, int slots, int slot_bytes, int u0, int span, int pw,
                                           int per)
{
    // ---- joins inside the CTA -------------------------------------------------------------------
    // Job 0 is the item that began before the CTA's range (parts 0 of warps 0 ..), job 1 + w the one
    // that warp w's range cut (its part 1, parts 0 of the warps after it).
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t part_ml = (int64_t)gridDim.x * 2 * R * D;
    const unsigned live = __ballot_sync(0xffffffffu, lane <= W && s_job[lane <= W ? lane : 0].rows > 0);
    if (live == 0)
        return;
    const int k = lane & 15;                          // a half warp's lane: a part, and 4 of 64 values
    const unsigned half = 0xffffu << (lane & 16);
    constexpr int SEG = D / 64;                       // half warps to a row
    bool cut = false;  // some item goes on in another CTA
    int tail = -1;     // the item that goes on after this CTA's range
    {
        const int njobs = __popc(live);
        unsigned left = live;
        int jj = -1, seen = 0;
        for (int i = tid >> 4; i < njobs * R * SEG; i += 2 * W) {
            while (seen <= i / (R * SEG)) {
                jj = __ffs(left) - 1;
                left &= left - 1;
                ++seen;
            }
            const int r = i / SEG % R, d = i % SEG * 64 + 4 * k;
            const int start = s_job[jj].start, end = s_job[jj].end;
            if (r >= s_job[jj].rows)
                continue;
            const int wa = max(0, jj - 1), wb = (min(end, span) - 1) / pw;
            // lane k has part k's maximum and sum, and makes its factor
            const float2 ml = wa + k <= wb ? s_ml[((wa + k) * 2 + (k == 0 && jj > 0)) * R + r] : make_float2(ATT_NONE, 0.0f);
            float M = ml.x;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                M = fmaxf(M, __shfl_xor_sync(half, M, o));
            const float f = ex2(ml.x - M);
            float L = ml.y * f;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                L += __shfl_xor_sync(half, L, o);
            float y[4] = {};
#pragma unroll 4
            for (int w = wa; w <= wb; ++w) {
                const bool one = w == wa && jj > 0;
                const float fw = __shfl_sync(half, f, (lane & 16) + w - wa);
                float v[4];
                load_f32(v, reinterpret_cast<const float *>(one ? smem + w * ring : smem + slots + w * slot_bytes) +
                                r * D + d);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] = fmaf(v[e], fw, y[e]);
            }
            if (start >= 0 && end <= span) {
                const float g1 = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    y[e] *= g1;
                store_f32(a.out + row_offset(a, s_job[jj].row0, s_job[jj].head, s_job[jj].first + r, a.out_stride, D) + d, y);
                if (LSE && a.lse && d == 0)
                    store_lse(a, s_job[jj].row0, s_job[jj].head, s_job[jj].first + r, M, L);
            } else {
                const int64_t at = ((int64_t)blockIdx.x * 2 + (start < 0 ? 0 : 1)) * R + r;
                store_f32(a.part + at * D + d, y);
                if (d == 0)
                    reinterpret_cast<float2 *>(a.part + part_ml)[at] = make_float2(M, L);
            }
        }
        for (unsigned x = live; x; x &= x - 1) {
            const int i = __ffs(x) - 1;
            if (s_job[i].end > span)
                tail = i;
        }
        cut = (live & 1) || tail >= 0;
    }
    if (!cut)
        return;

    // ---- joins between CTAs: the one that comes last adds the parts, in their order ---------------
    // At most two items are cut: job 0, and the tail.
    __syncthreads();
    if (tid < 2) {
        const int jj = tid == 0 ? ((live & 1) ? 0 : -1) : tail == 0 ? -1 : tail;
        int last = 0;
        if (jj >= 0) {
            const int c0 = (u0 + s_job[jj].start) / per, c1 = (u0 + s_job[jj].end - 1) / per;
            // releases the CTA's parts (ordered before it by the barrier) and acquires the others'
            unsigned come;
            asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(come) : "l"(a.ctr + c0) : "memory");
            last = come == (unsigned)(c1 - c0);
            if (last)
                a.ctr[c0] = 0;  // every part has come: left as it was found
        }
        s_last[tid] = last ? jj + 1 : 0;
    }
    __syncthreads();
    // A half warp takes 64 values of a row from every NG-th part; its maxima and sums and its first
    // values are in flight together.
    constexpr int TASKS = R * SEG, NG = 2 * W / TASKS > 0 ? 2 * W / TASKS : 1, AHEAD = 4;
    float4 *s_y = reinterpret_cast<float4 *>(smem);  // [NG][R * D / 4]
    for (int x = 0; x < 2; ++x) {
        if (!s_last[x])
            continue;
        const Job j = s_job[s_last[x] - 1];
        const int c0 = (u0 + j.start) / per, parts = (u0 + j.end - 1) / per - c0 + 1;
        // part i lies with CTA c0 + i, as its part 1 if the item began there
        auto slot = [&](int i) { return ((int64_t)(c0 + i) * 2 + (i == 0)) * R; };
        const float2 *ml = reinterpret_cast<const float2 *>(a.part + part_ml);
        for (int i = tid >> 4; i < NG * TASKS; i += 2 * W) {
            const int n0 = i / TASKS, r = i / SEG % R, e4 = i % SEG * 16 + k;
            if (r >= j.rows)
                continue;
            auto value = [&](int q) { return __ldcg(reinterpret_cast<const float4 *>(a.part + (slot(q) + r) * D) + e4); };
            float4 v[AHEAD];
            float vm[AHEAD];
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
                if (n0 + q * NG < parts) {
                    v[q] = value(n0 + q * NG);
                    vm[q] = __ldcg(&ml[slot(n0 + q * NG) + r]).x;
                }
            float M = ATT_NONE, L = 0.0f;  // the lane's parts k, k + 16, .., then all
            for (int q = k; q < parts; q += 16) {
                const float2 w = __ldcg(&ml[slot(q) + r]);
                const float mn = fmaxf(M, w.x);
                L = fmaf(w.y, ex2(w.x - mn), L * ex2(M - mn));
                M = mn;
            }
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) {
                const float m2 = __shfl_xor_sync(half, M, o), l2 = __shfl_xor_sync(half, L, o), mn = fmaxf(M, m2);
                // the same expression on both lanes of a pair: the same bits
                L = fmaf(fminf(M, m2) == M ? L : l2, ex2(fminf(M, m2) - mn), fminf(M, m2) == M ? l2 : L);
                M = mn;
            }
            float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto add = [&](const float4 &u, float m) {
                const float f = ex2(m - M);
                y.x = fmaf(u.x, f, y.x), y.y = fmaf(u.y, f, y.y), y.z = fmaf(u.z, f, y.z), y.w = fmaf(u.w, f, y.w);
            };
#pragma unroll
            for (int q = 0; q < AHEAD; ++q)
                if (n0 + q * NG < parts)
                    add(v[q], vm[q]);
#pragma unroll 4
            for (int q = n0 + AHEAD * NG; q < parts; q += NG)
                add(value(q), __ldcg(&ml[slot(q) + r]).x);
            if (LSE && a.lse && n0 == 0 && e4 == 0)
                store_lse(a, j.row0, j.head, j.first + r, M, L);
            const float g1 = L == 0.0f ? 0.0f : 1.0f / L;
            y.x *= g1, y.y *= g1, y.z *= g1, y.w *= g1;
            if (NG > 1)
                s_y[(n0 * R + r) * (D / 4) + e4] = y;
            else
                *reinterpret_cast<float4 *>(a.out + row_offset(a, j.row0, j.head, j.first + r, a.out_stride, D) + 4 * e4) = y;
        }
        if (NG > 1) {
            __syncthreads();
            for (int e = tid; e < j.rows * (D / 4); e += W * 32) {
                float4 z = s_y[e];
#pragma unroll
                for (int n = 1; n < NG; ++n) {
                    const float4 u = s_y[n * R * (D / 4) + e];
                    z.x += u.x, z.y += u.y, z.z += u.z, z.w += u.w;
                }
                const int r = e / (D / 4);
                *reinterpret_cast<float4 *>(a.out + row_offset(a, j.row0, j.head, j.first + r, a.out_stride, D) +
                                            e % (D / 4) * 4) = z;
            }
            __syncthreads();
        }
    }
}

}  // namespace qmd
