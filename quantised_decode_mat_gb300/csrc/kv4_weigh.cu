// kv4_weigh.cu -- the attention weight that each token of the 4-bit cache gets.
//
// weight_j = (weight_j, or 0 where j is one of the call's own rows) + sum over the rows that see j and the query
// heads of the key/value head of e^(s_j - lse), s_j = scale q . K_j and lse attention's.  With the log-sum-exp
// known there is nothing to keep from one slot to the next and no value to read: half of the cache, and 8 bytes a slot.
//
// A unit is 32 slots of a sequence and key/value head, with all its rows, R = 4, 8 or 16 of them at a time.  The line of all
// units is cut into equal ranges for the warps of one CTA per SM.  The scores are kv4_mma.cuh's; a lane adds its rows'
// weights of four slots, and three exchanges leave every lane with the sum of one slot.
//
// More rows than R (TEAM: a prompt's last ones): a range belongs to a team of 2, 4 or 8 warps of a CTA, each of which
// takes every team-th group of rows through all of it; their sums meet in shared memory, a few units at a time, and
// are added in the groups' order.  (One warp taking the groups one after the other has its pipeline of copies and its
// queries anew for each: 8 groups over 16010 slots 62 us.)
//
// Measured: 24 sequences of 2080 slots, 32 heads over 8 of 128, 14.0 us (32 MB: 2.3 TB/s; 5 units a warp behind the same
// 5 us of launch and lookups that a single unit takes); a prompt's last 32 rows over 16010 slots 48.5 us (4.2 GFLOP, as
// two f16 parts each 8.4 on mma.sync).
//
// Either way a slot's weight is only ever touched by one warp at a time, in one order: no atomics, the same bits every time.
// The exponent's two terms are rounded at their own size in log2 units (half a step of f32 is 2^-19 from 32 on) before they are
// subtracted: with sums |scale| |q| |K| of 26 and log-sum-exps up to 32 a weight is off by up to 3.4 * 2^-20 of itself, 1.2 to 2.0 *
// 2^-20 root mean square (64 to 256 dimensions).
#include <climits>
#include <mutex>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4_mma.cuh"

namespace qmd {

struct Weigh4Args : AttnArgs {
    Units4Args units;
    float *weight;
    int team;  // warps to a range
};

template <int D, int R, bool TEAM>
struct Weigh4Cfg {
    using T = Tile4<D>;
    static constexpr int W = D == 256 ? (R == 4 ? 12 : 8) : R == 4 || D == 64 ? 16 : R == 8 ? 12 : 8;
    // (24 x 2080 slots, a row each: 14.0, 14.5, 15.0 us with 2, 3, 4; asking for a unit is some 60 instructions of one lane)
    static constexpr int STAGES = !TEAM ? 2 : D == 256 ? 3 : 4;
    static constexpr int RING = STAGES * Units4<D, STAGES, false>::STAGE;
    static constexpr int CHUNK = 8;  // units whose sums a team's warps lay down before they are added (4: 50.8, 8: 48.5 us)
    static constexpr int PART = TEAM ? CHUNK * 128 : 0;
    static constexpr int FIXED = W * (RING + 512 + PART) + W * (8 * STAGES + 8);
    static_assert(RING % (4 * D) == 0, "rings begin where the swizzle does");
    static_assert(FIXED + 256 + (QMD_KV_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits beside the sums of the most sequences");
};

// A barrier of one of a CTA's teams of warps.
__device__ __forceinline__ void team_barrier(int id, int warps)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id + 1), "r"(warps * 32) : "memory");
}

template <int D, int R, bool TEAM>
__global__ void __launch_bounds__(Weigh4Cfg<D, R, TEAM>::W * 32, 1)
    kv4_weigh_kernel(const Weigh4Args a, const __grid_constant__ Maps4 maps)
{
    using C = Weigh4Cfg<D, R, TEAM>;
    using T = Tile4<D>;
    using Q = Cols4<R>;
    constexpr int W = C::W, S = C::STAGES, LR = Q::LR;
    extern __shared__ __align__(1024) unsigned char smem[];
    float *s_part = reinterpret_cast<float *>(smem + W * C::RING);                   // [W][CHUNK][32]
    int2 *s_list = reinterpret_cast<int2 *>(smem + W * (C::RING + C::PART));          // [W][64]
    uint64_t *s_bar = reinterpret_cast<uint64_t *>(s_list + W * 64);  // [W][STAGES]
    int64_t *s_warp = reinterpret_cast<int64_t *>(s_bar + W * S);                     // [W]
    int *s_pre = reinterpret_cast<int *>(s_warp + W);                                 // [seqs + 1]

    const KvParams &p = a.kv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t bar0 = smem_addr(s_bar + warp * S);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < S; ++i)
            mbar_init(bar0 + 8 * i, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    pdl_launch_dependents();
    pdl_wait();
    if ((smem_addr(smem) & 1023u) != 0) {  // the copies' swizzle counts from 1024-byte boundaries
        atomicOr(p.err, (unsigned)ERRBIT_PLAN);
        return;
    }
    __syncwarp();

    // the 16-token blocks [lo, hi) of a sequence that any of its rows sees or owns
    auto first_of = [&](const KvSeq &q) { return row_begin(a, row_end(q, 0)) / KV_BLOCK; };
    auto end_of = [&](const KvSeq &q) { return (q.len + KV_BLOCK - 1) / KV_BLOCK; };
    auto units_of = [&](const KvSeq &q) {
        return q.n == 0 ? (int64_t)0 : (int64_t)(((end_of(q) + 1) >> 1) - (first_of(q) >> 1)) * p.heads;
    };
    const UnitLine line = unit_line<W>(p, units_of, s_warp, s_pre);
    if (line.too_many) {
        kv_index_error(p);
        return;
    }
    // the warps' (or teams') ranges, of all CTAs: short calls spread over the SMs
    const int team = TEAM ? a.team : 1, mate = TEAM ? warp & (team - 1) : 0;
    const int units = line.units, ranges = gridDim.x * (W / team);
    const int pw = (units + ranges - 1) / ranges;
    const int64_t u64 = (int64_t)(warp / team * (int)gridDim.x + (int)blockIdx.x) * pw;
    if (u64 >= units)
        return;
    int u = (int)u64;
    const int w1 = (int)min((int64_t)units, u64 + pw);
    bool dead = false;  // a copy did not land in time: what follows is left out

    Units4<D, S, false> kv = {a, a.units, maps, smem_addr(smem + warp * C::RING), bar0};
    kv.list = s_list + warp * 64;
    uint32_t lane_at[T::LOADS];
#pragma unroll
    for (int x = 0; x < T::LOADS; ++x)
        lane_at[x] = T::at(lane, x);

    const unsigned live = line_live(line);
    int pre, count;
    int s = line_find(line, p, u, s_pre, &pre, &count);
    const int of_head = count / a.by_heads;
    int head = (u - pre) / of_head, b0 = (u - pre) % of_head;
    while (u < w1) {
        const KvSeq sq = kv_seq(p, s);
        const int lo = first_of(sq), hi = end_of(sq), nb = ((hi + 1) >> 1) - (lo >> 1);
        const int cnt = min(nb - b0, w1 - u);
        const int first_blk = 2 * ((lo >> 1) + b0);
        const int own = max(0, sq.len - sq.n);  // the first of the rows' own slots
        // a slot's place among the weights, and whether it has one
        auto place = [&](int blk, int j, int64_t &at) {
            at = (int64_t)max(blk, 0) * KV_BLOCK + j % KV_BLOCK;
            return blk >= 0 && j < sq.len && j >= lo * KV_BLOCK;
        };
        for (int cg0 = 0; cg0 * R < sq.n * a.group; cg0 += team) {
            const int cg = cg0 + mate;
            const bool mine = cg * R < sq.n * a.group;  // (without TEAM always)
            const int rows = min(R, sq.n * a.group - cg * R);
            Query4<D, R> qf;
            float lse[LR];
            if (mine && !dead) {
                kv.begin(s, head, lo, hi, first_blk, cnt);
                qf.load(a.q, [&](int r) { return row_offset(a, sq.row0, head, cg * R + r, a.q_stride, D); }, rows, a.scale_log2e);
#pragma unroll
                for (int i = 0; i < LR; ++i)
                    lse[i] = a.lse[row_offset(a, sq.row0, head, cg * R + min(Q::row(i, t), rows - 1), a.group * p.heads, 1)] *
                             1.4426950408889634f;
            }
            auto query = [&](int i) { return make_uint4(qf.f[4 * i], qf.f[4 * i + 1], qf.f[4 * i + 2], qf.f[4 * i + 3]); };
            const int all_to = row_end(sq, cg * R / a.by_group);
            const int all_from = row_begin(a, row_end(sq, (cg * R + rows - 1) / a.by_group));
            // the lane's slot of a unit is that of h = t >> 1, e = t & 1
            const int my_slot = 16 * (t >> 1) + 8 * (t & 1) + g;

            for (int c0 = 0; c0 < cnt; c0 += TEAM ? C::CHUNK : cnt) {
                const int c1 = TEAM ? min(cnt, c0 + C::CHUNK) : cnt;
                for (int idx = c0; idx < c1 && mine && !dead; ++idx) {
                    if (!kv.next(idx)) {
                        kv.drain();
                        dead = true;
                        break;
                    }
                    const int pos = (first_blk + 2 * idx) * KV_BLOCK;
                    int64_t at;
                    bool here = false;
                    float old = 0.0f;
                    if constexpr (!TEAM) {
                        const int2 b = kv.blocks(idx);
                        here = place(t >> 1 ? b.y : b.x, pos + my_slot, at);
                        if (here && (cg > 0 || pos + my_slot < own))
                            old = a.weight[at];
                    }
                    const uint32_t codes = kv.stage();
                    const unsigned char *scales = smem + (codes + kv.SCALES - smem_addr(smem));
                    float sum[2][2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float sc[LR][2];
                        scores4<D, R>(sc, codes + h * 16 * T::ROW, scales + h * 16 * T::G * 2, lane_at, query, qf.scale);
                        const bool whole = pos >= all_from && pos + KV4_UNIT <= all_to;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            sum[h][e] = 0.0f;
#pragma unroll
                            for (int i = 0; i < LR; ++i) {
                                bool sees = Q::row(i, t) < rows;
                                if (!whole) {
                                    const int j = pos + 16 * h + 8 * e + g;
                                    const int end = row_end(sq, (cg * R + min(Q::row(i, t), rows - 1)) / a.by_group);
                                    sees &= j >= row_begin(a, end) && j < end;
                                }
                                const float w = ex2(sc[i][e] - lse[i]);
                                sum[h][e] += sees ? w : 0.0f;
                            }
                        }
                    }
                    kv.advance();
                    // over the four lanes of a slot, each ending with one of their four slots
                    float keep[2], give[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        keep[e] = t & 2 ? sum[1][e] : sum[0][e];
                        give[e] = t & 2 ? sum[0][e] : sum[1][e];
                        keep[e] += __shfl_xor_sync(0xffffffffu, give[e], 2);
                    }
                    const float one = (t & 1 ? keep[1] : keep[0]) + __shfl_xor_sync(0xffffffffu, t & 1 ? keep[0] : keep[1], 1);
                    if constexpr (TEAM)
                        s_part[(warp * C::CHUNK + idx - c0) * 32 + my_slot] = one;
                    else if (here)
                        a.weight[at] = old + one;
                }
                if constexpr (TEAM) {
                    // a warp of the team adds each unit's parts, in their order.  (One whose copies failed adds nothing.)
                    if (dead)
                        for (int i = 0; i < C::CHUNK; ++i)
                            s_part[(warp * C::CHUNK + i) * 32 + lane] = 0.0f;
                    team_barrier(warp / team, team);
                    for (int idx = c0 + mate; idx < c1; idx += team) {
                        const int j = (first_blk + 2 * idx) * KV_BLOCK + lane;
                        int64_t at;
                        if (place(kv.look_up_in(s, head, lo, hi, j / KV_BLOCK), j, at)) {
                            float sum = cg0 > 0 || j < own ? a.weight[at] : 0.0f;
                            for (int m = 0; m < team && (cg0 + m) * R < sq.n * a.group; ++m)
                                sum += s_part[((warp - mate + m) * C::CHUNK + idx - c0) * 32 + lane];
                            a.weight[at] = sum;
                        }
                    }
                    team_barrier(warp / team, team);
                }
            }
            if (!TEAM && dead)
                return;
        }
        u += cnt;
        b0 = 0;
        if (u < w1 && ++head == p.heads) {
            head = 0;
            s = line_next(p, live, s, s_pre);
        }
    }
}

template <int D, int R, bool TEAM>
static qmd_status launch_weigh4(const Weigh4Args &a, const DeviceInfo &dev, cudaStream_t s)
{
    using C = Weigh4Cfg<D, R, TEAM>;
    const size_t smem = C::FIXED + ((size_t)a.kv.seqs + 1) * sizeof(int);
    if (smem + 256 > (size_t)dev.smem_optin)
        return QMD_ERR_SHAPE;
    {
        static std::mutex mu;
        static bool opted[64] = {false};
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[dev.device]) {
            const cudaError_t e = cudaFuncSetAttribute(kv4_weigh_kernel<D, R, TEAM>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       dev.smem_optin - 256);
            if (e != cudaSuccess)
                return fail(QMD_ERR_LAUNCH, "kv4_weigh smem attribute", e);
            opted[dev.device] = true;
        }
    }
    Maps4 maps = {};
    const qmd_status st = kv4_map(&maps.k, a.kv.k, a.kv, D, a.units.pairs);
    if (st != QMD_OK)
        return st;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)dev.sm_count);
    cfg.blockDim = dim3(C::W * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_weigh_kernel<D, R, TEAM>, a, maps);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv4_weigh launch", e);
}

qmd_status launch_kv4_weigh(const Kv4Params &kv, int head_dim, const float *q, int64_t q_stride, int q_heads,
                            float scale, int64_t window, const float *lse, float *weight, const DeviceInfo &dev,
                            cudaStream_t s)
{
    Weigh4Args a;
    static_cast<AttnArgs &>(a) = attn_args(kv, q, q_stride, q_heads, scale, window, nullptr, 0, nullptr, dev);
    a.lse = const_cast<float *>(lse);
    a.units = {kv.ks4, nullptr, kv.page_blocks % 2 == 0};
    a.weight = weight;
    // the least of 4, 8, 16 (8 at 256 dimensions) that holds a sequence's rows of one key/value head; for more, a team
    // of as many warps as there are groups of them, to a power of two, up to 8 (a CTA of the widest instance)
    const int64_t rows = (int64_t)a.group * kv.max_q, most = head_dim == 256 ? 8 : 16;
    a.team = 1;
    while (a.team < 8 && a.team * most < rows)
        a.team *= 2;
    if (head_dim == 64)
        return rows <= 4    ? launch_weigh4<64, 4, false>(a, dev, s)
               : rows <= 8  ? launch_weigh4<64, 8, false>(a, dev, s)
               : rows <= 16 ? launch_weigh4<64, 16, false>(a, dev, s)
                            : launch_weigh4<64, 16, true>(a, dev, s);
    if (head_dim == 128)
        return rows <= 4    ? launch_weigh4<128, 4, false>(a, dev, s)
               : rows <= 8  ? launch_weigh4<128, 8, false>(a, dev, s)
               : rows <= 16 ? launch_weigh4<128, 16, false>(a, dev, s)
                            : launch_weigh4<128, 16, true>(a, dev, s);
    return rows <= 4   ? launch_weigh4<256, 4, false>(a, dev, s)
           : rows <= 8 ? launch_weigh4<256, 8, false>(a, dev, s)
                       : launch_weigh4<256, 8, true>(a, dev, s);
}

}  // namespace qmd
