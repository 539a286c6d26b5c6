// kv4_weigh.cu -- the attention weight that each token of the 4-bit cache gets.
//
// weight_j = (weight_j, or 0 where j is one of the call's own rows) + sum over the rows that see j and the query
// heads of the key/value head of e^(s_j - lse), s_j = scale q . K_j and lse attention's.  With the log-sum-exp
// known there is nothing to keep from one slot to the next and no value to read: half of the cache, and 8 bytes a slot.
//
// A unit is 32 slots of a sequence and key/value head, with all its rows.  The line of all units is cut into
// equal ranges for one CTA per SM and its warps; a range takes its rows in groups of R = 4, 8 or 16, one after the
// other (their keys come from L2 again), so a slot's weight is only ever touched by one warp, in one order: no atomics,
// the same bits every time.  The scores are kv4_mma.cuh's; a lane adds its rows' weights of four slots, and
// three exchanges leave every lane with the sum of one slot.
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
};

template <int D, int R>
struct Weigh4Cfg {
    using T = Tile4<D>;
    static constexpr int W = D == 256 ? (R == 4 ? 12 : 8) : R == 4 || D == 64 ? 16 : R == 8 ? 12 : 8;
    static constexpr int STAGES = D == 256 ? 3 : 4;
    static constexpr int RING = STAGES * Units4<D, STAGES, false>::STAGE;
    static constexpr int FIXED = W * (RING + 512) + W * (8 * STAGES + 8);
    static_assert(RING % (4 * D) == 0, "rings begin where the swizzle does");
    static_assert(FIXED + 256 + (QMD_KV_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits beside the sums of the most sequences");
};

template <int D, int R>
__global__ void __launch_bounds__(Weigh4Cfg<D, R>::W * 32, 1)
    kv4_weigh_kernel(const Weigh4Args a, const __grid_constant__ Maps4 maps)
{
    using C = Weigh4Cfg<D, R>;
    using T = Tile4<D>;
    using Q = Cols4<R>;
    constexpr int W = C::W, S = C::STAGES, LR = Q::LR;
    extern __shared__ __align__(1024) unsigned char smem[];
    int2 *s_list = reinterpret_cast<int2 *>(smem + W * C::RING);  // [W][64]
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
    // the warps' ranges, of all CTAs: short calls spread over the SMs
    const int units = line.units, warps = gridDim.x * W;
    const int pw = (units + warps - 1) / warps;
    int64_t u64 = (int64_t)(warp * (int)gridDim.x + (int)blockIdx.x) * pw;
    if (u64 >= units)
        return;
    int u = (int)u64;
    const int w1 = (int)min((int64_t)units, u64 + pw);

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
        for (int cg = 0; cg * R < sq.n * a.group; ++cg) {
            kv.begin(s, head, lo, hi, first_blk, cnt);
            const int rows = min(R, sq.n * a.group - cg * R);
            Query4<D, R> qf;
            qf.load(a.q, [&](int r) { return row_offset(a, sq.row0, head, cg * R + r, a.q_stride, D); }, rows, a.scale_log2e);
            auto query = [&](int i) { return make_uint4(qf.f[4 * i], qf.f[4 * i + 1], qf.f[4 * i + 2], qf.f[4 * i + 3]); };
            float lse[LR];
#pragma unroll
            for (int i = 0; i < LR; ++i)
                lse[i] = a.lse[row_offset(a, sq.row0, head, cg * R + min(Q::row(i, t), rows - 1), a.group * p.heads, 1)] *
                         1.4426950408889634f;
            const int all_to = row_end(sq, cg * R / a.by_group);
            const int all_from = row_begin(a, row_end(sq, (cg * R + rows - 1) / a.by_group));

            for (int idx = 0; idx < cnt; ++idx) {
                if (!kv.next(idx)) {
                    kv.drain();
                    return;
                }
                const int pos = (first_blk + 2 * idx) * KV_BLOCK;
                // this lane's slot: that of h = t >> 1, e = t & 1
                const int mine = pos + 16 * (t >> 1) + 8 * (t & 1) + g, blk = t >> 1 ? kv.blocks(idx).y : kv.blocks(idx).x;
                float *at = a.weight + (int64_t)max(blk, 0) * KV_BLOCK + 8 * (t & 1) + g;
                const bool here = blk >= 0 && mine < sq.len && mine >= lo * KV_BLOCK;
                const float old = here && (cg > 0 || mine < own) ? *at : 0.0f;

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
                if (here)
                    *at = old + one;
            }
        }
        u += cnt;
        b0 = 0;
        if (u < w1 && ++head == p.heads) {
            head = 0;
            s = line_next(p, live, s, s_pre);
        }
    }
}

template <int D, int R>
static qmd_status launch_weigh4(const Weigh4Args &a, const DeviceInfo &dev, cudaStream_t s)
{
    using C = Weigh4Cfg<D, R>;
    const size_t smem = C::FIXED + ((size_t)a.kv.seqs + 1) * sizeof(int);
    if (smem + 256 > (size_t)dev.smem_optin)
        return QMD_ERR_SHAPE;
    {
        static std::mutex mu;
        static bool opted[64] = {false};
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[dev.device]) {
            const cudaError_t e = cudaFuncSetAttribute(kv4_weigh_kernel<D, R>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_weigh_kernel<D, R>, a, maps);
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
    const int64_t rows = (int64_t)a.group * kv.max_q;
    if (head_dim == 64)
        return rows <= 4   ? launch_weigh4<64, 4>(a, dev, s)
               : rows <= 8 ? launch_weigh4<64, 8>(a, dev, s)
                           : launch_weigh4<64, 16>(a, dev, s);
    if (head_dim == 128)
        return rows <= 4   ? launch_weigh4<128, 4>(a, dev, s)
               : rows <= 8 ? launch_weigh4<128, 8>(a, dev, s)
                           : launch_weigh4<128, 16>(a, dev, s);
    return rows <= 4 ? launch_weigh4<256, 4>(a, dev, s) : launch_weigh4<256, 8>(a, dev, s);
}

}  // namespace qmd
