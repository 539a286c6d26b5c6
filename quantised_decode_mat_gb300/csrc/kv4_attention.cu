// kv4_attention.cu -- attention of a decode step's rows over the paged 4-bit key/value cache.
//
// Per row and query head, over the slots j that it sees:  out = sum_j e^(s_j - m) V_j / sum_j e^(s_j - m),
// s_j = scale q . K_j, lse = m + ln sum_j e^(s_j - m).  One pass over the cache.
//
// Work as in kv_attention.cu: an item is up to R = 4, 8 or 16 query rows of one sequence and key/value head, a
// unit 32 slots of an item; the line of all units is cut into equal ranges for one CTA per SM and its warps, and
// items that were cut are joined in the CTA and, through the workspace, between CTAs.
//
// A unit.  S = K Q^T as kv4_mma.cuh has it.  Then O^T += V^T P^T, the head's dimensions the 16 rows: the weights
// move from the first product's layout to the second's by 8 x 8 transposes between lanes (movmatrix).  A value
// scale belongs to a slot and a group of 32 dimensions, so the weights are multiplied by it, for each group
// its own operand, as two f16 parts of 11 bits.
//
// Reference.  Weights are taken over 2^ref, an integer for each query row, such that weight times |scale| stays
// under 2^16 (what f16 holds) and weights under 2^46; it moves up only when one of these is passed, to leave
// the largest product in (2^12, 2^14] (then every sum is rescaled, exactly).  What two f16 parts lose is then
// at most 2^-22 of a product, or, where the parts are subnormal and each is rounded to a multiple of 2^-24, 2^-36 of the
// largest that the row has met.  (A scale without weight does not count.)  Where slots of scale zero have the weight, the
// reference leaves theirs at 2^43 at least, and 2^-67 of it is lost at most.
//
// Loads: per unit a warp asks for the keys' and the values' codes by tiled tensor copies (swizzled, so that
// ldmatrix meets no bank conflicts) and for their scales by plain bulk copies, into a ring of STAGES units.
// A page of an even number of 16-token blocks holds whole units: one copy of 32 rows instead of two of 16.  Rings of two
// units and as many warps as registers allow: at 128 dimensions and 4 rows 16 warps 72.4 us, 12 with two or three
// units 76.0 (40 sequences of 1500-14011 tokens); 8 rows 12 warps 68.4, 8 warps 76.9 (24 x 8100, 8 heads to one).
//
// Measured: those 40 sequences (32 heads over 8 of 128, 343 MB) 74 us, 4.6 TB/s, 0.68 of the copy rate: 9 us of lookups
// and joins, then 5.4 TB/s.  Instructions bound it: 653 a unit, of them 288 that make codes f16 (without these 64 us;
// without either product 62, which is the copies).  One sequence of 32768 20.7 us, of 19 5.2 us; 16 rows to a head (12 x
// 8100, 4 rows each) 66.8 us.
#include <climits>
#include <mutex>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4_mma.cuh"

namespace qmd {

struct Attn4Args : AttnArgs {
    Units4Args units;
};

template <int D, int R>
struct Attn4Cfg {
    using T = Tile4<D>;
    static constexpr int W = D == 256 ? (R == 4 ? 8 : 6) : R == 4 ? 16 : D == 64 ? (R == 8 ? 12 : 8) : R == 8 ? 12 : 8;
    static constexpr int STAGES = D == 64 ? 4 : D == 256 || R != 8 ? 2 : 3;
    static constexpr int RING = STAGES * Units4<D, STAGES, true>::STAGE;
    static constexpr int SLOT = R * D * 4;
    static constexpr bool QS = D == 256 || (D == 128 && R == 16);  // query fragments in shared memory
    static constexpr int QN = Query4<D, R>::N;
    static constexpr int QBYTES = QS ? QN * 128 : 0;
    static_assert(RING >= SLOT, "a warp's last part lies in its ring");
    static_assert(RING % (4 * D) == 0, "rings begin where the swizzle does");
    static constexpr int BAR = 8 * STAGES;
    static constexpr int FIXED = W * (RING + SLOT + QBYTES + 512 + 32) + 2 * W * R * 8 + (W + 1) * 32 + W * (BAR + 8) + 8 + 16;
    static_assert(FIXED + 256 + (QMD_KV_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits beside the sums of the most sequences");
};

struct Item4 {  // what a warp needs of its item after its units
    int row0, n;           // the sequence's first row and rows
    int units, at, count;  // the item's units, the first of them in the warp's range, and how many
    int rows;              // query rows
    unsigned live;         // the sequences that have units, of up to 32
    int pad;
};

constexpr float A4_TOP = 60000.0f;  // how large a weight times scale may get
constexpr float A4_LOG = 14.0f;     // and (log2) may be where the reference moves
constexpr float A4_WEIGHT = 44.0f;  // likewise a weight alone, whose limit is 2^2 above

// The least k with |d| < 2^k, for an f16 scale; 16 where it is not finite.
__device__ __forceinline__ float scale4_log2(float d)
{
    return (float)min((int)(__float_as_uint(d) >> 23 & 255u) - 126, 16);
}

template <int D, int R>
__global__ void __launch_bounds__(Attn4Cfg<D, R>::W * 32, 1)
    kv4_attention_kernel(const Attn4Args a, const __grid_constant__ Maps4 maps)
{
    using C = Attn4Cfg<D, R>;
    using T = Tile4<D>;
    using Q = Cols4<R>;
    constexpr int W = C::W, S = C::STAGES, G = T::G, LR = Q::LR, NT = Q::NT;
    extern __shared__ __align__(1024) unsigned char smem[];
    constexpr int SLOTS = W * C::RING, QS0 = SLOTS + W * C::SLOT;
    int2 *s_list = reinterpret_cast<int2 *>(smem + QS0 + W * C::QBYTES);    // [W][64]
    Item4 *s_item = reinterpret_cast<Item4 *>(s_list + W * 64);             // [W]
    float2 *s_ml = reinterpret_cast<float2 *>(s_item + W);                  // [W][2][R] maximum, weight sum
    Job *s_job = reinterpret_cast<Job *>(s_ml + 2 * W * R);                 // [1 + W]
    uint64_t *s_bar = reinterpret_cast<uint64_t *>(s_job + W + 1);          // [W][STAGES]
    int64_t *s_warp = reinterpret_cast<int64_t *>(s_bar + W * S);           // [W]
    int *s_last = reinterpret_cast<int *>(s_warp + W);                      // [2]
    int *s_range = s_last + 2;                                              // u0, span, pw, per
    int *s_pre = s_range + 4;                                               // [seqs + 1] units before a sequence

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
        s_job[1 + warp].rows = 0;
        if (warp == 0)
            s_job[0].rows = 0;
    }
    pdl_launch_dependents();
    pdl_wait();
    if ((smem_addr(smem) & 1023u) != 0) {  // the copies' swizzle counts from 1024-byte boundaries
        atomicOr(p.err, (unsigned)ERRBIT_PLAN);
        return;
    }
    __syncwarp();

    // ---- the line of units, this CTA's range, this warp's range ---------------------------------
    auto units_in = [](const Group &gr) { return max(1, ((gr.hi + 1) >> 1) - (gr.lo >> 1)); };
    auto units_of = [&](const KvSeq &q) {
        int64_t u = 0;
        for (int cg = 0; cg * R < q.n * a.group; ++cg)
            u += units_in(group_of<R>(a, q, cg));
        return u * p.heads;
    };
    const UnitLine line = unit_line<W>(p, units_of, s_warp, s_pre);
    const int units = line.units;
    if (line.too_many) {  // more units than a launch counts
        kv_index_error(p);
        return;
    }
    // at least a unit for every warp, so that short items are cut inside a CTA, not between CTAs
    const int per = max(W, (units - 1) / a.by_grid + 1);
    if ((int64_t)blockIdx.x * per >= units)
        return;
    const int u0 = blockIdx.x * per;
    const int span = min(units - u0, per), pw = (span + W - 1) / W;
    if (tid == 0)
        s_range[0] = u0, s_range[1] = span, s_range[2] = pw, s_range[3] = per;  // (the joins read them again: registers are few in between)
    const unsigned live = line_live(line);
    if (lane == 0)
        s_item[warp].live = live;
    int u = warp * pw;  // from here on counted from u0
    const int w1 = min(span, u + pw);

    Units4<D, S, true> kv = {a, a.units, maps, smem_addr(smem + warp * C::RING), bar0};
    kv.list = s_list + warp * 64;
    uint32_t lane_at[T::LOADS];
#pragma unroll
    for (int x = 0; x < T::LOADS; ++x)
        lane_at[x] = T::at(lane, x);
    bool dead = false;                // a copy did not land in time

    int s = 0, cg = 0, head = 0, b0 = 0;  // the item of unit u, and the unit's place in it
    if (u < w1) {
        int pre, count;
        s = line_find(line, p, u0 + u, s_pre, &pre, &count);
        int rem = u0 + u - pre;
        const KvSeq sq = kv_seq(p, s);
        // the row groups of a head lie together: they read the same keys and values
        const int of_head = count / a.by_heads;
        head = rem / of_head;
        rem -= head * of_head;
        for (;; ++cg) {
            const int nb = units_in(group_of<R>(a, sq, cg));
            if (rem < nb)
                break;
            rem -= nb;
        }
        b0 = rem;
    }
    while (u < w1) {
        const KvSeq sq = kv_seq(p, s);
        const Group gr = group_of<R>(a, sq, cg);
        const int lo2 = gr.lo >> 1, hi2 = (gr.hi + 1) >> 1;
        int real;  // units of this item in the range that hold slots
        {
            const int nb = max(1, hi2 - lo2), cnt = min(nb - b0, w1 - u);
            real = min(cnt, hi2 - lo2 - b0);
            __syncwarp();  // every lane has read the last item's
            if (lane == 0)
                s_item[warp] = {sq.row0, sq.n, nb, b0, cnt, gr.rows, s_item[warp].live};  // (registers are few in between)
            __syncwarp();
        }

        const int first_blk = 2 * (lo2 + b0);
        kv.begin(s, head, gr.lo, gr.hi, first_blk, real);
        Query4<D, R> qf;
        qf.load(a.q, [&](int r) { return row_offset(a, sq.row0, head, cg * R + r, a.q_stride, D); }, gr.rows, a.scale_log2e);
        uint4 *q_keep = reinterpret_cast<uint4 *>(smem + QS0 + warp * C::QBYTES) + lane;
        if constexpr (C::QS) {
#pragma unroll
            for (int i = 0; i < C::QN / 4; ++i)
                q_keep[i * 32] = make_uint4(qf.f[4 * i], qf.f[4 * i + 1], qf.f[4 * i + 2], qf.f[4 * i + 3]);
        }
        auto query = [&](int i) {
            if constexpr (C::QS)
                return q_keep[i * 32];
            else
                return make_uint4(qf.f[4 * i], qf.f[4 * i + 1], qf.f[4 * i + 2], qf.f[4 * i + 3]);
        };
        // slots in [all_from, all_to) are seen by every row of the group
        const int all_to = row_end(sq, cg * R / a.by_group);
        const int all_from = row_begin(a, row_end(sq, (cg * R + gr.rows - 1) / a.by_group));

        float o[NT][D / 16][4];
        float ref[LR], l[LR];
#pragma unroll
        for (int i = 0; i < LR; ++i)
            ref[i] = ATT_NONE, l[i] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
                o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.0f;

        for (int idx = 0; idx < real; ++idx) {
            if (!kv.next(idx)) {
                dead = true;
                break;
            }
            const uint32_t codes = kv.stage();
            const unsigned char *scales = smem + (codes + kv.SCALES - smem_addr(smem));
            float sc[2][LR][2];
#pragma unroll
            for (int h = 0; h < 2; ++h)
                scores4<D, R>(sc[h], codes + h * 16 * T::ROW, scales + h * 16 * G * 2, lane_at, query, qf.scale);
            uint32_t dv[2][2][G / 2];  // the values' scales, of slots 16 h + g + 8 e
#pragma unroll
            for (int h = 0; h < 2; ++h)
                load_scales<D>(dv[h], scales + T::SCALES + h * 16 * G * 2, g);

            const int pos = (first_blk + 2 * idx) * KV_BLOCK;
            unsigned poison = 0;
            if (pos < all_from || pos + KV4_UNIT > all_to || kv.misses(idx)) {
                const int2 at = kv.blocks(idx);
                // some slot is not there, or not seen by some row: bit 2 h + e of these is the lane's slot (h, e)
                unsigned any = 0, all = 15, bad = 0;
#pragma unroll
                for (int i = 0; i < LR; ++i) {
                    const int end = row_end(sq, (cg * R + min(Q::row(i, t), gr.rows - 1)) / a.by_group) - (pos + g);
                    const int begin = row_begin(a, end + pos + g) - (pos + g);
                    unsigned sees = 0;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if ((h ? at.y : at.x) >= 0 && 16 * h + 8 * e >= begin && 16 * h + 8 * e < end)
                                sees |= 1u << (2 * h + e);
                            else
                                sc[h][i][e] = -INFINITY;
                    any |= sees;
                    all &= sees;
                    poison |= sees << (4 * i);
                }
                // a scale that is not finite must not reach rows that do not see its slot: where some of the lane's do
                // not, it is 0 and the others' values are made NaN below
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const unsigned bit = 1u << (2 * h + e);
#pragma unroll
                        for (int i = 0; i < G / 2; ++i) {
                            const uint32_t top = dv[h][e][i] & 0x7c007c00u;
                            if ((top & 0x7c00u) == 0x7c00u || top >> 16 == 0x7c00u)
                                bad |= bit;
                        }
                        if (!(any & bit) || (bad & ~all & bit))
#pragma unroll
                            for (int i = 0; i < G / 2; ++i)
                                dv[h][e][i] = 0;
                    }
                poison &= (bad & ~all) * 0x1111u;
            }
            // Is a row's reference passed?  (By a bound on every weight times scale of this lane's four slots.)
            __half2 most = __habs2(as_half2(dv[0][0][0]));
#pragma unroll
            for (int i = 1; i < 2 * G; ++i)
                most = __hmax2(most, __habs2(as_half2(dv[i / G][i / (G / 2) & 1][i % (G / 2)])));
            const float2 most2 = __half22float2(most);
            const float most1 = fmaxf(most2.x, most2.y);
            bool up = false;
#pragma unroll
            for (int i = 0; i < LR; ++i) {
                const float x = fmaxf(fmaxf(sc[0][i][0], sc[0][i][1]), fmaxf(sc[1][i][0], sc[1][i][1])) - ref[i];
                up |= x > A4_WEIGHT + 2.0f || ex2(x) * most1 > A4_TOP;
            }
            if (__any_sync(0xffffffffu, up)) {
                float lg[2][2];  // the slots' largest |scale|: the least k with |d| < 2^k, at most 2^16
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        __half2 m = __habs2(as_half2(dv[h][e][0]));
#pragma unroll
                        for (int i = 1; i < G / 2; ++i)
                            m = __hmax2(m, __habs2(as_half2(dv[h][e][i])));
                        const float2 m2 = __half22float2(m);
                        lg[h][e] = fmaxf(scale4_log2(fmaxf(m2.x, m2.y)) - A4_LOG, -A4_WEIGHT);
                    }
                float f[LR];
#pragma unroll
                for (int i = 0; i < LR; ++i) {
                    float top = fmaxf(fmaxf(sc[0][i][0] + lg[0][0], sc[0][i][1] + lg[0][1]),
                                      fmaxf(sc[1][i][0] + lg[1][0], sc[1][i][1] + lg[1][1]));
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    const float now = top > ref[i] ? ceilf(top) : ref[i];
                    f[i] = pow2(ref[i] - now);
                    ref[i] = now;
                    l[i] *= f[i];
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[n][i][e] *= f[R == 4 ? 0 : 2 * n + (e & 1)];
            }
            float w[2][LR][2];
#pragma unroll
            for (int i = 0; i < LR; ++i) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        w[h][i][e] = ex2(sc[h][i][e] - ref[i]);
                l[i] += (w[0][i][0] + w[0][i][1]) + (w[1][i][0] + w[1][i][1]);
            }
            if (poison) {
#pragma unroll
                for (int i = 0; i < LR; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (poison >> (4 * i + 2 * h + e) & 1)
                                w[h][i][e] = NAN;
            }

            // the second product: V^T P^T, 16 slots at a time, for each group its own weights
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t v[2][G];
                load_words<D, true>(v, codes + T::CODES + h * 16 * T::ROW, lane_at);
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    uint32_t x[4], y[4];
                    unpack4_f16(x, v[0][i]);
                    unpack4_f16(y, v[1][i]);
                    const uint32_t first[4] = {x[0], x[1], y[0], y[1]}, second[4] = {x[2], x[3], y[2], y[3]};
                    uint32_t q[LR][2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float2 two = halves(dv[h][e][i / 2]);
                        const float d = i & 1 ? two.y : two.x;
#pragma unroll
                        for (int j = 0; j < LR; ++j) {
                            const float x = w[h][j][e] * d, hi = first_bits(x);
                            q[j][e] = pack_f16(hi, x - hi);
                        }
                    }
                    if constexpr (R == 4) {
                        const uint32_t b0 = transpose_8x8(q[0][0]), b1 = transpose_8x8(q[0][1]);
                        mma_16816(o[0][2 * i], first, b0, b1);
                        mma_16816(o[0][2 * i + 1], second, b0, b1);
                    } else {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            uint32_t bh[2], bl[2];  // the first parts of two rows, and the second
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t q0 = q[(2 * n) % LR][e], q1 = q[(2 * n + 1) % LR][e];
                                bh[e] = transpose_8x8(__byte_perm(q0, q1, 0x5410));
                                bl[e] = transpose_8x8(__byte_perm(q0, q1, 0x7632));
                            }
                            mma_16816(o[n][2 * i], first, bl[0], bl[1]);
                            mma_16816(o[n][2 * i + 1], second, bl[0], bl[1]);
                            mma_16816(o[n][2 * i], first, bh[0], bh[1]);
                            mma_16816(o[n][2 * i + 1], second, bh[0], bh[1]);
                        }
                    }
                }
            }
            kv.advance();
        }
        if (dead) {
            kv.drain();  // the rest is left out
            break;
        }

        // ---- the item's part: finished, or laid down for the join --------------------------------
        const Item4 it = s_item[warp];
        const int row0 = it.row0, nb = it.units, cnt = it.count;
        b0 = it.at;
        const bool done = b0 == 0 && cnt == nb;
        const int part = b0 > 0 ? 0 : 1;
        float *dst = reinterpret_cast<float *>(part == 0 ? smem + SLOTS + warp * C::SLOT : smem + warp * C::RING);
        if (part == 1 && !done)
            __syncwarp();  // every lane has read the ring
#pragma unroll
        for (int i = 0; i < LR; ++i) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1)
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            const int r = Q::row(i, t);
            if (!done && g == 0)
                s_ml[(warp * 2 + part) * R + r] = make_float2(ref[i], l[i]);
            if (done && r >= it.rows)
                continue;
            if (done && a.lse && g == 0)
                store_lse(a, row0, head, cg * R + r, ref[i], l[i]);
            const float f = done ? (l[i] == 0.0f ? 0.0f : 1.0f / l[i]) : 1.0f;
            float *to = (done ? a.out + row_offset(a, row0, head, cg * R + r, a.out_stride, D) : dst + r * D) + 4 * g;
#pragma unroll
            for (int j = 0; j < G; ++j) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float(&c)[4] = o[R == 4 ? 0 : i / 2][2 * j + (e >> 1)];
                    y[e] = (R == 4 ? c[2 * (e & 1)] + c[2 * (e & 1) + 1] : c[2 * (e & 1) + (i & 1)]) * f;
                }
                store_f32(to + 32 * j, y);
            }
        }
        // the item's first cut in this CTA makes the job of joining it
        if (!done && lane == 0 && (part == 1 || warp == 0)) {
            Job &j = s_job[part == 1 ? 1 + warp : 0];
            j.start = u - b0;
            j.end = u - b0 + nb;
            j.row0 = row0;
            j.first = cg * R;
            j.head = head;
            j.rows = it.rows;
        }
        u += cnt;
        b0 = 0;
        if (u < w1 && ++cg * R >= it.n * a.group) {  // on to the next head, or the next sequence with rows
            cg = 0;
            if (++head == p.heads) {
                head = 0;
                s = line_next(p, it.live, s, s_pre);
            }
        }
    }
    __syncthreads();
    join_parts<D, R, W, true>(a, s_job, s_ml, s_last, smem, C::RING, SLOTS, C::SLOT, s_range[0], s_range[1], s_range[2],
                              s_range[3]);
}

template <int D, int R>
static qmd_status launch_att4(const Attn4Args &a, const DeviceInfo &dev, cudaStream_t s)
{
    using C = Attn4Cfg<D, R>;
    const size_t smem = C::FIXED + ((size_t)a.kv.seqs + 1) * sizeof(int);
    if (smem + 256 > (size_t)dev.smem_optin)
        return QMD_ERR_SHAPE;
    {
        static std::mutex mu;
        static bool opted[64] = {false};
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[dev.device]) {
            const cudaError_t e = cudaFuncSetAttribute(kv4_attention_kernel<D, R>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, dev.smem_optin - 256);
            if (e != cudaSuccess)
                return fail(QMD_ERR_LAUNCH, "kv4_attention smem attribute", e);
            opted[dev.device] = true;
        }
    }
    Maps4 maps;
    qmd_status st = kv4_map(&maps.k, a.kv.k, a.kv, D, a.units.pairs);
    if (st == QMD_OK)
        st = kv4_map(&maps.v, a.kv.v, a.kv, D, a.units.pairs);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_attention_kernel<D, R>, a, maps);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv4_attention launch", e);
}

qmd_status launch_kv4_attention(const Kv4Params &kv, int head_dim, const float *q, int64_t q_stride, int q_heads,
                                float scale, int64_t window, float *out, int64_t out_stride, float *lse, void *ws,
                                const DeviceInfo &dev, cudaStream_t s)
{
    Attn4Args a;
    static_cast<AttnArgs &>(a) = attn_args(kv, q, q_stride, q_heads, scale, window, out, out_stride, ws, dev);
    a.lse = lse;
    a.units = {kv.ks4, kv.vs4, kv.page_blocks % 2 == 0};
    // rows per item: 4 or 8 where that holds a sequence's rows of one key/value head; of more, 16 where they make whole
    // pairs of groups of 8 (16 rows, 12 x 8100: 66.5 us, 69.8 in eights; 32 rows, 8 x 3000: 41.4 and 42.5), else 8 (20 rows, 8 x
    // 3000: 34.1 us, 39.6 in sixteens, of which the last would be more than half empty)
    const int64_t rows = (int64_t)a.group * kv.max_q;
    const bool eights = (rows + 7) / 8 & 1;
    if (head_dim == 64)
        return rows <= 4 ? launch_att4<64, 4>(a, dev, s) : eights ? launch_att4<64, 8>(a, dev, s) : launch_att4<64, 16>(a, dev, s);
    if (head_dim == 128)
        return rows <= 4 ? launch_att4<128, 4>(a, dev, s)
               : eights  ? launch_att4<128, 8>(a, dev, s)
                         : launch_att4<128, 16>(a, dev, s);
    return rows <= 4 ? launch_att4<256, 4>(a, dev, s) : launch_att4<256, 8>(a, dev, s);
}

}  // namespace qmd
