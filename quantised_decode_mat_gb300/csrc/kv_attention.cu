// kv_attention.cu -- attention of a decode step's rows over the paged 8-bit key/value cache.
//
// "Language models on the device: the cajeta-llm kernels", §2.5: attention over the key/value
// cache, 1, 4 or 8 query heads to a key/value head.  Per row at position p and query head, over the
// positions j that it sees:  out = sum_j e^(s_j - m) V[j] / sum_j e^(s_j - m),  s_j = scale q . K[j].
//
// One pass over the cache, which bounds it: a decode row does 2 multiply-adds per byte read.
//
// Work.  An item is up to R = 4, 8 or 16 query rows (rows x heads that share a key/value head) of one
// sequence and one key/value head; a unit is one block of 16 positions of an item.  The units of
// all items stand in one line (sequence, head, row group, block), which is cut into equal ranges
// for one CTA per SM and these into equal ranges for the CTA's warps, whatever the sequences'
// lengths: no work list, no launch that depends on lengths held on the device.  An item inside one
// warp's range is finished by that warp; one cut inside a CTA is joined through shared memory; one
// cut between CTAs through the workspace, by the CTA that comes last (a counter per CTA; nobody
// waits).  The joins add in the order of the parts, so the bits do not depend on who comes last.
//
// A unit.  Both products run on mma.sync m16n8k16 (f16 in, f32 sums).  f32 values go in as two f16
// parts, the first 11 bits and the next 11, and the codes, integers of 8 bits, enter exactly.  Up to 4
// query rows (R = 4): S^T = K Q^T and O^T += V^T P^T, positions or the head's dimensions the 16 rows and
// query rows the 8 columns, a column to each part (the second 2^11 times larger); P^T moves from the
// first product's layout to the second's by an 8 x 8 transpose between lanes (movmatrix).  More
// (R = 8, 16): S = Q K^T and O += P V, the parts as rows 0-7 and 8-15, or as two products into the
// same sums; these are half as many registers, and P is already laid out as the operand it becomes.
// (tcgen05 wants its operands in shared memory and 128 rows: the codes would be widened and written
// there at twice the bytes for rows that a decode step does not have.)  The order of the head's
// dimensions inside a product is free, so a lane takes 16 neighbouring bytes of a key for four
// products, and of four values' rows 16 neighbouring dimensions; the sums then hold 16 neighbouring
// outputs.  A code c becomes an f16 by bytes: c + 128 under the exponent byte 0x64 is 1024 + c + 128,
// less 1152.
//
// Each query row has two references.  The sum of weights is kept over 2^m, m a running maximum of the
// scores s (log2 units, rounded up to an integer).  The sums of values are kept over 2^(m + e): with d < 2^k
// a block's scale, 2^(m + e) is at or above the largest 2^(s + k) met so far.  What f16 holds is thus small
// only against what the row has already summed: a large scale without weight takes no bits from a small
// one that has it (one reference for all scales lost 1.5e-2 of the result at scales 2^24 apart).  The
// references move only when a weight passes one of them by more than 2^8 (then every sum is rescaled);
// until then weights are at most 2^8, which f32 and the f16 parts have room for.
//
// Loads: a lane asks for each block's keys and values by tiled tensor copies (TMA) into a ring of
// STAGES blocks per warp in shared memory, 4 KB a block (head_dim 128), an mbarrier to a stage.  The
// copies swizzle the rows' 16-byte pieces, and rows are dealt to lanes so that the eight lanes that
// read shared memory together meet eight different pieces: no bank conflicts.  Page numbers and
// scales are looked up 32 blocks at a time, a lane each, a chunk ahead.
//
// Measured: 48 sequences of 2500-12301 tokens (32 heads over 8 of 128) 123-125 us, 6.3 TB/s, 0.94 of the
// copy rate; per-lane cp.async instead of tensor copies 166 us, with or without the arithmetic.  One
// sequence of 32768 22.2 us, of 17 8.5 us: lookups that wait for each other, and the joins.  16 rows to a
// head (16 x 8100 tokens, 4 rows each) 75.5 us against 40 for the bytes: 8 warps to an SM are few for it.
#include <climits>
#include <cstring>
#include <mutex>

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"
#include "tensor_map.h"

namespace qmd {

// n / d for 0 <= n < 2^31 and a divisor that the host knows, by a product: floor(n m / 2^shift)
// with m = ceil(2^shift / d), shift = 31 + ceil(log2 d) (an integer division is some 40 dependent
// instructions, and there are a dozen before a warp's first load).
struct FastDiv {
    unsigned d, m, shift;
};

static FastDiv fast_div(unsigned d)
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
};

// Warps, ring depth and shared memory of an instance.
template <int D, int R>
struct AttnCfg {
    // up to 4 query rows: columns of the products, two to a row; up to 8 or 16: their rows
    static constexpr bool WIDE = R > 4;
    // Warps: as many as registers and shared memory hold (at 128 dimensions and 4 rows 16 with rings of
    // 2 against 14 with rings of 3: 1 x 32768 23.0 against 25.2 us, 48 ragged sequences 124 against 127;
    // at 256 and 4 rows 8 against 6: 16 x 8100 90.6 against 104 us).
    static constexpr int W = D == 256 ? (R == 4 ? 8 : 6) : R == 4 ? 16 : D == 64 ? (R == 8 ? 16 : 12) : R == 8 ? 12 : 8;
    static constexpr int STAGES = D == 256 || (D == 128 && R == 4) ? 2 : 3;
    static constexpr int META = 64 * 16;  // block index and scales of two chunks of 32 blocks
    static constexpr int BOX = D < 128 ? D : 128;  // bytes of a row that one copy takes
    static constexpr int TILE = 16 * BOX;          // a copy: BOX bytes of 16 rows
    static constexpr int BLOCK_BYTES = 32 * D;  // keys and values of 16 positions
    static constexpr int RING = STAGES * BLOCK_BYTES;
    static constexpr int SLOT = R * D * 4;
    // query fragments stay in registers but for 256 dimensions, whose sums take 64 or 128 of them
    static constexpr bool QS = D == 256;
    static constexpr int QBYTES = QS ? R * D * 4 : 0;  // two f16 parts
    static constexpr int QN = D / 16 * (R == 4 ? 2 : R == 8 ? 4 : 8);  // registers of them
    static_assert(RING >= SLOT, "a warp's last part lies in its ring");
    // rings, first parts, query fragments, maxima and sums of 2 W parts, jobs, barriers, scans
    static constexpr int FIXED = W * (RING + SLOT + QBYTES + META) + 2 * W * R * 8 + (W + 1) * 32 + W * (STAGES + 1) * 8 + 8;
    static_assert(FIXED + 256 + (QMD_KV_MAX_SEQS + 1) * 4 <= 227 * 1024, "fits beside the sums of the most sequences");
};

constexpr int ATT_MAX_ROWS_FLOATS = 16 * 128;  // the largest R x D of an instance (8 x 256 is the same)
constexpr float ATT_NONE = -3.0e38f;           // the maximum before any score
constexpr float ATT_SLACK = 8.0f;              // how far (log2) a weight may pass its reference
// e before any value, and the least: an output under 2^-113 may have fewer bits
constexpr float ATT_LOW = -120.0f;
// How far a block's k may pass e: what e^x loses under 2^-126 is 2^-46 of the reference then.  Scales up to
// twice as far apart lower m.
constexpr float ATT_APART = 80.0f;

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

// Two bytes of w (biased by 128), picked by sel over (w, 0x64646464), as codes in f16.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t codes_f16(uint32_t w)
{
    const uint32_t u = __byte_perm(w, 0x64646464u, SEL);
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
    const __half2 c = __hsub2(*reinterpret_cast<const __half2 *>(&u), bias);
    return *reinterpret_cast<const uint32_t *>(&c);
}

// x and y as two f16 each: the first 11 bits, and the rest 2^11 times larger (in the upper half).
__device__ __forceinline__ void split_f16(float x, float y, uint32_t &px, uint32_t &py)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 b = __half22float2(h);
    const __half2 l = __floats2half2_rn((x - b.x) * 2048.0f, (y - b.y) * 2048.0f);
    const uint32_t hw = *reinterpret_cast<const uint32_t *>(&h), lw = *reinterpret_cast<const uint32_t *>(&l);
    px = __byte_perm(hw, lw, 0x5410);
    py = __byte_perm(hw, lw, 0x7632);
}

// The same as two pairs, the rest at its own size: for values up to 2^15 that matter down to 2^-31 of
// the largest.
__device__ __forceinline__ void split_pairs(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 b = __half22float2(h);
    const __half2 l = __floats2half2_rn(x - b.x, y - b.y);
    hi = *reinterpret_cast<const uint32_t *>(&h);
    lo = *reinterpret_cast<const uint32_t *>(&l);
}

constexpr float LOW_PART = 1.0f / 2048.0f;

// The least k (at most 127) with |d| < 2^k, for a value scale d down to 2^-126; 256 where d is not finite.
__device__ __forceinline__ float scale_log2(float d)
{
    const int ex = (int)(__float_as_uint(d) >> 23 & 255u);
    return ex == 255 ? 256.0f : (float)min(ex - 126, 127);
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

struct AttnMaps {  // the pools as [block][16][head_dim] bytes
    CUtensorMap k, v;
};

template <int D, int R>
__global__ void __launch_bounds__(AttnCfg<D, R>::W * 32, 1)
    kv_attention_kernel(const AttnArgs a, const __grid_constant__ AttnMaps maps)
{
    using C = AttnCfg<D, R>;
    constexpr int W = C::W, S = C::STAGES;
    constexpr int KH = D / 64;   // 64-byte parts of a key, 16 bytes to a lane
    constexpr int MT = D / 16;   // 16-row tiles of V^T
    constexpr bool WIDE = C::WIDE;
    constexpr int QR = R == 16 ? 2 : 1;          // query rows whose scores a lane holds
    constexpr int OT = WIDE ? 2 * MT : MT, CT = WIDE ? 2 : 1;  // tiles of sums, of scores
    constexpr int VW = D / 32;   // words of a value row that a lane holds
    extern __shared__ __align__(1024) unsigned char smem[];
    float2 *s_ml = reinterpret_cast<float2 *>(smem + W * (C::RING + C::SLOT + C::QBYTES + C::META));  // [W][2][R] maximum, weight sum
    Job *s_job = reinterpret_cast<Job *>(s_ml + 2 * W * R);                      // [1 + W]
    uint64_t *s_bar = reinterpret_cast<uint64_t *>(s_job + W + 1);               // [W][STAGES]
    int64_t *s_warp = reinterpret_cast<int64_t *>(s_bar + W * S);                // [W]
    int *s_last = reinterpret_cast<int *>(s_warp + W);                           // [2]
    int *s_pre = s_last + 2;                                                     // [seqs + 1] units before a sequence

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

    // ---- the line of units: an exclusive sum over the sequences ------------------------------
    if (lane == 0) {
        s_job[1 + warp].rows = 0;
        if (warp == 0)
            s_job[0].rows = 0;
    }
    auto units_of = [&](const KvSeq &q) {
        int64_t u = 0;
        for (int cg = 0; cg * R < q.n * a.group; ++cg) {
            const Group gr = group_of<R>(a, q, cg);
            u += max(1, gr.hi - gr.lo);
        }
        return u * p.heads;
    };
    // up to 32 sequences: every warp for itself, a lane a sequence; else through shared memory
    const bool few = p.seqs <= 32;
    int my_pre = 0, my_units = 0;
    int units = 0;
    bool too_many = false;
    if (few) {
        int64_t u = lane < p.seqs ? units_of(kv_seq(p, lane)) : 0;
        my_units = (int)min(u, (int64_t)INT_MAX);
        const bool big = __any_sync(0xffffffffu, u > INT_MAX / 32);  // the 32-bit sum may run over
        if (big) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                u += __shfl_xor_sync(0xffffffffu, u, o);
            too_many = u > INT_MAX;
        }
        unsigned sum = (unsigned)my_units;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o)
                sum += x;
        }
        my_pre = (int)(sum - (unsigned)my_units);
        units = (int)__shfl_sync(0xffffffffu, sum, 31);
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
        units = (int)total;
        too_many = total > INT_MAX;
        if (tid == 0)
            s_pre[p.seqs] = units;
        __syncthreads();
    }
    if (too_many) {  // more blocks than a launch counts
        kv_index_error(p);
        return;
    }
    // ---- this CTA's range, this warp's range ---------------------------------------------------
    // at least a unit for every warp, so that short items are cut inside a CTA, not between CTAs
    const int per = max(W, (units - 1) / a.by_grid + 1);
    if ((int64_t)blockIdx.x * per >= units)
        return;
    const int u0 = blockIdx.x * per;
    const int span = min(units - u0, per), pw = (span + W - 1) / W;
    int u = warp * pw;  // from here on counted from u0
    const int w1 = min(span, u + pw);

    unsigned char *ring = smem + warp * C::RING;
    const uint32_t ring_a = smem_addr(ring);
    uint32_t use = 0, use_phase = 0;  // the ring stage of the next block to read, and its barrier's phase
    bool dead = false;                // a copy did not land in time
    // Lane (g, t) reads row rho of a tile's upper and lower 8 rows of keys, 16-byte pieces 4 h + t.
    // Rows of 128 bytes: the copies put piece c of row r at c ^ (r & 7); lanes 0-7 hold rows 0 and 4
    // (pieces apart by 4), so rho swaps g's lowest and highest bits' places.  Rows of 64 bytes: at
    // c ^ (r >> 1 & 3), and the rows' own 64 bytes keep neighbours apart.
    const int rho = D > 64 ? (g >> 1) | (g & 1) << 2 : g;
    const uint32_t k_at = D > 64 ? rho * 128 + ((t ^ rho) << 4) : g * 64 + ((t ^ (g >> 1 & 3)) << 4);
    // ... and of values rows (positions) v0, v0 + v1, v0 + 8, v0 + v1 + 8: those that rho deals to
    // columns 2 t, 2 t + 1, 2 t + 8, 2 t + 9, dimensions 16 rho + 0..15 (of a 64-wide head 8 g + 0..7).
    const uint32_t v_at = D > 64 ? t * 128 + ((rho ^ t) << 4) : 2 * t * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
    int4 *meta = reinterpret_cast<int4 *>(smem + W * (C::RING + C::SLOT + C::QBYTES) + warp * C::META);

    int s = 0, cg = 0, head = 0, b0 = 0;  // the item of unit u, and the unit's block in it
    if (u < w1) {
        const int at = u0 + u;
        int pre;
        if (few) {
            s = 31 - __clz(__ballot_sync(0xffffffffu, my_units > 0 && my_pre <= at));
            pre = __shfl_sync(0xffffffffu, my_pre, s);
        } else {
            int lo = 0, hi = p.seqs;  // s_pre[lo] <= at < s_pre[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_pre[mid] <= at)
                    lo = mid;
                else
                    hi = mid;
            }
            s = lo;
            pre = s_pre[s];
        }
        int rem = at - pre;
        const KvSeq sq = kv_seq(p, s);
        // the row groups of a head lie together: they read the same keys and values
        const int of_head = (few ? __shfl_sync(0xffffffffu, my_units, s) : s_pre[s + 1] - pre) / a.by_heads;
        head = rem / of_head;
        rem -= head * of_head;
        for (;; ++cg) {
            const Group gr = group_of<R>(a, sq, cg);
            const int nb = max(1, gr.hi - gr.lo);
            if (rem < nb)
                break;
            rem -= nb;
        }
        b0 = rem;
    }
    while (u < w1) {
        const KvSeq sq = kv_seq(p, s);
        const Group gr = group_of<R>(a, sq, cg);
        const int nb = max(1, gr.hi - gr.lo);
        const int cnt = min(nb - b0, w1 - u);              // units of this item in the range
        const int real = min(cnt, gr.hi - gr.lo - b0);          // those that hold positions

        // pages and scales, 32 blocks at a time: block index in the pool, or -1
        const int first_blk = gr.lo + b0;
        auto page_of = [&](int i) -> int {  // of the item's i-th block here; INT_MIN past the end
            return i < real ? p.table[(int64_t)s * p.table_stride + (first_blk + i) / a.by_blocks] : INT_MIN;
        };
        auto block_of = [&](int i, int page) -> int {
            if (page < 0 || page >= p.pages) {
                if (page != INT_MIN)
                    kv_index_error(p);
                return -1;
            }
            const int blk = first_blk + i;
            return (page * p.heads + head - blk / a.by_blocks) * p.page_blocks + blk;
        };
        int page_n = page_of(lane);
        // lane (g, t) takes dimensions 64 h + 16 t + 0..15 of a query row: that of column g (two columns to
        // a row), or rows g and g + 8; past the rows the last one again
        float x[QR][KH][16];
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            const int r = cg * R + min(WIDE ? g + 8 * i : g >> 1, gr.rows - 1);
            const float *qp = a.q + row_offset(a, sq.row0, head, r, a.q_stride, D) + 16 * t;
#pragma unroll
            for (int h = 0; h < KH; ++h)
                load_f32(x[i][h], qp + 64 * h);
        }
        int bi_n = block_of(lane, page_n);
        fence_proxy_async_smem();
        __syncwarp();  // every lane has read the last item's ring and meta

        auto issue = [&](int j, int bi, uint32_t stage) {  // copy the item's j-th block, bi, into a ring stage
            if (j < real && lane == 0) {
                const uint32_t dst = ring_a + stage * C::BLOCK_BYTES, bar = bar0 + 8 * stage;
                mbar_arrive_expect_tx(bar, bi >= 0 ? C::BLOCK_BYTES : 0);  // (nothing to wait for)
                if (bi >= 0) {
#pragma unroll
                    for (int x = 0; x < D / C::BOX; ++x) {
                        load_tile(dst + x * C::TILE, &maps.k, x * C::BOX, bi, bar);
                        load_tile(dst + 16 * D + x * C::TILE, &maps.v, x * C::BOX, bi, bar);
                    }
                }
            }
        };
        uint32_t put = use;  // the ring stage of the next block to ask for
#pragma unroll
        for (int j = 0; j < S - 1; ++j) {
            issue(j, __shfl_sync(0xffffffffu, bi_n, j), put);
            put = put + 1 == S ? 0 : put + 1;
        }
        float ks_n = bi_n >= 0 ? p.ks[bi_n] : 0.0f, vs_n = bi_n >= 0 ? p.vs[bi_n] : 0.0f;
        auto put_meta = [&](int at) {
            meta[at] = make_int4(bi_n, __float_as_int(ks_n), __float_as_int(vs_n), __float_as_int(scale_log2(vs_n)));
        };
        put_meta(lane);
        __syncwarp();

        // ---- the queries as two f16 parts ------------------------------------------------------
        uint32_t qf[C::QN];   // of word w of part h: [4 h + w][column] or [4 h + w][row, dimension]
        float qscale[QR];     // of query row t, or rows g and g + 8
#pragma unroll
        for (int i = 0; i < QR; ++i) {
            float top = 0.0f;
#pragma unroll
            for (int h = 0; h < KH; ++h)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    top = fmaxf(top, fabsf(x[i][h][e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // q times a power of two: the largest value in [0.5, 1), or in [2^14, 2^15)
            const int ex = (int)(__float_as_uint(top) >> 23);
            const int field = WIDE ? min(253, 268 - ex) : min(253, max(1, 253 - ex));
            const float f = __uint_as_float((uint32_t)field << 23);
            const float back = __uint_as_float((uint32_t)(254 - field) << 23) * a.scale_log2e;
#pragma unroll
            for (int h = 0; h < KH; ++h)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float x0 = x[i][h][4 * w + 2 * e] * f, x1 = x[i][h][4 * w + 2 * e + 1] * f;
                        uint32_t hi, lo;
                        if constexpr (!WIDE) {
                            split_f16(x0, x1, lo, hi);
                            qf[(4 * h + w) * 2 + e] = __byte_perm(lo, hi, (g & 1) ? 0x7632 : 0x5410);
                        } else {
                            split_pairs(x0, x1, hi, lo);
                            if constexpr (R == 8) {  // rows 0-7 the first parts, rows 8-15 the second
                                qf[(4 * h + w) * 4 + 2 * e] = hi;
                                qf[(4 * h + w) * 4 + 2 * e + 1] = lo;
                            } else {
                                qf[(4 * h + w) * 8 + 2 * e + i] = hi;
                                qf[(4 * h + w) * 8 + 4 + 2 * e + i] = lo;
                            }
                        }
                    }
            qscale[i] = WIDE ? back : __shfl_sync(0xffffffffu, back, 8 * t);
        }
        uint4 *q_keep = reinterpret_cast<uint4 *>(smem + W * (C::RING + C::SLOT) + warp * C::QBYTES) + lane;
        if constexpr (C::QS) {
#pragma unroll
            for (int i = 0; i < C::QN / 4; ++i)
                q_keep[i * 32] = make_uint4(qf[4 * i], qf[4 * i + 1], qf[4 * i + 2], qf[4 * i + 3]);
        }
        auto query = [&](int i) {  // registers 4 i .. 4 i + 3 of the fragments
            if constexpr (C::QS)
                return q_keep[i * 32];
            else
                return make_uint4(qf[4 * i], qf[4 * i + 1], qf[4 * i + 2], qf[4 * i + 3]);
        };
        // positions in [all_from, all_to) are seen by every row of the group
        const int all_to = row_end(sq, cg * R / a.by_group);
        const int all_from = row_begin(a, row_end(sq, (cg * R + gr.rows - 1) / a.by_group));

        float o[OT][4];
        float m[QR], ve8[QR], vinv[QR], l[QR];  // the references: m, e + ATT_SLACK, 2^-e; the weights' sum
        // wide rows' weights times 2^6 besides, so that what f16 loses below its smallest value is 2^-31 of
        // the reference
        constexpr float LIFT = WIDE ? 64.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < QR; ++i)
            m[i] = ATT_NONE, ve8[i] = ATT_LOW + ATT_SLACK, vinv[i] = 0.0f, l[i] = 0.0f;
#pragma unroll
        for (int i = 0; i < OT; ++i)
            o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        // the first product of the block in a ring stage: K Q^T (16 positions by columns), or Q K^T (rows
        // by two tiles of 8 positions)
        auto scores = [&](float (&c)[CT][4], const unsigned char *st) {
            float c2[CT][4] = {};  // twice as many chains of sums (at 8 rows the registers cost more)
#pragma unroll
            for (int i = 0; i < CT; ++i)
                c[i][0] = c[i][1] = c[i][2] = c[i][3] = 0.0f;
#pragma unroll
            for (int h = 0; h < KH; ++h) {
                const unsigned char *kp = st + (h >> 1) * C::TILE + (k_at ^ (h & 1) << 6);
                const uint4 ka = lds128(kp), kb = lds128(kp + 8 * C::BOX);
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int w2 = 0; w2 < 4; w2 += 2) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t x = wa[w2 + e] ^ 0x80808080u, y = wb[w2 + e] ^ 0x80808080u;
                        f[e][0] = codes_f16<0x4140>(x), f[e][1] = codes_f16<0x4140>(y);
                        f[e][2] = codes_f16<0x4342>(x), f[e][3] = codes_f16<0x4342>(y);
                    }
                    if constexpr (!WIDE) {
                        const uint4 qv = query(2 * h + w2 / 2);
                        mma_16816(c[0], f[0], qv.x, qv.y);
                        mma_16816(c2[0], f[1], qv.z, qv.w);
                    } else {
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int part = 0; part < R / 8; ++part) {
                                const uint4 qv = query((4 * h + w2 + e) * (R / 8) + part);
                                const uint32_t qa[4] = {qv.x, qv.y, qv.z, qv.w};
                                mma_16816(part ? c2[0] : c[0], qa, f[e][0], f[e][2]);
                                mma_16816(part ? c2[CT - 1] : c[CT - 1], qa, f[e][1], f[e][3]);
                            }
                    }
                }
            }
            if constexpr (R != 8)
#pragma unroll
                for (int i = 0; i < CT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        c[i][e] += c2[i][e];
        };
        float c[CT][4];
        // wait for the block in a stage
        auto landed = [&](uint32_t stage, uint32_t phase) {
            if (__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * stage, phase, a.wait_ns)))
                return true;
            dead = true;
            return false;
        };
        for (int idx = 0; idx < real && !dead; ++idx) {
            if ((idx & 7) == 0 && (idx | 31) + 1 < real) {  // the next 32 blocks, a step of their lookup at a time
                const int i = (idx | 31) + 1 + lane;
                if ((idx & 24) == 0) {
                    page_n = page_of(i);
                } else if ((idx & 24) == 8) {
                    bi_n = block_of(i, page_n);
                    ks_n = bi_n >= 0 ? p.ks[bi_n] : 0.0f, vs_n = bi_n >= 0 ? p.vs[bi_n] : 0.0f;
                } else if ((idx & 24) == 16) {
                    __syncwarp();
                    put_meta(i & 63);
                    __syncwarp();
                }
            }
            const uint32_t next = use + 1 == S ? 0 : use + 1, next_phase = next == 0 ? use_phase ^ 1u : use_phase;
            fence_proxy_async_smem();
            __syncwarp();  // every lane has read the stage that is asked for again
            issue(idx + S - 1, meta[(idx + S - 1) & 63].x, put);
            put = put + 1 == S ? 0 : put + 1;
            if (!landed(use, use_phase))
                break;
            scores(c, ring + use * C::BLOCK_BYTES);
            const int4 md = meta[idx & 63];
            const int bi = md.x;
            const float ks = __int_as_float(md.y), vs = __int_as_float(md.z), vk = __int_as_float(md.w);
            const unsigned char *st = ring + use * C::BLOCK_BYTES;

            // The scores in log2 units.  sc[i][e] is of query row t at position pos + rho + 8 e; or of row
            // g + 8 i at position pos + 8 (e >> 1) + (what rho deals to column 2 t + (e & 1)).
            constexpr int SN = WIDE ? 4 : 2;
            const int pos = (first_blk + idx) * KV_BLOCK;
            const bool whole = pos >= all_from && pos + KV_BLOCK <= all_to && bi >= 0;
            float sc[QR][SN];
            bool up = false;
            float vr[QR];  // the block's scale over 2^e
#pragma unroll
            for (int i = 0; i < QR; ++i) {
                const float f = qscale[i] * ks;
                if constexpr (!WIDE) {
                    sc[i][0] = fmaf(c[0][1], LOW_PART, c[0][0]) * f;
                    sc[i][1] = fmaf(c[0][3], LOW_PART, c[0][2]) * f;
                } else {
#pragma unroll
                    for (int e = 0; e < SN; ++e)
                        sc[i][e] = (R == 8 ? c[CT * e / SN][e & 1] + c[CT * e / SN][2 + (e & 1)]
                                           : c[CT * e / SN][2 * i + (e & 1)]) * f;
                }
                if (!whole) {
                    const int end = row_end(sq, (cg * R + min(WIDE ? g + 8 * i : t, gr.rows - 1)) / a.by_group);
                    const int begin = row_begin(a, end);
#pragma unroll
                    for (int e = 0; e < SN; ++e) {
                        const int j = pos + (!WIDE ? rho + 8 * e : 8 * (e >> 1) + (D > 64 ? t + 4 * (e & 1) : 2 * t + (e & 1)));
                        if (bi < 0 || j < begin || j >= end)
                            sc[i][e] = -INFINITY;
                    }
                }
                vr[i] = vs * vinv[i];
                const float room = ve8[i] - vk, most = m[i] + fminf(ATT_SLACK, room);
                up |= room < ATT_SLACK - ATT_APART;
#pragma unroll
                for (int e = 0; e < SN; ++e)
                    up |= sc[i][e] > most;
            }
            if (__any_sync(0xffffffffu, up)) {
                float fo[QR];
#pragma unroll
                for (int i = 0; i < QR; ++i) {
                    float top = sc[i][0];
#pragma unroll
                    for (int e = 1; e < SN; ++e)
                        top = fmaxf(top, sc[i][e]);
                    // over the lanes that hold the row's other positions
#pragma unroll
                    for (int x = WIDE ? 1 : 4; x < (WIDE ? 4 : 32); x <<= 1)
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    // integers, so that e moves by what m moves and 2^(m + e) stays where it is
                    const float mn = top > m[i] ? ceilf(top) : m[i], ve = ve8[i] - ATT_SLACK;
                    const float k = top > -INFINITY ? vk : ATT_LOW;  // (a row that does not see the block keeps its references)
                    const float en = fmaxf(fmaxf(ve + (m[i] - mn), ceilf(top - mn + k)), fmaxf(ATT_LOW, k - 2.0f * ATT_APART));
                    // a scale further above 2^e than e^x reaches: m that much lower, and e higher
                    const float low = fmaxf(k - en - ATT_APART, 0.0f);
                    l[i] *= pow2(m[i] - mn + low);
                    fo[i] = pow2(m[i] - mn + (ve - en));
                    m[i] = mn - low;
                    ve8[i] = en + low + ATT_SLACK;
                    vinv[i] = pow2(1.0f - (en + low)) * (0.5f * LIFT);
                    // 0 for a row that does not see the block, whose scale may not be finite
                    vr[i] = k == vk ? vs * vinv[i] : 0.0f;
                }
#pragma unroll
                for (int i = 0; i < OT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[i][e] *= fo[R == 16 ? e >> 1 : 0];
            }
            // the weights, as the second product's operand: columns, or rows
            uint32_t pb[WIDE ? R / 8 : 1][4];
#pragma unroll
            for (int i = 0; i < QR; ++i) {
                float w[SN];
#pragma unroll
                for (int e = 0; e < SN; ++e) {
                    w[e] = ex2(sc[i][e] - m[i]);
                    l[i] += w[e];
                    w[e] *= vr[i];
                }
                if constexpr (!WIDE) {
                    uint32_t a0, a1;
                    split_f16(w[0], w[1], a0, a1);
                    pb[0][0] = transpose_8x8(a0);
                    pb[0][1] = transpose_8x8(a1);
                } else {
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        uint32_t hi, lo;
                        split_pairs(w[(2 * n) % SN], w[(2 * n + 1) % SN], hi, lo);
                        if constexpr (R == 8) {
                            pb[0][2 * n] = hi;
                            pb[0][2 * n + 1] = lo;
                        } else {
                            pb[0][2 * n + i] = hi;
                            pb[(R / 8) - 1][2 * n + i] = lo;
                        }
                    }
                }
            }

            // the second product: V^T P^T (16 dimensions by columns), or P V (rows by 8 dimensions)
            const unsigned char *sv = st + 16 * D;
#pragma unroll
            for (int y = 0; y < (VW + 3) / 4; ++y) {
                uint32_t v[4][VW < 4 ? VW : 4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if constexpr (D == 64) {
                        const uint2 q2 = *reinterpret_cast<const uint2 *>(sv + v_at + (x & 1) * 64 + (x >> 1) * 512);
                        v[x][0] = q2.x, v[x][1] = q2.y;
                    } else {
                        const uint4 q4 = lds128(sv + y * C::TILE + ((x & 1) ? (v_at ^ 64) + 512 : v_at) + (x >> 1) * 1024);
                        v[x][0] = q4.x, v[x][1] = q4.y, v[x][2] = q4.z, v[x][3] = q4.w;
                    }
                }
#pragma unroll
                for (int w = 0; w < (VW < 4 ? VW : 4); ++w) {
                    const uint32_t x0 = v[0][w] ^ 0x80808080u, x1 = v[1][w] ^ 0x80808080u;
                    const uint32_t x2 = v[2][w] ^ 0x80808080u, x3 = v[3][w] ^ 0x80808080u;
                    const uint32_t e01 = __byte_perm(x0, x1, 0x5140), e23 = __byte_perm(x2, x3, 0x5140);
                    const uint32_t f01 = __byte_perm(x0, x1, 0x7362), f23 = __byte_perm(x2, x3, 0x7362);
                    const uint32_t fa[4] = {codes_f16<0x4140>(e01), codes_f16<0x4342>(e01), codes_f16<0x4140>(e23),
                                            codes_f16<0x4342>(e23)};
                    const uint32_t fb[4] = {codes_f16<0x4140>(f01), codes_f16<0x4342>(f01), codes_f16<0x4140>(f23),
                                            codes_f16<0x4342>(f23)};
                    const int i = 8 * y + 2 * w;
                    if constexpr (!WIDE) {
                        mma_16816(o[i], fa, pb[0][0], pb[0][1]);
                        mma_16816(o[i + 1], fb, pb[0][0], pb[0][1]);
                    } else {
#pragma unroll
                        for (int part = 0; part < R / 8; ++part) {
                            mma_16816(o[(2 * i) % OT], pb[part % (WIDE ? R / 8 : 1)], fa[0], fa[2]);
                            mma_16816(o[(2 * i + 1) % OT], pb[part % (WIDE ? R / 8 : 1)], fa[1], fa[3]);
                            mma_16816(o[(2 * i + 2) % OT], pb[part % (WIDE ? R / 8 : 1)], fb[0], fb[2]);
                            mma_16816(o[(2 * i + 3) % OT], pb[part % (WIDE ? R / 8 : 1)], fb[1], fb[3]);
                        }
                    }
                }
            }
            use = next;
            use_phase = next_phase;
        }
        if (dead) {
            // flag it, wait (bounded) for this warp's copies that may be in flight, leave the rest out
            if (lane == 0) {
                atomicOr(p.err, (unsigned)ERRBIT_QMV_WAIT);
                for (int i = 0; i < S; ++i) {
                    if (!mbar_wait_bounded(bar0 + 8 * use, use_phase, a.wait_ns)) {
                        atomicOr(p.err, (unsigned)ERRBIT_DRAIN_WAIT);
                        break;
                    }
                    use = use + 1 == S ? 0 : use + 1;
                    use_phase = use == 0 ? use_phase ^ 1u : use_phase;
                }
            }
            __syncwarp();
            break;
        }

        // ---- the item's part: finished, or laid down for the join --------------------------------
        const bool done = b0 == 0 && cnt == nb;
        const int part = b0 > 0 ? 0 : 1;
        float *dst = reinterpret_cast<float *>(part == 0 ? smem + W * C::RING + warp * C::SLOT : ring);
        if (part == 1 && !done)
            __syncwarp();  // every lane has read the ring
#pragma unroll
        for (int i = 0; i < QR; ++i) {
#pragma unroll
            for (int x = WIDE ? 1 : 4; x < (WIDE ? 4 : 32); x <<= 1)
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], x);
            const int r = WIDE ? g + 8 * i : t;
            const float f = (done ? (l[i] == 0.0f ? 0.0f : 1.0f / l[i]) : 1.0f) * (1.0f / LIFT), fe = pow2(ve8[i] - ATT_SLACK);
            if (!done && (WIDE ? t : g) == 0)
                s_ml[(warp * 2 + part) * R + r] = make_float2(m[i], l[i]);
            if (done && r >= gr.rows)
                continue;
            float *to = done ? a.out + row_offset(a, sq.row0, head, cg * R + r, a.out_stride, D) : dst + r * D;
            // runs of RUN neighbouring dimensions: 16 of those that rho deals to a lane (of a 64-wide head
            // 8), for columns 2 t and 2 t + 1 where rows are rows
            constexpr int RUN = D == 64 ? 8 : 16;
#pragma unroll
            for (int n = 0; n < (WIDE ? 2 : 1); ++n) {
                const int piece = WIDE ? (D == 64 ? 2 * t + n : t + 4 * n) : rho;
#pragma unroll
                for (int d = 0; d < D / 8; d += 4) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = (!WIDE ? fmaf(o[(d + e) / 2 % OT][((d + e) & 1) * 2 + 1], LOW_PART, o[(d + e) / 2 % OT][((d + e) & 1) * 2])
                                : R == 8 ? o[(d + e) % OT][n] + o[(d + e) % OT][2 + n]
                                         : o[(d + e) % OT][2 * i + n]) * f * fe;
                    *reinterpret_cast<float4 *>(to + d / RUN * 128 + piece * RUN + d % RUN) = make_float4(y[0], y[1], y[2], y[3]);
                }
            }
        }
        // the item's first cut in this CTA makes the job of joining it
        if (!done && lane == 0 && (part == 1 || warp == 0)) {
            Job &j = s_job[part == 1 ? 1 + warp : 0];
            j.start = u - b0;
            j.end = u - b0 + nb;
            j.row0 = sq.row0;
            j.first = cg * R;
            j.head = head;
            j.rows = gr.rows;
        }
        u += cnt;
        b0 = 0;
        if (u < w1 && ++cg * R >= sq.n * a.group) {  // on to the next head, or the next sequence with rows
            cg = 0;
            if (++head == p.heads) {
                head = 0;
                if (few) {
                    s = __ffs(__ballot_sync(0xffffffffu, my_units > 0) & ~((2u << s) - 1)) - 1;
                } else {
                    do
                        ++s;
                    while (s_pre[s + 1] == s_pre[s]);
                }
            }
        }
    }
    __syncthreads();

    // ---- joins inside the CTA -------------------------------------------------------------------
    // Job 0 is the item that began before the CTA's range (parts 0 of warps 0 ..), job 1 + w the one
    // that warp w's range cut (its part 1, parts 0 of the warps after it).
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
                load_f32(v, reinterpret_cast<const float *>(one ? smem + w * C::RING : smem + W * C::RING + w * C::SLOT) +
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

template <int D, int R>
static qmd_status launch_att(const AttnArgs &a, const DeviceInfo &dev, cudaStream_t s)
{
    using C = AttnCfg<D, R>;
    const size_t smem = C::FIXED + ((size_t)a.kv.seqs + 1) * sizeof(int);
    if (smem + 256 > (size_t)dev.smem_optin)
        return QMD_ERR_SHAPE;
    {
        static std::mutex mu;
        static bool opted[64] = {false};
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[dev.device]) {
            const cudaError_t e = cudaFuncSetAttribute(kv_attention_kernel<D, R>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, dev.smem_optin - 256);
            if (e != cudaSuccess)
                return fail(QMD_ERR_LAUNCH, "kv_attention smem attribute", e);
            opted[dev.device] = true;
        }
    }
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc)
        return fail(QMD_ERR_LAUNCH, "cuTensorMapEncodeTiled entry point", cudaErrorNotSupported);
    AttnMaps maps;
    const cuuint64_t dim[3] = {(cuuint64_t)D, KV_BLOCK, (cuuint64_t)a.kv.pages * a.kv.heads * a.kv.page_blocks};
    const cuuint64_t str[2] = {(cuuint64_t)D, (cuuint64_t)D * KV_BLOCK};
    const cuuint32_t box[3] = {(cuuint32_t)C::BOX, KV_BLOCK, 1}, one[3] = {1, 1, 1};
    for (int i = 0; i < 2; ++i)
        if (enc(i ? &maps.v : &maps.k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, i ? a.kv.v : a.kv.k, dim, str, box, one,
                CU_TENSOR_MAP_INTERLEAVE_NONE, D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return fail(QMD_ERR_LAUNCH, "tensor map of the cache", cudaErrorInvalidValue);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, R>, a, maps);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv_attention launch", e);
}

// counters (a CTA each, to a multiple of 16 bytes), then the parts and their maxima and sums
static size_t counter_bytes(const DeviceInfo &dev) { return ((size_t)dev.sm_count * 4 + 15) / 16 * 16; }

size_t kv_attention_workspace(const DeviceInfo &dev)
{
    return counter_bytes(dev) + (size_t)dev.sm_count * 2 * (ATT_MAX_ROWS_FLOATS + 16 * 2) * 4;
}

qmd_status launch_kv_attention(const KvParams &kv, int head_dim, const float *q, int64_t q_stride, int q_heads,
                               float scale, int64_t window, float *out, int64_t out_stride, void *ws,
                               const DeviceInfo &dev, cudaStream_t s)
{
    const AttnArgs a = {kv, q, out, reinterpret_cast<float *>(static_cast<char *>(ws) + counter_bytes(dev)),
                        static_cast<unsigned *>(ws), q_stride, out_stride, window, wait_limit_ns(), q_heads / kv.heads,
                        fast_div((unsigned)(q_heads / kv.heads)), fast_div((unsigned)kv.page_blocks),
                        fast_div((unsigned)kv.heads), fast_div((unsigned)dev.sm_count),
                        scale * 1.4426950408889634f};
    // rows per item: the least of 4, 8, 16 that holds a sequence's rows of one key/value head
    const int64_t rows = (int64_t)a.group * kv.max_q;
    if (head_dim == 64)
        return rows <= 4 ? launch_att<64, 4>(a, dev, s) : rows <= 8 ? launch_att<64, 8>(a, dev, s) : launch_att<64, 16>(a, dev, s);
    if (head_dim == 128)
        return rows <= 4   ? launch_att<128, 4>(a, dev, s)
               : rows <= 8 ? launch_att<128, 8>(a, dev, s)
                           : launch_att<128, 16>(a, dev, s);
    return rows <= 4 ? launch_att<256, 4>(a, dev, s) : launch_att<256, 8>(a, dev, s);
}

}  // namespace qmd
