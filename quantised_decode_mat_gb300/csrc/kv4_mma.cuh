// kv4_mma.cuh -- the products with the 4-bit cache on the tensor cores, which attention and its weights share.
//
// S = K Q^T of 16 slots on mma.sync m16n8k16 (f16 in, f32 sums), slots the 16 rows and query rows the 8
// columns.  f32 queries go in as two f16 parts, the first 11 bits and the next 11; a code c enters exactly, as c - 8.  Up
// to 4 query rows (R = 4) have two columns each, one to a part; of 8 or 16 rows both parts are multiplied
// into the same sums.  A group of 32 dimensions is two steps of 16; its sums are multiplied by its scale in f32,
// which is exact but for one rounding.
//
// Layout: as rows of head_dim / 2 bytes lie in memory, the 8 x 8 matrices that ldmatrix takes (16 bytes of 8
// rows: a group of 8 tokens) give lane (g, t) word t of row g, dimensions 32 i + 8 t .. + 7: the operand of two
// steps, as the order of the dimensions inside a group is free.  Transposed, they give it half-word g of rows 2 t
// and 2 t + 1: dimensions 32 i + 4 g .. + 3 of two tokens, which is the operand V^T.  So nothing is permuted in
// memory, and a word's 8 codes become four f16 pairs by the same nine instructions for both.
//
// Subnormal f16 (a masked nibble as it is, c 2^-24) would save four of the nine; the tensor cores align what they
// add to the largest product with such a factor counted as 2^-14, which costs the sums 7 to 10 bits.
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"
#include "kv_attn.cuh"
#include "tensor_map.h"

namespace qmd {

constexpr int KV4_UNIT = 32;  // slots that are worked on together

// How a row of codes of a D-dimensional head lies in shared memory after a tensor copy of KV4_UNIT rows.
template <int D>
struct Tile4 {
    static constexpr int ROW = D / 2, G = D / KV4_GROUP;
    static constexpr int CODES = KV4_UNIT * ROW, SCALES = KV4_UNIT * G * 2;  // bytes of a unit's keys (or values)
    static constexpr int LOADS = G < 4 ? 1 : G / 2;  // ldmatrix (of four matrices) for 16 slots
    // Where lane l's row of ldmatrix x of 16 slots lies: the copies swizzle 16-byte pieces (by 32, 64 or 128
    // bytes, as a row is long), so the 8 rows of a matrix lie in different banks.
    static __device__ __forceinline__ uint32_t at(int l, int x)
    {
        const int r = l & 7, m = l >> 3;
        if constexpr (D == 64)  // matrices: groups 0, 1 of slots 0-7, then of 8-15
            return ((m >> 1) * 8 + r) * 32 + (((m & 1) ^ (r >> 2)) << 4);
        else if constexpr (D == 128)  // groups 0-3 of slots 8 x ..
            return (x * 8 + r) * 64 + ((m ^ (r >> 1)) << 4);
        else  // groups 4 (x & 1) .. + 3 of slots 8 (x >> 1) ..
            return ((x >> 1) * 8 + r) * 128 + (((4 * (x & 1) + m) ^ r) << 4);
    }
};

template <bool TRANS>
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr)
{
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// The words of 16 slots at addr (with the lane's part of it), w[e][i]: of slots 8 e .. and group i.
template <int D, bool TRANS>
__device__ __forceinline__ void load_words(uint32_t (&w)[2][Tile4<D>::G], uint32_t base, const uint32_t (&lane_at)[Tile4<D>::LOADS])
{
#pragma unroll
    for (int x = 0; x < Tile4<D>::LOADS; ++x) {
        uint32_t r[4];
        ldmatrix_x4<TRANS>(r, base + lane_at[x]);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            if constexpr (D == 64)
                w[m >> 1][m & 1] = r[m];
            else if constexpr (D == 128)
                w[x][m] = r[m];
            else
                w[x >> 1][4 * (x & 1) + m] = r[m];
        }
    }
}

// (a & b) | c in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}

// A word's codes, less 8, as f16 pairs: f[n] holds nibbles n and n + 4.  (Whole bytes by __byte_perm in place of the
// upper nibbles, with what multiplies them adjusted, came to an instruction more a word.)
__device__ __forceinline__ void unpack4_f16(uint32_t (&f)[4], uint32_t w)
{
    // a nibble under the exponent of 1024 is 1024 + c, or 1024 + 16 c where it is the second
    const __half2 low = __half2half2(__ushort_as_half(0xe408));   // -1032
    const __half2 by16 = __half2half2(__ushort_as_half(0x2c00));  // 1 / 16
    const __half2 high = __half2half2(__ushort_as_half(0xd480));  // -72
#pragma unroll
    for (int n = 0; n < 4; n += 2) {
        const uint32_t v = n ? w >> 8 : w;
        const uint32_t x = and_or(v, 0x000f000fu, 0x64006400u), y = and_or(v, 0x00f000f0u, 0x64006400u);
        const __half2 a = __hadd2(*reinterpret_cast<const __half2 *>(&x), low);
        const __half2 b = __hfma2(*reinterpret_cast<const __half2 *>(&y), by16, high);
        f[n] = *reinterpret_cast<const uint32_t *>(&a);
        f[n + 1] = *reinterpret_cast<const uint32_t *>(&b);
    }
}

// How R query rows are columns of the products.
template <int R>
struct Cols4 {
    static constexpr int NT = R == 4 ? 1 : R / 8;         // tiles of 8 columns
    static constexpr int PARTS = R == 4 ? 1 : 2;          // products into the same sums
    static constexpr int LR = R == 4 ? 1 : 2 * NT;        // query rows whose scores a lane holds
    // the i-th query row of lane t
    static __device__ __forceinline__ int row(int i, int t) { return R == 4 ? t : (i >> 1) * 8 + 2 * t + (i & 1); }
};

// f32 values x, y as their first 11 bits (exact in f16 down to 2^-14) and the rest.
__device__ __forceinline__ float first_bits(float x) { return __uint_as_float(__float_as_uint(x) & 0xffffe000u); }

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }

// The query fragments of a warp's item: [tile][group][step of 16][part][2] registers.
template <int D, int R>
struct Query4 {
    using C = Cols4<R>;
    static constexpr int G = D / KV4_GROUP, N = C::NT * G * 4 * C::PARTS;
    uint32_t f[N];
    float scale[C::LR];  // what a lane's rows' sums are multiplied by for scores in log2 units

    // rows: those the item has (past them the last one again); offset(r): where query row r begins
    template <class Offset>
    __device__ __forceinline__ void load(const float *q, Offset offset, int rows, float scale_log2e)
    {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
            const float *p = q + offset(min(R == 4 ? g >> 1 : nt * 8 + g, rows - 1)) + 8 * t;
            float x[G][8], top = 0.0f;
#pragma unroll
            for (int i = 0; i < G; ++i)
                load_f32(x[i], p + 32 * i);
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    top = fmaxf(top, fabsf(x[i][e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // q times a power of two: the largest value in [2^14, 2^15)
            const int field = min(253, 268 - (int)(__float_as_uint(top) >> 23));
            const float by = __uint_as_float((uint32_t)field << 23);
            const float back = __uint_as_float((uint32_t)(254 - field) << 23) * scale_log2e;
#pragma unroll
            for (int i = 0; i < G; ++i)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float u = x[i][2 * s + b] * by, v = x[i][2 * s + b + 4] * by;
                        const __half2 h = __floats2half2_rn(u, v);
                        const float2 back2 = __half22float2(h);
                        const uint32_t hi = *reinterpret_cast<const uint32_t *>(&h), lo = pack_f16(u - back2.x, v - back2.y);
                        const int at = (((nt * G + i) * 2 + s) * C::PARTS) * 2 + b;
                        if constexpr (R == 4) {
                            f[at] = (g & 1) ? lo : hi;
                        } else {
                            f[at] = hi;
                            f[at + 2] = lo;
                        }
                    }
            if constexpr (R == 4) {
                scale[0] = __shfl_sync(0xffffffffu, back, 8 * t);
            } else {
                scale[2 * nt] = __shfl_sync(0xffffffffu, back, 8 * t);
                scale[2 * nt + 1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
            }
        }
    }
};

// Scales of a lane's slots g and g + 8 of 16 slots whose scales begin at p: [e][pair of groups].
template <int D>
__device__ __forceinline__ void load_scales(uint32_t (&d)[2][Tile4<D>::G / 2], const unsigned char *p, int g)
{
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const unsigned char *q = p + (g + 8 * e) * (D / KV4_GROUP * 2);
        if constexpr (D == 64) {
            d[e][0] = *reinterpret_cast<const uint32_t *>(q);
        } else if constexpr (D == 128) {
            const uint2 v = *reinterpret_cast<const uint2 *>(q);
            d[e][0] = v.x, d[e][1] = v.y;
        } else {
            const uint4 v = lds128(q);
            d[e][0] = v.x, d[e][1] = v.y, d[e][2] = v.z, d[e][3] = v.w;
        }
    }
}

__device__ __forceinline__ float2 halves(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2 *>(&w)); }

// The scores of 16 slots in log2 units: s[i][e] of the lane's i-th query row and slot g + 8 e.  query(j) gives
// fragments 4 j .. 4 j + 3.
template <int D, int R, class QueryAt>
__device__ __forceinline__ void scores4(float (&s)[Cols4<R>::LR][2], uint32_t codes, const unsigned char *scales,
                                        const uint32_t (&lane_at)[Tile4<D>::LOADS], QueryAt query,
                                        const float (&qscale)[Cols4<R>::LR])
{
    using C = Cols4<R>;
    constexpr int G = Tile4<D>::G;
    const int g = (threadIdx.x & 31) >> 2;
    uint32_t w[2][G], d[2][G / 2];
    load_words<D, false>(w, codes, lane_at);
    load_scales<D>(d, scales, g);
#pragma unroll
    for (int i = 0; i < C::LR; ++i)
        s[i][0] = s[i][1] = 0.0f;
#pragma unroll
    for (int i = 0; i < G; ++i) {
        uint32_t a[4], b[4];
        unpack4_f16(a, w[0][i]);
        unpack4_f16(b, w[1][i]);
        const uint32_t first[4] = {a[0], b[0], a[1], b[1]}, second[4] = {a[2], b[2], a[3], b[3]};
        const float2 d0 = halves(d[0][i / 2]), d1 = halves(d[1][i / 2]);
        const float da = i & 1 ? d0.y : d0.x, db = i & 1 ? d1.y : d1.x;
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
            float c[4] = {};
            if constexpr (R == 4) {
                const uint4 q = query(i);
                mma_16816(c, first, q.x, q.y);
                mma_16816(c, second, q.z, q.w);
                s[0][0] = fmaf(c[0] + c[1], da, s[0][0]);
                s[0][1] = fmaf(c[2] + c[3], db, s[0][1]);
            } else {
                const uint4 q0 = query((nt * G + i) * 2), q1 = query((nt * G + i) * 2 + 1);
                mma_16816(c, first, q0.z, q0.w);
                mma_16816(c, second, q1.z, q1.w);
                mma_16816(c, first, q0.x, q0.y);
                mma_16816(c, second, q1.x, q1.y);
                s[2 * nt][0] = fmaf(c[0], da, s[2 * nt][0]);
                s[2 * nt + 1][0] = fmaf(c[1], da, s[2 * nt + 1][0]);
                s[2 * nt][1] = fmaf(c[2], db, s[2 * nt][1]);
                s[2 * nt + 1][1] = fmaf(c[3], db, s[2 * nt + 1][1]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < C::LR; ++i)
        s[i][0] *= qscale[i], s[i][1] *= qscale[i];
}

// An untiled copy of `bytes` bytes (a multiple of 16) with the default L2 policy.
__device__ __forceinline__ void load_bytes(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// What a kernel over the 4-bit cache's units is given.
struct Units4Args {
    const __half *ks4, *vs4;
    int pairs;  // a page holds whole units (an even number of 16-token blocks)
};

struct Maps4 {  // the pools as [block][16][head_dim / 2] bytes
    CUtensorMap k, v;
};

// A warp's way through the units of its items: pages looked up 32 units at a time, a lane each, and copies into a
// ring of S units of shared memory, S - 1 ahead: codes by tiled tensor copies, scales by plain bulk copies,
// keys and (VALUES) values.  A whole warp makes every call.
template <int D, int S, bool VALUES>
struct Units4 {
    using T = Tile4<D>;
    static constexpr int KV = VALUES ? 2 : 1;
    // a stage: codes of keys and values, then their scales, up to where the swizzle begins anew
    static constexpr int SCALES = KV * T::CODES, STAGE = (SCALES + KV * T::SCALES + 4 * D - 1) / (4 * D) * (4 * D);
    const AttnArgs &a;
    const Units4Args &u;
    const Maps4 &maps;
    uint32_t ring, bars;          // this warp's, in shared memory
    uint32_t use = 0, phase = 0;  // the stage to read next, its barrier's phase
    int seq = 0, head = 0, lo = 0, hi = 0, first = 0, count = 0;
    int2 *list;         // of 64 units, in shared memory: their two blocks in the pool, or -1
    unsigned gone = 0, gone_next = 0;  // of this chunk of 32 units and of the next: those that miss a block

    // Where 16-token block blk of a sequence's head lies in the pool, or -1 if it is not in [lo, hi) or its page is bad.
    __device__ __forceinline__ int look_up_in(int seq, int head, int lo, int hi, int blk) const
    {
        if (blk < lo || blk >= hi)
            return -1;
        const int col = blk / a.by_blocks, page = a.kv.table[seq * a.kv.table_stride + col];
        if (page < 0 || page >= a.kv.pages) {
            kv_index_error(a.kv);
            return -1;
        }
        return (page * a.kv.heads + head - col) * a.kv.page_blocks + blk;
    }
    __device__ __forceinline__ int block_of(int blk) const { return look_up_in(seq, head, lo, hi, blk); }
    __device__ __forceinline__ int2 look_up(int i) const
    {
        int2 b = make_int2(-1, -1);
        if (i < count) {
            const int blk = first + 2 * i;
            if (u.pairs) {  // both blocks lie in one page, whichever of them is seen
                const int seen = max(blk, lo);
                b.x = block_of(seen);
                if (b.x >= 0)
                    b.x -= seen - blk;
                b.y = b.x >= 0 ? b.x + 1 : -1;
            } else {
                b.x = block_of(blk);
                b.y = block_of(blk + 1);
            }
        }
        return b;
    }
    __device__ __forceinline__ uint32_t stage() const { return ring + use * STAGE; }
    // Look up 32 units from the i-th on, a lane each; those that miss a block.
    __device__ __forceinline__ unsigned look_up_32(int i) const
    {
        const int lane = threadIdx.x & 31;
        const int2 b = look_up(i + lane);
        list[(i & 32) + lane] = b;
        return __ballot_sync(0xffffffffu, b.x < 0 || b.y < 0);
    }
    __device__ __forceinline__ void ask(int i, uint32_t put) const  // lane 0: for the item's i-th unit, into a stage
    {
        constexpr int HC = T::CODES / 2, HS = T::SCALES / 2;
        const int2 b = list[i & 63];
        const uint32_t bar = bars + 8 * put, dst = ring + put * STAGE;
        mbar_arrive_expect_tx(bar, (b.x >= 0 ? KV * (HC + HS) : 0) + (b.y >= 0 ? KV * (HC + HS) : 0));
        if (u.pairs) {
            if (b.x >= 0) {
                load_tile(dst, &maps.k, 0, b.x, bar);
                load_bytes(dst + SCALES, u.ks4 + (int64_t)b.x * (HS / 2), 2 * HS, bar);
                if constexpr (VALUES) {
                    load_tile(dst + T::CODES, &maps.v, 0, b.x, bar);
                    load_bytes(dst + SCALES + T::SCALES, u.vs4 + (int64_t)b.x * (HS / 2), 2 * HS, bar);
                }
            }
        } else {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const int one = h ? b.y : b.x;
                if (one < 0)
                    continue;
                load_tile(dst + h * HC, &maps.k, 0, one, bar);
                load_bytes(dst + SCALES + h * HS, u.ks4 + (int64_t)one * (HS / 2), HS, bar);
                if constexpr (VALUES) {
                    load_tile(dst + T::CODES + h * HC, &maps.v, 0, one, bar);
                    load_bytes(dst + SCALES + T::SCALES + h * HS, u.vs4 + (int64_t)one * (HS / 2), HS, bar);
                }
            }
        }
    }
    // An item's units: `count` of them from 16-token block `first` (even) on, of which [lo, hi) are seen.
    __device__ __forceinline__ void begin(int seq_, int head_, int lo_, int hi_, int first_, int count_)
    {
        seq = seq_, head = head_, lo = lo_, hi = hi_, first = first_, count = count_;
        __syncwarp();  // every lane has read the last item's list
        gone = look_up_32(0);
        fence_proxy_async_smem();
        __syncwarp();  // the list is written, and the last item's stages are read
        if ((threadIdx.x & 31) == 0) {
#pragma unroll 1
            for (int i = 0; i < min(S - 1, count); ++i)
                ask(i, use + i < S ? use + i : use + i - S);
        }
    }
    // Ask for the unit S - 1 ahead, and wait for unit i; false if it did not come in time.
    __device__ __forceinline__ bool next(int i)
    {
        if ((i & 15) == 0 && i > 0) {
            if (!(i & 16))
                gone = gone_next;
            else if (i + 16 < count)  // half way through a chunk the next is looked up
                gone_next = look_up_32(i + 16);
        }
        fence_proxy_async_smem();
        __syncwarp();  // every lane has read the stage that is asked for again
        if ((threadIdx.x & 31) == 0 && i + S - 1 < count)
            ask(i + S - 1, use == 0 ? S - 1 : use - 1);
        return __all_sync(0xffffffffu, mbar_wait_bounded(bars + 8 * use, phase, a.wait_ns));
    }
    __device__ __forceinline__ bool misses(int i) const { return gone >> (i & 31) & 1; }  // a block of unit i
    __device__ __forceinline__ int2 blocks(int i) const { return list[i & 63]; }
    __device__ __forceinline__ void advance()
    {
        use = use + 1 == S ? 0 : use + 1;
        phase = use == 0 ? phase ^ 1u : phase;
    }
    // After a wait that gave up: flag it, and wait (bounded) for the copies that may be in flight.
    __device__ __forceinline__ void drain()
    {
        if ((threadIdx.x & 31) == 0) {
            atomicOr(a.kv.err, (unsigned)ERRBIT_QMV_WAIT);
            for (int i = 0; i < S; ++i) {
                if (!mbar_wait_bounded(bars + 8 * use, phase, a.wait_ns)) {
                    atomicOr(a.kv.err, (unsigned)ERRBIT_DRAIN_WAIT);
                    break;
                }
                advance();
            }
        }
        __syncwarp();
    }
};

// A unit's keys, or values, as a tensor of 16-row blocks; a copy takes a unit or, where pages do not hold whole ones,
// a block, swizzled as its rows are long.
static inline qmd_status kv4_map(CUtensorMap *map, const void *base, const KvParams &kv, int head_dim, bool pairs)
{
    const TensorMapEncodeFn enc = tensor_map_encoder();
    if (!enc)
        return fail(QMD_ERR_LAUNCH, "cuTensorMapEncodeTiled entry point", cudaErrorNotSupported);
    const cuuint64_t row = (cuuint64_t)head_dim / 2;
    const cuuint64_t dim[3] = {row, KV_BLOCK, (cuuint64_t)kv.pages * kv.heads * kv.page_blocks}, str[2] = {row, row * KV_BLOCK};
    const cuuint32_t box[3] = {(cuuint32_t)row, KV_BLOCK, pairs ? 2u : 1u}, one[3] = {1, 1, 1};
    const CUtensorMapSwizzle swizzle = row == 32   ? CU_TENSOR_MAP_SWIZZLE_32B
                                       : row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                   : CU_TENSOR_MAP_SWIZZLE_128B;
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dim, str, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? QMD_OK
               : fail(QMD_ERR_LAUNCH, "tensor map of the 4-bit cache", cudaErrorInvalidValue);
}

}  // namespace qmd
