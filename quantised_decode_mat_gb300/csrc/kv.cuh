// kv.cuh -- what the key/value cache kernels share: the call's parameters, and the lookups in the
// caller's device arrays with the checks that keep a bad entry from becoming a bad address.
//
// A cache page holds, for each key/value head, page_tokens x head_dim int8 codes and one f32 scale
// for each block of 16 tokens; the blocks of one head lie one after the other, so a block is
// 16 x head_dim contiguous bytes and never crosses a page.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "internal.h"

namespace qmd {

constexpr int KV_BLOCK = QMD_KV_BLOCK;
constexpr int KV_MAX_LEN = 1 << 30;  // so that positions rounded up to a block stay in 31 bits

struct KvParams {
    int8_t *k, *v;
    float *ks, *vs;
    const int32_t *table, *len, *q_start;
    int64_t table_stride, rows, pages;
    int heads, page_blocks;  // key/value heads; blocks per page
    int seqs, max_q;
    unsigned *err;
};

struct KvSeq {
    int row0, n, len;  // first row, rows, tokens; n = 0 for a sequence left out
};

__device__ __forceinline__ void kv_index_error(const KvParams &p)
{
    atomicOr(p.err, (unsigned)ERRBIT_INDEX);
}

// Sequence s as the device arrays describe it; one whose entries are out of range is left out.
__device__ __forceinline__ KvSeq kv_seq(const KvParams &p, int s)
{
    KvSeq q;
    int end;
    if (p.q_start) {
        q.row0 = p.q_start[s];
        end = p.q_start[s + 1];
    } else {
        q.row0 = s * p.max_q;
        end = q.row0 + p.max_q;
    }
    q.len = p.len[s];
    q.n = end - q.row0;
    const bool ok = q.row0 >= 0 && end >= q.row0 && end <= p.rows && q.n <= p.max_q && q.len >= 0 &&
                    q.len <= KV_MAX_LEN && q.len <= p.table_stride * p.page_blocks * KV_BLOCK;
    if (!ok) {
        kv_index_error(p);
        q.row0 = q.n = q.len = 0;
    }
    return q;
}

// The page of block `blk` (16 positions) of sequence s, or -1 for one outside the pool.
__device__ __forceinline__ int kv_page(const KvParams &p, int s, int blk)
{
    const int32_t page = p.table[(int64_t)s * p.table_stride + blk / p.page_blocks];
    if (page < 0 || page >= p.pages) {
        kv_index_error(p);
        return -1;
    }
    return page;
}

// Where that block of a head lies in the pool, counted in blocks: its scale's place; its codes begin
// 16 * head_dim times as far.
__device__ __forceinline__ int64_t kv_block_offset(const KvParams &p, int page, int head, int blk)
{
    return ((int64_t)page * p.heads + head) * p.page_blocks + blk % p.page_blocks;
}

// The sequence that owns row t: the last one whose first row is at or before t.
__device__ __forceinline__ int kv_row_seq(const KvParams &p, int t)
{
    if (!p.q_start)
        return min(t / p.max_q, p.seqs - 1);
    int lo = 0, hi = p.seqs;  // q_start[lo] <= t < q_start[hi], as far as the array is in order
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.q_start[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <int N>
__device__ __forceinline__ void load_f32(float (&x)[N], const float *p)
{
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 a = *reinterpret_cast<const float4 *>(p + i);
            x[i] = a.x, x[i + 1] = a.y, x[i + 2] = a.z, x[i + 3] = a.w;
        }
    } else {
        static_assert(N == 2, "2 or a multiple of 4 values");
        const float2 a = *reinterpret_cast<const float2 *>(p);
        x[0] = a.x, x[1] = a.y;
    }
}

template <int N>
__device__ __forceinline__ void store_f32(float *p, const float (&x)[N])
{
    static_assert(N % 4 == 0, "a multiple of 4 values");
#pragma unroll
    for (int i = 0; i < N; i += 4)
        *reinterpret_cast<float4 *>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}

// N int8 codes at p as f32 (exact).
template <int N>
__device__ __forceinline__ void load_codes(float (&x)[N], const int8_t *p)
{
    static_assert(N % 4 == 0, "a multiple of 4 codes");
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const char4 a = *reinterpret_cast<const char4 *>(p + i);
        x[i] = (float)a.x, x[i + 1] = (float)a.y, x[i + 2] = (float)a.z, x[i + 3] = (float)a.w;
    }
}

}  // namespace qmd
