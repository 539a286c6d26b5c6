// kv4.cuh -- the 4-bit key/value cache's parameters and codes.
//
// A token's head is head_dim / 2 bytes of codes, dimension 2 i in the low four bits of byte i, and an f16
// scale d for each group of 32 dimensions; a value is d (c - 8).
#pragma once

#include <cstdint>
#include <cuda_fp16.h>

#include "kv.cuh"

namespace qmd {

constexpr int KV4_GROUP = QMD_KV4_GROUP;

struct Kv4Params : KvParams {  // k and v: bytes of codes; ks and vs are not used
    __half *ks4, *vs4;
};

// Where slot `pos` of a head lies in the pool, counted in tokens: that of its weight; its codes begin
// head_dim / 2 bytes times as far, its scales head_dim / 32 f16 times.
__device__ __forceinline__ int64_t kv4_token(const KvParams &p, int page, int head, int pos)
{
    return ((int64_t)page * p.heads + head) * p.page_blocks * KV_BLOCK + pos % (p.page_blocks * KV_BLOCK);
}

// N codes, less 8, of the N / 2 bytes in w (exact).
template <int N>
__device__ __forceinline__ void unpack4(float (&x)[N], uint32_t w)
{
    static_assert(N <= 8, "a word holds 8 codes");
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = (float)((int)(w >> 4 * i & 15u) - 8);
}

}  // namespace qmd
