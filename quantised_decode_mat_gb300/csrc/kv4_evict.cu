// kv4_evict.cu -- taking the tokens with the least attention weight out of the 4-bit cache.
//
// Per sequence and key/value head, of the slots between the first `sinks` and the last `recent` those with the
// largest weights stay (of equal ones the earlier); what stays moves to the front in its order.  A token moves
// whole, codes, scales and weight, so nothing is rounded again.
//
// Split.  Four CTAs to a sequence and head, a cluster.  Each moves its part of every row that stays (half of the keys'
// bytes or of the values'), which lies in nobody else's way, and (SPLIT) selects among its quarter of the slots; where
// tables are short each selects among all for itself, which takes less than the cluster's meetings (12 x 8 heads of
// 1088 slots: 16.2 us against 28.4 with quarters; 8 heads of 24000: 24.9 against 18.8).
// The host decides, by the page table's width: it does not know the lengths.  So short sequences behind a wide table take the
// quarters, and shared memory for its width (those 12 x 8 heads: 15.1 us up to 4096 slots of table, 36.3 from there on, 37.8
// behind 131072, where the list has room for a whole block).
//
// Selection.  Weights become whole numbers in their order, kept in shared memory, four neighbouring slots to a thread and
// row of them (of more slots than a block of it holds, the blocks are read again for each pass).  The number that
// just stays is found by three histograms, of 11, 11 and 10 bits, each over the numbers that agree with what was
// found so far, summed over the cluster (SPLIT) by reading the others' shared memory; it ends early when a bin is taken whole.
//
// Moving, a block of slots at a time: counts of each row and warp, one scan, and ballots give every slot that stays its
// place in the list, which with SPLIT each CTA writes into all four.  A token's place is never behind its slot, and places and
// slots both rise, so a token may be written once all that come before it have been read: a round of tokens is read,
// the CTA meets, the round is written; the next round's reads may pass these writes.  Weights are moved by one
// CTA, after the barrier behind which all have read theirs.
//
// Bound: latency (some twenty dependent steps), and for few sequences what their few SMs move.  8 heads of 24000 slots to
// 2048: 18.8 us; 12 x 8 heads of 1088 to 1024: 14.9 us, half of it the moves (28 MB).
#include <mutex>
#include <type_traits>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "kv_attn.cuh"
#include "ptx.cuh"

namespace qmd {

struct Evict4Args {
    Kv4Params kv;
    float *weight;
    int keep, sinks, recent;
    int block;  // slots worked on together, at most 4 * ROWS * THREADS a share
    FastDiv by_tokens;
    int32_t *len_out, *kept;
};

constexpr int EVICT_PARTS = 4;   // CTAs to a sequence and head
constexpr int EVICT_BINS = 2048;

// Weights as whole numbers in their order: -0 as 0, NaN below everything.  (0 is no weight's key.)
constexpr unsigned EVICT_STAYS = 0xffffffffu, EVICT_NONE = 0xfffffffeu;  // nor are these

__device__ __forceinline__ unsigned weight_key(float w)
{
    if (w != w)
        return 1;
    const unsigned b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ int warp_scan(int x)  // inclusive
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o)
            x += y;
    }
    return x;
}

// All threads of the cluster meet; what they wrote to shared memory before is seen after.
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

// Where this CTA's shared memory at p lies in that of the cluster's `rank`-th.
__device__ __forceinline__ uint32_t in_cta(const void *p, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ int4 load_remote4(uint32_t at)
{
    int4 v;
    asm volatile("ld.shared::cluster.v4.s32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void store_remote16(uint32_t at, uint16_t v)
{
    asm volatile("st.shared::cluster.u16 [%0], %1;" ::"r"(at), "h"(v) : "memory");
}

// ROWS: times four keys to a thread.  SPLIT: each CTA of a cluster has a quarter of the slots.
template <int D, int THREADS, int ROWS, bool SPLIT>
__global__ void __cluster_dims__(EVICT_PARTS, 1, 1) __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1)
    kv4_evict_kernel(const Evict4Args a)
{
    constexpr int W = THREADS / 32, SHARES = SPLIT ? EVICT_PARTS : 1, PLACES = (ROWS * W + 31) / 32 * 32;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *s_key = reinterpret_cast<uint4 *>(smem);                      // of this CTA's share of a block
    uint16_t *s_src = reinterpret_cast<uint16_t *>(s_key + a.block / (4 * SHARES));  // slots that stay, counted from the block's first
    __shared__ __align__(16) int s_hists[2][EVICT_BINS], s_all[4];
    __shared__ int s_sum[W], s_found[3];
    __shared__ int s_count[PLACES], s_place[PLACES], s_take[PLACES];
    const Kv4Params &p = a.kv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, block = a.block;
    const int item = blockIdx.x / EVICT_PARTS, part = blockIdx.x % EVICT_PARTS;
    const int s = item / p.heads, head = item % p.heads;
    pdl_launch_dependents();
    pdl_wait();
    const int tokens = p.page_blocks * KV_BLOCK;
    const int32_t *table = p.table + (int64_t)s * p.table_stride;
    int len = p.len[s];
    bool ok = len >= 0 && len <= KV_MAX_LEN && len <= p.table_stride * tokens;
    if (!ok)
        len = 0;
    bool bad = false;
    for (int i = tid; i < (len + tokens - 1) / a.by_tokens; i += THREADS)
        bad |= table[i] < 0 || table[i] >= p.pages;
    ok = !__syncthreads_or(bad) && ok;
    if (part == 0 && tid == 0) {
        if (!ok)
            kv_index_error(p);
        if (head == 0)
            a.len_out[s] = ok ? min(len, a.keep) : len;
    }
    int32_t *kept = a.kept && part == 0 ? a.kept + (int64_t)item * a.keep : nullptr;
    if (!ok || len <= a.keep) {  // the same for the whole cluster
        if (kept)
            for (int i = tid; i < a.keep; i += THREADS)
                kept[i] = ok && i < len ? i : -1;
        return;
    }
    auto token = [&](int j) {
        const int col = j / a.by_tokens;
        return ((int64_t)table[col] * p.heads + head - col) * tokens + j;
    };

    // ---- which weight just stays -----------------------------------------------------------------
    const int m0 = a.sinks, m1 = len - a.recent;
    // slots that stay anyway have a key above all weights', those behind the last one below them
    auto key_at = [&](int j, float w) { return j >= len ? 0u : j < m0 || j >= m1 ? EVICT_STAYS : weight_key(w); };
    // the share of block b that this CTA has: slots c0 .. c0 + n - 1, n a multiple of 128
    int b0 = -1, c0 = 0, n = 0;
    auto load = [&](int b) {
        if (b0 == b)
            return;
        b0 = b;
        n = (min(block, len - b) + SHARES * 128 - 1) / (SHARES * 128) * 128;
        c0 = SPLIT ? b + part * n : b;
        __syncthreads();  // the last one's keys are read
#pragma unroll 4
        for (int j = 4 * tid; j < n; j += 4 * THREADS) {
            float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (c0 + j < min(len, b + block))  // (a page's tokens are a multiple of 16)
                w = *reinterpret_cast<const float4 *>(a.weight + token(c0 + j));
            s_key[j / 4] = make_uint4(key_at(c0 + j, w.x), key_at(c0 + j + 1, w.y), key_at(c0 + j + 2, w.z), key_at(c0 + j + 3, w.w));
        }
        __syncthreads();
    };
    // a row's keys of this thread (behind the share's last slot there are none)
    auto keys = [&](int r) {
        const int i = r * THREADS + tid;
        return 4 * i < n ? s_key[i] : make_uint4(0, 0, 0, 0);
    };
    auto meet = [] {  // those who have shares
        if constexpr (SPLIT)
            cluster_barrier();
        else
            __syncthreads();
    };
    int need = a.keep - a.sinks - a.recent;  // of slots [m0, m1)
    // keys from `above` on stay, and the first `need` that are `equal`
    unsigned above = EVICT_STAYS, equal = EVICT_NONE;
    if (need > 0) {
        unsigned prefix = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            // (two by turns: the others may still read the last pass's)
            int *s_hist = s_hists[pass & 1];
            for (int i = tid; i < EVICT_BINS; i += THREADS)
                s_hist[i] = 0;
            __syncthreads();
            for (int b = 0; b < len; b += block) {
                load(b);
                auto count = [&](unsigned k) {  // larger keys first; 0 is no weight
                    if (k != 0 && (pass == 0 ? k != EVICT_STAYS : k >> (shift + bits) == prefix))
                        atomicAdd(&s_hist[(1 << bits) - 1 - (int)(k >> shift & ((1u << bits) - 1))], 1);
                };
#pragma unroll 1
                for (int r = 0; 4 * r * THREADS < n; ++r) {
                    const uint4 k = keys(r);
                    count(k.x), count(k.y), count(k.z), count(k.w);
                }
            }
            meet();
            // the bin in which the need-th lies: a scan over threads of EVICT_BINS / THREADS bins each, of all shares
            constexpr int E = EVICT_BINS / THREADS;
            int h[E], sum = 0;
#pragma unroll
            for (int e = 0; e < E; e += 4) {
                h[e] = h[e + 1] = h[e + 2] = h[e + 3] = 0;
#pragma unroll
                for (int c = 0; c < SHARES; ++c) {
                    const int *at = s_hist + tid * E + e;
                    const int4 v = SPLIT ? load_remote4(in_cta(at, c)) : *reinterpret_cast<const int4 *>(at);
                    h[e] += v.x, h[e + 1] += v.y, h[e + 2] += v.z, h[e + 3] += v.w;
                }
                sum += (h[e] + h[e + 1]) + (h[e + 2] + h[e + 3]);
            }
            const int inc = warp_scan(sum);
            if (lane == 31)
                s_sum[warp] = inc;
            __syncthreads();
            const int others = warp_scan(lane < W ? s_sum[lane < W ? lane : 0] : 0);
            int before = inc - sum + (warp ? __shfl_sync(0xffffffffu, others, warp - 1) : 0);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                if (before < need && need <= before + h[e]) {
                    s_found[0] = (1 << bits) - 1 - (tid * E + e);
                    s_found[1] = need - before;
                    s_found[2] = h[e];
                }
                before += h[e];
            }
            __syncthreads();
            prefix = prefix << bits | (unsigned)s_found[0];
            need = s_found[1];
            above = prefix << shift;
            if (need == s_found[2]) {  // the bin stays whole
                need = 0;
                break;
            }
            if (pass == 2)
                equal = above++;
        }
    }

    // ---- what stays, block by block, and its move ------------------------------------------------
    constexpr int PP = D / 64;                 // 16-byte pieces of a row in this part
    const bool is_v = part & 1;
    uint4 *codes = reinterpret_cast<uint4 *>(is_v ? p.v : p.k) + (part >> 1) * PP;
    using Scales = std::conditional_t<D == 64, uint32_t, std::conditional_t<D == 128, uint2, uint4>>;
    Scales *scales = reinterpret_cast<Scales *>(is_v ? p.vs4 : p.ks4);
    const bool moves_scales = part < 2, moves_weights = part == 3;
    constexpr int M = D < 256 ? 2 : 1, ROUND = M * THREADS;  // rows read before they are written
    const unsigned below = (1u << lane) - 1;
    int place = 0;
    for (int b = 0; b < len; b += block) {
        load(b);
        __syncthreads();
#pragma unroll 1
        for (int r = 0; r < ROWS; ++r) {
            const uint4 k = keys(r);
            // those that stay in the low half, those that are just equal in the high
            int m = (k.x >= above) + (k.y >= above) + (k.z >= above) + (k.w >= above);
            m += ((k.x == equal) + (k.y == equal) + (k.z == equal) + (k.w == equal)) << 16;
            m = __reduce_add_sync(0xffffffffu, m);
            if (lane == 0)
                s_count[r * W + warp] = m;
        }
        if (tid >= ROWS * W && tid < PLACES)
            s_count[tid] = 0;
        __syncthreads();
        constexpr int E = PLACES / 32;
        int m[E], same = 0, stay = 0;
        if (warp == 0) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
                m[e] = s_count[lane * E + e];
                same += m[e] >> 16;
                stay += m[e] & 0xffff;
            }
            const int all_same = __reduce_add_sync(0xffffffffu, same), all_stay = __reduce_add_sync(0xffffffffu, stay);
            if (lane == 0)
                s_all[0] = all_stay, s_all[1] = all_same;
        }
        meet();  // (behind which, too, the others have read the last block's list)
        // this CTA's first place, and how many of its equals stay: the shares lie one after the other
        int first = 0, room = 0, total = 0, taken = 0;
#pragma unroll
        for (int c = 0; c < SHARES; ++c) {
            const int4 v = SPLIT ? load_remote4(in_cta(s_all, c)) : *reinterpret_cast<const int4 *>(s_all);
            const int take = max(0, min(v.y, need - taken));
            if (!SPLIT || c == part)
                first = total, room = take;
            total += v.x + take;
            taken += take;
        }
        total = min(total, a.keep - place);
        if (warp == 0) {  // in the slots' order: row after row, warp after warp
            int same_before = warp_scan(same) - same, take[E], sum = stay;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                take[e] = max(0, min(m[e] >> 16, room - same_before));
                same_before += m[e] >> 16;
                sum += take[e];
            }
            int at = first + warp_scan(sum) - sum;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s_place[lane * E + e] = at;
                s_take[lane * E + e] = take[e];
                at += (m[e] & 0xffff) + take[e];
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int r = 0; 4 * r * THREADS < n; ++r) {
            const uint4 k4 = keys(r);
            const unsigned k[4] = {k4.x, k4.y, k4.z, k4.w};
            const int left = s_take[r * W + warp];
            bool stays[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                stays[c] = k[c] >= above;
            if (left > 0) {  // the first of those that are just equal
                int rank = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    rank += __popc(__ballot_sync(0xffffffffu, k[c] == equal) & below);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (k[c] == equal)
                        stays[c] |= rank++ < left;
            }
            int at = s_place[r * W + warp];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                at += __popc(__ballot_sync(0xffffffffu, stays[c]) & below);
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (stays[c]) {
                    const uint16_t j = (uint16_t)(c0 - b + 4 * (r * THREADS + tid) + c);
                    if constexpr (SPLIT) {
#pragma unroll
                        for (int to = 0; to < EVICT_PARTS; ++to)
                            store_remote16(in_cta(s_src + at, to), j);
                    } else {
                        s_src[at] = j;
                    }
                    ++at;
                }
        }
        need -= taken;
        cluster_barrier();  // the list is whole, and this block's weights are read
        if (kept)
            for (int i = tid; i < total; i += THREADS)
                kept[place + i] = b + s_src[i];
        for (int i0 = 0; i0 < total; i0 += ROUND) {
            const int n = min(ROUND, total - i0);
            if (b + s_src[i0 + n - 1] == place + i0 + n - 1)  // all of them are where they stay
                continue;
            // a thread a row: its sector of codes, and its scales or its weight
            uint4 x[M][PP];
            Scales d[M];
            float w[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int i = tid + m * THREADS;
                if (i < n) {
                    const int64_t from = token(b + s_src[i0 + i]);
#pragma unroll
                    for (int e = 0; e < PP; ++e)
                        x[m][e] = codes[from * (D / 32) + e];
                    if (moves_scales)
                        d[m] = scales[from];
                    if (moves_weights)
                        w[m] = a.weight[from];
                }
            }
            __syncthreads();
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const int i = tid + m * THREADS;
                if (i < n) {
                    const int64_t to = token(place + i0 + i);
#pragma unroll
                    for (int e = 0; e < PP; ++e)
                        codes[to * (D / 32) + e] = x[m][e];
                    if (moves_scales)
                        scales[to] = d[m];
                    if (moves_weights)
                        a.weight[to] = w[m];
                }
            }
        }
        place += total;
    }
}

template <int D, int THREADS, int ROWS, bool SPLIT>
static qmd_status launch_evict4(Evict4Args a, const DeviceInfo &dev, cudaStream_t s)
{
    // a block: as many slots as the page table has room for, up to what the threads take; a list of those that stay
    constexpr int SHARES = SPLIT ? EVICT_PARTS : 1, MOST = SHARES * THREADS * 4 * ROWS;
    static_assert(MOST <= 65536, "listed in 16 bits");
    const int64_t room = a.kv.table_stride * a.kv.page_blocks * KV_BLOCK;
    a.block = room < MOST ? (int)((room + 511) / 512 * 512) : MOST;  // (shares of whole 128s)
    // (blocks that are read more than once could be written by someone in between: then any number may stay)
    const int list = a.keep < a.block && room <= MOST ? a.keep : a.block;
    const size_t smem = (size_t)a.block * 4 / SHARES + (list * 2 + 15) / 16 * 16;
    {   // with what the kernel declares itself (18016 bytes, SPLIT) a launch may pass 48 KB from 31 KB on: asked for
        // once per device, whatever the first call's size
        static std::mutex mu;
        static bool opted[64] = {false};
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[dev.device]) {
            const cudaError_t e = cudaFuncSetAttribute(kv4_evict_kernel<D, THREADS, ROWS, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       MOST * 4 / SHARES + MOST * 2);
            if (e != cudaSuccess)
                return fail(QMD_ERR_LAUNCH, "kv4_evict smem attribute", e);
            opted[dev.device] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.kv.seqs * a.kv.heads * EVICT_PARTS));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_evict_kernel<D, THREADS, ROWS, SPLIT>, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv4_evict launch", e);
}

qmd_status launch_kv4_evict(const Kv4Params &kv, int head_dim, float *weight, int keep, int sinks, int recent,
                            int32_t *len_out, int32_t *kept, const DeviceInfo &dev, cudaStream_t s)
{
    const int tokens = kv.page_blocks * KV_BLOCK;
    const Evict4Args a = {kv, weight, keep, sinks, recent, 0, fast_div((unsigned)tokens), len_out, kept};
    // short tables: small CTAs, many to an SM
    const bool small = kv.table_stride * tokens <= 4096;
    switch (head_dim) {
    case 64: return small ? launch_evict4<64, 256, 4, false>(a, dev, s) : launch_evict4<64, 512, 8, true>(a, dev, s);
    case 128: return small ? launch_evict4<128, 256, 4, false>(a, dev, s) : launch_evict4<128, 512, 8, true>(a, dev, s);
    default: return small ? launch_evict4<256, 256, 4, false>(a, dev, s) : launch_evict4<256, 512, 8, true>(a, dev, s);
    }
}

}  // namespace qmd
