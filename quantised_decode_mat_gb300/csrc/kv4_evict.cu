// kv4_evict.cu -- taking the tokens with the least attention weight out of the 4-bit cache.
//
// Per sequence and key/value head, of the slots between the first `sinks` and the last `recent` those with the
// largest weights stay (of equal ones the earlier); what stays moves to the front in its order.  A token moves
// whole, codes, scales and weight, so nothing is rounded again.
//
// Selection.  Weights become whole numbers in their order, kept in shared memory, four neighbouring slots to a thread and
// row of them (of more slots than a block of it holds, the blocks are read again for each pass).  The number that
// just stays is found by three histograms in shared memory, of 11, 11 and 10 bits, each over the numbers that agree
// with what was found so far; it ends early when a bin is taken whole.
//
// Moving, a block of slots at a time: ballots give each warp its counts, one scan over rows and warps the places, and
// the ballots again the list of what stays.  A token's place is never behind its slot, and places and slots both
// rise, so a token may be written once all that come before it have been read: a round of tokens is read, the CTA
// meets, the round is written; the next round's reads may pass these writes.
//
// Split.  Four CTAs to a sequence and head, a cluster: each selects for itself, and moves its part of every row
// (half of the keys' bytes or of the values'), which lies in nobody else's way.  Weights, which all four have
// to have read, are moved by one of them, after a barrier of the cluster in each block.
//
// Bound: latency (some ten dependent steps), and for few sequences what their few SMs move.
#include <mutex>
#include <set>
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
    int block;  // slots worked on together, at most 4 * ROWS * THREADS
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

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// ROWS: times four keys to a thread
template <int D, int THREADS, int ROWS>
__global__ void __cluster_dims__(EVICT_PARTS, 1, 1) __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1)
    kv4_evict_kernel(const Evict4Args a)
{
    constexpr int W = THREADS / 32, PLACES = ROWS * W;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4 *s_key = reinterpret_cast<uint4 *>(smem);                     // of a block's slots, [block / 4]
    uint16_t *s_src = reinterpret_cast<uint16_t *>(s_key + a.block / 4);  // those that stay, counted from the block's first
    __shared__ int s_hist[EVICT_BINS], s_sum[W], s_found[3];
    __shared__ int s_count[PLACES], s_place[PLACES], s_take[PLACES], s_total[2];
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
    int b0 = -1;  // the block whose keys are in shared memory
    auto load = [&](int b) {
        if (b0 == b)
            return;
        b0 = b;
        __syncthreads();  // the last one's are read
#pragma unroll 4
        for (int j = 4 * tid; j < block; j += 4 * THREADS) {
            float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (b + j < len)  // (a page's tokens are a multiple of 16)
                w = *reinterpret_cast<const float4 *>(a.weight + token(b + j));
            s_key[j / 4] = make_uint4(key_at(b + j, w.x), key_at(b + j + 1, w.y), key_at(b + j + 2, w.z), key_at(b + j + 3, w.w));
        }
        __syncthreads();
    };
    auto rows = [&] { return (min(block, len - b0) + 4 * THREADS - 1) / (4 * THREADS); };
    // a row's keys of this thread (behind the block's last slot there are none)
    auto keys = [&](int r) {
        const int i = r * THREADS + tid;
        return 4 * i < block ? s_key[i] : make_uint4(0, 0, 0, 0);
    };
    int need = a.keep - a.sinks - a.recent;  // of slots [m0, m1)
    // keys from `above` on stay, and the first `need` that are `equal`
    unsigned above = EVICT_STAYS, equal = EVICT_NONE;
    if (need > 0) {
        unsigned prefix = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < EVICT_BINS; i += THREADS)
                s_hist[i] = 0;
            __syncthreads();
            for (int b = 0; b < len; b += block) {
                load(b);
                auto count = [&](unsigned k) {  // larger keys first; 0 is no weight
                    if (k != 0 && (pass == 0 ? k != EVICT_STAYS : k >> (shift + bits) == prefix))
                        atomicAdd(&s_hist[(1 << bits) - 1 - (int)(k >> shift & ((1u << bits) - 1))], 1);
                };
                const int n = rows();
#pragma unroll 1
                for (int r = 0; r < n; ++r) {
                    const uint4 k = keys(r);
                    count(k.x), count(k.y), count(k.z), count(k.w);
                }
            }
            __syncthreads();
            // the bin in which the need-th lies: a scan over threads of EVICT_BINS / THREADS bins each
            constexpr int E = EVICT_BINS / THREADS;
            int h[E], sum = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                sum += h[e] = s_hist[tid * E + e];
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
        __syncthreads();  // the last block's list is read
        const int n_rows = rows();
#pragma unroll 1
        for (int r = 0; r < ROWS; ++r) {
            const uint4 k = r < n_rows ? keys(r) : make_uint4(0, 0, 0, 0);
            // those that stay in the low half, those that are just equal in the high
            int n = (k.x >= above) + (k.y >= above) + (k.z >= above) + (k.w >= above);
            n += ((k.x == equal) + (k.y == equal) + (k.z == equal) + (k.w == equal)) << 16;
            n = __reduce_add_sync(0xffffffffu, n);
            if (lane == 0)
                s_count[r * W + warp] = n;
        }
        __syncthreads();
        if (warp == 0) {  // in the slots' order: row after row, warp after warp
            constexpr int E = PLACES / 32;
            int n[E], same = 0, stay = 0;
#pragma unroll
            for (int e = 0; e < E; ++e)
                same += (n[e] = s_count[lane * E + e]) >> 16;
            int same_before = warp_scan(same) - same, take[E];
#pragma unroll
            for (int e = 0; e < E; ++e) {
                take[e] = max(0, min(n[e] >> 16, need - same_before));
                same_before += n[e] >> 16;
                stay += (n[e] & 0xffff) + take[e];
            }
            const int upto = warp_scan(stay);
            int at = upto - stay, taken = 0;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                s_place[lane * E + e] = at;
                s_take[lane * E + e] = take[e];
                at += (n[e] & 0xffff) + take[e];
                taken += take[e];
            }
            taken = __reduce_add_sync(0xffffffffu, taken);
            if (lane == 31)
                s_total[0] = upto, s_total[1] = taken;
        }
        __syncthreads();
        const int total = min(s_total[0], a.keep - place);
#pragma unroll 1
        for (int r = 0; r < n_rows; ++r) {
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
                if (stays[c])
                    s_src[at++] = (uint16_t)(4 * (r * THREADS + tid) + c);
        }
        need -= s_total[1];
        __syncthreads();
        cluster_arrive();  // this block's weights are read
        if (kept)
            for (int i = tid; i < total; i += THREADS)
                kept[place + i] = b + s_src[i];
        cluster_wait();
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

template <int D, int THREADS, int ROWS>
static qmd_status launch_evict4(Evict4Args a, cudaStream_t s)
{
    // a block: as many slots as the page table has room for, up to what the threads take; a list of those that stay
    constexpr int MOST = THREADS * 4 * ROWS;
    static_assert(MOST <= 65536, "listed in 16 bits");
    const int64_t room = a.kv.table_stride * a.kv.page_blocks * KV_BLOCK;
    a.block = (int)(room < MOST ? room : MOST);
    // (blocks that are read more than once could be written by someone in between: then any number may stay)
    const int list = a.keep < a.block && room <= MOST ? a.keep : a.block;
    const size_t smem = (size_t)a.block * 4 + (list * 2 + 15) / 16 * 16;
    if (smem > 32 * 1024) {  // (48 KB with what the kernel declares itself need no asking)
        static std::mutex mu;
        static std::set<int> opted;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess)
            return QMD_ERR_DEVICE;
        std::lock_guard<std::mutex> lock(mu);
        if (!opted.count(dev)) {
            const cudaError_t e = cudaFuncSetAttribute(kv4_evict_kernel<D, THREADS, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       MOST * 6);
            if (e != cudaSuccess)
                return fail(QMD_ERR_LAUNCH, "kv4_evict smem attribute", e);
            opted.insert(dev);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_evict_kernel<D, THREADS, ROWS>, a);
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
    case 64: return small ? launch_evict4<64, 256, 4>(a, s) : launch_evict4<64, 1024, 8>(a, s);
    case 128: return small ? launch_evict4<128, 256, 4>(a, s) : launch_evict4<128, 1024, 8>(a, s);
    default: return small ? launch_evict4<256, 256, 4>(a, s) : launch_evict4<256, 1024, 8>(a, s);
    }
}

}  // namespace qmd
