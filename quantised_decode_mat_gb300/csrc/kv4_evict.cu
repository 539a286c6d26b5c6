// kv4_evict.cu -- taking the tokens with the least attention weight out of the 4-bit cache.
//
// Per sequence and key/value head, of the slots between the first `sinks` and the last `recent` those with the
// largest weights stay (of equal ones the earlier); what stays moves to the front in its order.  A token moves
// whole, codes, scales and weight, so nothing is rounded again.
//
// Selection.  Weights become whole numbers in their order, kept in shared memory (those past CAP are read again).
// The number that just stays is found by three histograms, of 11, 11 and 10 bits, each over the numbers
// that agree with what was found so far; it ends early when a bin is taken whole.
//
// Moving.  A window of slots at a time (all of them, where the list of what stays fits): ballots give each warp its
// counts, one scan over the warps the places, and a second round of ballots the list.  A token's place is never behind
// its slot, and places and slots both rise, so a token may be written once all that come before it have been
// read: a round of tokens is read, the CTA meets, the round is written; the next round's reads may pass these writes.
//
// Split.  Four CTAs to a sequence and head, a cluster: each selects for itself, and moves its part of every row
// (half of the keys' bytes or of the values'), which lies in nobody else's way.  Weights, which all four have
// to have read, are moved by one of them, after a barrier of the cluster in each window.
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
    int cap, list;  // weights, and slots that stay, that shared memory holds (multiples of 16)
    FastDiv by_tokens;
    int32_t *len_out, *kept;
};

constexpr int EVICT_PARTS = 4;   // CTAs to a sequence and head
constexpr int EVICT_BINS = 2048;
constexpr int EVICT_LIST = 8192; // slots that stay, of a window
constexpr int EVICT_CAP = 32768;

// Weights as whole numbers in their order: -0 as 0, NaN below everything.
__device__ __forceinline__ unsigned weight_key(float w)
{
    if (w != w)
        return 0;
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

template <int D, int THREADS>
__global__ void __cluster_dims__(EVICT_PARTS, 1, 1) __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1)
    kv4_evict_kernel(const Evict4Args a)
{
    constexpr int W = THREADS / 32;
    extern __shared__ __align__(16) unsigned s_key[];  // [cap], then [list] slots that stay
    __shared__ int s_hist[EVICT_BINS], s_sum[W], s_equal[W], s_found[3];
    const Kv4Params &p = a.kv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = blockIdx.x / EVICT_PARTS, part = blockIdx.x % EVICT_PARTS;
    const int s = item / p.heads, head = item % p.heads;
    int *s_src = reinterpret_cast<int *>(s_key + a.cap);
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
    // four at a time (a page's tokens are a multiple of 16)
#pragma unroll 4
    for (int j = 4 * tid; j < min(len, a.cap); j += 4 * THREADS) {
        const float4 w = *reinterpret_cast<const float4 *>(a.weight + token(j));
        *reinterpret_cast<uint4 *>(s_key + j) = make_uint4(weight_key(w.x), weight_key(w.y), weight_key(w.z), weight_key(w.w));
    }
    __syncthreads();
    auto key_of = [&](int j) { return j < a.cap ? s_key[j] : weight_key(a.weight[token(j)]); };
    const int m0 = a.sinks, m1 = len - a.recent;
    int need = a.keep - a.sinks - a.recent;  // of slots [m0, m1)
    unsigned above = 0xffffffffu, equal = 0;  // keys from `above` on stay, and the first `need` that are `equal`
    if (need > 0) {
        unsigned prefix = 0;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < EVICT_BINS; i += THREADS)
                s_hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int j = m0 + tid; j < m1; j += THREADS) {
                const unsigned k = key_of(j);
                if (pass == 0 || k >> (shift + bits) == prefix)  // larger keys first
                    atomicAdd(&s_hist[(1 << bits) - 1 - (int)(k >> shift & ((1u << bits) - 1))], 1);
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

    // ---- what stays, window by window, and its move ------------------------------------------------
    constexpr int PP = D / 64;                 // 16-byte pieces of a row in this part
    const bool is_v = part & 1;
    uint4 *codes = reinterpret_cast<uint4 *>(is_v ? p.v : p.k) + (part >> 1) * PP;
    using Scales = std::conditional_t<D == 64, uint32_t, std::conditional_t<D == 128, uint2, uint4>>;
    Scales *scales = reinterpret_cast<Scales *>(is_v ? p.vs4 : p.ks4);
    const bool moves_scales = part < 2, moves_weights = part == 3;
    constexpr int M = (THREADS == 256 ? 4 : 2) / (D == 256 ? 2 : 1), ROUND = M * THREADS;  // rows read before they are written
    const int window = a.keep <= a.list ? (len + 32 * W - 1) / (32 * W) * (32 * W) : a.list / (32 * W) * (32 * W);
    const int steps = window / (32 * W);  // times 32 slots of a warp
    int place = 0;
    for (int w0 = 0; w0 < len; w0 += window) {
        const int j0 = w0 + warp * 32 * steps + lane;
        auto stays = [&](int j, bool &same) {  // surely; or if there is room for one that is just equal
            same = false;
            if (j < m0 || j >= m1)
                return j < len;
            const unsigned k = key_of(j);
            same = need > 0 && k == equal;
            return k >= above;
        };
        int n_stay = 0, n_same = 0;
#pragma unroll 4
        for (int i = 0; i < steps; ++i) {
            bool same;
            n_stay += __popc(__ballot_sync(0xffffffffu, stays(j0 + 32 * i, same)));
            n_same += __popc(__ballot_sync(0xffffffffu, same));
        }
        __syncthreads();  // the last window's list and sums are read
        if (lane == 0)
            s_sum[warp] = n_stay, s_equal[warp] = n_same;
        __syncthreads();
        const int their_same = lane < W ? s_equal[lane < W ? lane : 0] : 0;
        const int same_before = warp_scan(their_same) - their_same;
        const int take = max(0, min(their_same, need - same_before));
        const int theirs = (lane < W ? s_sum[lane < W ? lane : 0] : 0) + take;
        const int upto = warp_scan(theirs), taken = warp_scan(take);
        const int total = __shfl_sync(0xffffffffu, upto, 31);
        int at = __shfl_sync(0xffffffffu, upto - theirs, warp), left = __shfl_sync(0xffffffffu, take, warp);
        for (int i = 0; i < steps; ++i) {
            bool same;
            unsigned mine = __ballot_sync(0xffffffffu, stays(j0 + 32 * i, same));
            const unsigned eq = __ballot_sync(0xffffffffu, same);
            const unsigned first = __ballot_sync(0xffffffffu, same && __popc(eq & ((1u << lane) - 1)) < left);
            left -= __popc(first);
            mine |= first;
            if (mine >> lane & 1)
                s_src[at + __popc(mine & ((1u << lane) - 1))] = j0 + 32 * i;
            at += __popc(mine);
        }
        need -= __shfl_sync(0xffffffffu, taken, 31);
        __syncthreads();
        cluster_arrive();  // this window's weights are read
        if (kept)
            for (int i = tid; i < total; i += THREADS)
                kept[place + i] = s_src[i];
        cluster_wait();
        for (int i0 = 0; i0 < total; i0 += ROUND) {
            const int n = min(ROUND, total - i0);
            if (s_src[i0 + n - 1] == place + i0 + n - 1)  // all of them are where they stay
                continue;
            uint4 x[M * PP];
            Scales d[M];
            float w[M];
#pragma unroll
            for (int e = 0; e < M * PP; ++e) {
                const int i = (tid + e * THREADS) / PP, piece = (tid + e * THREADS) % PP;
                if (i < n)
                    x[e] = codes[token(s_src[i0 + i]) * (D / 32) + piece];
            }
#pragma unroll
            for (int e = 0; e < M; ++e) {
                const int i = tid + e * THREADS;
                if (i < n && moves_scales)
                    d[e] = scales[token(s_src[i0 + i])];
                if (i < n && moves_weights)
                    w[e] = a.weight[token(s_src[i0 + i])];
            }
            __syncthreads();
#pragma unroll
            for (int e = 0; e < M * PP; ++e) {
                const int i = (tid + e * THREADS) / PP, piece = (tid + e * THREADS) % PP;
                if (i < n)
                    codes[token(place + i0 + i) * (D / 32) + piece] = x[e];
            }
#pragma unroll
            for (int e = 0; e < M; ++e) {
                const int i = tid + e * THREADS;
                if (i < n && moves_scales)
                    scales[token(place + i0 + i)] = d[e];
                if (i < n && moves_weights)
                    a.weight[token(place + i0 + i)] = w[e];
            }
        }
        place += total;
    }
}

template <int D, int THREADS>
static qmd_status launch_evict4(Evict4Args a, cudaStream_t s)
{
    // shared memory for as many weights as the page table's columns can hold, up to EVICT_CAP
    const int64_t most = a.kv.table_stride * a.kv.page_blocks * KV_BLOCK;
    a.cap = (int)(most < EVICT_CAP ? most : EVICT_CAP);
    a.list = (int)(most < EVICT_LIST ? (most + THREADS - 1) / THREADS * THREADS : EVICT_LIST);
    const size_t smem = ((size_t)a.cap + a.list) * 4;
    if (smem > 32 * 1024) {  // (48 KB with what the kernel declares itself need no asking)
        static std::mutex mu;
        static std::set<int> opted;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess)
            return QMD_ERR_DEVICE;
        std::lock_guard<std::mutex> lock(mu);
        if (!opted.count(dev)) {
            const cudaError_t e = cudaFuncSetAttribute(kv4_evict_kernel<D, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (EVICT_CAP + EVICT_LIST) * 4);
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kv4_evict_kernel<D, THREADS>, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv4_evict launch", e);
}

qmd_status launch_kv4_evict(const Kv4Params &kv, int head_dim, float *weight, int keep, int sinks, int recent,
                            int32_t *len_out, int32_t *kept, const DeviceInfo &dev, cudaStream_t s)
{
    const int tokens = kv.page_blocks * KV_BLOCK;
    const Evict4Args a = {kv, weight, keep, sinks, recent, 0, 0, fast_div((unsigned)tokens), len_out, kept};
    // short tables: small CTAs, many to an SM
    const bool small = kv.table_stride * tokens <= 4096;
    switch (head_dim) {
    case 64: return small ? launch_evict4<64, 256>(a, s) : launch_evict4<64, 1024>(a, s);
    case 128: return small ? launch_evict4<128, 256>(a, s) : launch_evict4<128, 1024>(a, s);
    default: return small ? launch_evict4<256, 256>(a, s) : launch_evict4<256, 1024>(a, s);
    }
}

}  // namespace qmd
