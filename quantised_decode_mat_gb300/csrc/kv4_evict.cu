// kv4_evict.cu -- taking the tokens with the least attention weight out of the 4-bit cache.
//
// Per sequence and key/value head, of the slots between the first `sinks` and the last `recent` those with the
// largest weights stay (of equal ones the earlier); what stays moves to the front in its order.  A token moves
// whole, codes, scales and weight, so nothing is rounded again.
//
// A CTA to a sequence and head.  The weight that just stays is found bit by bit, counting; then chunks of slots
// in order: a running sum over what stays gives the places.  A token's place is never behind its slot, so a
// chunk that is read before any of it is written disturbs none that comes after it.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace qmd {

struct Evict4Args {
    Kv4Params kv;
    float *weight;
    int keep, sinks, recent;
    int32_t *len_out, *kept;
};

constexpr int EVICT_THREADS = 512;

// Weights as whole numbers in their order: -0 as 0, NaN below everything.
__device__ __forceinline__ unsigned weight_key(float w)
{
    if (w != w)
        return 0;
    const unsigned b = __float_as_uint(w + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the CTA, and this thread's exclusive sum.
__device__ __forceinline__ int block_scan(int x, int *s_sum, int *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int sum = x;
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o)
            sum += y;
    }
    __syncthreads();
    if (lane == 31)
        s_sum[warp] = sum;
    __syncthreads();
    int base = 0, all = 0;
    for (int w = 0; w < EVICT_THREADS / 32; ++w) {
        if (w < warp)
            base += s_sum[w];
        all += s_sum[w];
    }
    *total = all;
    return base + sum - x;
}

template <int D>
__global__ void __launch_bounds__(EVICT_THREADS) kv4_evict_kernel(const Evict4Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    __shared__ int s_sum[EVICT_THREADS / 32], s_src[EVICT_THREADS];
    const Kv4Params &p = a.kv;
    const int s = blockIdx.x / p.heads, head = blockIdx.x % p.heads, tid = threadIdx.x;
    const int tokens = p.page_blocks * KV_BLOCK;
    const int32_t *table = p.table + (int64_t)s * p.table_stride;
    int len = p.len[s];
    bool ok = len >= 0 && len <= KV_MAX_LEN && len <= p.table_stride * tokens;
    if (!ok)
        len = 0;
    bool bad = false;
    for (int i = tid; i < (len + tokens - 1) / tokens; i += EVICT_THREADS)
        bad |= table[i] < 0 || table[i] >= p.pages;
    bad = __syncthreads_or(bad);
    ok = ok && !bad;
    if (!ok && tid == 0)
        kv_index_error(p);
    if (head == 0 && tid == 0)
        a.len_out[s] = ok ? min(len, a.keep) : len;
    int32_t *kept = a.kept ? a.kept + (int64_t)blockIdx.x * a.keep : nullptr;
    if (!ok || len <= a.keep) {
        if (kept)
            for (int i = tid; i < a.keep; i += EVICT_THREADS)
                kept[i] = ok && i < len ? i : -1;
        return;
    }
    auto token = [&](int j) { return kv4_token(p, table[j / tokens], head, j); };
    const int need = a.keep - a.sinks - a.recent, m0 = a.sinks, m1 = len - a.recent;
    // the largest key that at least `need` have or pass
    unsigned key = 0;
    for (int bit = 31; bit >= 0; --bit) {
        const unsigned with = key | 1u << bit;
        int n = 0, total;
        for (int j = m0 + tid; j < m1; j += EVICT_THREADS)
            n += weight_key(a.weight[token(j)]) >= with;
        block_scan(n, s_sum, &total);
        if (total >= need)
            key = with;
    }
    int above = 0;
    {
        int n = 0;
        for (int j = m0 + tid; j < m1; j += EVICT_THREADS)
            n += weight_key(a.weight[token(j)]) > key;
        block_scan(n, s_sum, &above);
    }
    int equal_left = need - above, place = 0;
    for (int j0 = 0; j0 < len; j0 += EVICT_THREADS) {
        const int j = j0 + tid;
        bool stay = j < len && (j < m0 || j >= m1), equal = false;
        if (j >= m0 && j < m1) {
            const unsigned k = weight_key(a.weight[token(j)]);
            stay = k > key;
            equal = k == key;
        }
        int total;
        const int before = block_scan(equal, s_sum, &total);
        if (equal && before < equal_left)
            stay = true;
        equal_left = max(0, equal_left - total);
        const int at = block_scan(stay, s_sum, &total);
        __syncthreads();
        if (stay)
            s_src[at] = j;
        __syncthreads();
        if (kept)
            for (int i = tid; i < total; i += EVICT_THREADS)
                kept[place + i] = s_src[i];
        // words of a token: codes of K and V, their scales, the weight
        constexpr int C = D / 8, S = D / 64, W = 2 * C + 2 * S + 1;
        for (int i0 = 0; i0 < total * W; i0 += EVICT_THREADS) {
            const int i = i0 + tid;
            uint32_t *to = nullptr, x = 0;
            if (i < total * W) {
                const int w = i % W;
                const int64_t src = token(s_src[i / W]), dst = token(place + i / W);
                auto word = [&](int64_t t) {
                    return w < C           ? reinterpret_cast<uint32_t *>(p.k) + t * C + w
                           : w < 2 * C     ? reinterpret_cast<uint32_t *>(p.v) + t * C + w - C
                           : w < 2 * C + S ? reinterpret_cast<uint32_t *>(p.ks4) + t * S + w - 2 * C
                           : w < W - 1     ? reinterpret_cast<uint32_t *>(p.vs4) + t * S + w - 2 * C - S
                                           : reinterpret_cast<uint32_t *>(a.weight) + t;
                };
                to = word(dst);
                x = *word(src);
            }
            __syncthreads();
            if (to)
                *to = x;
        }
        __syncthreads();
        place += total;
    }
}

qmd_status launch_kv4_evict(const Kv4Params &kv, int head_dim, float *weight, int keep, int sinks, int recent,
                            int32_t *len_out, int32_t *kept, const DeviceInfo &dev, cudaStream_t s)
{
    const Evict4Args a = {kv, weight, keep, sinks, recent, len_out, kept};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(kv.seqs * kv.heads));
    cfg.blockDim = dim3(EVICT_THREADS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = head_dim == 64    ? cudaLaunchKernelEx(&cfg, kv4_evict_kernel<64>, a)
                          : head_dim == 128 ? cudaLaunchKernelEx(&cfg, kv4_evict_kernel<128>, a)
                                            : cudaLaunchKernelEx(&cfg, kv4_evict_kernel<256>, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv4_evict launch", e);
}

}  // namespace qmd
