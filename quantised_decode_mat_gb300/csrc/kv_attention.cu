// kv_attention.cu -- attention of a decode step's rows over the paged 8-bit key/value cache.
//
// "Language models on the device: the cajeta-llm kernels", §2.5: attention over the key/value
// cache, 1, 4 or 8 query heads to a key/value head.  Per row at position p and query head, over the
// positions j that it sees:  out = sum_j e^(s_j - m) V[j] / sum_j e^(s_j - m),  s_j = scale q . K[j].
// One pass with a running maximum m and sum.
//
// Plain form: one warp per (row, query head), a position at a time.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace qmd {

struct AttnArgs {
    KvParams kv;
    const float *q;
    float *out;
    int64_t q_stride, out_stride, window;
    int q_heads;
    float scale;
};

template <int D>
__global__ void __launch_bounds__(32) kv_attention_kernel(const AttnArgs a)
{
    constexpr int E = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const KvParams &p = a.kv;
    const int lane = threadIdx.x;
    const int s = blockIdx.x / p.max_q, i = blockIdx.x % p.max_q, h = blockIdx.y;
    const int g = h / (a.q_heads / p.heads);
    const KvSeq sq = kv_seq(p, s);
    if (i >= sq.n)
        return;
    const int64_t row = sq.row0 + i;
    float x[E], o[E] = {};
    load_f32(x, a.q + row * a.q_stride + h * D + E * lane);
    const int pos = sq.len - sq.n + i;
    const int begin = a.window > 0 && pos + 1 > a.window ? (int)(pos + 1 - a.window) : 0;
    float m = -INFINITY, l = 0.0f;
    for (int j = begin; j <= pos; ++j) {
        const int page = kv_page(p, s, j / KV_BLOCK);
        if (page < 0)
            continue;
        const int64_t blk = kv_block_offset(p, page, g, j / KV_BLOCK);
        float c[E];
        load_codes(c, p.k + (blk * KV_BLOCK + j % KV_BLOCK) * D + E * lane);
        float t = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e)
            t = fmaf(x[e], c[e], t);
#pragma unroll
        for (int w = 16; w > 0; w >>= 1)
            t += __shfl_xor_sync(0xffffffffu, t, w);
        t *= p.ks[blk] * a.scale;
        const float mn = fmaxf(m, t), f = m == mn ? 1.0f : expf(m - mn), w = p.vs[blk], pr = expf(t - mn);
        m = mn;
        l = l * f + pr;
        load_codes(c, p.v + (blk * KV_BLOCK + j % KV_BLOCK) * D + E * lane);
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[e] = fmaf(pr * w, c[e], o[e] * f);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        o[e] = l == 0.0f ? 0.0f : o[e] / l;
    store_f32(a.out + row * a.out_stride + h * D + E * lane, o);
}

qmd_status launch_kv_attention(const KvParams &kv, int head_dim, const float *q, int64_t q_stride, int q_heads,
                               float scale, int64_t window, float *out, int64_t out_stride, void *ws,
                               const DeviceInfo &dev, cudaStream_t s)
{
    (void)ws, (void)dev;
    const AttnArgs a = {kv, q, out, q_stride, out_stride, window, q_heads, scale};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)kv.seqs * (unsigned)kv.max_q, (unsigned)q_heads);
    cfg.blockDim = dim3(32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = head_dim == 64    ? cudaLaunchKernelEx(&cfg, kv_attention_kernel<64>, a)
                          : head_dim == 128 ? cudaLaunchKernelEx(&cfg, kv_attention_kernel<128>, a)
                                            : cudaLaunchKernelEx(&cfg, kv_attention_kernel<256>, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "kv_attention launch", e);
}

size_t kv_attention_workspace(const DeviceInfo &dev)
{
    (void)dev;
    return 4096;
}

}  // namespace qmd
