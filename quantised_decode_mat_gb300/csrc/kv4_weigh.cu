// kv4_weigh.cu -- the attention weight that each token of the 4-bit cache gets: weight_j += sum of
// e^(s_j - lse) over rows and heads.  A warp to 32 slots of a key/value head, a lane a slot.
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace qmd {

struct Weigh4Args {
    Kv4Params kv;
    const float *q;
    float *out, *lse;
    float *weight;
    int64_t q_stride, out_stride, window;
    int q_heads;
    float scale;
};

template <int D>
__device__ float dot4(const float *q, const uint8_t *codes, const __half *scales)
{
    float s = 0.0f;
    for (int g = 0; g < D / KV4_GROUP; ++g) {
        float part = 0.0f;
        for (int w = 0; w < 4; ++w) {
            float x[8];
            unpack4(x, reinterpret_cast<const uint32_t *>(codes)[4 * g + w]);
            for (int e = 0; e < 8; ++e)
                part = fmaf(x[e], q[32 * g + 8 * w + e], part);
        }
        s = fmaf(part, __half2float(scales[g]), s);
    }
    return s;
}

template <int D>
__global__ void __launch_bounds__(128) kv4_weigh_kernel(const Weigh4Args a)
{
    pdl_launch_dependents();
    pdl_wait();
    const Kv4Params &p = a.kv;
    const int lane = threadIdx.x & 31, G = a.q_heads / p.heads;
    const int s = blockIdx.y / p.heads, head = blockIdx.y % p.heads;
    const KvSeq sq = kv_seq(p, s);
    if (sq.n == 0)
        return;
    const int first = a.window > 0 ? (int)max((int64_t)0, sq.len - sq.n + 1 - a.window) : 0;
    for (int j = (blockIdx.x * 4 + (threadIdx.x >> 5)) * 32 + lane; j < sq.len; j += gridDim.x * 128) {
        const bool is_new = j >= sq.len - sq.n;
        if (j < first && !is_new)
            continue;
        const int page = kv_page(p, s, j / KV_BLOCK);
        if (page < 0)
            continue;
        const int64_t tok = kv4_token(p, page, head, j);
        float w = is_new ? 0.0f : a.weight[tok];
        for (int i = 0; i < sq.n; ++i) {
            const int end = sq.len - sq.n + 1 + i;
            if (j >= end || (a.window > 0 && j < end - a.window))
                continue;
            for (int g = 0; g < G; ++g) {
                const int h = head * G + g;
                const float sc = a.scale * dot4<D>(a.q + (sq.row0 + i) * a.q_stride + h * D,
                                                   reinterpret_cast<const uint8_t *>(p.k) + tok * (D / 2),
                                                   p.ks4 + tok * (D / KV4_GROUP));
                w += expf(sc - a.lse[(int64_t)(sq.row0 + i) * a.q_heads + h]);
            }
        }
        a.weight[tok] = w;
    }
}

static qmd_status launch4(void (*kernel)(const Weigh4Args), const Weigh4Args &a, dim3 grid, const char *what, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, what, e);
}

qmd_status launch_kv4_weigh(const Kv4Params &kv, int head_dim, const float *q, int64_t q_stride, int q_heads,
                            float scale, int64_t window, const float *lse, float *weight, const DeviceInfo &dev,
                            cudaStream_t s)
{
    const Weigh4Args a = {kv, q, nullptr, const_cast<float *>(lse), weight, q_stride, 0, window, q_heads, scale};
    const dim3 grid(64, (unsigned)(kv.seqs * kv.heads));
    return head_dim == 64    ? launch4(kv4_weigh_kernel<64>, a, grid, "kv4_weigh launch", s)
           : head_dim == 128 ? launch4(kv4_weigh_kernel<128>, a, grid, "kv4_weigh launch", s)
                             : launch4(kv4_weigh_kernel<256>, a, grid, "kv4_weigh launch", s);
}

}  // namespace qmd
