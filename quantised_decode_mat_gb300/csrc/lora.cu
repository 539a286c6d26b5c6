// lora.cu -- low-rank adapters of several requests beside a shared projection:
//     out[v] = base[v] + scale[a] * (B[a] (A[a] x[v])),  a = adapter[v]
// in f32, A and B f16 or bf16 (widened exactly).
//
// Plain form: a CTA per (vector, 256 rows) computes A x for itself, then its rows.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace qmd {

struct LoraArgs {
    const float *x, *base;
    const void *A, *B;
    const float *scale;
    const int32_t *adapter;
    float *out;
    int64_t rows;
    int K, rank, adapters;
    unsigned *err;
};

__device__ __forceinline__ float2 widen(uint32_t w, __half) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
__device__ __forceinline__ float2 widen(uint32_t w, __nv_bfloat16)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

template <class T>
__global__ void __launch_bounds__(256) lora_add_kernel(const LoraArgs a)
{
    __shared__ float t[QMD_LORA_MAX_RANK];
    pdl_launch_dependents();
    pdl_wait();
    const int v = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int id = a.adapter[v];
    if (id >= a.adapters && threadIdx.x == 0)
        atomicOr(a.err, (unsigned)ERRBIT_INDEX);
    const bool on = id >= 0 && id < a.adapters;
    if (on) {
        for (int r = warp; r < a.rank; r += 8) {
            const uint4 *w = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.A) + ((int64_t)id * a.rank + r) * a.K);
            const float4 *x = reinterpret_cast<const float4 *>(a.x + (int64_t)v * a.K);
            float acc = 0.0f;
            for (int i = lane; i < a.K / 8; i += 32) {
                const uint4 u = w[i];
                const float4 x0 = x[2 * i], x1 = x[2 * i + 1];
                float2 f = widen(u.x, T());
                acc = fmaf(f.x, x0.x, fmaf(f.y, x0.y, acc));
                f = widen(u.y, T());
                acc = fmaf(f.x, x0.z, fmaf(f.y, x0.w, acc));
                f = widen(u.z, T());
                acc = fmaf(f.x, x1.x, fmaf(f.y, x1.y, acc));
                f = widen(u.w, T());
                acc = fmaf(f.x, x1.z, fmaf(f.y, x1.w, acc));
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                acc += __shfl_xor_sync(0xffffffffu, acc, o);
            if (lane == 0)
                t[r] = acc;
        }
    }
    __syncthreads();
    if (row >= a.rows)
        return;
    float y = a.base[v * a.rows + row];
    if (on) {
        const uint4 *w = reinterpret_cast<const uint4 *>(static_cast<const T *>(a.B) + ((int64_t)id * a.rows + row) * a.rank);
        float acc = 0.0f;
        for (int i = 0; i < a.rank / 8; ++i) {
            const uint4 u = w[i];
            const uint32_t c[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = widen(c[e], T());
                acc = fmaf(f.x, t[8 * i + 2 * e], fmaf(f.y, t[8 * i + 2 * e + 1], acc));
            }
        }
        y = fmaf(a.scale[id], acc, y);
    }
    a.out[v * a.rows + row] = y;
}

qmd_status launch_lora_add(qmd_half type, const float *x, const float *base, const void *A, const void *B,
                           const float *scale, const int32_t *adapter, float *out, int64_t K, int64_t rows, int rank,
                           int adapters, int batch, const DeviceInfo &dev, unsigned *err, cudaStream_t s)
{
    (void)dev;
    const LoraArgs a = {x, base, A, B, scale, adapter, out, rows, (int)K, rank, adapters, err};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((rows + 255) / 256), (unsigned)batch);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = type == QMD_F16 ? cudaLaunchKernelEx(&cfg, lora_add_kernel<__half>, a)
                                          : cudaLaunchKernelEx(&cfg, lora_add_kernel<__nv_bfloat16>, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "lora_add launch", e);
}

}  // namespace qmd
