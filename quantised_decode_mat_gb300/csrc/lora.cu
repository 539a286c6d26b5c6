// lora.cu -- low-rank adapters of several requests beside a shared projection:
//     out[v] = base[v] + scale[a] * (B[a] (A[a] x[v])),  a = adapter[v]
// in f32, A and B f16 or bf16 (widened exactly).
//
// Bound: the adapters' bytes, each read once where they are large (64 x (4096 + 28672) x 2 bytes a
// vector); two dependent passes over little data where they are small, so what counts is one
// launch and every load that can be in flight early.
//
// A cluster of 8 CTAs serves one vector and a share of its rows.  Each CTA multiplies its eighth of
// x with all rows of A, the partial sums go to all 8 CTAs' shared memory, and after the cluster's
// barrier each CTA adds the eighths in order and multiplies its rows of B, whose first loads were
// issued before the barrier.  With few vectors several clusters share a vector's rows; each then
// computes A x for itself (A is small beside B, and comes from L2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace qmd {

constexpr int LORA_CLUSTER = 8;
constexpr int LORA_WARPS = 16;
constexpr int LORA_AHEAD = 4;  // 16-byte loads of B a lane has in flight before the barrier, and after it

struct LoraArgs {
    const float *x, *base;
    const void *A, *B;
    const float *scale;
    const int32_t *adapter;
    float *out;
    int rows, K, rank, adapters;
    int shares;       // clusters per vector
    int lanes_shift;  // log2 of the lanes that share a row of B
    unsigned *err;
};

__device__ __forceinline__ float2 widen(uint32_t w, __half) { return __half22float2(*reinterpret_cast<__half2 *>(&w)); }
__device__ __forceinline__ float2 widen(uint32_t w, __nv_bfloat16)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// acc + the product of 8 weights and 8 values
template <class T>
__device__ __forceinline__ float dot8(const uint4 &u, const float4 &a, const float4 &b, float acc)
{
    float2 f = widen(u.x, T());
    acc = fmaf(f.x, a.x, acc), acc = fmaf(f.y, a.y, acc);
    f = widen(u.y, T());
    acc = fmaf(f.x, a.z, acc), acc = fmaf(f.y, a.w, acc);
    f = widen(u.z, T());
    acc = fmaf(f.x, b.x, acc), acc = fmaf(f.y, b.y, acc);
    f = widen(u.w, T());
    return fmaf(f.y, b.w, fmaf(f.x, b.z, acc));
}

// NR: rows of A that a warp multiplies (rank / 16, rounded up)
template <class T, int NR>
__global__ void __launch_bounds__(LORA_WARPS * 32, 1) lora_add_kernel(const LoraArgs a)
{
    __shared__ __align__(16) float s_part[LORA_CLUSTER][QMD_LORA_MAX_RANK];
    __shared__ __align__(16) float s_t[QMD_LORA_MAX_RANK];
    // every CTA of the cluster runs before its shared memory is written from another
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x % LORA_CLUSTER, cl = blockIdx.x / LORA_CLUSTER;
    const int v = cl / a.shares, share = cl % a.shares;
    const int id = a.adapter[v];
    const bool on = id >= 0 && id < a.adapters;
    if (id >= a.adapters && threadIdx.x == 0)
        atomicOr(a.err, (unsigned)ERRBIT_INDEX);
    const float *base = a.base + (int64_t)v * a.rows;
    float *out = a.out + (int64_t)v * a.rows;
    // this CTA's rows
    const int part = share * LORA_CLUSTER + c, parts = a.shares * LORA_CLUSTER;
    const int r0 = (int)((int64_t)a.rows * part / parts), r1 = (int)((int64_t)a.rows * (part + 1) / parts);
    if (!on) {  // the whole cluster takes this way
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if (out != base)
            for (int i = r0 + (int)threadIdx.x; i < r1; i += LORA_WARPS * 32)
                out[i] = base[i];
        return;
    }

    // ---- A x over this CTA's eighth of K, in pieces of 32 ---------------------------------------
    const int pieces = a.K / 32;
    const int k0 = pieces * c / LORA_CLUSTER * 32, k1 = pieces * (c + 1) / LORA_CLUSTER * 32;
    const T *A = static_cast<const T *>(a.A) + (int64_t)id * a.rank * a.K;
    const float *x = a.x + (int64_t)v * a.K;
    float acc[NR] = {};
    for (int k = k0 + 8 * lane; k < k1; k += 256) {
        uint4 u[NR];
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = warp + LORA_WARPS * i;
            u[i] = r < a.rank ? *reinterpret_cast<const uint4 *>(A + (int64_t)r * a.K + k) : make_uint4(0, 0, 0, 0);
        }
        const float4 x0 = *reinterpret_cast<const float4 *>(x + k), x1 = *reinterpret_cast<const float4 *>(x + k + 4);
#pragma unroll
        for (int i = 0; i < NR; ++i)
            if (warp + LORA_WARPS * i < a.rank)  // (x may be NaN or infinite: 0 times it is not 0)
                acc[i] = dot8<T>(u[i], x0, x1, acc[i]);
    }

    // the first loads of this CTA's rows of B, while the sums meet
    const int per = 1 << a.lanes_shift, sub = lane & (per - 1), chunks = a.rank / 8;
    const int step = LORA_WARPS * 32 >> a.lanes_shift;  // rows the CTA takes at once
    const int my = r0 + (int)(threadIdx.x >> a.lanes_shift);
    const T *B = static_cast<const T *>(a.B) + (int64_t)id * a.rows * a.rank;
    auto load_b = [&](int row, int ch) { return *reinterpret_cast<const uint4 *>(B + (int64_t)row * a.rank + 8 * ch); };
    uint4 w[LORA_AHEAD];
#pragma unroll
    for (int i = 0; i < LORA_AHEAD; ++i)
        if (my + i * step < r1)
            w[i] = load_b(my + i * step, sub);

#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    if (lane < LORA_CLUSTER) {
#pragma unroll
        for (int i = 0; i < NR; ++i) {
            const int r = warp + LORA_WARPS * i;
            if (r < a.rank) {
                uint32_t at;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(&s_part[c][r])), "r"(lane));
                asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(acc[i]) : "memory");
            }
        }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    if ((int)threadIdx.x < a.rank) {
        float t = s_part[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < LORA_CLUSTER; ++i)
            t += s_part[i][threadIdx.x];
        s_t[threadIdx.x] = t;
    }
    __syncthreads();

    // ---- this CTA's rows of B --------------------------------------------------------------------
    const float s = a.scale[id];
    const float4 *t4 = reinterpret_cast<const float4 *>(s_t);
    const float4 ta = t4[2 * sub], tb = t4[2 * sub + 1];  // the lane's first piece, the only one of most ranks
    const int first = r0 + (warp * 32 >> a.lanes_shift);  // the warp's first row
    for (int off = 0; first + off < r1; off += LORA_AHEAD * step) {
        const int row = my + off;
        float y[LORA_AHEAD];
#pragma unroll
        for (int i = 0; i < LORA_AHEAD; ++i) {
            const int r = row + i * step;
            y[i] = 0.0f;
            if (r < r1) {
                y[i] = dot8<T>(w[i], ta, tb, 0.0f);
                for (int ch = sub + per; ch < chunks; ch += per)
                    y[i] = dot8<T>(load_b(r, ch), t4[2 * ch], t4[2 * ch + 1], y[i]);
            }
        }
        // the next rows' loads
#pragma unroll
        for (int i = 0; i < LORA_AHEAD; ++i)
            if (row + (LORA_AHEAD + i) * step < r1)
                w[i] = load_b(row + (LORA_AHEAD + i) * step, sub);
#pragma unroll
        for (int i = 0; i < LORA_AHEAD; ++i) {
            for (int o = per >> 1; o > 0; o >>= 1)
                y[i] += __shfl_xor_sync(0xffffffffu, y[i], o);
            const int r = row + i * step;
            if (sub == 0 && r < r1)
                out[r] = fmaf(s, y[i], base[r]);
        }
    }
}

template <class T, int NR>
static cudaError_t launch_lora(const LoraArgs &a, int batch, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * a.shares * LORA_CLUSTER));
    cfg.blockDim = dim3(LORA_WARPS * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = LORA_CLUSTER;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, lora_add_kernel<T, NR>, a);
}

template <class T>
static cudaError_t launch_lora_rank(const LoraArgs &a, int batch, cudaStream_t s)
{
    const int nr = (a.rank + LORA_WARPS - 1) / LORA_WARPS;
    return nr <= 1   ? launch_lora<T, 1>(a, batch, s)
           : nr <= 2 ? launch_lora<T, 2>(a, batch, s)
           : nr <= 4 ? launch_lora<T, 4>(a, batch, s)
                     : launch_lora<T, 8>(a, batch, s);
}

qmd_status launch_lora_add(qmd_half type, const float *x, const float *base, const void *A, const void *B,
                           const float *scale, const int32_t *adapter, float *out, int64_t K, int64_t rows, int rank,
                           int adapters, int batch, const DeviceInfo &dev, unsigned *err, cudaStream_t s)
{
    LoraArgs a = {x, base, A, B, scale, adapter, out, (int)rows, (int)K, rank, adapters, 1, 0, err};
    // clusters per vector: as many as fill the SMs, while a CTA keeps at least 64 rows
    const int most = (int)((rows + 64 * LORA_CLUSTER - 1) / (64 * LORA_CLUSTER));
    a.shares = dev.sm_count / LORA_CLUSTER / batch;
    a.shares = a.shares < 1 ? 1 : a.shares > most ? most : a.shares;
    // lanes to a row of B: the largest power of two that divides the row's 16-byte pieces
    while (a.lanes_shift < 4 && (rank / 8) % (2 << a.lanes_shift) == 0)
        ++a.lanes_shift;
    const cudaError_t e = type == QMD_F16 ? launch_lora_rank<__half>(a, batch, s) : launch_lora_rank<__nv_bfloat16>(a, batch, s);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "lora_add launch", e);
}

}  // namespace qmd
