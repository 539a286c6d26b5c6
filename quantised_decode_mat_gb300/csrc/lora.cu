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
// barrier each CTA adds the eighths in order and multiplies its rows of B.  Those come by bulk
// copies, 4 KB of whole rows at a time into a ring of each warp, the first of them asked for before
// A x is begun.  With few vectors several clusters share a vector's rows; each then computes A x for
// itself (A is small beside B, and comes from L2).
//
// B (A x) runs on the tensor cores (mma.sync m16n8k16, 16 rows of B by columns that hold the parts
// of t = A x: two f16 parts of t over a power of two, or three bf16 parts, 22 or 24 bits; f32 sums):
// as f32 multiply-adds it took 45 instructions for 512 bytes and set the time (8 adapters of rank 64
// on 28672 x 4096: 13.2 us).  The order of the ranks inside a product is free, so a lane takes 16
// neighbouring bytes of a row for two products.
#include <mutex>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace qmd {

constexpr int LORA_CLUSTER = 8;
constexpr int LORA_WARPS = 16;
constexpr int LORA_STAGES = 2;
constexpr int LORA_CHUNK = 4096;                // bytes of B's rows that a copy takes, at most
constexpr int LORA_CHUNK_ROWS = LORA_CHUNK / 16;  // and the most rows in them
constexpr int LORA_STAGE_BYTES = LORA_CHUNK + LORA_CHUNK_ROWS * 4;  // with the rows' base values
constexpr int LORA_SMEM = LORA_WARPS * LORA_STAGES * LORA_STAGE_BYTES;

struct LoraArgs {
    const float *x, *base;
    const void *A, *B;
    const float *scale;
    const int32_t *adapter;
    float *out;
    int rows, K, rank, adapters;
    int shares;       // clusters per vector
    int chunk_rows;   // rows of B in a full copy
    unsigned *err;
    uint64_t wait_ns;
};

// bulk_copy_g2s with the default L2 policy: adapters are read again in the next step.
__device__ __forceinline__ void load_chunk(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

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

// The parts of a value of t that columns 0, 1 (and 2) hold.  The second is 2^11 (bf16: 2^8) times larger than
// it counts, the third 2^16: as large as the first, so that none runs out of exponents before it.
constexpr float LORA_LOW = 1.0f / 2048.0f, LORA_LOW_BF16 = 1.0f / 256.0f;
__device__ __forceinline__ uint32_t part_bits(float x, int col, __half)
{
    const __half h = __float2half_rn(x), l = __float2half_rn((x - __half2float(h)) * 2048.0f);
    return __half_as_ushort(col == 0 ? h : col == 1 ? l : __half(0.0f));
}
__device__ __forceinline__ uint32_t part_bits(float x, int col, __nv_bfloat16)
{
    const __nv_bfloat16 h = __float2bfloat16_rn(x);
    const float r = (x - __bfloat162float(h)) * 256.0f;
    const __nv_bfloat16 m = __float2bfloat16_rn(r), l = __float2bfloat16_rn((r - __bfloat162float(m)) * 256.0f);
    return __bfloat16_as_ushort(col == 0 ? h : col == 1 ? m : col == 2 ? l : __nv_bfloat16(0.0f));
}

__device__ __forceinline__ void mma_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __half)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_half(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, __nv_bfloat16)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NR: rows of A that a warp multiplies (rank / 16, rounded up)
template <class T, int NR>
__global__ void __launch_bounds__(LORA_WARPS * 32, 1) lora_add_kernel(const LoraArgs a)
{
    __shared__ __align__(16) float s_part[LORA_CLUSTER][QMD_LORA_MAX_RANK];
    __shared__ __align__(16) float s_t[QMD_LORA_MAX_RANK];
    __shared__ __align__(8) uint64_t s_bar[LORA_WARPS][LORA_STAGES];
    extern __shared__ __align__(16) unsigned char s_ring[];
    // every CTA of the cluster runs before its shared memory is written from another
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t bar0 = smem_addr(&s_bar[warp][0]);
    if (lane == 0) {
#pragma unroll
        for (int i = 0; i < LORA_STAGES; ++i)
            mbar_init(bar0 + 8 * i, 1);
        fence_barrier_init();
    }
    __syncwarp();
    pdl_launch_dependents();
    pdl_wait();
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

    // ---- this warp's chunks of the CTA's rows of B, and of base -----------------------------------
    const T *B = static_cast<const T *>(a.B) + (int64_t)id * a.rows * a.rank;
    unsigned char *ring = s_ring + warp * LORA_STAGES * LORA_STAGE_BYTES;
    const int nchunks = (r1 - r0 + a.chunk_rows - 1) / a.chunk_rows;
    auto ask = [&](int j) {  // chunk j of the CTA into this warp's stage (j / LORA_WARPS) % LORA_STAGES
        if (j < nchunks) {
            const int stage = j / LORA_WARPS % LORA_STAGES;
            const int row = r0 + j * a.chunk_rows, n = min(a.chunk_rows, r1 - row);
            const uint32_t dst = smem_addr(ring + stage * LORA_STAGE_BYTES);
            if (lane == 0) {
                const uint32_t bytes = (uint32_t)(n * a.rank * 2);
                mbar_arrive_expect_tx(bar0 + 8 * stage, bytes);
                load_chunk(dst, B + (int64_t)row * a.rank, bytes, bar0 + 8 * stage);
            }
            for (int i = lane; i < n; i += 32)
                asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + LORA_CHUNK + 4 * i), "l"(base + row + i)
                             : "memory");
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < LORA_STAGES; ++i)
        ask(warp + i * LORA_WARPS);

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
    // Lane (g, t) holds column g of the products' second operand: the parts of ranks 8 (t + 4 i) + 0..7
    // of group i, zeros past the rank and in the columns without a part.
    constexpr bool F16 = sizeof(T) == 2 && __is_same(T, __half);
    constexpr int NI = (NR * LORA_WARPS + 31) / 32;  // groups of 32 ranks
    const int g = lane >> 2, q = lane & 3, pieces_b = a.rank / 8;
    // f16: t is taken over a power of two, its largest value in [0.5, 1).  Sums go back by a product of their
    // own: that power times the adapter's scale may leave f32 where the result does not.
    float up = 1.0f, back = 1.0f;
    if constexpr (F16) {
        unsigned top = 0;  // |t|'s order is that of its bits
        for (int i = lane; i < a.rank; i += 32)
            top = max(top, __float_as_uint(s_t[i]) & 0x7fffffffu);
        const int ex = min(252, (int)(__reduce_max_sync(0xffffffffu, top) >> 23));
        up = __uint_as_float((uint32_t)(253 - ex) << 23);
        back = __uint_as_float((uint32_t)max(1, ex + 1) << 23);
    }
    uint32_t tb[NI][4];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const int r = 8 * (q + 4 * i) + 2 * w;
            tb[i][w] = q + 4 * i < pieces_b
                           ? part_bits(s_t[r] * up, g, T()) | part_bits(s_t[r + 1] * up, g, T()) << 16 : 0u;
        }
    uint32_t phase = 0;
    for (int j = warp, stage = 0; j < nchunks; j += LORA_WARPS) {
        asm volatile("cp.async.wait_group %0;" ::"n"(LORA_STAGES - 1) : "memory");
        if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar0 + 8 * stage, phase, a.wait_ns))) {
            // flag it, wait (bounded) for the copies that may be in flight, leave the rest out
            if (lane == 0) {
                atomicOr(a.err, (unsigned)ERRBIT_QMV_WAIT);
                for (int i = 0; i < LORA_STAGES && j + i * LORA_WARPS < nchunks; ++i) {
                    if (!mbar_wait_bounded(bar0 + 8 * stage, phase, a.wait_ns))
                        atomicOr(a.err, (unsigned)ERRBIT_DRAIN_WAIT);
                    stage = stage + 1 == LORA_STAGES ? 0 : stage + 1;
                    phase = stage == 0 ? phase ^ 1u : phase;
                }
            }
            break;
        }
        __syncwarp();  // every lane's base values have landed
        const unsigned char *st = ring + stage * LORA_STAGE_BYTES;
        const float *bs = reinterpret_cast<const float *>(st + LORA_CHUNK);
        const int row = r0 + j * a.chunk_rows, n = min(a.chunk_rows, r1 - row);
        for (int r = 0; r < n; r += 16) {
            // rows r + g and r + g + 8 (past n the last row again, not written)
            float c[4] = {};
            const unsigned char *wa = st + min(r + g, n - 1) * a.rank * 2, *wb = st + min(r + g + 8, n - 1) * a.rank * 2;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const bool has = q + 4 * i < pieces_b;
                const uint4 x0 = has ? lds128(wa + 16 * (q + 4 * i)) : make_uint4(0, 0, 0, 0);
                const uint4 x1 = has ? lds128(wb + 16 * (q + 4 * i)) : make_uint4(0, 0, 0, 0);
                const uint32_t f0[4] = {x0.x, x1.x, x0.y, x1.y}, f1[4] = {x0.z, x1.z, x0.w, x1.w};
                mma_half(c, f0, tb[i][0], tb[i][1], T());
                mma_half(c, f1, tb[i][2], tb[i][3], T());
            }
            float ya, yb;
            if constexpr (F16) {
                ya = fmaf(c[1], LORA_LOW, c[0]) * back;
                yb = fmaf(c[3], LORA_LOW, c[2]) * back;
            } else {
                ya = fmaf(fmaf(__shfl_down_sync(0xffffffffu, c[0], 1), LORA_LOW_BF16, c[1]), LORA_LOW_BF16, c[0]);
                yb = fmaf(fmaf(__shfl_down_sync(0xffffffffu, c[2], 1), LORA_LOW_BF16, c[3]), LORA_LOW_BF16, c[2]);
            }
            if (q == 0 && r + g < n)
                out[row + r + g] = fmaf(s, ya, bs[r + g]);
            if (q == 0 && r + g + 8 < n)
                out[row + r + g + 8] = fmaf(s, yb, bs[r + g + 8]);
        }
        fence_proxy_async_smem();
        __syncwarp();  // every lane has read the stage that is asked for again
        ask(j + LORA_STAGES * LORA_WARPS);
        stage = stage + 1 == LORA_STAGES ? 0 : stage + 1;
        phase = stage == 0 ? phase ^ 1u : phase;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <class T, int NR>
static cudaError_t launch_lora(const LoraArgs &a, int batch, int device, cudaStream_t s)
{
    {
        // opt in to the rings' shared memory once per device; host threads may race here
        static std::mutex mu;
        static bool opted[64] = {false};
        std::lock_guard<std::mutex> lock(mu);
        if (!opted[device]) {
            const cudaError_t e =
                cudaFuncSetAttribute(lora_add_kernel<T, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, LORA_SMEM);
            if (e != cudaSuccess)
                return e;
            opted[device] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(batch * a.shares * LORA_CLUSTER));
    cfg.blockDim = dim3(LORA_WARPS * 32);
    cfg.dynamicSmemBytes = LORA_SMEM;
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
static cudaError_t launch_lora_rank(const LoraArgs &a, int batch, int device, cudaStream_t s)
{
    const int nr = (a.rank + LORA_WARPS - 1) / LORA_WARPS;
    return nr <= 1   ? launch_lora<T, 1>(a, batch, device, s)
           : nr <= 2 ? launch_lora<T, 2>(a, batch, device, s)
           : nr <= 4 ? launch_lora<T, 4>(a, batch, device, s)
                     : launch_lora<T, 8>(a, batch, device, s);
}

qmd_status launch_lora_add(qmd_half type, const float *x, const float *base, const void *A, const void *B,
                           const float *scale, const int32_t *adapter, float *out, int64_t K, int64_t rows, int rank,
                           int adapters, int batch, const DeviceInfo &dev, unsigned *err, cudaStream_t s)
{
    LoraArgs a = {x, base, A, B, scale, adapter, out, (int)rows, (int)K, rank, adapters, 1, LORA_CHUNK / (rank * 2), err, wait_limit_ns()};
    // clusters per vector: as many as fill the SMs, while a CTA keeps at least 64 rows
    const int most = (int)((rows + 64 * LORA_CLUSTER - 1) / (64 * LORA_CLUSTER));
    a.shares = dev.sm_count / LORA_CLUSTER / batch;
    a.shares = a.shares < 1 ? 1 : a.shares > most ? most : a.shares;
    const cudaError_t e = type == QMD_F16 ? launch_lora_rank<__half>(a, batch, dev.device, s)
                                          : launch_lora_rank<__nv_bfloat16>(a, batch, dev.device, s);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, "lora_add launch", e);
}

}  // namespace qmd
