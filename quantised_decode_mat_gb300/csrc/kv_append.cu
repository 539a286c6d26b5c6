// kv_append.cu -- storing rotated keys and values in the paged 8-bit cache, and reading rows back.
//
// "Language models on the device: the cajeta-llm kernels", §2.6 lists rope among the kernels of a
// layer; here the rotation of queries and keys, the quantisation and the store are one launch.
//
// Mathematics: per pair (a, b) of a head at position p, a' = a c - b s and b' = b c + a s with the
// table's c, s of p; per block of 16 positions and head, d = max |x| / 127 over the block's new
// rows (and the scale that its earlier positions have), code = rne(x / d) taken as x * (1 / d).
// Codes are decided by rounding, so every f32 operation is rounded on its own (explicit _rn
// intrinsics): the same inputs give the same codes as any other program that does these steps.
//
// Layout: a CTA looks up a chunk of 16 rows -- the sequence, position and page of each, once --
// and its warps take tasks: one (block, head, K or V) or one query (row, head) each.  A row is the
// leader of a block if it is the first of the call's rows in it; the block's task is done by the
// leader's chunk, so no two warps touch a block's scale and no atomics are needed.  Lane l owns
// head_dim / 32 neighbouring values; a rotation partner half a head away comes by a shuffle.
//
// Bound: memory for prompts (11739 rows of 32 + 2 x 8 heads of 128: 95 us for 511 MB, 5.4 TB/s; with
// their blocks read back 131, 121 and 160 us at 4, 8 and 16 query heads a task; a read back of 32000
// rows 61 us, 5.4 TB/s, with streaming stores 72), launch latency for single tokens (8 rows 3.5 us).
#include <mutex>
#include <set>
#include <utility>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace qmd {

constexpr int APP_WARPS = 4;
constexpr int APP_CHUNK = 16;  // rows a CTA looks up
constexpr int APP_HEADS = 8;   // query heads of a task: their loads in flight together, the table's row read once

struct KvRow {
    int seq;   // -1: a row that no sequence owns
    int pos;
    int page;  // of its position; -1 if outside the pool
    int left;  // rows of the sequence from this one on
    int lead;  // the first of the call's rows in its block
};

// Fill rows[0..16) for the chunk and order[] with the chunk's leaders; all threads call it.
__device__ __forceinline__ void chunk_rows(const KvParams &p, int64_t t0, KvRow *rows, int *order, int *count)
{
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        KvRow r = {-1, 0, -1, 0, 0};
        const int64_t t = t0 + lane;
        if (lane < APP_CHUNK && t < p.rows) {
            const int s = kv_row_seq(p, (int)t);
            const KvSeq q = kv_seq(p, s);
            if (t >= q.row0 && t < q.row0 + q.n) {
                const int pos = q.len - q.n + (int)(t - q.row0);
                if (q.len < q.n) {  // a sequence shorter than its rows; one without tokens pads the batch
                    if (q.len > 0)
                        kv_index_error(p);
                } else {
                    r.seq = s;
                    r.pos = pos;
                    r.page = kv_page(p, s, pos / KV_BLOCK);
                    r.left = q.row0 + q.n - (int)t;
                    r.lead = t == q.row0 || pos % KV_BLOCK == 0;
                }
            }
        }
        if (lane < APP_CHUNK)
            rows[lane] = r;
        const unsigned m = __ballot_sync(0xffffffffu, r.seq >= 0 && r.page >= 0 && r.lead);
        if (lane == 0)
            *count = __popc(m);
        if (m >> lane & 1)
            order[__popc(m & ((1u << lane) - 1))] = lane;
    }
    __syncthreads();
}

struct RopeArgs {
    const float *table;
    int64_t rows;
    int rot, pairs;
};

// This lane's cosines and sines of a position.
template <int E>
struct Angles {
    float c[E], s[E];
};

template <int E>
__device__ __forceinline__ void load_angles(Angles<E> &a, const RopeArgs &r, int pos, int lane)
{
    const float *row = r.table + (int64_t)pos * r.rot;
    const int half = r.rot >> 1;
    if (r.pairs == QMD_ROPE_HALVES) {
        const int off = half / E;  // lanes between the two of a pair
        if (lane < 2 * off) {
            const int at = E * (lane < off ? lane : lane - off);
            load_f32(a.c, row + at);
            load_f32(a.s, row + half + at);
        }
    } else if (E * lane < r.rot) {
        float c[E / 2], s[E / 2];
        load_f32(c, row + E / 2 * lane);
        load_f32(s, row + half + E / 2 * lane);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            a.c[i] = c[i], a.s[i] = s[i];
    }
}

// Rotate this lane's E values of a head (the warp holds the head).
template <int E>
__device__ __forceinline__ void rotate(float (&x)[E], const RopeArgs &r, const Angles<E> &a, int lane)
{
    if (r.pairs == QMD_ROPE_HALVES) {
        const int off = (r.rot >> 1) / E;
        const bool first = lane < off, second = !first && lane < 2 * off;
        float o[E];
#pragma unroll
        for (int i = 0; i < E; ++i)
            o[i] = __shfl_sync(0xffffffffu, x[i], first ? lane + off : second ? lane - off : lane);
        if (first || second) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float xc = __fmul_rn(x[i], a.c[i]), os = __fmul_rn(o[i], a.s[i]);
                x[i] = first ? __fsub_rn(xc, os) : __fadd_rn(xc, os);
            }
        }
    } else if (E * lane < r.rot) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(p, a.c[i]), __fmul_rn(q, a.s[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(q, a.c[i]), __fmul_rn(p, a.s[i]));
        }
    }
}

template <int E>
__device__ __forceinline__ void store_codes(int8_t *p, const float (&x)[E], float inv)
{
    uint32_t w[(E + 3) / 4] = {};
#pragma unroll
    for (int i = 0; i < E; ++i) {
        // NaN (an infinite value times 0) becomes 0
        const int q = min(127, max(-127, __float2int_rn(__fmul_rn(x[i], inv))));
        w[i / 4] |= (uint32_t)(q & 255) << (8 * (i % 4));
    }
    if constexpr (E == 2) {
        *reinterpret_cast<uint16_t *>(p) = (uint16_t)w[0];
    } else {
#pragma unroll
        for (int i = 0; i < E / 4; ++i)
            reinterpret_cast<uint32_t *>(p)[i] = w[i];
    }
}

struct AppendArgs {
    KvParams kv;
    RopeArgs rope;
    const float *k, *v, *q;
    float *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    int q_heads;
};

template <int D>
__global__ void __launch_bounds__(APP_WARPS * 32) kv_append_kernel(const AppendArgs a)
{
    constexpr int E = D / 32;
    constexpr int RB = 4;  // rows whose loads are in flight together
    extern __shared__ __align__(16) float s_x[];  // [warps][16][D]: a block's new rows until its scale is known
    __shared__ KvRow s_row[APP_CHUNK];
    __shared__ int s_order[APP_CHUNK], s_count;
    pdl_launch_dependents();
    pdl_wait();
    const KvParams &p = a.kv;
    const int64_t t0 = (int64_t)blockIdx.x * APP_CHUNK;
    chunk_rows(p, t0, s_row, s_order, &s_count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int blocks = s_count * p.heads * 2;
    const int groups = (a.q_heads + APP_HEADS - 1) / APP_HEADS;
    const int tasks = blocks + (a.q ? APP_CHUNK * groups : 0);
    for (int task = blockIdx.y * APP_WARPS + warp; task < tasks; task += gridDim.y * APP_WARPS) {
        if (task >= blocks) {  // APP_HEADS query heads of a row
            const int i = (task - blocks) / groups, h = (task - blocks) % groups * APP_HEADS;
            const KvRow r = s_row[i];
            if (r.seq < 0)
                continue;
            if (a.rope.table && r.pos >= a.rope.rows) {
                kv_index_error(p);
                continue;
            }
            const float *src = a.q + (t0 + i) * a.q_stride + h * D + E * lane;
            float *dst = a.q_out + (t0 + i) * a.q_out_stride + h * D + E * lane;
            float x[APP_HEADS][E];
#pragma unroll
            for (int j = 0; j < APP_HEADS; ++j)
                if (h + j < a.q_heads)
                    load_f32(x[j], src + j * D);
            Angles<E> ang;
            if (a.rope.table)
                load_angles(ang, a.rope, r.pos, lane);
#pragma unroll
            for (int j = 0; j < APP_HEADS; ++j)
                if (h + j < a.q_heads) {
                    if (a.rope.table)
                        rotate(x[j], a.rope, ang, lane);
                    store_f32(dst + j * D, x[j]);
                }
            continue;
        }
        const int i = s_order[task / (2 * p.heads)], h = task / 2 % p.heads;
        const bool is_v = task & 1;
        const KvRow r = s_row[i];
        const bool turn = a.rope.table && !is_v;
        const int tok0 = r.pos % KV_BLOCK;
        int m = min(KV_BLOCK - tok0, r.left);
        if (a.rope.table && r.pos + m > a.rope.rows) {  // positions past the table are not stored
            kv_index_error(p);
            m = (int)(a.rope.rows - r.pos);
            if (m <= 0)
                continue;
        }
        const float *src = (is_v ? a.v + (t0 + i) * a.v_stride : a.k + (t0 + i) * a.k_stride) + h * D + E * lane;
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        const int64_t blk = kv_block_offset(p, r.page, h, r.pos / KV_BLOCK);
        int8_t *codes = (is_v ? p.v : p.k) + blk * (KV_BLOCK * D) + E * lane;
        float *scale = (is_v ? p.vs : p.ks) + blk;

        float *keep = s_x + warp * KV_BLOCK * D + E * lane;  // each lane reads back its own
        float top = 0.0f;
        for (int j0 = 0; j0 < m; j0 += RB) {
            float x[RB][E];
            Angles<E> ang[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                if (j0 + j < m) {
                    load_f32(x[j], src + (j0 + j) * stride);
                    if (turn)
                        load_angles(ang[j], a.rope, r.pos + j0 + j, lane);
                }
#pragma unroll
            for (int j = 0; j < RB; ++j)
                if (j0 + j < m) {
                    if (turn)
                        rotate(x[j], a.rope, ang[j], lane);
                    store_f32(keep + (j0 + j) * D, x[j]);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        top = fmaxf(top, fabsf(x[j][e]));
                }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float d0 = tok0 > 0 ? *scale : 0.0f;
        const float d = fmaxf(d0, top < 1e-30f ? 0.0f : __fdiv_rn(top, 127.0f));
        const float inv = d > 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
        if (d > d0) {
            // the block's earlier tokens in steps of the larger scale
#pragma unroll 2
            for (int j = 0; j < tok0; ++j) {
                float y[E];
                load_codes(y, codes + j * D);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    y[e] = __fmul_rn(y[e], d0);
                store_codes(codes + j * D, y, inv);
            }
        }
#pragma unroll 4
        for (int j = 0; j < m; ++j) {
            float x[E];
            load_f32(x, keep + j * D);
            store_codes(codes + (tok0 + j) * D, x, inv);
        }
        __syncwarp();  // every lane has read the old scale
        if (lane == 0)
            *scale = d;
    }
}

constexpr int READ_HEADS = 4;

struct ReadArgs {
    KvParams kv;
    float *k, *v;
    int64_t k_stride, v_stride;
};

template <int D>
__global__ void __launch_bounds__(APP_WARPS * 32) kv_read_kernel(const ReadArgs a)
{
    constexpr int E = D / 32;
    __shared__ KvRow s_row[APP_CHUNK];
    __shared__ int s_order[APP_CHUNK], s_count;
    pdl_launch_dependents();
    pdl_wait();
    const KvParams &p = a.kv;
    const int64_t t0 = (int64_t)blockIdx.x * APP_CHUNK;
    chunk_rows(p, t0, s_row, s_order, &s_count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // a warp takes READ_HEADS neighbouring heads of a row, keys or values: their loads in flight together
    const int groups = (p.heads + READ_HEADS - 1) / READ_HEADS;
    const int tasks = APP_CHUNK * groups * 2;
    for (int task = blockIdx.y * APP_WARPS + warp; task < tasks; task += gridDim.y * APP_WARPS) {
        const int i = task / (2 * groups), h = task / 2 % groups * READ_HEADS;
        const bool is_v = task & 1;
        const KvRow r = s_row[i];
        float *out = is_v ? a.v : a.k;
        if (r.seq < 0 || r.page < 0 || !out)
            continue;
        const int64_t blk = kv_block_offset(p, r.page, h, r.pos / KV_BLOCK);
        const int8_t *codes = (is_v ? p.v : p.k) + (blk * KV_BLOCK + r.pos % KV_BLOCK) * D + E * lane;
        const float *scale = (is_v ? p.vs : p.ks) + blk;
        float x[READ_HEADS][E], d[READ_HEADS];
#pragma unroll
        for (int j = 0; j < READ_HEADS; ++j)
            if (h + j < p.heads) {
                load_codes(x[j], codes + (int64_t)j * p.page_blocks * (KV_BLOCK * D));
                d[j] = scale[j * p.page_blocks];
            }
        float *dst = out + (t0 + i) * (is_v ? a.v_stride : a.k_stride) + h * D + E * lane;
#pragma unroll
        for (int j = 0; j < READ_HEADS; ++j)
            if (h + j < p.heads) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[j][e] = __fmul_rn(x[j][e], d[j]);
                store_f32(dst + j * D, x[j]);
            }
    }
}

// CTAs per chunk: enough that every task has a warp while the launch has no more than a few waves.
static unsigned chunk_ctas(int64_t chunks, int64_t tasks, int sms)
{
    int64_t y = (tasks + APP_WARPS - 1) / APP_WARPS;
    const int64_t most = (int64_t)sms * 16 / chunks;
    if (y > most)
        y = most;
    return (unsigned)(y < 1 ? 1 : y > 65535 ? 65535 : y);
}

template <class Args>
static qmd_status launch_chunks(void (*kernel)(const Args), const Args &a, int64_t tasks, int sms, size_t smem,
                                const char *what, cudaStream_t s)
{
    if (smem > 48 * 1024) {
        // opt in once per device and kernel; host threads may race here
        static std::mutex mu;
        static std::set<std::pair<int, const void *>> opted;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess)
            return QMD_ERR_DEVICE;
        std::lock_guard<std::mutex> lock(mu);
        if (opted.insert({dev, reinterpret_cast<const void *>(kernel)}).second) {
            const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e != cudaSuccess) {
                opted.erase({dev, reinterpret_cast<const void *>(kernel)});
                return fail(QMD_ERR_LAUNCH, what, e);
            }
        }
    }
    const int64_t chunks = (a.kv.rows + APP_CHUNK - 1) / APP_CHUNK;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)chunks, chunk_ctas(chunks, tasks, sms));
    cfg.blockDim = dim3(APP_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = (launch_flags() & LAUNCH_NO_PDL) ? 0 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
    return e == cudaSuccess ? QMD_OK : fail(QMD_ERR_LAUNCH, what, e);
}

qmd_status launch_kv_append(const KvParams &kv, int head_dim, const float *k, int64_t k_stride, const float *v,
                            int64_t v_stride, const float *q, int64_t q_stride, int q_heads, float *q_out,
                            int64_t q_out_stride, const float *rope, int64_t rope_rows, int rot, int pairs, int sms,
                            cudaStream_t s)
{
    const AppendArgs a = {kv, {rope, rope_rows, rot, pairs}, k, v, q, q_out, k_stride, v_stride, q_stride,
                          q_out_stride, q_heads};
    const int64_t rows = kv.rows < APP_CHUNK ? kv.rows : APP_CHUNK;
    const int64_t tasks = rows * (2 * kv.heads + (q_heads + APP_HEADS - 1) / APP_HEADS);
    const size_t smem = (size_t)APP_WARPS * KV_BLOCK * head_dim * 4;
    return head_dim == 64    ? launch_chunks(kv_append_kernel<64>, a, tasks, sms, smem, "kv_append launch", s)
           : head_dim == 128 ? launch_chunks(kv_append_kernel<128>, a, tasks, sms, smem, "kv_append launch", s)
                             : launch_chunks(kv_append_kernel<256>, a, tasks, sms, smem, "kv_append launch", s);
}

qmd_status launch_kv_read(const KvParams &kv, int head_dim, float *k, int64_t k_stride, float *v, int64_t v_stride,
                          int sms, cudaStream_t s)
{
    const ReadArgs a = {kv, k, v, k_stride, v_stride};
    const int64_t rows = kv.rows < APP_CHUNK ? kv.rows : APP_CHUNK;
    const int64_t tasks = rows * 2 * ((kv.heads + READ_HEADS - 1) / READ_HEADS);
    return head_dim == 64    ? launch_chunks(kv_read_kernel<64>, a, tasks, sms, 0, "kv_read launch", s)
           : head_dim == 128 ? launch_chunks(kv_read_kernel<128>, a, tasks, sms, 0, "kv_read launch", s)
                             : launch_chunks(kv_read_kernel<256>, a, tasks, sms, 0, "kv_read launch", s);
}

}  // namespace qmd
