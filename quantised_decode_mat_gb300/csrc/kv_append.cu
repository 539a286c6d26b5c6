// kv_append.cu -- storing rotated keys and values in the paged 8-bit cache, and reading rows back.
//
// "Language models on the device: the cajeta-llm kernels", §2.6 lists rope among the kernels of a
// layer; here the rotation of queries and keys, the quantisation and the store are one launch.
//
// Mathematics: per pair (a, b) of a head at position p, a' = a c - b s and b' = b c + a s with the
// table's c, s of p; per block of 16 positions and head, d = max |x| / 127 over the block's new
// rows (and the size of the scale that its earlier positions have), code = rne(x / d) taken as
// x * (1 / d) and held in -127 .. 127.
// Codes are decided by rounding, so every f32 operation is rounded on its own (explicit _rn
// intrinsics): the same inputs give the same codes as any other program that does these steps.
//
// Layout: a CTA looks up a chunk of 32 rows -- the sequence, position and page of each, once --
// and its warps take tasks: a block of one head's K or V (two heads of 64), or 1024 query values of a
// row.  A row is the
// leader of a block if it is the first of the call's rows in it; the block's task is done by the
// leader's chunk, so no two warps touch a block's scale and no atomics are needed.  A lane owns 4 or 8
// neighbouring values of a head; a rotation partner half a head away comes by a shuffle.  A block's new
// rows wait in shared memory until its scale is known.
//
// Bound: memory for prompts (11739 rows of 32 + 2 x 8 heads of 128: 95 us for 511 MB, 5.4 TB/s; with
// their blocks read back 131, 121 and 160 us at 4, 8 and 16 query heads a task; the rows by cp.async, all
// in flight, 122; a read back of 32000 rows 56 us, 5.9 TB/s; streaming stores cost a fifth of that),
// launch latency for single tokens (8 rows 3.5 us).  Chunks of 16 rows: 1 to 8 % more for appends.
// 64-wide heads two to a warp: 40 us against 47 with one (8 bytes a lane); 256-wide ones with 2 rows in
// flight 143 against 153 with 4 (registers).
#include <mutex>
#include <set>
#include <utility>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"
#include "ptx.cuh"

namespace qmd {

constexpr int APP_WARPS = 4;
constexpr int APP_CHUNK = 32;  // rows a CTA looks up, a lane each

// How a warp holds heads: E neighbouring values to a lane (16 bytes at least), so one head, or two of 64.
template <int D>
struct HeadLanes {
    static constexpr int LPH = D < 128 ? D / 4 : 32;  // lanes to a head
    static constexpr int HPW = 32 / LPH;              // heads to a warp
    static constexpr int E = D / LPH;
    static constexpr int QN = 32 / E;                 // loads of a query task in flight together (4 KB)
    static constexpr int RN = 16 / E;                 // and of a read
};

struct KvRow {
    int seq;   // -1: a row that no sequence owns
    int pos;
    int page;  // of its position; -1 if outside the pool
    int left;  // rows of the sequence from this one on
    int lead;  // the first of the call's rows in its block
};

// Fill rows[] for the chunk and order[] with the chunk's leaders; all threads call it.
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
__device__ __forceinline__ void load_angles(Angles<E> &a, const RopeArgs &r, int pos, int l)
{
    const float *row = r.table + (int64_t)pos * r.rot;
    const int half = r.rot >> 1;
    if (r.pairs == QMD_ROPE_HALVES) {
        const int off = half / E;  // lanes between the two of a pair
        if (l < 2 * off) {
            const int at = E * (l < off ? l : l - off);
            load_f32(a.c, row + at);
            load_f32(a.s, row + half + at);
        }
    } else if (E * l < r.rot) {
        float c[E / 2], s[E / 2];
        load_f32(c, row + E / 2 * l);
        load_f32(s, row + half + E / 2 * l);
#pragma unroll
        for (int i = 0; i < E / 2; ++i)
            a.c[i] = c[i], a.s[i] = s[i];
    }
}

// Rotate this lane's E values of a head, of which it is lane l; o: the values of the lane half a
// rotation away (not used for adjacent pairs).
template <int E>
__device__ __forceinline__ void rotate(float (&x)[E], const float (&o)[E], const RopeArgs &r, const Angles<E> &a, int l)
{
    if (r.pairs == QMD_ROPE_HALVES) {
        const int off = (r.rot >> 1) / E;
        const bool first = l < off;
        if (l < 2 * off) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float xc = __fmul_rn(x[i], a.c[i]), os = __fmul_rn(o[i], a.s[i]);
                x[i] = first ? __fsub_rn(xc, os) : __fadd_rn(xc, os);
            }
        }
    } else if (E * l < r.rot) {
#pragma unroll
        for (int i = 0; i < E / 2; ++i) {
            const float p = x[2 * i], q = x[2 * i + 1];
            x[2 * i] = __fsub_rn(__fmul_rn(p, a.c[i]), __fmul_rn(q, a.s[i]));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(q, a.c[i]), __fmul_rn(p, a.s[i]));
        }
    }
}

// The lane of its head that holds the other halves of lane l's pairs (l itself where it has none).
template <int E>
__device__ __forceinline__ int partner(const RopeArgs &r, int l)
{
    const int off = r.pairs == QMD_ROPE_HALVES ? (r.rot >> 1) / E : 0;
    return l < off ? l + off : l < 2 * off ? l - off : l;
}

// The codes of E values: x * inv held in -127 .. 127 and rounded to the nearest even integer by adding
// 1.5 * 2^23 (unit 1), which leaves it in the low byte.  Both bounds are needed: a block's scale may be one
// that the caller wrote, with codes of -128, or so small that a new value is thousands of its steps.  (0.7 % of a
// prompt's append; new rows held only under 1e-30, by a branch, cost 1.3 %.)
template <int E>
__device__ __forceinline__ void store_codes(int8_t *p, const float (&x)[E], float inv)
{
#pragma unroll
    for (int i = 0; i < E; i += 4) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            w[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fmul_rn(x[i + e], inv), -127.0f), 127.0f), 12582912.0f));
        *reinterpret_cast<uint32_t *>(p + i) =
            __byte_perm(__byte_perm(w[0], w[1], 0x5140u), __byte_perm(w[2], w[3], 0x5140u), 0x5410u);
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
__global__ void __launch_bounds__(APP_WARPS * 32, D == 256 ? 3 : 4) kv_append_kernel(const AppendArgs a)
{
    using H = HeadLanes<D>;
    constexpr int E = H::E;
    constexpr int RB = D == 256 ? 2 : 4;  // rows whose loads are in flight together
    extern __shared__ __align__(16) float s_x[];  // [warps][16][D * HPW]: a block's new rows until its scale is known
    __shared__ KvRow s_row[APP_CHUNK];
    __shared__ int s_order[APP_CHUNK], s_count;
    pdl_launch_dependents();
    pdl_wait();
    const KvParams &p = a.kv;
    const int64_t t0 = (int64_t)blockIdx.x * APP_CHUNK;
    chunk_rows(p, t0, s_row, s_order, &s_count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hl = lane / H::LPH, l = lane % H::LPH;  // which of the warp's heads, which lane of it
    const int other = hl * H::LPH + partner<E>(a.rope, l);  // the lane with the other halves of its pairs
    const int kv_groups = (p.heads + H::HPW - 1) / H::HPW;
    const int blocks = s_count * kv_groups * 2;
    const int groups = (a.q_heads + H::QN * H::HPW - 1) / (H::QN * H::HPW);
    const int tasks = blocks + (a.q ? APP_CHUNK * groups : 0);
    for (int task = blockIdx.y * APP_WARPS + warp; task < tasks; task += gridDim.y * APP_WARPS) {
        if (task >= blocks) {  // some query heads of a row: their loads in flight together, its angles read once
            const int i = (task - blocks) / groups, h = (task - blocks) % groups * (H::QN * H::HPW);
            const KvRow r = s_row[i];
            if (r.seq < 0)
                continue;
            if (a.rope.table && r.pos >= a.rope.rows) {
                kv_index_error(p);
                continue;
            }
            const float *src = a.q + (t0 + i) * a.q_stride + (h + hl) * D + E * l;
            float *dst = a.q_out + (t0 + i) * a.q_out_stride + (h + hl) * D + E * l;
            float x[H::QN][E];
#pragma unroll
            for (int j = 0; j < H::QN; ++j)
                if (h + hl + j * H::HPW < a.q_heads)
                    load_f32(x[j], src + j * H::HPW * D);
            Angles<E> ang;
            if (a.rope.table)
                load_angles(ang, a.rope, r.pos, l);
#pragma unroll
            for (int j = 0; j < H::QN; ++j)
                if (h + j * H::HPW < a.q_heads) {  // (the same for every lane)
                    if (a.rope.table) {
                        float o[E];
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            o[e] = __shfl_sync(0xffffffffu, x[j][e], other);
                        rotate(x[j], o, a.rope, ang, l);
                    }
                    if (h + hl + j * H::HPW < a.q_heads)
                        store_f32(dst + j * H::HPW * D, x[j]);
                }
            continue;
        }
        const int i = s_order[task / (2 * kv_groups)], h = task / 2 % kv_groups * H::HPW + hl;
        const bool is_v = task & 1, ok = h < p.heads;
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
        const int64_t stride = is_v ? a.v_stride : a.k_stride;
        const float *src = (is_v ? a.v : a.k) + (t0 + i) * stride + h * D + E * l;
        const int64_t blk = kv_block_offset(p, r.page, ok ? h : 0, r.pos / KV_BLOCK);
        int8_t *codes = (is_v ? p.v : p.k) + blk * (KV_BLOCK * D) + E * l;
        float *scale = (is_v ? p.vs : p.ks) + blk;

        // the block's new rows, RB at a time with their loads in flight together, wait in shared memory
        // until the scale is known; each lane reads back its own
        constexpr int ROW = D * H::HPW;
        float *keep = s_x + warp * KV_BLOCK * ROW + E * lane;
        const float d0 = ok && tok0 > 0 ? *scale : 0.0f;
        float top = 0.0f;
        for (int j0 = 0; j0 < m; j0 += RB) {
            float x[RB][E] = {};
            Angles<E> ang[RB];
#pragma unroll
            for (int j = 0; j < RB; ++j)
                if (j0 + j < m) {
                    if (ok)
                        load_f32(x[j], src + (j0 + j) * stride);
                    if (turn)
                        load_angles(ang[j], a.rope, r.pos + j0 + j, l);
                }
#pragma unroll
            for (int j = 0; j < RB; ++j)
                if (j0 + j < m) {  // (the same for every lane)
                    if (turn) {
                        float o[E];
#pragma unroll
                        for (int e = 0; e < E; ++e)
                            o[e] = __shfl_sync(0xffffffffu, x[j][e], other);
                        rotate(x[j], o, a.rope, ang[j], l);
                    }
                    store_f32(keep + (j0 + j) * ROW, x[j]);
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        top = fmaxf(top, fabsf(x[j][e]));
                }
        }
#pragma unroll
        for (int o = H::LPH / 2; o > 0; o >>= 1)
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // the scale's size counts, so that earlier values are kept whatever its sign; under 2^-128 its
        // reciprocal is held at the largest f32
        const float d = fmaxf(fabsf(d0), top < 1e-30f ? 0.0f : __fdiv_rn(top, 127.0f));
        const float inv = d > 0.0f ? fminf(__fdiv_rn(1.0f, d), 3.402823466e38f) : 0.0f;
        if (ok) {
            if (d != d0) {
                // the block's earlier tokens in steps of the new scale
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
                load_f32(x, keep + j * ROW);
                store_codes(codes + (tok0 + j) * D, x, inv);
            }
        }
        __syncwarp();  // every lane has read the old scale
        if (ok && l == 0)
            *scale = d;
    }
}

struct ReadArgs {
    KvParams kv;
    float *k, *v;
    int64_t k_stride, v_stride;
};

template <int D>
__global__ void __launch_bounds__(APP_WARPS * 32) kv_read_kernel(const ReadArgs a)
{
    using H = HeadLanes<D>;
    constexpr int E = H::E;
    __shared__ KvRow s_row[APP_CHUNK];
    __shared__ int s_order[APP_CHUNK], s_count;
    pdl_launch_dependents();
    pdl_wait();
    const KvParams &p = a.kv;
    const int64_t t0 = (int64_t)blockIdx.x * APP_CHUNK;
    chunk_rows(p, t0, s_row, s_order, &s_count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hl = lane / H::LPH, l = lane % H::LPH;
    // a warp takes some neighbouring heads of a row, keys or values: their loads in flight together
    const int groups = (p.heads + H::RN * H::HPW - 1) / (H::RN * H::HPW);
    const int tasks = APP_CHUNK * groups * 2;
    for (int task = blockIdx.y * APP_WARPS + warp; task < tasks; task += gridDim.y * APP_WARPS) {
        const int i = task / (2 * groups), h = task / 2 % groups * (H::RN * H::HPW) + hl;
        const bool is_v = task & 1;
        const KvRow r = s_row[i];
        float *out = is_v ? a.v : a.k;
        if (r.seq < 0 || r.page < 0 || !out)
            continue;
        const int64_t blk = kv_block_offset(p, r.page, h, r.pos / KV_BLOCK);
        const int8_t *codes = (is_v ? p.v : p.k) + (blk * KV_BLOCK + r.pos % KV_BLOCK) * D + E * l;
        const float *scale = (is_v ? p.vs : p.ks) + blk;
        float x[H::RN][E], d[H::RN];
#pragma unroll
        for (int j = 0; j < H::RN; ++j)
            if (h + j * H::HPW < p.heads) {
                load_codes(x[j], codes + (int64_t)j * H::HPW * p.page_blocks * (KV_BLOCK * D));
                d[j] = scale[j * H::HPW * p.page_blocks];
            }
        float *dst = out + (t0 + i) * (is_v ? a.v_stride : a.k_stride) + h * D + E * l;
#pragma unroll
        for (int j = 0; j < H::RN; ++j)
            if (h + j * H::HPW < p.heads) {
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[j][e] = __fmul_rn(x[j][e], d[j]);
                store_f32(dst + j * H::HPW * D, x[j]);
            }
    }
}

// CTAs per chunk: enough that every task has a warp, while the launch has no more than `per_sm` CTAs an
// SM.  Appends 16: 5400 rows of 16 + 2 x 16 heads of 128 and their read back take 64 us, 69 with 10 or 24.
// Reads 32: 16000 rows of 8 heads of 256 take 59 us, 69 with 16, 63 with 24, 60 with 48.
static unsigned chunk_ctas(int64_t chunks, int64_t tasks, int sms, int per_sm)
{
    int64_t y = (tasks + APP_WARPS - 1) / APP_WARPS;
    const int64_t most = (int64_t)sms * per_sm / chunks;
    if (y > most)
        y = most;
    return (unsigned)(y < 1 ? 1 : y > 65535 ? 65535 : y);
}

template <class Args>
static qmd_status launch_chunks(void (*kernel)(const Args), const Args &a, int64_t tasks, int sms, int per_sm, size_t smem,
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
    cfg.gridDim = dim3((unsigned)chunks, chunk_ctas(chunks, tasks, sms, per_sm));
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
    const int64_t tasks = rows * (2 * kv.heads + (q_heads * head_dim + 1023) / 1024);
    const size_t smem = (size_t)APP_WARPS * KV_BLOCK * (head_dim < 128 ? 128 : head_dim) * 4;
    return head_dim == 64    ? launch_chunks(kv_append_kernel<64>, a, tasks, sms, 16, smem, "kv_append launch", s)
           : head_dim == 128 ? launch_chunks(kv_append_kernel<128>, a, tasks, sms, 16, smem, "kv_append launch", s)
                             : launch_chunks(kv_append_kernel<256>, a, tasks, sms, 16, smem, "kv_append launch", s);
}

qmd_status launch_kv_read(const KvParams &kv, int head_dim, float *k, int64_t k_stride, float *v, int64_t v_stride,
                          int sms, cudaStream_t s)
{
    const ReadArgs a = {kv, k, v, k_stride, v_stride};
    const int64_t rows = kv.rows < APP_CHUNK ? kv.rows : APP_CHUNK;
    const int64_t tasks = rows * 2 * ((kv.heads * head_dim + 511) / 512);
    return head_dim == 64    ? launch_chunks(kv_read_kernel<64>, a, tasks, sms, 32, 0, "kv_read launch", s)
           : head_dim == 128 ? launch_chunks(kv_read_kernel<128>, a, tasks, sms, 32, 0, "kv_read launch", s)
                             : launch_chunks(kv_read_kernel<256>, a, tasks, sms, 32, 0, "kv_read launch", s);
}

}  // namespace qmd
