// kv_rows.cuh -- what the calls share that take a batch's rows one by one (appends and reads of either cache):
// the rows of a chunk, the rotation, and the launch over chunks.
#pragma once

#include <mutex>
#include <set>
#include <utility>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"

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

}  // namespace qmd
