// kv4_append.cu -- storing rotated keys and values in the 4-bit cache, and reading rows back.
//
// Mathematics: the rotation of kv_append.cu, by a position that may run ahead of the slot; then per group of 32
// values d = f16(top / -8), top the value of largest size (of several the first), and code
// clamp(rne(x * (1 / d)), -8, 7) + 8.  Codes are decided by rounding, so every f32 operation is rounded on its own.
//
// Layout: a CTA looks up a chunk of 32 rows, and its warps take tasks: some neighbouring heads of a row's
// queries, keys or values, whose loads are in flight together and whose angles are read once.  A lane owns 4 or
// 8 neighbouring values of a head, a group is 8 or 4 lanes.  Rows do not depend on each other (a scale belongs to
// one token), so nothing waits for a block and nothing is written twice.
//
// Bound: memory for prompts (11739 rows of 32 + 2 x 8 heads of 128: 97 to 105 us for 500 MB, 4.8 to 5.1 TB/s, seven
// eighths of it queries in and out; their read back 24 us, 4.5 TB/s, of loads that are 64 bytes of codes to a warp), launch
// latency for single tokens (8 rows 4.0 us, read back 2.8).
#include <cuda_runtime.h>

#include "internal.h"
#include "kv4.cuh"
#include "kv_rows.cuh"
#include "ptx.cuh"

namespace qmd {

struct Append4Args {
    Kv4Params kv;
    RopeArgs rope;
    const float *k, *v, *q;
    float *q_out;
    int64_t k_stride, v_stride, q_stride, q_out_stride;
    int q_heads;
    const int32_t *positions;
};

// Codes and scale of this lane's E values of a group, which LANES neighbouring lanes hold.  Every lane of the warp
// calls it.
template <int E>
__device__ __forceinline__ void quantise4(const float (&x)[E], uint32_t &codes, __half &scale)
{
    constexpr int LANES = KV4_GROUP / E;
    const int lane = threadIdx.x & 31;
    float most = fabsf(x[0]), top = x[0];
#pragma unroll
    for (int e = 1; e < E; ++e)
        if (fabsf(x[e]) > most)
            most = fabsf(x[e]), top = x[e];
    float all = most;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1)
        all = fmaxf(all, __shfl_xor_sync(0xffffffffu, all, o));
    // the first lane of the group that has it
    const unsigned has = __ballot_sync(0xffffffffu, most == all) >> (lane & ~(LANES - 1)) & ((1u << LANES) - 1);
    top = __shfl_sync(0xffffffffu, top, (lane & ~(LANES - 1)) + max(__ffs(has) - 1, 0));
    scale = __float2half_rn(fminf(fmaxf(__fmul_rn(top, -0.125f), -65504.0f), 65504.0f));
    const float d = __half2float(scale), inv = d != 0.0f ? __fdiv_rn(1.0f, d) : 0.0f;
    // 1.5 * 2^23 + 8: rounds to the nearest even integer and leaves the code in the lowest bits, zeros above
    // them up to the 22nd; sixteen times the next code and so on then add up in the low half
    uint32_t w[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
        w[e] = __float_as_uint(__fadd_rn(fminf(fmaxf(__fmul_rn(x[e], inv), -8.0f), 7.0f), 12582920.0f));
    codes = 0;
#pragma unroll
    for (int e = 0; e < E; e += 4)
        codes |= ((w[e] + w[e + 1] * 16 + w[e + 2] * 256 + w[e + 3] * 4096) & 0xffffu) << 4 * e;
}

template <int D>
__global__ void __launch_bounds__(APP_WARPS * 32) kv4_append_kernel(const Append4Args a)
{
    using H = HeadLanes<D>;
    constexpr int E = H::E, N = H::RN;  // heads (two 64-wide ones) of a task
    __shared__ KvRow s_row[APP_CHUNK];
    __shared__ int s_order[APP_CHUNK], s_count;
    pdl_launch_dependents();
    pdl_wait();
    const Kv4Params &p = a.kv;
    const int64_t t0 = (int64_t)blockIdx.x * APP_CHUNK;
    chunk_rows(p, t0, s_row, s_order, &s_count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hl = lane / H::LPH, l = lane % H::LPH;
    const int other = hl * H::LPH + partner<E>(a.rope, l);
    const int kv_groups = (p.heads + N * H::HPW - 1) / (N * H::HPW);
    const int q_groups = (a.q_heads + N * H::HPW - 1) / (N * H::HPW);
    const int of_row = 2 * kv_groups + q_groups, tasks = (int)min((int64_t)APP_CHUNK, p.rows - t0) * of_row;
    for (int task = blockIdx.y * APP_WARPS + warp; task < tasks; task += gridDim.y * APP_WARPS) {
        const int i = task / of_row, part = task % of_row;
        const int kind = part < kv_groups ? 0 : part < 2 * kv_groups ? 1 : 2;  // keys, values, queries
        const int h = (part - kind * kv_groups) * (N * H::HPW) + hl, heads = kind == 2 ? a.q_heads : p.heads;
        const KvRow r = s_row[i];
        if (r.seq < 0 || (kind != 2 && r.page < 0))
            continue;
        int at = r.pos;
        if (a.rope.table) {
            if (a.positions)
                at = a.positions[t0 + i];
            if (at < 0 || at >= a.rope.rows) {
                kv_index_error(p);
                continue;
            }
        }
        const int64_t stride = kind == 0 ? a.k_stride : kind == 1 ? a.v_stride : a.q_stride;
        const float *src = (kind == 0 ? a.k : kind == 1 ? a.v : a.q) + (t0 + i) * stride + h * D + E * l;
        float x[N][E];
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (h + j * H::HPW < heads)
                load_f32(x[j], src + j * H::HPW * D);
            else
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[j][e] = 0.0f;
        if (a.rope.table && kind != 1) {
            Angles<E> ang;
            load_angles(ang, a.rope, at, l);
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (h - hl + j * H::HPW < heads) {  // (the same for every lane)
                    float o[E];
#pragma unroll
                    for (int e = 0; e < E; ++e)
                        o[e] = __shfl_sync(0xffffffffu, x[j][e], other);
                    rotate(x[j], o, a.rope, ang, l);
                }
        }
        if (kind == 2) {
            float *dst = a.q_out + (t0 + i) * a.q_out_stride + h * D + E * l;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (h + j * H::HPW < heads)
                    store_f32(dst + j * H::HPW * D, x[j]);
            continue;
        }
        uint8_t *codes = reinterpret_cast<uint8_t *>(kind ? p.v : p.k);
        __half *scales = kind ? p.vs4 : p.ks4;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (h - hl + j * H::HPW < heads) {
                uint32_t c;
                __half d;
                quantise4(x[j], c, d);
                if (h + j * H::HPW < heads) {
                    const int64_t tok = kv4_token(p, r.page, h + j * H::HPW, r.pos);
                    uint8_t *to = codes + tok * (D / 2) + E / 2 * l;
                    if constexpr (E == 4)
                        *reinterpret_cast<uint16_t *>(to) = (uint16_t)c;
                    else
                        *reinterpret_cast<uint32_t *>(to) = c;
                    if (l % (KV4_GROUP / E) == 0)
                        scales[tok * (D / KV4_GROUP) + l / (KV4_GROUP / E)] = d;
                }
            }
    }
}

struct Read4Args {
    Kv4Params kv;
    float *k, *v;
    int64_t k_stride, v_stride;
};

// N: heads (two 64-wide ones) of a task, whose loads are in flight together.
template <int D, int N>
__global__ void __launch_bounds__(APP_WARPS * 32) kv4_read_kernel(const Read4Args a)
{
    using H = HeadLanes<D>;
    constexpr int E = H::E;
    __shared__ KvRow s_row[APP_CHUNK];
    __shared__ int s_order[APP_CHUNK], s_count;
    pdl_launch_dependents();
    pdl_wait();
    const Kv4Params &p = a.kv;
    const int64_t t0 = (int64_t)blockIdx.x * APP_CHUNK;
    chunk_rows(p, t0, s_row, s_order, &s_count);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int hl = lane / H::LPH, l = lane % H::LPH;
    const int groups = (p.heads + N * H::HPW - 1) / (N * H::HPW);
    const int tasks = (int)min((int64_t)APP_CHUNK, p.rows - t0) * groups * 2;
    for (int task = blockIdx.y * APP_WARPS + warp; task < tasks; task += gridDim.y * APP_WARPS) {
        const int i = task / (2 * groups), h = task / 2 % groups * (N * H::HPW) + hl;
        const bool is_v = task & 1;
        const KvRow r = s_row[i];
        float *out = is_v ? a.v : a.k;
        if (r.seq < 0 || r.page < 0 || !out)
            continue;
        const uint8_t *codes = reinterpret_cast<const uint8_t *>(is_v ? p.v : p.k);
        const __half *scales = is_v ? p.vs4 : p.ks4;
        uint32_t c[N];
        __half d[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (h + j * H::HPW < p.heads) {
                const int64_t tok = kv4_token(p, r.page, h + j * H::HPW, r.pos);
                const uint8_t *from = codes + tok * (D / 2) + E / 2 * l;
                c[j] = E == 4 ? *reinterpret_cast<const uint16_t *>(from) : *reinterpret_cast<const uint32_t *>(from);
                d[j] = scales[tok * (D / KV4_GROUP) + l / (KV4_GROUP / E)];
            }
        float *dst = out + (t0 + i) * (is_v ? a.v_stride : a.k_stride) + h * D + E * l;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (h + j * H::HPW < p.heads) {
                float x[E];
                unpack4(x, c[j]);
#pragma unroll
                for (int e = 0; e < E; ++e)
                    x[e] *= __half2float(d[j]);
                store_f32(dst + j * H::HPW * D, x);
            }
    }
}

qmd_status launch_kv4_append(const Kv4Params &kv, int head_dim, const float *k, int64_t k_stride, const float *v,
                             int64_t v_stride, const float *q, int64_t q_stride, int q_heads, float *q_out,
                             int64_t q_out_stride, const float *rope, int64_t rope_rows, int rot, int pairs,
                             const int32_t *positions, int sms, cudaStream_t s)
{
    const Append4Args a = {kv, {rope, rope_rows, rot, pairs}, k, v, q, q_out, k_stride, v_stride, q_stride,
                           q_out_stride, q_heads, positions};
    const int64_t rows = kv.rows < APP_CHUNK ? kv.rows : APP_CHUNK;
    // 2 KB a task: 8 rows 4.4 us, 5.7 with 4 KB; prompts the same
    const int64_t tasks = rows * (2 * ((kv.heads * head_dim + 511) / 512) + (q_heads * head_dim + 511) / 512);
    return head_dim == 64    ? launch_chunks(kv4_append_kernel<64>, a, tasks, sms, 16, 0, "kv4_append launch", s)
           : head_dim == 128 ? launch_chunks(kv4_append_kernel<128>, a, tasks, sms, 16, 0, "kv4_append launch", s)
                             : launch_chunks(kv4_append_kernel<256>, a, tasks, sms, 16, 0, "kv4_append launch", s);
}

qmd_status launch_kv4_read(const Kv4Params &kv, int head_dim, float *k, int64_t k_stride, float *v, int64_t v_stride,
                           int sms, cudaStream_t s)
{
    const Read4Args a = {kv, k, v, k_stride, v_stride};
    const int64_t rows = kv.rows < APP_CHUNK ? kv.rows : APP_CHUNK;
    // 4 KB a task where there are many: 12288 rows of 8 heads of 128 23 us, 25 with 2 KB, but 8 rows 3.6 against 3.0
    const bool many = kv.rows * kv.heads * head_dim >= 1 << 21;
    const int64_t tasks = rows * 2 * ((kv.heads * head_dim + (many ? 1023 : 511)) / (many ? 1024 : 512));
    void (*kernel)(Read4Args) =
        head_dim == 64    ? (many ? kv4_read_kernel<64, HeadLanes<64>::QN> : kv4_read_kernel<64, HeadLanes<64>::RN>)
        : head_dim == 128 ? (many ? kv4_read_kernel<128, HeadLanes<128>::QN> : kv4_read_kernel<128, HeadLanes<128>::RN>)
                          : (many ? kv4_read_kernel<256, HeadLanes<256>::QN> : kv4_read_kernel<256, HeadLanes<256>::RN>);
    return launch_chunks(kernel, a, tasks, sms, 32, 0, "kv4_read launch", s);
}

}  // namespace qmd
