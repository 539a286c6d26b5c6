// api_kv.cu -- the C ABI of the key/value cache calls and of the adapters: argument validation on
// the host, before anything is launched, with the same named statuses as api.cu.
#include <cmath>
#include <numeric>

#include <cuda_runtime.h>

#include "internal.h"
#include "kv.cuh"

namespace qmd {
namespace {

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Do [a, a + na) and [b, b + nb) bytes overlap?
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a), pb = reinterpret_cast<uintptr_t>(b);
    return a && b && pa < pb + nb && pb < pa + na;
}

// `rows` rows of `width` f32 values, a stride apart.
struct Rows {
    const void *p;
    int64_t stride, width;
};

// Bytes from the first value of `rows` rows of `width` f32 values to the end of the last.
inline size_t extent(int64_t rows, int64_t stride, int64_t width) { return ((size_t)(rows - 1) * stride + width) * 4; }

// Do a's and b's rows overlap?  Parts of one wider buffer lie between each other's rows: every byte of
// a's rows is 0 .. its width past a's first value, counted modulo the greatest common divisor of the
// strides, so b's rows are apart from them if they fall behind that and end before the next one begins.
// With equal strides that decides it; with others rows that interleave some other way count as overlapping.
bool rows_overlap(const Rows &a, const Rows &b, int64_t rows)
{
    if (!a.p || !b.p || !overlaps(a.p, extent(rows, a.stride, a.width), b.p, extent(rows, b.stride, b.width)))
        return false;
    if (rows == 1)
        return true;
    const int64_t period = std::gcd(a.stride, b.stride) * 4;
    const intptr_t apart = (intptr_t)reinterpret_cast<uintptr_t>(b.p) - (intptr_t)reinterpret_cast<uintptr_t>(a.p);
    const int64_t at = (apart % period + period) % period;
    return at < a.width * 4 || at + b.width * 4 > period;
}

// A row stride that keeps 16-byte alignment, holds a row, and cannot overflow an offset.
inline bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 4 == 0 && stride < ((int64_t)1 << 36); }

qmd_status check_kv(const qmd_kv_cache *c, const qmd_kv_batch *b, bool want_k, bool want_v, KvParams *kv)
{
    if (!c || !b || (want_k && (!c->k || !c->k_scale)) || (want_v && (!c->v || !c->v_scale)) || !b->page_table ||
        !b->kv_len)
        return QMD_ERR_NULL;
    if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->page_tokens < KV_BLOCK ||
        c->page_tokens > 65536 || c->page_tokens % KV_BLOCK != 0 || c->kv_heads < 1 || c->kv_heads > 1024 ||
        c->pages < 1 || c->pages > 0x7fffffff ||
        c->pages * c->kv_heads > 0x7fffffff / (c->page_tokens / KV_BLOCK))  // blocks are counted in 31 bits
        return QMD_ERR_SHAPE;
    if (b->seqs < 1 || b->seqs > QMD_KV_MAX_SEQS || b->max_q < 1 || b->max_q > (1 << 20) || b->rows < 1 ||
        b->rows > (1 << 24) || b->table_stride < 1 || b->table_stride > (1 << 24))
        return QMD_ERR_SHAPE;
    if (!b->q_start && (int64_t)b->seqs * b->max_q > b->rows)
        return QMD_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
        !aligned(b->page_table, 4) || !aligned(b->kv_len, 4) || !aligned(b->q_start, 4))
        return QMD_ERR_MISALIGNED;
    kv->k = c->k;
    kv->v = c->v;
    kv->ks = c->k_scale;
    kv->vs = c->v_scale;
    kv->table = b->page_table;
    kv->len = b->kv_len;
    kv->q_start = b->q_start;
    kv->table_stride = b->table_stride;
    kv->rows = b->rows;
    kv->pages = c->pages;
    kv->heads = c->kv_heads;
    kv->page_blocks = c->page_tokens / KV_BLOCK;
    kv->seqs = b->seqs;
    kv->max_q = b->max_q;
    kv->err = nullptr;
    return QMD_OK;
}

}  // namespace
}  // namespace qmd

using namespace qmd;

extern "C" {

qmd_status qmd_kv_append(const qmd_kv_cache *cache, const qmd_kv_batch *batch, const float *k, int64_t k_stride,
                         const float *v, int64_t v_stride, const float *q, int64_t q_stride, int q_heads,
                         float *q_out, int64_t q_out_stride, const float *rope, int64_t rope_rows, int rot,
                         qmd_rope_pairs pairs, void *stream)
{
    KvParams kv;
    qmd_status st = check_kv(cache, batch, true, true, &kv);
    if (st != QMD_OK)
        return st;
    if (!k || !v)
        return QMD_ERR_NULL;
    const int D = cache->head_dim;
    const int64_t T = batch->rows, kw = (int64_t)kv.heads * D;
    if (!stride_ok(k_stride, kw) || !stride_ok(v_stride, kw))
        return QMD_ERR_SHAPE;
    if ((q != nullptr) != (q_out != nullptr) || (q == nullptr) != (q_heads == 0))
        return QMD_ERR_VALUE;
    const int64_t qw = (int64_t)q_heads * D;
    if (q && (q_heads < 1 || q_heads > 65536 || !stride_ok(q_stride, qw) || !stride_ok(q_out_stride, qw)))
        return QMD_ERR_SHAPE;
    if (rope ? rot < 32 || rot > D || rot % 32 != 0 || rope_rows < 1 || rope_rows > ((int64_t)1 << 31) : rot != 0)
        return QMD_ERR_SHAPE;
    if (pairs != QMD_ROPE_HALVES && pairs != QMD_ROPE_ADJACENT)
        return QMD_ERR_VALUE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(rope, 16))
        return QMD_ERR_MISALIGNED;
    if (q) {  // q_out may be q itself; in place or not, it is written while k, v and the table are read
        const Rows out = {q_out, q_out_stride, qw};
        const bool in_place = q_out == q && q_out_stride == q_stride;
        if ((!in_place && rows_overlap(out, {q, q_stride, qw}, T)) || rows_overlap(out, {k, k_stride, kw}, T) ||
            rows_overlap(out, {v, v_stride, kw}, T) ||
            (rope && overlaps(q_out, extent(T, q_out_stride, qw), rope, extent(rope_rows, rot, rot))))
            return QMD_ERR_VALUE;
    }
    DeviceInfo dev;
    if ((st = current_device(&dev)) != QMD_OK)
        return st;
    if (!(kv.err = device_error_word()))
        return QMD_ERR_DEVICE;
    return launch_kv_append(kv, D, k, k_stride, v, v_stride, q, q_stride, q_heads, q_out, q_out_stride, rope, rope_rows,
                            rot, pairs, dev.sm_count, static_cast<cudaStream_t>(stream));
}

qmd_status qmd_kv_read(const qmd_kv_cache *cache, const qmd_kv_batch *batch, float *k_out, int64_t k_stride,
                       float *v_out, int64_t v_stride, void *stream)
{
    KvParams kv;
    if (!k_out && !v_out)
        return QMD_ERR_NULL;
    qmd_status st = check_kv(cache, batch, k_out != nullptr, v_out != nullptr, &kv);
    if (st != QMD_OK)
        return st;
    const int64_t T = batch->rows, kw = (int64_t)kv.heads * cache->head_dim;
    if ((k_out && !stride_ok(k_stride, kw)) || (v_out && !stride_ok(v_stride, kw)))
        return QMD_ERR_SHAPE;
    if (!aligned(k_out, 16) || !aligned(v_out, 16))
        return QMD_ERR_MISALIGNED;
    if (rows_overlap({k_out, k_stride, kw}, {v_out, v_stride, kw}, T))
        return QMD_ERR_VALUE;
    DeviceInfo dev;
    if ((st = current_device(&dev)) != QMD_OK)
        return st;
    if (!(kv.err = device_error_word()))
        return QMD_ERR_DEVICE;
    return launch_kv_read(kv, cache->head_dim, k_out, k_stride, v_out, v_stride, dev.sm_count,
                          static_cast<cudaStream_t>(stream));
}

qmd_status qmd_kv_attention(const qmd_kv_cache *cache, const qmd_kv_batch *batch, const float *q, int64_t q_stride,
                            int q_heads, float scale, int64_t window, float *out, int64_t out_stride, void *workspace,
                            void *stream)
{
    KvParams kv;
    qmd_status st = check_kv(cache, batch, true, true, &kv);
    if (st != QMD_OK)
        return st;
    if (!q || !out || !workspace)
        return QMD_ERR_NULL;
    const int64_t qw = (int64_t)q_heads * cache->head_dim;
    if (q_heads < 1 || q_heads % kv.heads != 0 || q_heads / kv.heads > 64 || !stride_ok(q_stride, qw) ||
        !stride_ok(out_stride, qw))
        return QMD_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16))
        return QMD_ERR_MISALIGNED;
    if (!std::isfinite(scale) || window < 0 ||
        rows_overlap({out, out_stride, qw}, {q, q_stride, qw}, batch->rows))
        return QMD_ERR_VALUE;
    DeviceInfo dev;
    if ((st = current_device(&dev)) != QMD_OK)
        return st;
    if (!(kv.err = device_error_word()))
        return QMD_ERR_DEVICE;
    return launch_kv_attention(kv, cache->head_dim, q, q_stride, q_heads, scale, window, out, out_stride, workspace,
                               dev, static_cast<cudaStream_t>(stream));
}

size_t qmd_kv_workspace_bytes(void)
{
    DeviceInfo dev;
    return current_device(&dev) == QMD_OK ? kv_attention_workspace(dev) : 0;
}

qmd_status qmd_lora_add(qmd_half type, const float *x, const float *base, const void *A, const void *B,
                        const float *scale, const int32_t *adapter, float *out, int64_t K, int64_t rows, int rank,
                        int adapters, int batch, void *stream)
{
    if (type != QMD_F16 && type != QMD_BF16)
        return QMD_ERR_FORMAT;
    if (!x || !base || !A || !B || !scale || !adapter || !out)
        return QMD_ERR_NULL;
    if (K < QMD_QK || K > 65536)
        return QMD_ERR_SHAPE;
    if (K % QMD_QK != 0)
        return QMD_ERR_K_NOT_MULTIPLE_OF_256;
    if (batch < 1 || batch > QMD_MAX_BATCH)
        return QMD_ERR_BATCH;
    if (rows < 1 || rows > (1 << 24) || rank < 8 || rank > QMD_LORA_MAX_RANK || rank % 8 != 0 || adapters < 1 ||
        adapters > (1 << 20))
        return QMD_ERR_SHAPE;
    if (!aligned(x, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(base, 4) || !aligned(out, 4) ||
        !aligned(scale, 4) || !aligned(adapter, 4))
        return QMD_ERR_MISALIGNED;
    const size_t yb = (size_t)batch * rows * 4;
    if (overlaps(out, yb, x, (size_t)batch * K * 4) || (out != base && overlaps(out, yb, base, yb)))
        return QMD_ERR_VALUE;
    DeviceInfo dev;
    qmd_status st = current_device(&dev);
    if (st != QMD_OK)
        return st;
    unsigned *err = device_error_word();
    if (!err)
        return QMD_ERR_DEVICE;
    return launch_lora_add(type, x, base, A, B, scale, adapter, out, K, rows, rank, adapters, batch, dev, err,
                           static_cast<cudaStream_t>(stream));
}

}  // extern "C"
