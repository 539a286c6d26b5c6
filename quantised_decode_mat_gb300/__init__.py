"""Thin Python binding of libqmd (ctypes): decode-time Q4_K / Q6_K x q8_K mat-vec on GB300, and
the operators of a decode step around it (the 8-bit key/value cache, low-rank adapters).

Argument marshalling only.  Every step of the computation runs in the library's CUDA kernels;
torch supplies device memory and streams.  The functions here carry the C ABI's names
(qmd_q8k_pack -> q8k_pack, qmd_qmatvec -> qmatvec, ...) and raise QmdError on any status
other than QMD_OK.  There is no CPU path: if libqmd.so is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqmd.so")

QMD_QK = 256
QMD_MAX_BATCH = 8
QMD_WORKSPACE_BYTES = 4096
Q4_K = 12
Q5_K = 13
Q6_K_SPLIT = 14
QMD_KV_BLOCK = 16
ROPE_HALVES, ROPE_ADJACENT = 0, 1
F16, BF16 = 1, 2

STATUS = {
    0: "QMD_OK",
    1: "QMD_ERR_NULL",
    2: "QMD_ERR_FORMAT",
    3: "QMD_ERR_K_NOT_MULTIPLE_OF_256",
    4: "QMD_ERR_BATCH",
    5: "QMD_ERR_MISALIGNED",
    6: "QMD_ERR_SHAPE",
    7: "QMD_ERR_LAUNCH",
    8: "QMD_ERR_DEVICE_TIMEOUT",
    9: "QMD_ERR_DEVICE",
    10: "QMD_ERR_VALUE",
    11: "QMD_ERR_INDEX",
}


class QmdError(RuntimeError):
    def __init__(self, status: int, detail: str = ""):
        self.status = status
        self.name = STATUS.get(status, f"status {status}")
        super().__init__(self.name + (f": {detail}" if detail else ""))


class Q8KPtrs(ctypes.Structure):
    _fields_ = [("qs", ctypes.c_void_p), ("d", ctypes.c_void_p), ("bsums", ctypes.c_void_p)]


class KVCachePtrs(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("kv_heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int)]


class KVBatchPtrs(ctypes.Structure):
    _fields_ = [("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("q_start", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64), ("rows", ctypes.c_int64), ("seqs", ctypes.c_int),
                ("max_q", ctypes.c_int)]


_lib = None


def lib(path: str | None = None) -> ctypes.CDLL:
    """Load libqmd.so (raises if it has not been built).  `path` loads another build of the same
    library instead (the traced build, libqmd_trace.so); it must come before the first load."""
    global _lib
    if _lib is not None and path is not None and path != _lib._name:
        raise RuntimeError(f"{_lib._name} is already loaded")
    if _lib is None:
        path = path or LIB_PATH
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'` "
                "or `python -m quantised_decode_mat_gb300.build`")
        L = ctypes.CDLL(path)
        i64, i32, vp, u64 = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_uint64
        ip = ctypes.POINTER(ctypes.c_int)
        sizep = ctypes.POINTER(ctypes.c_size_t)
        cp, bp = ctypes.POINTER(KVCachePtrs), ctypes.POINTER(KVBatchPtrs)
        sigs = {
            "qmd_q8k_pack": ([vp, Q8KPtrs, i64, i32, vp], i32),
            "qmd_rmsnorm_q8k_pack": ([vp, vp, vp, ctypes.c_float, vp, Q8KPtrs, i64, i32, vp], i32),
            "qmd_qmatvec": ([i32, vp, vp, Q8KPtrs, vp, i64, i64, i32, vp], i32),
            "qmd_qmatvec_x": ([i32, vp, vp, vp, Q8KPtrs, vp, i64, i64, i32, vp], i32),
            "qmd_qmatvec_ws": ([i32, vp, vp, Q8KPtrs, vp, i64, i64, i32, vp, vp], i32),
            "qmd_qmatvec_x_ws": ([i32, vp, vp, vp, Q8KPtrs, vp, i64, i64, i32, vp, vp], i32),
            "qmd_qmatvec_x_static": ([i32, vp, vp, vp, Q8KPtrs, vp, i64, i64, i32, vp], i32),
            "qmd_qmatvec_rmsnorm_x": ([i32, vp, vp, vp, vp, vp, ctypes.c_float, vp, Q8KPtrs, vp, i64, i64, i32, vp],
                                      i32),
            "qmd_q6k_prefix_stride": ([i64], i64),
            "qmd_q6k_split_bytes": ([i64, i64, sizep, sizep], i32),
            "qmd_bind_q6k": ([vp, vp, vp, i64, i64, vp], i32),
            "qmd_bind_q4k": ([vp, i64, i64], i32),
            "qmd_bind_q5k": ([vp, i64, i64], i32),
            "qmd_status_str": ([i32], ctypes.c_char_p),
            "qmd_last_error_detail": ([], ctypes.c_char_p),
            "qmd_get_device_error": ([vp], i32),
            "qmd_set_wait_limit_ns": ([u64], None),
            "qmd_qmatvec_launch_info": ([i32, i64, i64, i32, ip, ip, ip, ip, ip], i32),
            "qmd_qmatvec_launch_kernel": ([i32, i64, i64, i32], i32),
            "qmd_debug_qmatvec_dump": ([i32, vp, vp, Q8KPtrs, vp, i64, i64, i32, vp, vp, vp], i32),
            "qmd_debug_wait_timeout": ([u64, vp], i32),
            "qmd_measure_alu": ([ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)], i32),
            "qmd_measure_read_bw": ([vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_double)], i32),
            "qmd_debug_set_plan": ([i32, i32, i32, i32], None),
            "qmd_debug_set_launch_flags": ([ctypes.c_uint], None),
            "qmd_debug_set_dynamic_tiles": ([i32], None),
            "qmd_debug_set_split_k": ([i32], None),
            "qmd_version": ([], i32),
            "qmd_kv_append": ([cp, bp, vp, i64, vp, i64, vp, i64, i32, vp, i64, vp, i64, i32, i32, vp], i32),
            "qmd_kv_read": ([cp, bp, vp, i64, vp, i64, vp], i32),
            "qmd_kv_attention": ([cp, bp, vp, i64, i32, ctypes.c_float, i64, vp, i64, vp, vp], i32),
            "qmd_kv_workspace_bytes": ([], ctypes.c_size_t),
            "qmd_lora_add": ([i32, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, vp], i32),
        }
        if hasattr(L, "qmd_debug_trace"):  # the traced build (include/qmd_trace.h)
            sigs["qmd_debug_trace"] = ([vp, i64], i32)
            sigs["qmd_debug_trace_launches"] = ([vp, vp, i64], i64)
        for name, (args, res) in sigs.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _check(st: int) -> None:
    if st != 0:
        detail = lib().qmd_last_error_detail()
        raise QmdError(st, detail.decode() if detail else "")


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


@dataclass
class Q8K:
    """q8_K-packed activations (torch tensors on one CUDA device): qs int8 [B, K], d f32 [B, nb],
    bsums int16 [B, nb, 8]."""
    qs: "object"
    d: "object"
    bsums: "object"

    @property
    def batch(self) -> int:
        return self.qs.shape[0]

    @property
    def K(self) -> int:
        return self.qs.shape[1]

    def ptrs(self) -> Q8KPtrs:
        return Q8KPtrs(_ptr(self.qs), _ptr(self.d), _ptr(self.bsums))

    @staticmethod
    def empty(batch: int, K: int, device="cuda") -> "Q8K":
        import torch
        nb = K // QMD_QK
        return Q8K(torch.empty((batch, K), dtype=torch.int8, device=device),
                   torch.empty((batch, nb), dtype=torch.float32, device=device),
                   torch.empty((batch, nb, 8), dtype=torch.int16, device=device))


def q8k_pack(x, out: Q8K | None = None, stream=None) -> Q8K:
    """qmd_q8k_pack: x f32 [batch, K] (CUDA, contiguous) -> Q8K."""
    batch, K = x.shape
    if out is None:
        out = Q8K.empty(batch, K, x.device)
    _check(lib().qmd_q8k_pack(_ptr(x), out.ptrs(), K, batch, _stream(stream)))
    return out


def rmsnorm_q8k_pack(x, r, g, eps: float, h_out=None, out: Q8K | None = None, stream=None) -> Q8K:
    """qmd_rmsnorm_q8k_pack: h = x + r (r may be None), n = RMSNorm(h) * g, packed to q8_K.
    x, r, h_out f32 [batch, K]; g f32 [K].  h_out (optional, may be x or r) receives h."""
    batch, K = x.shape
    if out is None:
        out = Q8K.empty(batch, K, x.device)
    _check(lib().qmd_rmsnorm_q8k_pack(_ptr(x), _ptr(r), _ptr(g), float(eps), _ptr(h_out), out.ptrs(), K, batch,
                                      _stream(stream)))
    return out


def workspace(device="cuda"):
    """A zeroed scheduling workspace for qmatvec / qmatvec_x (QMD_WORKSPACE_BYTES on `device`).
    Calls ordered in one stream may share it; concurrent calls need their own."""
    import torch
    return torch.zeros(QMD_WORKSPACE_BYTES // 4, dtype=torch.int32, device=device)


def qmatvec(fmt: int, W, W_aux, xq: Q8K, y=None, rows: int | None = None, stream=None, workspace=None):
    """qmd_qmatvec (qmd_qmatvec_ws with a workspace): y f32 [batch, rows] = W (fmt) x xq.  W is the
    uint8 weight tensor whose first dimension is rows; W_aux the Q6_K prefix (None for Q4_K)."""
    import torch
    rows = W.shape[0] if rows is None else rows
    if y is None:
        y = torch.empty((xq.batch, rows), dtype=torch.float32, device=xq.qs.device)
    if workspace is None:
        _check(lib().qmd_qmatvec(fmt, _ptr(W), _ptr(W_aux), xq.ptrs(), _ptr(y), rows, xq.K, xq.batch,
                                 _stream(stream)))
    else:
        _check(lib().qmd_qmatvec_ws(fmt, _ptr(W), _ptr(W_aux), xq.ptrs(), _ptr(y), rows, xq.K, xq.batch,
                                    _ptr(workspace), _stream(stream)))
    return y


def qmatvec_x(fmt: int, W, W_aux, x, y=None, rows: int | None = None, xq_out: Q8K | None = None,
              stream=None, workspace=None):
    """qmd_qmatvec_x (qmd_qmatvec_x_ws with a workspace): y f32 [batch, rows] = W (fmt) x
    q8k_pack(x), packing inside the kernel.  x: f32 [batch, K].  xq_out: optional Q8K that
    receives the packed activations."""
    import torch
    rows = W.shape[0] if rows is None else rows
    batch, K = x.shape
    if y is None:
        y = torch.empty((batch, rows), dtype=torch.float32, device=x.device)
    out = xq_out.ptrs() if xq_out is not None else Q8KPtrs(None, None, None)
    if workspace is None:
        _check(lib().qmd_qmatvec_x(fmt, _ptr(W), _ptr(W_aux), _ptr(x), out, _ptr(y), rows, K, batch,
                                   _stream(stream)))
    else:
        _check(lib().qmd_qmatvec_x_ws(fmt, _ptr(W), _ptr(W_aux), _ptr(x), out, _ptr(y), rows, K, batch,
                                      _ptr(workspace), _stream(stream)))
    return y


def qmatvec_x_static(fmt: int, W, W_aux, x, y=None, rows: int | None = None, xq_out: Q8K | None = None,
                     stream=None):
    """qmd_qmatvec_x_static: qmatvec_x scheduled through the library's own static workspace, for
    callers that cannot allocate; calls that overlap on the GPU race on that workspace."""
    import torch
    rows = W.shape[0] if rows is None else rows
    batch, K = x.shape
    if y is None:
        y = torch.empty((batch, rows), dtype=torch.float32, device=x.device)
    out = xq_out.ptrs() if xq_out is not None else Q8KPtrs(None, None, None)
    _check(lib().qmd_qmatvec_x_static(fmt, _ptr(W), _ptr(W_aux), _ptr(x), out, _ptr(y), rows, K, batch,
                                      _stream(stream)))
    return y


def qmatvec_rmsnorm_x(fmt: int, W, W_aux, x, r, g, eps: float, h_out=None, y=None, rows: int | None = None,
                      xq_out: Q8K | None = None, stream=None):
    """qmd_qmatvec_rmsnorm_x: y f32 [batch, rows] = W (fmt) x rmsnorm_q8k_pack(x, r, g, eps), in one
    launch.  x, r (may be None), h_out (optional; must not overlap x, r or g) f32 [batch, K];
    g f32 [K]."""
    import torch
    rows = W.shape[0] if rows is None else rows
    batch, K = x.shape
    if y is None:
        y = torch.empty((batch, rows), dtype=torch.float32, device=x.device)
    out = xq_out.ptrs() if xq_out is not None else Q8KPtrs(None, None, None)
    _check(lib().qmd_qmatvec_rmsnorm_x(fmt, _ptr(W), _ptr(W_aux), _ptr(x), _ptr(r), _ptr(g), float(eps),
                                       _ptr(h_out), out, _ptr(y), rows, K, batch, _stream(stream)))
    return y


# ---- the key/value cache and the adapters ------------------------------------------------------


def _need(ok: bool, status: int, detail: str) -> None:
    if not ok:
        raise QmdError(status, detail)


# torch's names that every call below uses, looked up with the first cache or adapter call.
_F32 = _I32 = _device_now = _stream_now = None


def _torch_names() -> None:
    global _F32, _I32, _device_now, _stream_now
    import torch
    _F32, _I32 = torch.float32, torch.int32
    _device_now, _stream_now = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _stream_on(stream, index: int, what: str) -> int:
    """The stream of a call on the device with this index, which has to be the current one."""
    if index < 0 or index != _device_now():
        raise QmdError(9, f"{what} must be on the current CUDA device")
    if stream is None:
        return _stream_now(index)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, device, stream):
    """A new f32 tensor for a call on `stream`: its memory belongs to that stream."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream), device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=torch.float32, device=device)


# The checks below run on every call of a decode step's small operators: messages are made only for
# a refusal.
def _array(t, dtype, shape, index: int, what: str) -> int:
    """The address of a contiguous tensor of this type and shape on the device with this index."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise QmdError(2, f"{what}: {dtype} is wanted, got {t.dtype}")
    if t.shape != shape:
        raise QmdError(6, f"{what}: shape {tuple(shape)} is wanted, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise QmdError(6, f"{what} must be contiguous")
    raise QmdError(9, f"{what} is on {t.device}, not on the device of the others")


def _rows_of(t, rows: int, heads: int | None, dim: int, index: int, what: str) -> tuple[int, int]:
    """(heads, row stride) of f32 rows [rows or more, heads, dim] or [rows or more, heads * dim],
    strided by rows only."""
    if t.dtype is _F32 and t.get_device() == index:
        shape = t.shape
        if len(shape) == 3:
            n, h, d = shape
            a, b, c = t.stride()
            width, ok = h * d, d == dim and c == 1 and (b == dim or h == 1)
        elif len(shape) == 2:
            n, width = shape
            a, b = t.stride()
            ok = b == 1 and width % dim == 0
        else:
            ok = False
        if ok and n >= rows and (width > 0 if heads is None else width == heads * dim):
            return width // dim, a if n > 1 else (width + 3) // 4 * 4
    if t.dtype is not _F32:
        raise QmdError(2, f"{what}: float32 is wanted, got {t.dtype}")
    if t.get_device() != index:
        raise QmdError(9, f"{what} is on {t.device}, not on the cache's device")
    raise QmdError(6, f"{what}: {rows} or more rows of {heads or 'some'} heads of {dim} values are wanted, strided by "
                      f"rows only; got shape {tuple(t.shape)}, strides {tuple(t.stride())}")


class KVCache:
    """A paged 8-bit key/value cache: int8 codes [pages, kv_heads, page_tokens, head_dim] of keys and
    of values, and f32 scales [pages, kv_heads, page_tokens / 16].  A cached value is code * scale."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        _torch_names()
        _need(k.dim() == 4, 6, "k: [pages, kv_heads, page_tokens, head_dim] is wanted")
        pages, heads, tokens, dim = k.shape
        self.index = k.get_device()
        for t, what in ((k, "k"), (v, "v")):
            _array(t, torch.int8, k.shape, self.index, what)
        for t, what in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _array(t, torch.float32, (pages, heads, tokens // QMD_KV_BLOCK), self.index, what)
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.kv_heads, self.head_dim, self.device = heads, dim, k.device
        self.ptrs = KVCachePtrs(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), pages, heads, tokens, dim)

    @staticmethod
    def empty(pages: int, kv_heads: int, page_tokens: int, head_dim: int, device="cuda") -> "KVCache":
        import torch
        codes = [torch.zeros((pages, kv_heads, page_tokens, head_dim), dtype=torch.int8, device=device) for _ in "kv"]
        scales = [torch.zeros((pages, kv_heads, page_tokens // QMD_KV_BLOCK), device=device) for _ in "kv"]
        return KVCache(*codes, *scales)


class KVBatch:
    """The sequences of a call, for every layer of a step: page_table int32 [seqs, columns], kv_len
    int32 [seqs] (tokens in the cache, the call's rows counted in), and q_start int32 [seqs + 1] (the
    first row of each sequence, and the end of the last) with the most rows a sequence has and the
    rows of the call's tensors; without q_start every sequence has max_q rows."""

    def __init__(self, page_table, kv_len, q_start=None, max_q: int = 1, rows: int | None = None):
        _torch_names()
        _need(page_table.dim() == 2, 6, "page_table: [seqs, columns] is wanted")
        seqs = page_table.shape[0]
        self.index = page_table.get_device()
        _array(page_table, _I32, page_table.shape, self.index, "page_table")
        _array(kv_len, _I32, (seqs,), self.index, "kv_len")
        if q_start is not None:
            _array(q_start, _I32, (seqs + 1,), self.index, "q_start")
            _need(rows is not None, 6, "rows: the rows of the call's tensors are wanted with q_start")
        self.page_table, self.kv_len, self.q_start = page_table, kv_len, q_start
        self.max_q, self.rows = max_q, seqs * max_q if rows is None else rows
        # (ctypes would take them modulo 2^32 and 2^64; the library checks what fits)
        _need(abs(max_q) < 1 << 31 and abs(self.rows) < 1 << 63, 6, f"max_q {max_q}, rows {self.rows}")
        self.ptrs = KVBatchPtrs(_ptr(page_table), _ptr(kv_len), _ptr(q_start), page_table.shape[1], self.rows, seqs, max_q)


def _kv_stream(cache: KVCache, batch: KVBatch, stream) -> int:
    if batch.index != cache.index:
        raise QmdError(9, f"the batch is on {batch.page_table.device}, the cache on {cache.device}")
    return _stream_on(stream, cache.index, "the cache")


def rope_table(positions: int, rot: int, base: float = 10000.0, inv_freq=None, device="cuda"):
    """f32 [positions, rot]: the rot / 2 cosines and then the rot / 2 sines of each position's angles
    p * base^(-2 i / rot) (or p * inv_freq[i]), taken in 64 bits: made once, when a model is loaded."""
    import torch
    if inv_freq is None:
        inv_freq = base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device="cpu").detach()
    _need(inv_freq.shape == (rot // 2,), 6, f"inv_freq: {rot // 2} values are wanted")
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * inv_freq
    return torch.cat((angle.cos(), angle.sin()), 1).float().to(device)


def kv_append(cache: KVCache, batch: KVBatch, k, v, rope=None, q=None, q_out=None, pairs: int = ROPE_HALVES,
              stream=None):
    """qmd_kv_append: rotates the rows' keys and queries by the table's positions, quantises keys and
    values into the cache and returns the rotated queries (q_out, by default a new tensor; None
    without q).  k, v f32 [rows, kv_heads, head_dim], q f32 [rows, heads, head_dim], strided by rows
    only (parts of one fused projection's output); q_out may be q."""
    st = _kv_stream(cache, batch, stream)
    D, dev, T = cache.head_dim, cache.index, batch.rows
    _, ks = _rows_of(k, T, cache.kv_heads, D, dev, "k")
    _, vs = _rows_of(v, T, cache.kv_heads, D, dev, "v")
    _need(pairs == ROPE_HALVES or pairs == ROPE_ADJACENT, 10, "pairs: ROPE_HALVES or ROPE_ADJACENT")
    heads = qs = os_ = 0
    if q is not None:
        heads, qs = _rows_of(q, T, None, D, dev, "q")
        if q_out is None:
            q_out = _empty(q.shape, cache.device, stream)
        os_ = qs if q_out is q else _rows_of(q_out, T, heads, D, dev, "q_out")[1]
    n = rot = 0
    if rope is not None:
        _need(rope.dim() == 2, 6, "rope: [positions, rot] is wanted")
        n, rot = rope.shape
        _array(rope, _F32, (n, rot), dev, "rope")
    st = lib().qmd_kv_append(cache.ptrs, batch.ptrs, k.data_ptr(), ks, v.data_ptr(), vs, _ptr(q), qs, heads,
                             _ptr(q_out), os_, _ptr(rope), n, rot, pairs, st)
    if st:
        _check(st)
    return q_out


def kv_read(cache: KVCache, batch: KVBatch, k_out=None, v_out=None, stream=None, keys: bool = True, values: bool = True):
    """qmd_kv_read: the rows' keys and values as the cache holds them, code * scale, f32
    [rows, kv_heads, head_dim] each (new tensors by default).  keys=False or values=False leaves one of
    them out (None in its place)."""
    st = _kv_stream(cache, batch, stream)
    H, D, dev, T = cache.kv_heads, cache.head_dim, cache.index, batch.rows
    if not (keys and values):
        _need(keys or values, 1, "neither keys nor values are wanted")
        _need((keys or k_out is None) and (values or v_out is None), 10, "an output is given for what is left out")
    ks = vs = 0
    if keys:
        if k_out is None:
            k_out = _empty((T, H, D), cache.device, stream)
        _, ks = _rows_of(k_out, T, H, D, dev, "k_out")
    if values:
        if v_out is None:
            v_out = _empty((T, H, D), cache.device, stream)
        _, vs = _rows_of(v_out, T, H, D, dev, "v_out")
    st = lib().qmd_kv_read(cache.ptrs, batch.ptrs, _ptr(k_out), ks, _ptr(v_out), vs, st)
    if st:
        _check(st)
    return k_out, v_out


_workspace_words: dict = {}  # of qmd_kv_workspace_bytes on the devices called so far


def kv_workspace(device="cuda"):
    """A zeroed workspace for kv_attention on the current device.  Calls ordered in one stream may
    share it; calls that may run at the same time (other streams, two captured graphs) need their own."""
    import torch
    n = int(lib().qmd_kv_workspace_bytes())
    _need(n > 0, 9, "no usable device")
    return torch.zeros(n // 4, dtype=torch.int32, device=device)


def kv_attention(cache: KVCache, batch: KVBatch, q, scale: float, workspace, window: int = 0, out=None, stream=None):
    """qmd_kv_attention: attention of the rows' queries (rotated; f32 [rows, heads, head_dim], strided
    by rows only) over the cached keys and values of their sequences.  out f32, by default
    [rows, heads * head_dim]; rows that no sequence owns are not written."""
    st = _kv_stream(cache, batch, stream)
    D, dev, T = cache.head_dim, cache.index, batch.rows
    heads, qs = _rows_of(q, T, None, D, dev, "q")
    if window >> 63:
        raise QmdError(10, f"window: {window}")
    if out is None:
        out = _empty((T, heads * D), cache.device, stream)
    _, os_ = _rows_of(out, T, heads, D, dev, "out")
    L = lib()
    if dev not in _workspace_words:
        _workspace_words[dev] = (int(L.qmd_kv_workspace_bytes()) // 4,)
    ws = _array(workspace, _I32, _workspace_words[dev], dev, "workspace")
    st = L.qmd_kv_attention(cache.ptrs, batch.ptrs, q.data_ptr(), qs, heads, scale, window, out.data_ptr(), os_, ws, st)
    if st:
        _check(st)
    return out


def lora_add(x, base, A, B, adapter, scale, out=None, stream=None):
    """qmd_lora_add: out[v] = base[v] + scale[a] * (B[a] (A[a] x[v])) with a = adapter[v], or base[v]
    where a < 0.  x f32 [batch, K]; base, out f32 [batch, rows] (out may be base); A f16 or bf16
    [adapters, rank, K], B [adapters, rows, rank]; adapter int32 [batch]; scale f32 [adapters]."""
    import torch
    if _F32 is None:
        _torch_names()
    dev = x.get_device()
    st = _stream_on(stream, dev, "x")
    half = A.dtype
    if half is not torch.float16 and half is not torch.bfloat16:
        raise QmdError(2, f"A: float16 or bfloat16 is wanted, got {half}")
    if A.dim() != 3 or x.dim() != 2 or base.dim() != 2:
        raise QmdError(6, "x [batch, K], base [batch, rows] and A [adapters, rank, K] are wanted")
    (n, rank, K), (batch, rows) = A.shape, base.shape
    if out is None:
        out = _empty((batch, rows), x.device, stream)
    # all of it in one condition (seven tensors: a call of _array for each costs 1 us more); what is
    # wrong is found out below
    if not (x.dtype is base.dtype is scale.dtype is out.dtype is _F32 and B.dtype is half and adapter.dtype is _I32
            and x.shape == (batch, K) and B.shape == (n, rows, rank) and scale.shape == (n,) and adapter.shape == (batch,)
            and out.shape == (batch, rows) and x.is_contiguous() and base.is_contiguous() and A.is_contiguous()
            and B.is_contiguous() and scale.is_contiguous() and adapter.is_contiguous() and out.is_contiguous()
            and dev == base.get_device() == A.get_device() == B.get_device() == scale.get_device()
            == adapter.get_device() == out.get_device()):
        for t, dtype, shape, what in ((x, _F32, (batch, K), "x"), (base, _F32, (batch, rows), "base"), (A, half, A.shape, "A"),
                                      (B, half, (n, rows, rank), "B"), (scale, _F32, (n,), "scale"),
                                      (adapter, _I32, (batch,), "adapter"), (out, _F32, (batch, rows), "out")):
            _array(t, dtype, shape, dev, what)
    st = lib().qmd_lora_add(F16 if half is torch.float16 else BF16, x.data_ptr(), base.data_ptr(), A.data_ptr(), B.data_ptr(),
                            scale.data_ptr(), adapter.data_ptr(), out.data_ptr(), K, rows, rank, n, batch, st)
    if st:
        _check(st)
    return out


def q6k_prefix_stride(K: int) -> int:
    return int(lib().qmd_q6k_prefix_stride(K))


def q6k_split_bytes(rows: int, K: int) -> tuple[int, int]:
    b, p = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().qmd_q6k_split_bytes(rows, K, ctypes.byref(b), ctypes.byref(p)))
    return b.value, p.value


def bind_q6k(gguf, rows: int, K: int, body=None, prefix=None, stream=None):
    """qmd_bind_q6k: canonical Q6_K bytes (uint8 CUDA tensor, rows*nb*210) -> (body u8
    [rows, nb*208], prefix int16-typed f16 bits [rows, prefix_stride])."""
    import torch
    nb = K // QMD_QK
    if body is None:
        body = torch.empty((rows, nb * 208), dtype=torch.uint8, device=gguf.device)
    if prefix is None:
        prefix = torch.empty((rows, q6k_prefix_stride(K)), dtype=torch.int16, device=gguf.device)
    _check(lib().qmd_bind_q6k(_ptr(gguf), _ptr(body), _ptr(prefix), rows, K, _stream(stream)))
    return body, prefix


def bind_q4k(gguf, rows: int, K: int):
    """qmd_bind_q4k: checks the slab can be read in place as 32-bit words; returns it unchanged."""
    _check(lib().qmd_bind_q4k(_ptr(gguf), rows, K))
    return gguf


def bind_q5k(gguf, rows: int, K: int):
    """qmd_bind_q5k: checks the slab can be read in place; returns it unchanged."""
    _check(lib().qmd_bind_q5k(_ptr(gguf), rows, K))
    return gguf


def get_device_error(stream=None) -> None:
    """qmd_get_device_error: synchronise and raise QmdError if a kernel's bounded wait gave up."""
    _check(lib().qmd_get_device_error(_stream(stream)))


def set_wait_limit_ns(ns: int) -> None:
    lib().qmd_set_wait_limit_ns(int(ns))


def status_str(st: int) -> str:
    return lib().qmd_status_str(st).decode()


def launch_info(fmt: int, rows: int, K: int, batch: int) -> dict:
    vals = [ctypes.c_int() for _ in range(5)]
    _check(lib().qmd_qmatvec_launch_info(fmt, rows, K, batch, *[ctypes.byref(v) for v in vals]))
    return dict(zip(("grid", "threads", "smem_bytes", "stages", "rows_per_stage"), (v.value for v in vals)))


KERNELS = {0: "qmv_kernel", 1: "qmv_tc_kernel", 2: "qmv_rl_kernel", 3: "qmv_sk_kernel"}


def launch_kernel(fmt: int, rows: int, K: int, batch: int) -> str:
    """qmd_qmatvec_launch_kernel: the name of the kernel qmatvec runs for these sizes."""
    k = int(lib().qmd_qmatvec_launch_kernel(fmt, rows, K, batch))
    if k < 0:
        _check(-k)
    return KERNELS[k]


def debug_qmatvec_dump(fmt: int, W, W_aux, xq: Q8K, rows: int | None = None, stream=None):
    """qmd_debug_qmatvec_dump -> (y [B, rows], dots int32 [B, rows, nb, 16], sm int32 [B, rows, nb, 2])."""
    import torch
    rows = W.shape[0] if rows is None else rows
    dev = xq.qs.device
    nb = xq.K // QMD_QK
    y = torch.empty((xq.batch, rows), dtype=torch.float32, device=dev)
    dots = torch.zeros((xq.batch, rows, nb, 16), dtype=torch.int32, device=dev)
    sm = torch.zeros((xq.batch, rows, nb, 2), dtype=torch.int32, device=dev)
    _check(lib().qmd_debug_qmatvec_dump(fmt, _ptr(W), _ptr(W_aux), xq.ptrs(), _ptr(y), rows, xq.K,
                                        xq.batch, _ptr(dots), _ptr(sm), _stream(stream)))
    return y, dots, sm


def measure_alu() -> tuple[float, float]:
    """qmd_measure_alu: (dp4a instructions/s, mma.sync f16 FLOP/s) measured on this device."""
    d, m = ctypes.c_double(), ctypes.c_double()
    _check(lib().qmd_measure_alu(ctypes.byref(d), ctypes.byref(m)))
    return d.value, m.value


def measure_read_bw(buf) -> float:
    """qmd_measure_read_bw: bytes/s of read-only bulk streaming of `buf` (a CUDA tensor whose
    byte size is a multiple of 16; make it several times the L2)."""
    r = ctypes.c_double()
    _check(lib().qmd_measure_read_bw(_ptr(buf), buf.numel() * buf.element_size(), ctypes.byref(r)))
    return r.value


def debug_wait_timeout(limit_ns: int, stream=None) -> None:
    _check(lib().qmd_debug_wait_timeout(int(limit_ns), _stream(stream)))


def debug_set_plan(row_groups: int = 0, rows_per_stage: int = 0, max_stages: int = 0, ctas_per_sm: int = 0) -> None:
    lib().qmd_debug_set_plan(row_groups, rows_per_stage, max_stages, ctas_per_sm)


def debug_set_launch_flags(flags: int = 0) -> None:
    lib().qmd_debug_set_launch_flags(int(flags))


def debug_set_dynamic_tiles(per_mille: int = -1) -> None:
    lib().qmd_debug_set_dynamic_tiles(int(per_mille))


def debug_set_split_k(ctas: int = 0) -> None:
    """qmd_debug_set_split_k: split each row's blocks over `ctas` CTAs of a cluster (2..8); 0 restores the default."""
    lib().qmd_debug_set_split_k(int(ctas))


def version() -> int:
    return int(lib().qmd_version())
