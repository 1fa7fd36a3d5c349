"""Python binding of libqgemm (the C ABI in include/qgemm.h).

Argument marshalling only: every function takes torch tensors that already live
on the GPU, derives sizes from their shapes, passes raw device pointers and the
current CUDA stream to the C entry point of the same name, and raises
``QGError`` on a non-zero status. All arithmetic happens in the CUDA kernels of
the shared library; there is no other implementation to fall back to, and
loading fails loudly if the library has not been built.
"""
from __future__ import annotations

import ctypes as C
import os

QG_F32 = 0
QG_F16 = 1
Q4_0 = 2
Q8_0 = 8

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgemm.so")

EXPORTS = ("qg_status_str", "qgemv_q4_0", "qgemv_q8_0", "qgemm_cols", "qffn_gate_up_silu",
           "qmoe_workspace_bytes", "qmoe_experts", "qmoe_experts_noalloc", "qrepack",
           "qargmax_f32", "qtopk_f32", "qmoe_router", "qrope_plan", "qrope",
           "qkv_page_bytes", "qkv_append", "qkv_read", "qattn_workspace_bytes", "qattn_paged",
           "qg_kernel_launches", "qg_device_error",
           "qg_wait_selftest", "qg_last_cuda_error", "qg_last_cuda_error_string")

QG_MOE_NOALLOC_WS_BYTES = 1 << 20

# qg_status values (include/qgemm.h)
QG_OK, QG_ERR_NULL, QG_ERR_SHAPE, QG_ERR_ALIGN, QG_ERR_TYPE = 0, 1, 2, 3, 4
QG_ERR_WORKSPACE, QG_ERR_CUDA, QG_ERR_ALIAS = 5, 6, 7
STATUS = {QG_OK: "QG_OK", QG_ERR_NULL: "QG_ERR_NULL", QG_ERR_SHAPE: "QG_ERR_SHAPE",
          QG_ERR_ALIGN: "QG_ERR_ALIGN", QG_ERR_TYPE: "QG_ERR_TYPE",
          QG_ERR_WORKSPACE: "QG_ERR_WORKSPACE", QG_ERR_CUDA: "QG_ERR_CUDA",
          QG_ERR_ALIAS: "QG_ERR_ALIAS"}


class QGError(RuntimeError):
    def __init__(self, fn: str, status: int, msg: str):
        super().__init__(f"{fn}: {STATUS.get(status, status)} ({msg})")
        self.status = status


class QGExpert(C.Structure):
    _fields_ = [("qg", C.c_void_p), ("sg", C.c_void_p), ("qu", C.c_void_p),
                ("su", C.c_void_p), ("qd", C.c_void_p), ("sd", C.c_void_p)]


class QGRope(C.Structure):
    """A rotary plan (host memory), filled by qrope_plan."""
    _fields_ = [("rot_dim", C.c_int32), ("interleaved", C.c_int32), ("mscale", C.c_float),
                ("reserved", C.c_int32), ("step", C.c_uint64 * 128)]


class QGKVCache(C.Structure):
    """A paged key/value cache: device pointers and sizes (made by qkv_cache)."""
    _fields_ = [("pool", C.c_void_p), ("page_table", C.c_void_p), ("type", C.c_int32),
                ("n_kv_heads", C.c_int32), ("head_dim", C.c_int32), ("page_size", C.c_int32),
                ("n_pages", C.c_int32), ("max_pages", C.c_int32), ("n_seq", C.c_int32)]


# bits of the cache calls' error flag (include/qgemm.h)
QG_KV_BAD_SEQ, QG_KV_BAD_POS, QG_KV_BAD_PAGE = 1, 2, 4

_lib = None


def load(path: str | None = None):
    """Load libqgemm.so (built by ``gemm_q4_q8_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"libqgemm.so not built ({path}); run gemm_q4_q8_gb300.build.build()")
    L = C.CDLL(path)
    vp, i32, sz = C.c_void_p, C.c_int, C.c_size_t
    L.qg_status_str.argtypes = [i32]
    L.qg_status_str.restype = C.c_char_p
    gemv = [vp, vp, i32, i32, vp, i32, vp, vp, vp]
    L.qgemv_q4_0.argtypes = gemv
    L.qgemv_q8_0.argtypes = gemv
    L.qgemm_cols.argtypes = [i32] + gemv
    L.qffn_gate_up_silu.argtypes = [i32, vp, vp, vp, vp, i32, i32, vp, i32, vp, vp]
    L.qmoe_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.qmoe_workspace_bytes.restype = sz
    L.qmoe_experts.argtypes = [i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32,
                               C.POINTER(QGExpert), vp, i32, vp, vp, vp, sz, vp, vp, vp]
    L.qmoe_experts_noalloc.argtypes = [i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, vp, i32,
                                       C.POINTER(QGExpert), vp, i32, vp, vp, vp, vp, vp]
    L.qrepack.argtypes = [i32, vp, i32, i32, vp, vp, vp]
    L.qargmax_f32.argtypes = [vp, i32, i32, vp, vp, vp]
    L.qtopk_f32.argtypes = [vp, i32, i32, i32, vp, vp, vp]
    L.qmoe_router.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
    i64, f64 = C.c_int64, C.c_double
    rope, cache = C.POINTER(QGRope), C.POINTER(QGKVCache)
    L.qrope_plan.argtypes = [rope, i32, i32, f64, f64, i32, f64, f64, f64]
    L.qrope.argtypes = [rope, i32, vp, i64, vp, i32, i32, i32, i32, vp, i64, vp]
    L.qkv_page_bytes.argtypes = [i32, i32, i32, i32]
    L.qkv_page_bytes.restype = sz
    L.qkv_append.argtypes = [cache, rope, i32, vp, i64, vp, i64, vp, i64, i32, vp, vp, vp, i32, vp, vp]
    L.qkv_read.argtypes = [cache, vp, vp, i32, i32, vp, vp, vp, vp]
    L.qattn_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
    L.qattn_workspace_bytes.restype = sz
    L.qattn_paged.argtypes = [cache, vp, i32, i32, vp, i32, C.c_float, vp, vp, sz, vp, vp]
    L.qg_kernel_launches.argtypes = []
    L.qg_kernel_launches.restype = C.c_uint64
    L.qg_device_error.argtypes = [C.POINTER(C.c_int32)]
    L.qg_wait_selftest.argtypes = [C.POINTER(C.c_int32), vp]
    L.qg_last_cuda_error.argtypes = []
    L.qg_last_cuda_error_string.argtypes = []
    L.qg_last_cuda_error_string.restype = C.c_char_p
    for f in EXPORTS:
        if f not in ("qg_status_str", "qmoe_workspace_bytes", "qkv_page_bytes",
                     "qattn_workspace_bytes", "qg_kernel_launches", "qg_last_cuda_error_string"):
            getattr(L, f).restype = i32
    _lib = L
    return L


def _check(fn: str, st: int):
    if st != 0:
        msg = load().qg_status_str(st).decode()
        if st == QG_ERR_CUDA:  # name the CUDA error behind it
            msg += ": " + load().qg_last_cuda_error_string().decode()
        raise QGError(fn, st, msg)


def _ptr(t):
    return None if t is None else t.data_ptr()


_raw_stream = _device = None


def _stream(stream):
    """The stream's handle; None: the current stream of the current device."""
    global _raw_stream, _device
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    if _raw_stream is None:
        import torch
        torch.cuda.current_stream()  # sets torch's CUDA side up
        _device = torch._C._cuda_getDevice
        _raw_stream = torch._C._cuda_getCurrentRawStream  # last: another thread that sees it needs the other, too
    return _raw_stream(_device())  # the handle itself, without a Stream object (2.9 us against 0.1)


def qgemv_q4_0(nib, scl, x, y, y0=None, stream=None):
    """y[c] = y0[c] + W x[c]; nib uint8 [rows, k/2], scl f16-bits [rows, k/32],
    x f16 [ncols, k] (1..8 columns), y / y0 f32 [ncols, rows]."""
    rows, k = scl.shape[0], scl.shape[1] * 32
    _check("qgemv_q4_0", load().qgemv_q4_0(_ptr(nib), _ptr(scl), rows, k, _ptr(x), x.shape[0],
                                           _ptr(y0), _ptr(y), _stream(stream)))


def qgemv_q8_0(qs, scl, x, y, y0=None, stream=None):
    """As qgemv_q4_0 with int8 quants qs [rows, k]."""
    rows, k = scl.shape[0], scl.shape[1] * 32
    _check("qgemv_q8_0", load().qgemv_q8_0(_ptr(qs), _ptr(scl), rows, k, _ptr(x), x.shape[0],
                                           _ptr(y0), _ptr(y), _stream(stream)))


def qgemm_cols(qtype, q, scl, x, y, y0=None, stream=None):
    """y[c] = y0[c] + W x[c] for 1..16 columns."""
    rows, k = scl.shape[0], scl.shape[1] * 32
    _check("qgemm_cols", load().qgemm_cols(int(qtype), _ptr(q), _ptr(scl), rows, k, _ptr(x),
                                           x.shape[0], _ptr(y0), _ptr(y), _stream(stream)))


def qffn_gate_up_silu(qtype, qg, sg, qu, su, x, h, stream=None):
    """h[c] = f16(SiLU(Wg x[c]) * (Wu x[c])), h f16 [ncols, rows], 1..16 columns."""
    rows, k = sg.shape[0], sg.shape[1] * 32
    _check("qffn_gate_up_silu",
           load().qffn_gate_up_silu(int(qtype), _ptr(qg), _ptr(sg), _ptr(qu), _ptr(su), rows, k,
                                    _ptr(x), x.shape[0], _ptr(h), _stream(stream)))


def qmoe_workspace_bytes(n_expert, ffn, hidden, ncols, topk) -> int:
    return int(load().qmoe_workspace_bytes(n_expert, ffn, hidden, ncols, topk))


def qmoe_experts(qtype, qg, sg, qu, su, qd, sd, n_expert, ffn, hidden, ids, rw, x, y,
                 ws, y0=None, shared=None, err_flag=None, uniq_ids_out=None, stream=None):
    """Stacked-expert MoE layer; ``shared`` is None or a dict with keys
    qg, sg, qu, su, qd, sd (device tensors)."""
    sh = None
    if shared is not None:
        sh = C.pointer(QGExpert(*[_ptr(shared[n]) for n in ("qg", "sg", "qu", "su", "qd", "sd")]))
    ncols, topk = ids.shape
    _check("qmoe_experts",
           load().qmoe_experts(int(qtype), _ptr(qg), _ptr(sg), _ptr(qu), _ptr(su), _ptr(qd),
                               _ptr(sd), n_expert, ffn, hidden, _ptr(ids), _ptr(rw), topk, sh,
                               _ptr(x), ncols, _ptr(y0), _ptr(y), _ptr(ws),
                               ws.numel() * ws.element_size(), _ptr(err_flag),
                               _ptr(uniq_ids_out), _stream(stream)))


def qmoe_experts_noalloc(qtype, qg, sg, qu, su, qd, sd, n_expert, ffn, hidden, ids, rw, x, y,
                         y0=None, shared=None, err_flag=None, uniq_ids_out=None, stream=None):
    """qmoe_experts with the library's built-in workspace of QG_MOE_NOALLOC_WS_BYTES
    (no caller allocation): for callers that cannot allocate device memory. Every
    shape qmoe_experts accepts fits; calls that overlap on the GPU race on the
    shared workspace."""
    sh = None
    if shared is not None:
        sh = C.pointer(QGExpert(*[_ptr(shared[n]) for n in ("qg", "sg", "qu", "su", "qd", "sd")]))
    ncols, topk = ids.shape
    _check("qmoe_experts_noalloc",
           load().qmoe_experts_noalloc(int(qtype), _ptr(qg), _ptr(sg), _ptr(qu), _ptr(su),
                                       _ptr(qd), _ptr(sd), n_expert, ffn, hidden, _ptr(ids),
                                       _ptr(rw), topk, sh, _ptr(x), ncols, _ptr(y0), _ptr(y),
                                       _ptr(err_flag), _ptr(uniq_ids_out), _stream(stream)))


def qg_kernel_launches() -> int:
    """Kernels launched by the library so far in this process."""
    return int(load().qg_kernel_launches())


QG_DEV_ERR_WAIT = 1


def qg_device_error() -> int:
    """The current device's error word, then cleared (0: no error; bit
    QG_DEV_ERR_WAIT: a tensor-core kernel gave up a wait, so some call since
    the last read returned wrong outputs). Synchronises the device."""
    v = C.c_int32(0)
    _check("qg_device_error", load().qg_device_error(C.byref(v)))
    return int(v.value)


def qg_wait_selftest(stream=None) -> tuple[int, int]:
    """Run the bounded-wait self-test (about 4 s): two waits on an mbarrier
    phase that nothing completes, CTA scope then cluster scope. Returns per
    wait 1 if it completed, 0 if it gave up (both 0 when the bounds work);
    each wait that gives up sets QG_DEV_ERR_WAIT in the device error word."""
    v = (C.c_int32 * 2)()
    _check("qg_wait_selftest", load().qg_wait_selftest(v, _stream(stream)))
    return int(v[0]), int(v[1])


def qrepack(qtype, gguf, rows, k, q_out, scl_out, stream=None):
    """GGUF interleaved blocks (device bytes) -> quant and scale arrays."""
    _check("qrepack", load().qrepack(int(qtype), _ptr(gguf), rows, k, _ptr(q_out), _ptr(scl_out),
                                     _stream(stream)))


def qargmax_f32(x, idx_out, val_out=None, stream=None):
    """Greedy argmax of each row of f32 x [ncols, n] (numbers before NaN, larger
    first, ties by lower index): idx_out int32 [ncols], val_out f32 [ncols] or None."""
    ncols, n = x.shape
    _check("qargmax_f32", load().qargmax_f32(_ptr(x), n, ncols, _ptr(idx_out), _ptr(val_out),
                                             _stream(stream)))


def qtopk_f32(x, k, idx_out, val_out=None, stream=None):
    """The k first-ranked elements of each row of f32 x [ncols, n], in rank order
    (the argmax order): idx_out int32 [ncols, k], val_out f32 [ncols, k] or None."""
    ncols, n = x.shape
    _check("qtopk_f32", load().qtopk_f32(_ptr(x), n, ncols, int(k), _ptr(idx_out), _ptr(val_out),
                                         _stream(stream)))


def qmoe_router(w_router, x, topk, ids_out, rw_out, logits_out=None, stream=None):
    """MoE router: w_router f32 [n_expert, hidden], x f16 [ncols, hidden] ->
    ids_out int32 [ncols, topk] (largest logits, lowest id on ties), rw_out f32
    [ncols, topk] (softmax over them), logits_out None or f32 [ncols, n_expert]."""
    n_expert, hidden = w_router.shape
    _check("qmoe_router", load().qmoe_router(_ptr(w_router), _ptr(x), n_expert, hidden, x.shape[0],
                                             int(topk), _ptr(logits_out), _ptr(ids_out),
                                             _ptr(rw_out), _stream(stream)))


_ELEM = _INT32 = _FLOAT16 = None


def _dtypes():
    """torch's dtypes that the calls below take (torch is imported on first use)."""
    global _ELEM, _INT32, _FLOAT16
    import torch
    _FLOAT16 = torch.float16  # in this order: a thread that finds _ELEM or _INT32 set uses what stands before it, too
    _INT32 = torch.int32
    _ELEM = {torch.float32: QG_F32, torch.float16: QG_F16}


def _elem(t, name):
    """QG_F32 or QG_F16 of a tensor; the cache and rotary calls take nothing else."""
    if _ELEM is None:
        _dtypes()
    kind = _ELEM.get(t.dtype)
    if kind is None:
        raise ValueError(f"{name}: float32 or float16 expected, got {t.dtype}")
    return kind


def _rows(t, shape, name):
    """Token stride of a tensor of `shape` [ntok, heads, head_dim] whose heads are contiguous."""
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(shape)} expected, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and shape[2] > 1) or (s1 != shape[2] and shape[1] > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {t.stride()}")
    return s0


def _dense(t, name, dtype, shape):
    """Address of a contiguous tensor of the given dtype and shape."""
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: contiguous {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _int32s(t, name, n):
    """Address of n contiguous int32, None for None."""
    if t is None:
        return None
    if _INT32 is None:
        _dtypes()
    if t.dtype != _INT32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous int32 expected, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _flag(t):
    return None if t is None else _int32s(t, "err_flag", 1)


def qrope_plan(rot_dim, base=10000.0, interleaved=False, factor=1.0, orig_ctx=0, low_turns=1.0,
               high_turns=32.0, mscale=1.0) -> QGRope:
    """A rotary plan: pairs of the first rot_dim elements of a head turn by
    pos * base^(-2i/rot_dim), the slow ones by 1/factor of it (all of them when
    orig_ctx is 0). Host memory; keep it and pass it to any number of calls."""
    plan = QGRope()
    _check("qrope_plan", load().qrope_plan(C.byref(plan), rot_dim, int(interleaved), base, factor, orig_ctx,
                                           low_turns, high_turns, mscale))
    return plan


def qrope(plan, x, pos, y, stream=None):
    """Rotate x [ntok, heads, head_dim] (f32 or f16, any token stride) at int32
    positions pos [ntok] into y (f32 or f16; y may be x itself)."""
    shape = x.shape
    ntok, heads, d = shape
    st = (_lib or load()).qrope(plan, _elem(x, "x"), x.data_ptr(), _rows(x, shape, "x"), _int32s(pos, "pos", ntok),
                                ntok, heads, d, _elem(y, "y"), y.data_ptr(), _rows(y, shape, "y"), _stream(stream))
    if st:
        _check("qrope", st)


def qkv_page_bytes(qtype, n_kv_heads, head_dim, page_size) -> int:
    """Bytes of a cache page; 0 for sizes the cache does not take."""
    return int(load().qkv_page_bytes(int(qtype), n_kv_heads, head_dim, page_size))


def qkv_cache(qtype, pool, page_table, n_kv_heads, head_dim, page_size) -> QGKVCache:
    """The cache over a pool (contiguous, a whole number of pages, any type) and an
    int32 page_table [n_seq, max_pages]. It keeps both tensors alive."""
    page = qkv_page_bytes(qtype, n_kv_heads, head_dim, page_size)
    if page == 0:
        raise ValueError(f"qkv_cache: no cache of type {qtype}, {n_kv_heads} heads of {head_dim}, "
                         f"pages of {page_size}")
    nbytes = pool.numel() * pool.element_size()
    if not pool.is_contiguous() or nbytes % page:
        raise ValueError(f"pool: contiguous, a multiple of {page} bytes expected")
    n_seq, max_pages = page_table.shape
    c = QGKVCache(pool.data_ptr(), _int32s(page_table, "page_table", n_seq * max_pages), int(qtype), n_kv_heads,
                  head_dim, page_size, nbytes // page, max_pages, n_seq)
    c.tensors = (pool, page_table)
    return c


def qkv_append(cache, k, v, pos, seq=None, rope=None, q=None, q_out=None, err_flag=None, stream=None):
    """Write k, v [ntok, n_kv_heads, head_dim] (f32 or f16, any token stride) at
    int32 (seq, pos) [ntok]; with rope, k is rotated, and so is q [ntok, heads,
    head_dim], which goes to q_out (f16, contiguous). seq None: the tokens are
    the sequences' in turn, ntok / n_seq each."""
    kind, ntok, d = _elem(k, "k"), k.shape[0], cache.head_dim
    want = (ntok, cache.n_kv_heads, d)
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise ValueError("q, k and v must be of one type")
    qp = qo = None
    qs = heads = 0
    if q is not None:
        heads = q.shape[1]
        if q_out is None:
            raise ValueError("q needs a q_out")
        shape = (ntok, heads, d)
        qp, qs, qo = q.data_ptr(), _rows(q, shape, "q"), _dense(q_out, "q_out", _FLOAT16, shape)
    st = (_lib or load()).qkv_append(cache, rope, kind, k.data_ptr(), _rows(k, want, "k"), v.data_ptr(),
                                     _rows(v, want, "v"), qp, qs, heads, qo, _int32s(seq, "seq", ntok),
                                     _int32s(pos, "pos", ntok), ntok, _flag(err_flag), _stream(stream))
    if st:
        _check("qkv_append", st)


def qkv_read(cache, pos, k_out=None, v_out=None, seq=None, err_flag=None, stream=None):
    """Read the tokens at int32 (seq, pos) [ntok] back into k_out, v_out [ntok,
    n_kv_heads, head_dim] (f16 or f32, contiguous; either may be None)."""
    some = k_out if k_out is not None else v_out
    if some is None:
        return
    ntok, kind, dtype = pos.shape[0], _elem(some, "k_out / v_out"), some.dtype
    want = (ntok, cache.n_kv_heads, cache.head_dim)
    st = (_lib or load()).qkv_read(cache, _int32s(seq, "seq", ntok), _int32s(pos, "pos", ntok), ntok, kind,
                                   None if k_out is None else _dense(k_out, "k_out", dtype, want),
                                   None if v_out is None else _dense(v_out, "v_out", dtype, want), _flag(err_flag),
                                   _stream(stream))
    if st:
        _check("qkv_read", st)


def qattn_workspace_bytes(cache, n_heads, ncols) -> int:
    """Workspace bytes of qattn_paged over this cache; 0 for a shape it rejects."""
    return int(load().qattn_workspace_bytes(cache.n_seq, n_heads, cache.n_kv_heads, cache.head_dim, ncols))


def qattn_paged(cache, q, lens, y, ws, scale=None, window=0, err_flag=None, stream=None):
    """Attention of q f16 [n_seq, ncols, heads, head_dim], the last ncols tokens of
    each sequence, over the cached tokens of lens int32 [n_seq] (the new ones
    among them), causal, within `window` tokens if it is not 0; y f16 as q. scale
    None: 1 / sqrt(head_dim)."""
    shape = q.shape
    n, ncols, heads, d = shape
    if n != cache.n_seq or d != cache.head_dim:
        raise ValueError(f"q: [{cache.n_seq}, ncols, heads, {cache.head_dim}] expected, got {tuple(shape)}")
    if not ws.is_contiguous():
        raise ValueError("ws: contiguous workspace expected")
    lens_at = _int32s(lens, "lens", n)  # (sets the dtypes up)
    st = (_lib or load()).qattn_paged(cache, _dense(q, "q", _FLOAT16, shape), heads, ncols, lens_at, window,
                                      d ** -0.5 if scale is None else scale, _dense(y, "y", _FLOAT16, shape),
                                      ws.data_ptr(), ws.nbytes, _flag(err_flag), _stream(stream))
    if st:
        _check("qattn_paged", st)
