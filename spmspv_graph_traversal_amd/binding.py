"""ctypes binding of ``libdbs.so`` (declared in ``include/dbs.h``).

Argument marshalling only (that of the decode-step calls in C++, ``csrc/calls.cpp``): every step of the
computation runs in the HIP library.  Tensors are torch tensors on the current GPU (torch provides the
device memory and the stream); the functions carry the C names.  Importing
this module without the built library raises ``ImportError``, as does a decode-step call without
the built ``_calls.so`` (the sparse products do without it) — there is no
fallback.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdbs.so")

# status codes (dbs_status)
DBS_OK, DBS_ERR_INVALID_ARG, DBS_ERR_BAD_CSR, DBS_ERR_OUT_OF_MEMORY = 0, 1, 2, 3
DBS_ERR_DEVICE, DBS_ERR_UNSUPPORTED, DBS_ERR_BAD_VECTOR, DBS_ERR_TOO_LARGE = 4, 5, 6, 7
DBS_NOALLOC_SCRATCH_BYTES = 32 << 20
# dtypes, semirings, tile formats
DBS_F32, DBS_BF16, DBS_PATTERN = 0, 1, 2
DBS_PLUS_TIMES, DBS_OR_AND = 0, 1
DBS_TILE_COO, DBS_TILE_DENSE, DBS_TILE_FORCE_CSR, DBS_TILE_FORCE_CSC, DBS_TILE_CSR = 0, 1, 2, 3, 4
# options
DBS_OPT_PATH, DBS_OPT_TH3_NUM, DBS_OPT_TH3_DEN = 0, 1, 2
DBS_OPT_LOCAL_PUSH_CUTOFF, DBS_OPT_TIMING, DBS_OPT_CHECK = 3, 4, 5
DBS_OPT_PULL_WIDTH, DBS_OPT_PULL_SHARE = 6, 7
# activations, rotary layouts and frequency scalings, limits
DBS_ACT_SILU, DBS_ACT_GELU_TANH, DBS_ACT_RELU = 0, 1, 2
DBS_ROPE_HALF, DBS_ROPE_INTERLEAVED = 0, 1
DBS_ROPE_PLAIN, DBS_ROPE_LINEAR, DBS_ROPE_BASE, DBS_ROPE_BANDS, DBS_ROPE_RAMP = 0, 1, 2, 3, 4
DBS_Q4_MAX_TOKENS, DBS_Q4_MAX_ROWS, DBS_Q4_MAX_COLUMNS = 524288, 2147483520, 1 << 28
DBS_LOGITS_MAX_ROWS, DBS_ROPE_MAX_DIM, DBS_ROPE_MAX_ELEMENTS = 65535, 1024, 1 << 30
DBS_KV4_MAX_VALUE, DBS_KV4_MAX_DIM, DBS_KV4_MAX_CONTEXT = 65024.0, 256, 1 << 30
DBS_KV4_MAX_SEQUENCES, DBS_KV4_MAX_ROWS, DBS_KV4_MAX_WORKSPACE = 1 << 20, 1 << 24, 1 << 29
# exported arrays
(DBS_ARR_RB_PTR, DBS_ARR_T_CB, DBS_ARR_T_META, DBS_ARR_CB_PTR, DBS_ARR_CSC_RB, DBS_ARR_CSC2CSR,
 DBS_ARR_PAYLOAD, DBS_ARR_SEGMENTS, DBS_ARR_XMASK, DBS_ARR_ACTIVE, DBS_ARR_CSC_CM, DBS_ARR_PAT_SEGS,
 DBS_ARR_T_CBX, DBS_ARR_META2, DBS_ARR_PAT_M2) = range(15)

_ARR_DTYPES = {
    DBS_ARR_RB_PTR: np.uint32, DBS_ARR_T_CB: np.uint32, DBS_ARR_T_META: np.uint64,
    DBS_ARR_CB_PTR: np.uint32, DBS_ARR_CSC_RB: np.uint32, DBS_ARR_CSC2CSR: np.uint32,
    DBS_ARR_PAYLOAD: np.uint8, DBS_ARR_SEGMENTS: np.uint32, DBS_ARR_XMASK: np.uint16,
    DBS_ARR_ACTIVE: np.uint32, DBS_ARR_CSC_CM: np.uint16, DBS_ARR_PAT_SEGS: np.uint32,
    DBS_ARR_T_CBX: np.uint32, DBS_ARR_META2: np.uint64, DBS_ARR_PAT_M2: np.uint32,
}


class dbs_build_options(C.Structure):
    _fields_ = [(name, C.c_int32) for name in (
        "th0", "th1", "th2_num", "th2_den", "force_format", "seg_w_dense", "seg_w_csr",
        "seg_w_coo", "seg_cap")]


class dbs_stats(C.Structure):
    _fields_ = [
        ("m", C.c_int32), ("n", C.c_int32), ("mb", C.c_int32), ("nb", C.c_int32),
        ("nnz", C.c_int64), ("tiles", C.c_int64),
        ("tiles_by_format", C.c_int64 * 5), ("nnz_by_format", C.c_int64 * 5),
        ("segments", C.c_int64), ("payload_bytes", C.c_int64), ("index_bytes", C.c_int64),
        ("format_bytes", C.c_int64), ("build_peak_bytes", C.c_int64),
        ("last_path", C.c_int32), ("last_n_nzblk", C.c_int32), ("last_push_chunks", C.c_int64),
        ("last_meta_ms", C.c_float), ("last_compute_ms", C.c_float),
        ("timed_calls", C.c_int64), ("sum_meta_ms", C.c_double), ("sum_compute_ms", C.c_double),
        ("bfs_levels", C.c_int32), ("bfs_push_levels", C.c_int32), ("bfs_reached", C.c_int64),
        ("bfs_ms", C.c_float), ("bfs_kernel_ms", C.c_float),
    ]


class dbs_logits_params(C.Structure):
    _fields_ = [("hist_ptr", C.c_void_p), ("hist", C.c_void_p), ("hist_len", C.c_int64), ("hist_new", C.c_void_p),
                ("repetition", C.c_void_p), ("frequency", C.c_void_p), ("presence", C.c_void_p),
                ("bias_ptr", C.c_void_p), ("bias_idx", C.c_void_p), ("bias_val", C.c_void_p), ("bias_len", C.c_int64),
                ("mask", C.c_void_p), ("ldmask", C.c_int64)]


class dbs_rope_options(C.Structure):
    _fields_ = [("rot_dim", C.c_int32), ("scaling", C.c_int32), ("base", C.c_double), ("factor", C.c_double),
                ("low", C.c_double), ("high", C.c_double), ("context", C.c_double)]


class dbs_norm_part(C.Structure):
    _fields_ = [("x", C.c_void_p), ("x_token_stride", C.c_int64), ("x_head_stride", C.c_int64), ("out", C.c_void_p),
                ("out_token_stride", C.c_int64), ("out_head_stride", C.c_int64), ("heads", C.c_int32), ("weight", C.c_void_p)]


class dbs_kv4_view(C.Structure):
    """dbs_kv4_cache of the C ABI."""
    _fields_ = [("pool", C.c_void_p), ("page_stride", C.c_int64), ("pages", C.c_int32), ("page_tokens", C.c_int32),
                ("key_heads", C.c_int32), ("head_dim", C.c_int32), ("group", C.c_int32), ("sequences", C.c_int32),
                ("table_pages", C.c_int32), ("table", C.c_void_p), ("ldtable", C.c_int64), ("lens", C.c_void_p),
                ("new_ptr", C.c_void_p)]


EXPORTED = ["dbs_build_options_default", "dbs_build", "dbs_spmspv", "dbs_spmspv_dense",
            "dbs_spmspv_dense_threshold", "dbs_bfs", "dbs_bfs_noalloc",
            "dbs_set_option", "dbs_get_option", "dbs_get_stats", "dbs_copy_array", "dbs_free",
            "dbs_status_string", "dbs_probe_read",
            "dbs_q4_build", "dbs_q4_bytes", "dbs_q4_free", "dbs_q4_product", "dbs_q4_product_masked", "dbs_q4_gated",
            "dbs_logits_adjust", "dbs_rope", "dbs_rope_frequencies", "dbs_norm_rope",
            "dbs_kv4_page_bytes", "dbs_kv4_store", "dbs_kv4_attention_workspace", "dbs_kv4_attention"]


def load_library(path: str = LIB_PATH) -> C.CDLL:
    # torch first: its HIP runtime (SONAME libamdhip64.so.7) is then the one
    # the library binds to, so torch's allocations and streams are valid in
    # the library.  Loading the library first would pull in a second runtime.
    import torch  # noqa: F401

    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build the HIP library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = C.CDLL(path)
    vp, i32, i64 = C.c_void_p, C.c_int32, C.c_int64
    sig = {
        "dbs_build_options_default": [C.POINTER(dbs_build_options)],
        "dbs_build": [i32, i32, i64, vp, vp, vp, C.c_int, C.POINTER(dbs_build_options), vp,
                      C.POINTER(vp)],
        "dbs_spmspv": [vp, i32, vp, vp, C.c_int, vp, vp],
        "dbs_spmspv_dense": [vp, vp, C.c_int, vp, vp],
        "dbs_spmspv_dense_threshold": [vp, vp, C.c_float, C.c_int, vp, vp],
        "dbs_bfs": [vp, i32, vp, vp],
        "dbs_bfs_noalloc": [vp, i32, vp, vp],
        "dbs_set_option": [vp, i32, i64],
        "dbs_get_option": [vp, i32, C.POINTER(i64)],
        "dbs_get_stats": [vp, C.POINTER(dbs_stats)],
        "dbs_copy_array": [vp, i32, vp, i64, C.POINTER(i64)],
        "dbs_free": [vp],
        "dbs_probe_read": [vp, i64, vp, C.c_uint32, vp],
        "dbs_q4_build": [i32, i32, i32, vp, vp, C.c_int, vp, vp, C.POINTER(vp)],
        "dbs_q4_bytes": [vp, C.POINTER(i64)],
        "dbs_q4_free": [vp],
        "dbs_q4_product": [vp, i32, vp, C.c_int, i64, vp, C.c_int, i64, vp],
        "dbs_q4_product_masked": [vp, i32, vp, C.c_int, i64, vp, i64, C.c_float, vp, C.c_int, i64, vp],
        "dbs_q4_gated": [vp, vp, C.c_int, i32, vp, C.c_int, i64, vp, C.c_int, i64, vp],
        "dbs_logits_adjust": [i32, i32, vp, C.c_int, i64, C.c_char_p, vp, C.c_int, i64, vp],
        "dbs_rope": [i32, i32, i32, i32, C.c_int, vp, vp, C.c_float, i32, vp, C.c_int, i64, i64, vp, C.c_int, i64,
                     i64, vp],
        "dbs_norm_rope": [i32, i32, i32, C.c_int, vp, vp, C.c_float, C.c_float, vp, i32, C.c_int, C.c_int, C.c_int, vp],
        "dbs_kv4_page_bytes": [i32, i32, i32, i32, C.POINTER(i64)],
        "dbs_kv4_store": [vp, i32, vp, i64, i64, vp, i64, i64, C.c_int, vp, i64, i64, vp, i64, i64, C.c_int, vp],
        "dbs_kv4_attention_workspace": [vp, i32, i32, C.c_int, C.c_int, i32, i32, i32, C.POINTER(i64)],
        "dbs_kv4_attention": [vp, i32, i32, vp, C.c_int, i64, i64, vp, C.c_int, i64, i64, C.c_float, i32, i32, i32, vp, i64, vp],
        "dbs_rope_frequencies": [C.POINTER(dbs_rope_options), C.POINTER(C.c_double), C.POINTER(C.c_float)],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = C.c_int
    lib.dbs_status_string.argtypes = [C.c_int]
    lib.dbs_status_string.restype = C.c_char_p
    return lib


_lib = load_library()


class DBSError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _lib.dbs_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")


def _check(st: int, where: str) -> None:
    if st != DBS_OK:
        raise DBSError(st, where)


# torch (imported by load_library before the library) and its raw current
# stream getter, looked up once: the per-call wrappers run at a few us
import torch as _torch  # noqa: E402

_RAW_STREAM = getattr(_torch._C, "_cuda_getCurrentRawStream", None)
_Tensor = _torch.Tensor
_I32, _F32, _U8 = (_torch.int32,), (_torch.float32,), (_torch.uint8,)


def _ptr(t):
    # the argtypes are c_void_p: a plain int (or None) converts on the call
    return None if t is None else t.data_ptr()


def _stream(stream, device=None):
    """Raw HIP stream handle: the given stream, else the current stream of
    `device` (the call's output tensor's device), read without building a
    Stream object where torch offers that."""
    if stream is None:
        if _RAW_STREAM is not None and device is not None:
            idx = device.index
            return _RAW_STREAM(idx if idx is not None else _torch.cuda.current_device())
        stream = _torch.cuda.current_stream(device)
    return stream.cuda_stream


def _need(t, name, dtypes, numel=None):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


_BF16_DTYPES = (_torch.bfloat16, _torch.int16, _torch.uint16)


def _value_dtypes(dtype):
    if dtype == DBS_F32:
        return _F32
    if dtype == DBS_BF16:
        return _BF16_DTYPES
    return ()


class Matrix:
    """Owner of a dbs_handle; freed with the object or by dbs_free."""

    def __init__(self, handle: C.c_void_p, m: int, n: int, dtype: int):
        self.handle = handle
        self.m, self.n, self.dtype = m, n, dtype

    @property
    def q4_handle(self):
        raise TypeError("a 4-bit matrix (dbs_q4_build) is expected, not a sparse one")

    def __del__(self):
        try:
            dbs_free(self)
        except Exception:
            pass


def default_build_options() -> dbs_build_options:
    o = dbs_build_options()
    _check(_lib.dbs_build_options_default(C.byref(o)), "dbs_build_options_default")
    return o


def dbs_build(m, n, row_ptr, col_idx, val, dtype, options=None, stream=None) -> Matrix:
    import torch

    _need(row_ptr, "row_ptr", (torch.int32,), m + 1)
    _need(col_idx, "col_idx", (torch.int32,))
    nnz = col_idx.numel()
    if dtype != DBS_PATTERN:
        _need(val, "val", _value_dtypes(dtype), nnz)
    h = C.c_void_p()
    opt = C.byref(options) if options is not None else None
    st = _lib.dbs_build(int(m), int(n), int(nnz), _ptr(row_ptr), _ptr(col_idx),
                        _ptr(val) if dtype != DBS_PATTERN else None, int(dtype), opt,
                        _stream(stream), C.byref(h))
    _check(st, "dbs_build")
    return Matrix(h, int(m), int(n), int(dtype))


def dbs_spmspv(A: Matrix, x_idx, x_val, semiring, y, stream=None) -> None:
    _need(x_idx, "x_idx", _I32)
    if semiring == DBS_PLUS_TIMES:
        _need(x_val, "x_val", _value_dtypes(A.dtype), x_idx.numel())
        _need(y, "y", _F32, A.m)
        xv = x_val.data_ptr()
    else:
        _need(y, "y", _U8, A.m)
        xv = None
    st = _lib.dbs_spmspv(A.handle, x_idx.numel(), x_idx.data_ptr(), xv, int(semiring), y.data_ptr(),
                         _stream(stream, y.device))
    if st != DBS_OK:
        raise DBSError(st, "dbs_spmspv")


def dbs_spmspv_dense(A: Matrix, x, semiring, y, stream=None) -> None:
    import torch

    xd = _value_dtypes(A.dtype) if A.dtype != DBS_PATTERN else (torch.float32,)
    _need(x, "x", xd, A.n)
    _need(y, "y", (torch.float32,) if semiring == DBS_PLUS_TIMES else (torch.uint8,), A.m)
    _check(_lib.dbs_spmspv_dense(A.handle, _ptr(x), int(semiring), _ptr(y), _stream(stream, y.device)),
           "dbs_spmspv_dense")


def dbs_spmspv_dense_threshold(A: Matrix, x, threshold: float, semiring, y, stream=None) -> None:
    import torch

    xd = _value_dtypes(A.dtype) if A.dtype != DBS_PATTERN else (torch.float32,)
    _need(x, "x", xd, A.n)
    _need(y, "y", (torch.float32,) if semiring == DBS_PLUS_TIMES else (torch.uint8,), A.m)
    _check(_lib.dbs_spmspv_dense_threshold(A.handle, _ptr(x), float(threshold), int(semiring), _ptr(y),
                                           _stream(stream, y.device)), "dbs_spmspv_dense_threshold")


def dbs_bfs(A: Matrix, src: int, levels, stream=None) -> None:
    import torch

    _need(levels, "levels", (torch.int32,), A.m)
    _check(_lib.dbs_bfs(A.handle, int(src), _ptr(levels), _stream(stream, levels.device)), "dbs_bfs")


def dbs_bfs_noalloc(A: Matrix, src: int, levels, stream=None) -> None:
    """dbs_bfs without allocation: the run's scratch is the library's fixed
    per-device array (DBS_NOALLOC_SCRATCH_BYTES); DBS_ERR_TOO_LARGE above it."""
    import torch

    _need(levels, "levels", (torch.int32,), A.m)
    _check(_lib.dbs_bfs_noalloc(A.handle, int(src), _ptr(levels), _stream(stream, levels.device)),
           "dbs_bfs_noalloc")


def dbs_set_option(A: Matrix, option: int, value: int) -> None:
    _check(_lib.dbs_set_option(A.handle, int(option), int(value)), "dbs_set_option")


def dbs_get_option(A: Matrix, option: int) -> int:
    v = C.c_int64()
    _check(_lib.dbs_get_option(A.handle, int(option), C.byref(v)), "dbs_get_option")
    return int(v.value)


def dbs_get_stats(A: Matrix, allow_bad_vector: bool = False) -> dict:
    s = dbs_stats()
    st = _lib.dbs_get_stats(A.handle, C.byref(s))
    if not (allow_bad_vector and st == DBS_ERR_BAD_VECTOR):
        _check(st, "dbs_get_stats")
    out = {}
    for name, _ in dbs_stats._fields_:
        v = getattr(s, name)
        out[name] = list(v) if isinstance(v, C.Array) else v
    out["status"] = st
    return out


def dbs_copy_array(A: Matrix, which: int) -> np.ndarray:
    nbytes = C.c_int64()
    _check(_lib.dbs_copy_array(A.handle, int(which), None, 0, C.byref(nbytes)), "dbs_copy_array")
    dt = _ARR_DTYPES[which]
    out = np.empty(nbytes.value // np.dtype(dt).itemsize, dtype=dt)
    _check(_lib.dbs_copy_array(A.handle, int(which), out.ctypes.data_as(C.c_void_p), out.nbytes,
                               C.byref(nbytes)), "dbs_copy_array")
    return out


def dbs_probe_read(buf, sink, never: int = 0xFFFFFFFF, stream=None) -> None:
    """Read the CUDA tensor `buf` once through the library's streaming-read
    probe (a measurement helper); `sink` is a one-element int32 CUDA tensor
    written only if some thread's XOR of words equals `never`."""
    if not isinstance(buf, _Tensor) or not buf.is_cuda or not buf.is_contiguous():
        raise TypeError("buf must be a contiguous CUDA tensor")
    _need(sink, "sink", _I32, 1)
    _check(_lib.dbs_probe_read(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(),
                               int(never) & 0xFFFFFFFF, _stream(stream, buf.device)), "dbs_probe_read")


def dbs_free(A: Matrix) -> None:
    if A.handle is not None and A.handle.value:
        _check(_lib.dbs_free(A.handle), "dbs_free")
        A.handle = C.c_void_p()


# ---------------------------------------------------------------------------
# The steps of a decoded token around the sparse products.  Tensors of several
# tokens are [tokens, elements] with contiguous elements and any row stride;
# all tensors of a call are on the current device.  Nothing here records
# gradients.
# ---------------------------------------------------------------------------
_VECTOR = {_torch.float32: DBS_F32, _torch.bfloat16: DBS_BF16}


class _NoCalls:
    """In place of ``_calls.so``: a decode-step call says why it cannot run."""

    def __init__(self, why: str):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(self._why)


def _load_calls():
    path = os.path.join(_HERE, "_calls.so")
    if not os.path.exists(path):
        return _NoCalls(f"{path} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    try:
        from . import _calls
    except ImportError as e:  # built for another torch or interpreter
        return _NoCalls(f"{path} does not load, build it again: {e}")
    _calls.bind(*(C.cast(getattr(_lib, f), C.c_void_p).value for f in (
        "dbs_q4_product", "dbs_q4_product_masked", "dbs_q4_gated", "dbs_logits_adjust", "dbs_rope", "dbs_norm_rope",
        "dbs_kv4_page_bytes", "dbs_kv4_store", "dbs_kv4_attention_workspace", "dbs_kv4_attention")))
    return _calls


_calls = _load_calls()


class Q4Matrix:
    """Owner of a dbs_q4_handle; freed with the object or by dbs_q4_free."""

    def __init__(self, q4_handle: C.c_void_p, m: int, n: int, group: int):
        self.q4_handle = q4_handle
        self.m, self.n, self.group = m, n, group

    @property
    def handle(self):
        raise TypeError("a sparse matrix (dbs_build) is expected, not a 4-bit one")

    def __del__(self):
        try:
            dbs_q4_free(self)
        except Exception:
            pass


def dbs_q4_build(m, n, group, codes, scales, zeros=None, stream=None) -> Q4Matrix:
    """W[i, j] = scales[i, j // group] * (code[i, j] - zeros[i, j // group]) in 4 bits: codes uint8
    [m, ceil(n/2)] (even column in the low nibble), scales [m, ceil(n/group)] float32 or bfloat16, zeros uint8
    of that shape (each at most 15) or None (8)."""
    m, n, group = int(m), int(n), int(group)
    if group not in (32, 64, 128):
        raise ValueError(f"group {group}: 32, 64 or 128 expected")
    if m > DBS_Q4_MAX_ROWS or n > DBS_Q4_MAX_COLUMNS:  # here, since ctypes keeps the low 32 bits
        raise ValueError(f"{m} x {n} is too large: at most {DBS_Q4_MAX_ROWS} x {DBS_Q4_MAX_COLUMNS}")
    groups = (n + group - 1) // group
    _need(codes, "codes", (_torch.uint8,), m * ((n + 1) // 2))
    _need(scales, "scales", tuple(_VECTOR), m * groups)
    if zeros is not None:
        _need(zeros, "zeros", (_torch.uint8,), m * groups)
    for t, name in ((codes, "codes"), (scales, "scales"), (zeros, "zeros")):
        if t is not None and t.get_device() != _torch.cuda.current_device():
            raise ValueError(f"{name} is not on the current device")
    if getattr(stream, "device_index", codes.get_device()) != codes.get_device():
        raise ValueError(f"the stream is on device {stream.device_index}, the call runs on the current device, {codes.get_device()}")
    h = C.c_void_p()
    _check(_lib.dbs_q4_build(m, n, group, _ptr(codes), _ptr(scales), _VECTOR[scales.dtype], _ptr(zeros),
                             _stream(stream, codes.device), C.byref(h)), "dbs_q4_build")
    return Q4Matrix(h, m, n, group)


def dbs_q4_bytes(A: Q4Matrix) -> int:
    v = C.c_int64()
    _check(_lib.dbs_q4_bytes(A.q4_handle, C.byref(v)), "dbs_q4_bytes")
    return int(v.value)


def dbs_q4_free(A: Q4Matrix) -> None:
    if A.q4_handle is not None and A.q4_handle.value:
        _check(_lib.dbs_q4_free(A.q4_handle), "dbs_q4_free")
        A.q4_handle = C.c_void_p()


def dbs_q4_product(A: Q4Matrix, x, y, stream=None) -> None:
    """y[t] = W x[t]; x [n] or [tokens, n], y [m] or [tokens, m], each float32 or bfloat16."""
    st = _calls.q4_product(A.q4_handle.value, A.m, A.n, x, y, stream)
    if st:
        raise DBSError(st, "dbs_q4_product")


def dbs_q4_product_masked(A: Q4Matrix, x, row_mask, y, fill: float = float("-inf"), stream=None) -> None:
    """dbs_q4_product for the rows whose bit is set in row_mask (int32 words [tokens, ceil(m/32)]), `fill`
    elsewhere."""
    st = _calls.q4_product_masked(A.q4_handle.value, A.m, A.n, x, row_mask, fill, y, stream)
    if st:
        raise DBSError(st, "dbs_q4_product_masked")


def dbs_q4_gated(G: Q4Matrix, U: Q4Matrix, x, activation: int, y, stream=None) -> None:
    """y[t] = act(G x[t]) * (U x[t]) for two matrices of one shape, group and scale type."""
    st = _calls.q4_gated(G.q4_handle.value, U.q4_handle.value, G.m, G.n, x, activation, y, stream)
    if st:
        raise DBSError(st, "dbs_q4_gated")


def dbs_logits_adjust(logits, out, hist_ptr=None, hist=None, hist_new=None, repetition=None, frequency=None,
                      presence=None, bias_ptr=None, bias_idx=None, bias_val=None, mask=None, stream=None) -> None:
    """Penalties for repeated tokens, sparse biases and a bit mask on rows of logits ([vocab] or [rows, vocab]);
    `out` may be `logits`.  Lists are ragged: row b's history is hist[hist_ptr[b]:hist_ptr[b + 1]], of which the
    entries from hist_new[b] on count for frequency and presence; its biases likewise."""
    st = _calls.logits_adjust(logits, out, hist_ptr, hist, hist_new, repetition, frequency, presence, bias_ptr, bias_idx,
                              bias_val, mask, stream)
    if st:
        raise DBSError(st, "dbs_logits_adjust")


def dbs_rope(x, pos, freq, out, layout: int = DBS_ROPE_HALF, scale: float = 1.0, inverse: bool = False,
             stream=None) -> None:
    """Rotary positions on x [tokens, heads, head_dim] (any token and head stride) into `out`, which may be x:
    the first 2 * freq.numel() elements of each head are rotated by pos[token] * freq (int32 positions, float64
    frequencies, dbs_rope_frequencies), the others copied; tokens of negative position are left alone."""
    st = _calls.rope(x, pos, freq, out, layout, scale, inverse, stream)
    if st:
        raise DBSError(st, "dbs_rope")


def dbs_rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: int = DBS_ROPE_PLAIN, factor: float = 1.0,
                         low: float = 1.0, high: float = 4.0, context: float = 0.0):
    """(frequencies, scale) for dbs_rope: a float64 CPU tensor [rot_dim / 2] and the factor of the rotated
    elements (1 but for DBS_ROPE_RAMP)."""
    o = dbs_rope_options(int(rot_dim), int(scaling), float(base), float(factor), float(low), float(high), float(context))
    freq = _torch.empty(max(0, int(rot_dim)) // 2, dtype=_torch.float64)
    scale = C.c_float()
    _check(_lib.dbs_rope_frequencies(C.byref(o), C.cast(freq.data_ptr(), C.POINTER(C.c_double)) if freq.numel() else None,
                                     C.byref(scale)), "dbs_rope_frequencies")
    return freq, float(scale.value)


def dbs_norm_rope(q, k, q_weight, k_weight, pos, freq, q_out, k_out, eps: float = 1e-6, layout: int = DBS_ROPE_HALF,
                  scale: float = 1.0, stream=None) -> None:
    """Root mean square norms of the heads of q and k [tokens, heads, head_dim] with weights [head_dim] (or None: ones),
    then dbs_rope on them, into q_out and k_out, which may be q and k themselves.  k, k_weight and k_out may be None."""
    st = _calls.norm_rope(q, k, q_weight, k_weight, pos, freq, q_out, k_out, eps, layout, scale, stream)
    if st:
        raise DBSError(st, "dbs_norm_rope")


class KV4Cache:
    """The pages of a cache of 4-bit keys and values, and what they hold: `pool` is uint8 [pages, bytes], the caller's or
    one of dbs_kv4_cache's; the bytes of a page are those of dbs_kv4_page_bytes or more."""

    def __init__(self, pool, key_heads: int, head_dim: int, group: int, page_tokens: int):
        self.pool = pool
        self.key_heads, self.head_dim, self.group, self.page_tokens = key_heads, head_dim, group, page_tokens


def dbs_kv4_page_bytes(key_heads: int, head_dim: int, group: int, page_tokens: int) -> int:
    v = C.c_int64()
    for x in (key_heads, head_dim, group, page_tokens):  # here, since ctypes keeps the low 32 bits
        if not 0 <= int(x) < 1 << 31:
            raise ValueError(f"{x} is out of range")
    _check(_lib.dbs_kv4_page_bytes(int(key_heads), int(head_dim), int(group), int(page_tokens), C.byref(v)), "dbs_kv4_page_bytes")
    return int(v.value)


def dbs_kv4_cache(pages: int, key_heads: int, head_dim: int, group: int, page_tokens: int, pool=None) -> KV4Cache:
    """The description of `pages` pages of `page_tokens` tokens (16 to 256, a power of two) of key_heads heads of
    head_dim (a multiple of 8 up to 256) in groups of 32, 64 or 128 channels.  Without `pool` the pages are allocated on
    the current device; their tokens are undefined until dbs_kv4_store."""
    size = dbs_kv4_page_bytes(key_heads, head_dim, group, page_tokens)
    if pool is None:
        pool = _torch.empty(int(pages), size, dtype=_torch.uint8, device="cuda")
    elif not isinstance(pool, _Tensor) or not pool.is_cuda or pool.dtype != _torch.uint8:
        raise TypeError("pool must be a uint8 CUDA tensor")
    elif pool.dim() != 2 or pool.size(0) != pages or pool.size(1) < size or (pool.size(1) > 1 and pool.stride(1) != 1):
        raise ValueError(f"pool must be [{pages}, {size} or more] with contiguous pages")
    elif pool.size(0) > 1 and pool.stride(0) < pool.size(1):
        raise ValueError("pages of the pool overlap")
    return KV4Cache(pool, int(key_heads), int(head_dim), int(group), int(page_tokens))


def dbs_kv4_store(cache: KV4Cache, table, lens, k, v, new_ptr=None, k_out=None, v_out=None, stream=None) -> None:
    """Keys and values [tokens, key_heads, head_dim] of the new tokens into their pages: row new_ptr[b] + i is the i-th of
    sequence b's new tokens, the last ones of its lens[b] tokens, whose pages are table[b] (int32); without new_ptr every
    sequence has tokens / sequences new ones.  k_out and v_out receive what the cache now stands for."""
    st = _calls.kv4_store(cache.pool, cache.key_heads, cache.head_dim, cache.group, cache.page_tokens, table, lens, k, v,
                          new_ptr, k_out, v_out, stream)
    if st:
        raise DBSError(st, "dbs_kv4_store")


def dbs_kv4_attention(cache: KV4Cache, table, lens, q, out, new_ptr=None, window: int = 0, sinks: int = 0, scale=None,
                      max_len: int = 0, workspace=None, stream=None) -> None:
    """Attention of the new tokens, stored before, over their sequences: q and out [tokens, heads, head_dim].  A token at
    position i sees tokens j <= i and, with a window, of these j > i - window and j < sinks.  scale: 1/sqrt(head_dim)
    unless given.  max_len bounds lens (0: the table's room); it and the workspace (uint8, allocated for the call
    unless given) only tell how the work is cut: give the bound where it is far below the room.  Where the allocation
    fails the call raises torch.OutOfMemoryError; an empty workspace asks for none, and the work is not cut."""
    st = _calls.kv4_attention(cache.pool, cache.key_heads, cache.head_dim, cache.group, cache.page_tokens, table, lens, q, out,
                              new_ptr, window, sinks, scale, max_len, workspace, stream)
    if st:
        raise DBSError(st, "dbs_kv4_attention")


def dbs_kv4_attention_workspace(cache: KV4Cache, table, lens, q, out, new_ptr=None, window: int = 0, sinks: int = 0,
                                max_len: int = 0) -> int:
    """Bytes of the workspace that dbs_kv4_attention takes for these arguments."""
    return _calls.kv4_workspace(cache.pool, cache.key_heads, cache.head_dim, cache.group, cache.page_tokens, table, lens, q, out,
                                new_ptr, window, sinks, max_len)
