"""Thin binding over librd.so (include/rd.h): ctypes, and for the routed layer's calls, whose kernels run
for a few microseconds, the native module ``_rd`` (csrc/rd_torch.cpp).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  PyTorch supplies device memory and the current
stream.  There is no fallback: if the library is missing or a call fails,
an exception is raised.

Device scalars (``group_offset``, ``limit``) are passed as int32 tensors of
shape ``(1,)`` on the GPU, and ``group_sizes`` as an int32 GPU tensor, so a
call never reads device data on the host and can be captured in a HIP graph.
"""

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librd.so")

ABI_VERSION = 8
RD_OK, RD_EINVAL, RD_EUNSUPPORTED, RD_EHIP, RD_ESCRATCH = 0, 1, 2, 3, 4
RD_NOALLOC_SCRATCH_BYTES = 80 << 20
RD_BF16, RD_F32 = 0, 1
_DTYPES = {torch.bfloat16: RD_BF16, torch.float32: RD_F32}

EXPORTS = (
    "rd_abi_version",
    "rd_status_string",
    "rd_forward_workspace_size",
    "rd_forward",
    "rd_forward_noalloc",
    "rd_forward_trans_rhs",
    "rd_forward_trans_rhs_fp8",
    "rd_forward_fp8",
    "rd_forward_glu",
    "rd_trans_workspace_size",
    "rd_trans",
    "rd_trans_fp8",
    "rd_glu_fwd",
    "rd_glu_bwd",
    "rd_unsort_bwd_rows",
    "rd_zero_rows_from_limit",
    "rd_route",
    "rd_route_bwd",
    "rd_group_rows_workspace_size",
    "rd_group_rows",
    "rd_dispatch_rows",
    "rd_combine_rows",
    "rd_combine_rows_bwd",
    "rd_quantize_mx",
    "rd_dequantize_mx",
    "rd_forward_mx",
    "rd_glu_fwd_mx8",
    "rd_glu_bwd_mx8",
    "rd_tune_set",
    "rd_tune_tile_count",
)
RD_TUNE_FWD_TILE, RD_TUNE_TRANS_TILE, RD_TUNE_DECODE = 0, 1, 2
RD_SOFTMAX, RD_SIGMOID = 0, 1
_SCORES = {"softmax": RD_SOFTMAX, "sigmoid": RD_SIGMOID}
MX_BLOCK = 32  # elements that share one MX scale


class RDError(RuntimeError):
    """A nonzero status from librd.so."""


_lib = None


def library():
    """The loaded librd.so (loaded once, after torch's HIP runtime)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RDError(f"{LIB_PATH} is not built; run `python -m expert_ffn_ragged_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.rd_abi_version.restype = ctypes.c_int
    lib.rd_abi_version.argtypes = []
    lib.rd_status_string.restype = ctypes.c_char_p
    lib.rd_status_string.argtypes = [ctypes.c_int]
    lib.rd_forward_workspace_size.restype = sz
    lib.rd_forward_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    fwd = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp, sz, vp]
    for name in ("rd_forward", "rd_forward_trans_rhs"):
        getattr(lib, name).restype = ctypes.c_int
        getattr(lib, name).argtypes = fwd
    lib.rd_forward_noalloc.restype = ctypes.c_int
    lib.rd_forward_noalloc.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp]
    lib.rd_forward_trans_rhs_fp8.restype = ctypes.c_int
    lib.rd_forward_trans_rhs_fp8.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp]
    lib.rd_forward_fp8.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp]
    lib.rd_forward_glu.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, vp, i64, i64, i64, vp]
    lib.rd_trans_workspace_size.restype = sz
    lib.rd_trans_workspace_size.argtypes = [i64, i64, i64, i32]
    lib.rd_trans.restype = ctypes.c_int
    lib.rd_trans.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp, sz, vp]
    lib.rd_trans_fp8.argtypes = [vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp, sz, vp]
    lib.rd_glu_fwd.restype = ctypes.c_int
    lib.rd_glu_fwd.argtypes = [vp, vp, vp, i64, i64, vp]
    lib.rd_glu_bwd.restype = ctypes.c_int
    lib.rd_glu_bwd.argtypes = [vp, vp, vp, vp, i64, i64, vp]
    lib.rd_unsort_bwd_rows.restype = ctypes.c_int
    lib.rd_unsort_bwd_rows.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, vp]
    lib.rd_zero_rows_from_limit.restype = ctypes.c_int
    lib.rd_zero_rows_from_limit.argtypes = [vp, vp, i64, i64, vp]
    f32 = ctypes.c_float
    lib.rd_route.argtypes = [vp, i32, vp, vp, vp, vp, i64, i32, i32, i32, i32, i32, i32, f32, vp]
    lib.rd_route_bwd.argtypes = [vp, i32, vp, vp, vp, i64, i32, i32, i32, i32, f32, vp]
    lib.rd_group_rows_workspace_size.restype = sz
    lib.rd_group_rows_workspace_size.argtypes = [i64, i32]
    lib.rd_group_rows.argtypes = [vp, i64, i32, vp, vp, vp, vp, vp, sz, vp]
    lib.rd_dispatch_rows.argtypes = [vp, vp, vp, i64, i32, i64, i64, vp]
    lib.rd_combine_rows.argtypes = [vp, vp, vp, vp, i64, i32, i64, i64, vp]
    lib.rd_combine_rows_bwd.argtypes = [vp, vp, vp, vp, vp, vp, i64, i32, i64, i64, vp]
    lib.rd_quantize_mx.argtypes = [vp, i32, vp, vp, vp, i64, i64, i32, vp]
    lib.rd_dequantize_mx.argtypes = [vp, vp, vp, vp, i32, i64, i64, i32, vp]
    lib.rd_forward_mx.argtypes = [vp, vp, i32, vp, vp, vp, i32, vp, i32, vp, vp, i32, i64, i64, i64, vp]
    lib.rd_glu_fwd_mx8.argtypes = [vp, vp, vp, vp, vp, i64, i64, vp]
    lib.rd_glu_bwd_mx8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, vp]
    lib.rd_tune_set.restype = ctypes.c_int
    lib.rd_tune_set.argtypes = [i32, i32]
    lib.rd_tune_tile_count.restype = ctypes.c_int
    lib.rd_tune_tile_count.argtypes = []
    if lib.rd_abi_version() != ABI_VERSION:
        raise RDError("librd.so ABI version mismatch")
    _lib = lib
    return lib


_module = None


def _native():
    """The _rd module (loaded once, on first use)."""
    global _module
    if _module is None:
        library()  # checks the ABI's version
        try:
            from . import _rd
        except ImportError as e:
            raise RDError("_rd.so is not built or does not load; run `python -m expert_ffn_ragged_amd.build`") from e
        _rd.setup(RDError, torch.OutOfMemoryError, _raw_stream)
        _module = _rd
    return _module


def _check(status):
    if status != RD_OK:
        raise RDError(library().rd_status_string(status).decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream_handle(index):
    return torch.cuda.current_stream(index).cuda_stream


# The current stream's handle and the current device as torch's own launchers ask for them: under 0.2 us,
# where torch.cuda.current_stream() and a torch.cuda.device() block take 2 and 1.4 (a whole call takes 7).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream_handle)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _launch(fn, tensors, stream, *args):
    """Call C entry point ``fn(*args, stream)`` with the one GPU that every tensor of the call lives on
    made current (the library sizes its grids, and finds its per-GPU scratch, on the current device);
    ``stream`` None means that GPU's current torch stream."""
    dev = None
    for t in tensors:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"operands on {dev} and {t.device}: every tensor of a call must be on one GPU")
    if stream is None:
        handle = _raw_stream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"stream on {stream.device}, operands on {dev}")
    else:
        handle = stream.cuda_stream
    if _current_device() == dev.index:
        _check(fn(*args, handle))
    else:
        with torch.cuda.device(dev):
            _check(fn(*args, handle))


def _empty(shape, dtype, device, stream):
    """A new tensor for the kernels of a call on ``stream`` (None: torch's current one).

    It comes from that stream's memory: the current stream's may still be in use by work that was queued there
    before its tensor was freed, and nothing orders the call after that work.  The caller goes on with the tensor
    on the current stream, so the caching allocator waits for that one too when it is freed.
    """
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError(f"stream on {stream.device}, operands on {device}")
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def tile_count():
    """Number of grouped-GEMM tile shapes ``tuning`` accepts."""
    return library().rd_tune_tile_count()


@contextlib.contextmanager
def tuning(fwd_tile=None, trans_tile=None, decode=None):
    """Force tile shapes (0 .. tile_count() - 1) or turn the decode split path off (decode=False) for
    the calls made inside the block, for tile sweeps; the built-in choices come back on exit.
    Process-wide (rd_tune_set), so not for concurrent use from several threads."""
    lib = library()
    sets = [(RD_TUNE_FWD_TILE, fwd_tile), (RD_TUNE_TRANS_TILE, trans_tile),
            (RD_TUNE_DECODE, None if decode is None else int(bool(decode)))]
    try:
        for key, val in sets:
            if val is not None:
                _check(lib.rd_tune_set(key, int(val)))
        yield
    finally:
        lib.rd_tune_set(RD_TUNE_FWD_TILE, -1)
        lib.rd_tune_set(RD_TUNE_TRANS_TILE, -1)
        lib.rd_tune_set(RD_TUNE_DECODE, 1)


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on the GPU")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _scalar(t, name):
    if t is None:
        return None
    _need(t, name, torch.int32)
    if t.numel() != 1:
        raise ValueError(f"{name} must hold exactly one int32")
    return t


def ragged_dot(x, w, group_sizes, group_offset=None, limit=None, trans_rhs=False,
               out_dtype=torch.bfloat16, out=None, workspace=None, stream=None):
    """out[rows of local group j] = x[rows] @ w[j] (or @ w[j].T with trans_rhs).

    x: [m, k] bf16; w: [num_local, k, n] bf16 ([num_local, n, k] with trans_rhs);
    group_sizes: [G] int32 on the GPU; group_offset, limit: optional (1,) int32
    GPU tensors.  Rows below the limit outside the local window are +0; rows
    at or past the limit are left as they were in ``out`` (uninitialised when
    ``out`` is not given).  ``workspace``: optional uint8 GPU scratch; when the
    sizes call for one (decode shapes) and none of sufficient size is given,
    one is allocated.
    """
    _need(x, "x", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, 3)
    _need(group_sizes, "group_sizes", torch.int32, 1)
    group_offset = _scalar(group_offset, "group_offset")
    limit = _scalar(limit, "limit")
    m, k = x.shape
    gl = w.shape[0]
    if trans_rhs:
        n, kw = w.shape[1], w.shape[2]
    else:
        kw, n = w.shape[1], w.shape[2]
    if kw != k:
        raise ValueError("contraction sizes of x and w differ")
    if out is None:
        out = _empty((m, n), out_dtype, x.device, stream)
    _need(out, "out", out.dtype, 2)
    if tuple(out.shape) != (m, n) or out.dtype not in _DTYPES:
        raise ValueError("out must be [m, n] bf16 or float32")
    lib = library()
    ws_bytes = lib.rd_forward_workspace_size(m, k, n, gl, 1 if trans_rhs else 0)
    if ws_bytes and (workspace is None or workspace.numel() * workspace.element_size() < ws_bytes):
        workspace = _empty(ws_bytes, torch.uint8, x.device, stream)
    fn = lib.rd_forward_trans_rhs if trans_rhs else lib.rd_forward
    _launch(fn, (x, w, group_sizes, group_offset, limit, out, workspace if ws_bytes else None), stream,
            _ptr(x), _ptr(w), _ptr(group_sizes), group_sizes.numel(), _ptr(group_offset), gl, _ptr(limit), _ptr(out),
            _DTYPES[out.dtype], m, k, n, _ptr(workspace) if ws_bytes else None, ws_bytes)
    return out


def ragged_dot_noalloc(x, w, group_sizes, group_offset=None, limit=None, out=None, stream=None):
    """ragged_dot (plain form) through rd_forward_noalloc: the library allocates nothing (the decode
    path's partial sums live in its static per-GPU scratch); ``out`` ([m, n] bf16 or float32) should be
    given by callers that cannot allocate.  Calls overlapping on one GPU race on that scratch."""
    _need(x, "x", torch.bfloat16, 2)
    _need(w, "w", torch.bfloat16, 3)
    _need(group_sizes, "group_sizes", torch.int32, 1)
    group_offset = _scalar(group_offset, "group_offset")
    limit = _scalar(limit, "limit")
    m, k = x.shape
    gl, kw, n = w.shape
    if kw != k:
        raise ValueError("contraction sizes of x and w differ")
    if out is None:
        out = _empty((m, n), torch.bfloat16, x.device, stream)
    _need(out, "out", out.dtype, 2)
    if tuple(out.shape) != (m, n) or out.dtype not in _DTYPES:
        raise ValueError("out must be [m, n] bf16 or float32")
    _launch(library().rd_forward_noalloc, (x, w, group_sizes, group_offset, limit, out), stream,
            _ptr(x), _ptr(w), _ptr(group_sizes), group_sizes.numel(), _ptr(group_offset), gl, _ptr(limit), _ptr(out),
            _DTYPES[out.dtype], m, k, n)
    return out


def ragged_dot_fp8(x, w, group_sizes, group_offset=None, limit=None, trans_rhs=False, out_dtype=torch.bfloat16,
                   out=None, stream=None):
    """fp8 (E4M3) ragged_dot: out[rows of local group j] = x[rows] @ w[j] (trans_rhs: @ w[j].T).

    x: [m, k] torch.float8_e4m3fn; w: [num_local, k, n] (trans_rhs: [num_local, n, k]) float8_e4m3fn;
    float32 accumulation, one rounding to out_dtype.
    """
    _need(x, "x", torch.float8_e4m3fn, 2)
    _need(w, "w", torch.float8_e4m3fn, 3)
    _need(group_sizes, "group_sizes", torch.int32, 1)
    group_offset = _scalar(group_offset, "group_offset")
    limit = _scalar(limit, "limit")
    m, k = x.shape
    if trans_rhs:
        gl, n, kw = w.shape
    else:
        gl, kw, n = w.shape
    if kw != k:
        raise ValueError("contraction sizes of x and w differ")
    if out is None:
        out = _empty((m, n), out_dtype, x.device, stream)
    _need(out, "out", out.dtype, 2)
    if tuple(out.shape) != (m, n) or out.dtype not in _DTYPES:
        raise ValueError("out must be [m, n] bf16 or float32")
    fn = library().rd_forward_trans_rhs_fp8 if trans_rhs else library().rd_forward_fp8
    _launch(fn, (x, w, group_sizes, group_offset, limit, out), stream,
            _ptr(x), _ptr(w), _ptr(group_sizes), group_sizes.numel(), _ptr(group_offset), gl, _ptr(limit), _ptr(out),
            _DTYPES[out.dtype], m, k, n)
    return out


def trans_ragged_dot_fp8(x, dy, group_sizes, num_local=None, group_offset=None, limit=None,
                         out_dtype=torch.float32, out=None, workspace=None, row_split=True, stream=None):
    """fp8 (E4M3) trans_ragged_dot: dw[j] = x_j^T @ dy_j, float32 accumulation, one rounding to out_dtype.

    x: [m, k] and dy: [m, n] torch.float8_e4m3fn; returns [num_local, k, n].  ``workspace`` and
    ``row_split`` as for trans_ragged_dot (the same row split of long groups).
    """
    _need(x, "x", torch.float8_e4m3fn, 2)
    _need(dy, "dy", torch.float8_e4m3fn, 2)
    _need(group_sizes, "group_sizes", torch.int32, 1)
    group_offset = _scalar(group_offset, "group_offset")
    limit = _scalar(limit, "limit")
    m, k = x.shape
    if dy.shape[0] != m:
        raise ValueError("x and dy row counts differ")
    n = dy.shape[1]
    gl = group_sizes.numel() if num_local is None else int(num_local)
    if out is None:
        out = _empty((gl, k, n), out_dtype, x.device, stream)
    _need(out, "out", out.dtype, 3)
    if tuple(out.shape) != (gl, k, n) or out.dtype not in _DTYPES:
        raise ValueError("out must be [num_local, k, n] bf16 or float32")
    lib = library()
    ws_bytes = 0
    if row_split and workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
        ws_bytes = workspace.numel()
    elif row_split:
        ws_bytes = lib.rd_trans_workspace_size(m, k, n, gl)
        if ws_bytes:
            workspace = _empty(ws_bytes, torch.uint8, x.device, stream)
    _launch(lib.rd_trans_fp8, (x, dy, group_sizes, group_offset, limit, out, workspace if ws_bytes else None), stream,
            _ptr(x), _ptr(dy), _ptr(group_sizes), group_sizes.numel(), _ptr(group_offset), gl, _ptr(limit),
            _ptr(out), _DTYPES[out.dtype], m, k, n, _ptr(workspace) if ws_bytes else None, ws_bytes)
    return out


def glu_epilogue_supported(m, k, h):
    """Whether ragged_dot_glu takes these sizes: k % 64 == 0, h % 128 == 0, every operand under 4 GiB."""
    return k % 64 == 0 and h % 128 == 0 and h > 0 and m * k * 2 < 1 << 32 and k * 2 * h * 2 < 1 << 32


def ragged_dot_glu(x, wi, group_sizes, group_offset=None, limit=None, act=None, fused=None, want_fused=False,
                   stream=None):
    """The up-projection with the GLU as its epilogue: act = glu_fwd(ragged_dot(x, wi)), bit for bit.

    x: [m, k] bf16; wi: [num_local, k, 2h] bf16 ([gate | up] columns).  Returns act [m, h] bf16, or
    (act, fused) with the [gate | up] buffer fused [m, 2h] when want_fused (or a fused tensor) is given.
    Requires k % 64 == 0 and h % 128 == 0.
    """
    _need(x, "x", torch.bfloat16, 2)
    _need(wi, "wi", torch.bfloat16, 3)
    _need(group_sizes, "group_sizes", torch.int32, 1)
    group_offset = _scalar(group_offset, "group_offset")
    limit = _scalar(limit, "limit")
    m, k = x.shape
    gl, kw, h2 = wi.shape
    if kw != k or h2 % 2:
        raise ValueError("wi must be [num_local, k, 2h] with x's k")
    h = h2 // 2
    if act is None:
        act = _empty((m, h), torch.bfloat16, x.device, stream)
    _need(act, "act", torch.bfloat16, 2)
    if tuple(act.shape) != (m, h):
        raise ValueError("act must be [m, h]")
    if fused is None and want_fused:
        fused = _empty((m, h2), torch.bfloat16, x.device, stream)
    if fused is not None:
        _need(fused, "fused", torch.bfloat16, 2)
        if tuple(fused.shape) != (m, h2):
            raise ValueError("fused must be [m, 2h]")
    _launch(library().rd_forward_glu, (x, wi, group_sizes, group_offset, limit, act, fused), stream,
            _ptr(x), _ptr(wi), _ptr(group_sizes), group_sizes.numel(), _ptr(group_offset), gl, _ptr(limit),
            _ptr(act), _ptr(fused), m, k, h)
    return act if fused is None else (act, fused)


def trans_ragged_dot(x, dy, group_sizes, num_local=None, group_offset=None, limit=None,
                     out_dtype=torch.float32, out=None, workspace=None, row_split=True, stream=None):
    """dw[j] = x_j^T @ dy_j over the rows of local group j; [num_local, k, n].

    ``workspace``: optional uint8 GPU scratch for the row split of long groups, used as given (a
    smaller one than ``rd_trans_workspace_size`` splits fewer groups); without it one of that size is
    allocated.  ``row_split=False`` passes no workspace (no group is split).
    """
    _need(x, "x", torch.bfloat16, 2)
    _need(dy, "dy", torch.bfloat16, 2)
    _need(group_sizes, "group_sizes", torch.int32, 1)
    group_offset = _scalar(group_offset, "group_offset")
    limit = _scalar(limit, "limit")
    m, k = x.shape
    if dy.shape[0] != m:
        raise ValueError("x and dy must have the same rows")
    n = dy.shape[1]
    gl = group_sizes.numel() if num_local is None else int(num_local)
    if out is None:
        out = _empty((gl, k, n), out_dtype, x.device, stream)
    _need(out, "out", out.dtype, 3)
    if tuple(out.shape) != (gl, k, n) or out.dtype not in _DTYPES:
        raise ValueError("out must be [num_local, k, n] bf16 or float32")
    lib = library()
    ws_bytes = 0
    if row_split and workspace is not None:
        _need(workspace, "workspace", torch.uint8, 1)
        ws_bytes = workspace.numel()
    elif row_split:
        ws_bytes = lib.rd_trans_workspace_size(m, k, n, gl)
        if ws_bytes:
            workspace = _empty(ws_bytes, torch.uint8, x.device, stream)
    _launch(lib.rd_trans, (x, dy, group_sizes, group_offset, limit, out, workspace if ws_bytes else None), stream,
            _ptr(x), _ptr(dy), _ptr(group_sizes), group_sizes.numel(), _ptr(group_offset), gl, _ptr(limit),
            _ptr(out), _DTYPES[out.dtype], m, k, n, _ptr(workspace) if ws_bytes else None, ws_bytes)
    return out


def trans_workspace_size(m, k, n, num_local):
    """Bytes of workspace that let trans_ragged_dot split every group that qualifies (0: none can)."""
    return int(library().rd_trans_workspace_size(m, k, n, num_local))


def glu_fwd(fused, limit=None, out=None, stream=None):
    """out[r, c] = bf16(silu(gate) * up) for rows r < limit; fused is [rows, 2h] as [gate | up]."""
    _need(fused, "fused", torch.bfloat16, 2)
    limit = _scalar(limit, "limit")
    rows, two_h = fused.shape
    if two_h % 2:
        raise ValueError("fused width must be even")
    h = two_h // 2
    if out is None:
        out = _empty((rows, h), torch.bfloat16, fused.device, stream)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (rows, h):
        raise ValueError("out must be [rows, h]")
    _launch(library().rd_glu_fwd, (fused, limit, out), stream,
            _ptr(fused), _ptr(limit), _ptr(out), rows, h)
    return out


def glu_bwd(fused, d_out, limit=None, out=None, stream=None):
    """[d_gate | d_up] for rows r < limit, -0 written as +0; returns [rows, 2h] bf16."""
    _need(fused, "fused", torch.bfloat16, 2)
    _need(d_out, "d_out", torch.bfloat16, 2)
    limit = _scalar(limit, "limit")
    rows, two_h = fused.shape
    h = two_h // 2
    if tuple(d_out.shape) != (rows, h):
        raise ValueError("d_out must be [rows, h]")
    if out is None:
        out = _empty((rows, two_h), torch.bfloat16, fused.device, stream)
    _need(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (rows, two_h):
        raise ValueError("out must be [rows, 2h]")
    _launch(library().rd_glu_bwd, (fused, d_out, limit, out), stream,
            _ptr(fused), _ptr(d_out), _ptr(limit), _ptr(out), rows, h)
    return out


def unsort_bwd_rows(g, y, w, limit=None, grad=None, dot=None, stream=None):
    """(grad, dot) over rows r < limit: grad = bf16(f32(g) * w[r]), dot[r] = sum_c g[r, c] * y[r, c] (float32).

    g, y: [rows, hidden] bf16 in the packed buffer's row order; w: [rows] float32 routing weights.
    Rows at or past the limit are left as they were in ``grad`` and ``dot`` (uninitialised when not given).
    """
    _need(g, "g", torch.bfloat16, 2)
    _need(y, "y", torch.bfloat16, 2)
    _need(w, "w", torch.float32, 1)
    limit = _scalar(limit, "limit")
    rows, hidden = g.shape
    if tuple(y.shape) != (rows, hidden) or w.shape[0] != rows:
        raise ValueError("g and y must be [rows, hidden] and w [rows]")
    if grad is None:
        grad = _empty((rows, hidden), torch.bfloat16, g.device, stream)
    if dot is None:
        dot = _empty((rows,), torch.float32, g.device, stream)
    _need(grad, "grad", torch.bfloat16, 2)
    _need(dot, "dot", torch.float32, 1)
    if tuple(grad.shape) != (rows, hidden) or dot.shape[0] != rows:
        raise ValueError("grad must be [rows, hidden] and dot [rows]")
    _launch(library().rd_unsort_bwd_rows, (g, y, w, limit, grad, dot), stream,
            _ptr(g), _ptr(y), _ptr(w), _ptr(limit), _ptr(grad), _ptr(dot), rows, hidden)
    return grad, dot


def zero_rows_from_limit(buf, limit, stream=None):
    """Rows at or past ``limit`` (a (1,) int32 GPU tensor; None: nothing to do) of ``buf`` set to +0,
    in place; ``buf`` is a contiguous GPU tensor whose first dim is the rows.  Returns ``buf``."""
    if limit is None:
        return buf
    limit = _scalar(limit, "limit")
    if buf.device.type != "cuda" or not buf.is_contiguous() or buf.dim() < 1:
        raise ValueError("buf must be a contiguous GPU tensor")
    rows = buf.shape[0]
    row_bytes = buf[0].numel() * buf.element_size() if rows else 16
    _launch(library().rd_zero_rows_from_limit, (buf, limit), stream,
            _ptr(buf) if rows else None, _ptr(limit), rows, row_bytes)
    return buf


# ---------------------------------------------------------------- the routed expert layer


def _score(score):
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    return _SCORES[score]


def route(logits, top_k, bias=None, score="softmax", groups=1, top_groups=None, renormalize=False, scale=1.0,
          limit=None, weights=None, ids=None, stream=None):
    """(weights, ids) of the top_k experts of each token: [tokens, top_k] float32 and int32.

    logits: [tokens, experts] bf16 or float32; scores are their softmax or sigmoid.  ``bias`` ([experts]
    float32) is added to the scores for the choice only.  With ``groups`` > 1 only experts of the
    ``top_groups`` groups with the largest sums of their two best (biased) scores take part.  Ties go to the
    lower index; an expert whose logit is -inf is never chosen.  ``renormalize`` divides the weights by their
    sum; ``scale`` multiplies them.  Choices without an expert, and those of rows at or past ``limit``, have
    id -1 and weight 0.
    """
    return _native().route(logits, top_k, bias, _score(score), groups, groups if top_groups is None else top_groups,
                           bool(renormalize), scale, limit, weights, ids, stream)


def route_bwd(logits, ids, d_weights, score="softmax", renormalize=False, scale=1.0, out=None, stream=None):
    """Gradient of route's logits ([tokens, experts], their dtype) from that of its weights, for its choice ids."""
    return _native().route_bwd(logits, ids, d_weights, _score(score), bool(renormalize), scale, out, stream)


def group_rows_workspace_size(n, experts):
    """Bytes of workspace that group_rows needs for n slots."""
    return int(library().rd_group_rows_workspace_size(n, experts))


def group_rows(ids, experts, workspace=None, stream=None):
    """The stable sort of the slots (entries of ids, int32, any shape) by expert: (sizes, rows, slots, total).

    sizes [experts]: slots of each expert (the products' group_sizes); rows [n]: the slots in sorted order, those
    whose id is outside [0, experts) last; slots (ids' shape): each slot's row, -1 for those; total (1,): the rows
    that belong to an expert (a limit for the calls on the sorted buffer).  All int32.
    """
    return _native().group_rows(ids, experts, workspace, stream)


def dispatch_rows(x, slots, out=None, stream=None):
    """out[slots[t, i]] = x[t]: token rows ([tokens, hidden] bf16) to the rows of the expert-sorted buffer.

    Entries of slots outside out's rows are skipped; rows of out that no slot names are left as they were
    (uninitialised when ``out`` is not given: it then has tokens * top_k rows).
    """
    return _native().dispatch_rows(x, slots, out, stream)


def combine_rows(y, slots, weights=None, out=None, stream=None):
    """out[t] = sum_i weights[t, i] * y[slots[t, i]] (weights None: a plain sum), float32 sums, one rounding to bf16.

    y: [rows, hidden] bf16; slots, weights: [tokens, top_k] int32, float32.  Entries of slots outside y's rows
    add nothing.
    """
    return _native().combine_rows(y, slots, weights, out, stream)


def combine_rows_bwd(g, y, slots, weights, dy=None, dw=None, stream=None):
    """(dy, dw) of combine_rows from its output's gradient g [tokens, hidden]: dy[slots[t, i]] = weights[t, i] * g[t],
    dw[t, i] = <g[t], y[slots[t, i]]> (0 for an entry outside y's rows).

    Rows of dy that no slot names are left as they were (uninitialised when ``dy`` is not given).
    """
    return _native().combine_rows_bwd(g, y, slots, weights, dy, dw, stream)


def _out_bytes(dtype):
    """Bytes of an element of an output type."""
    if dtype not in _DTYPES:
        raise TypeError(f"out_dtype must be bfloat16 or float32, got {dtype}")
    return dtype.itemsize


def quantize_mx(x, bits=4, limit=None, codes=None, scales=None, stream=None):
    """(codes, scales): rows in MX 4-bit (E2M1) or 8-bit (E4M3) elements, 32 to a power-of-two scale.

    x: [..., cols] bf16 or float32, cols a multiple of 32.  codes: uint8 [..., cols / 2], the even element in
    the low half of its byte (bits 4), or float8_e4m3fn [..., cols] (bits 8); scales: uint8 [..., cols / 32],
    biased by 127, 255 for a block with an infinity or NaN.  ``limit`` counts rows of x seen as [rows, cols];
    rows at or past it are left as they were in the outputs (uninitialised when not given).
    """
    return _native().quantize_mx(x, bits, limit, codes, scales, stream)


def dequantize_mx(codes, scales, limit=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """The values that quantize_mx's codes and scales stand for, rounded once to out's dtype."""
    return _native().dequantize_mx(codes, scales, limit, _out_bytes(out_dtype), out, stream)


def ragged_dot_mx(x_codes, x_scales, w_codes, w_scales, group_sizes, group_offset=None, limit=None,
                  out_dtype=torch.bfloat16, out=None, stream=None):
    """ragged_dot (trans_rhs) on MX operands: out[rows of local group j] = x[rows] @ w[j].T on the codes' values.

    x_codes: [m, k / 2] uint8 (4 bits) or [m, k] float8_e4m3fn (8 bits), x_scales: [m, k / 32] uint8;
    w_codes: [num_local, n, k / 2] uint8, w_scales: [num_local, n, k / 32] uint8 (quantize_mx of a
    [num_local, n, k] weight); k a multiple of 128.  Float32 sums, one rounding to out_dtype; window and limit
    as ragged_dot.
    """
    return _native().ragged_dot_mx(x_codes, x_scales, w_codes, w_scales, group_sizes, group_offset, limit,
                                   _out_bytes(out_dtype), out, stream)


def glu_fwd_mx8(fused, limit=None, act=None, codes=None, scales=None, stream=None):
    """(act, codes, scales): glu_fwd of fused [rows, 2h] bf16, and fused itself in MX 8-bit elements (codes
    [rows, 2h] float8_e4m3fn, scales [rows, 2h / 32] uint8) as the residual of glu_bwd_mx8.  h % 32 == 0."""
    return _native().glu_fwd_mx8(fused, limit, act, codes, scales, stream)


def glu_bwd_mx8(codes, scales, d_act, limit=None, weights=None, rows=None, d_fused=None, act=None, dot=None,
                stream=None):
    """(d_fused, act, dot) from glu_fwd_mx8's residual and d_act, the gradient of the unweighted activation.

    Row r has slot s = rows[r] (group_rows' rows; r where it is None) and weight w = weights[s] (1 where weights
    is None): act[r] = w * silu(g) * u, d_fused[r] = w * d_act[r] times the GLU's derivatives,
    dot[s] = <d_act[r], silu(g) * u>.  weights: [slots] float32; dot: [slots] float32 (slots = number of weights,
    or of rows without them).  Rows at or past the limit, and the dots of their slots, are left as they were.
    """
    return _native().glu_bwd_mx8(codes, scales, d_act, limit, weights, rows, d_fused, act, dot, stream)
