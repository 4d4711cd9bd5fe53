"""Python binding of libaxonn_fc.so -- argument marshalling only.

Every function named ``axonn_*`` here calls the C entry point of the same
name (declared in include/axonn_fc.h); all arithmetic runs in the library's
CUDA kernels.  PyTorch supplies device memory and the current stream.  There
is no fallback: if the library is missing or cannot load, calls raise.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

from . import build as _build

OP_FWD, OP_DGRAD, OP_WGRAD = 0, 1, 2
OPS = {"fwd": OP_FWD, "dgrad": OP_DGRAD, "wgrad": OP_WGRAD}

A_T = 0x1
B_T = 0x2
ACCUM_F32 = 0x4
VGRID = 0x8
FULL_OPERANDS = 0x10
OUT_F32 = 0x20
ZSHARDED = 0x40
REDUCE_ADD = 0x80
VGRID_PARTIALS = 0x100
BIAS_F32 = 0x200
IN_F32 = 0x400
LSE_PARTS = 0x800

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

OK, ERR_INVALID_ARG, ERR_ALIGNMENT, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(7)
STATUS_NAMES = ["OK", "INVALID_ARG", "ALIGNMENT", "UNSUPPORTED", "WORKSPACE", "CUDA", "TIMEOUT"]

EXPORTS = ("axonn_fc_fwd", "axonn_fc_dgrad", "axonn_fc_wgrad", "axonn_fc_vgrid_static",
           "axonn_shards_gather", "axonn_fc_wgrad_zsharded", "axonn_goldfish_ce",
           "axonn_fc_fwd_epi", "axonn_fc_dgrad_epi", "axonn_epi_bwd", "axonn_epi_workspace_size",
           "axonn_dropout", "axonn_linear_ce", "axonn_linear_ce_workspace_size",
           "axonn_token_logprobs", "axonn_token_logprobs_bwd", "axonn_distill",
           "axonn_fc_workspace_size", "axonn_fc_tune", "axonn_tune_cache_save",
           "axonn_tune_cache_load", "axonn_tune_cache_clear", "axonn_tune_cache_size",
           "axonn_tune_lookup",
           "axonn_last_choice",
           "axonn_block_range", "axonn_fc_block_extents", "axonn_sync_status", "axonn_set_wait_timeout_ns",
           "axonn_debug_set_inject", "axonn_set_kernel_config", "axonn_num_kernel_configs",
           "axonn_set_streamk", "axonn_last_streamk_tiles", "axonn_set_swap", "axonn_last_swap",
           "axonn_set_pdl", "axonn_set_l2_budget", "axonn_l2_budget",
           "axonn_device_info",
           "axonn_kernel_config_name", "axonn_last_kernel_config", "axonn_last_error",
           "axonn_version")


class AxonnError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        name = STATUS_NAMES[status] if 0 <= status < len(STATUS_NAMES) else str(status)
        super().__init__(f"AXONN_ERR_{name}: {message}")


class Shape(ctypes.Structure):
    """axonn_fc_shape_t: layer sizes, 3D grid and block coordinate."""
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int64), ("N", ctypes.c_int64),
                ("gx", ctypes.c_int32), ("gy", ctypes.c_int32), ("gz", ctypes.c_int32),
                ("x", ctypes.c_int32), ("y", ctypes.c_int32), ("z", ctypes.c_int32)]

    def __init__(self, T, K, N, grid=(1, 1, 1), coords=(0, 0, 0)):
        super().__init__(T, K, N, *grid, *coords)


class Epilogue(ctypes.Structure):
    """axonn_epilogue_t: bias, activation, dropout and residual of a layer."""
    _fields_ = [("bias", ctypes.c_void_p), ("pre", ctypes.c_void_p), ("ld_pre", ctypes.c_int64),
                ("residual", ctypes.c_void_p), ("ld_residual", ctypes.c_int64),
                ("dbias", ctypes.c_void_p), ("rng", ctypes.c_void_p), ("act", ctypes.c_int32),
                ("p", ctypes.c_float)]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(path: str | None = None):
    """Load the built library (raises if it is absent)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or _build.LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"libaxonn_fc.so not built at {p}; run pmm_fc_layer_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i64, u32, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int32
        sz = ctypes.c_size_t
        sig = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(Shape), u32, vp, sz, vp]
        for name in ("axonn_fc_fwd", "axonn_fc_dgrad", "axonn_fc_wgrad"):
            f = getattr(lib, name)
            f.argtypes = sig
            f.restype = ctypes.c_int
        lib.axonn_shards_gather.argtypes = [ctypes.POINTER(vp), i32, i64, i64, i64, vp, i64, vp]
        lib.axonn_shards_gather.restype = ctypes.c_int
        lib.axonn_fc_wgrad_zsharded.argtypes = [vp, vp, ctypes.POINTER(vp), i64, i64, i64,
                                                ctypes.POINTER(Shape), u32, vp, sz, vp]
        lib.axonn_fc_wgrad_zsharded.restype = ctypes.c_int
        lib.axonn_goldfish_ce.argtypes = [vp, i64, vp, vp, i64, i64, i64, i32, i32, vp, vp, vp, vp,
                                          vp, i64, vp]
        lib.axonn_goldfish_ce.restype = ctypes.c_int
        epi = ctypes.POINTER(Epilogue)
        lib.axonn_fc_fwd_epi.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(Shape), u32, epi, vp]
        lib.axonn_fc_fwd_epi.restype = ctypes.c_int
        lib.axonn_fc_dgrad_epi.argtypes = [vp, vp, vp, i64, i64, i64, ctypes.POINTER(Shape), u32, epi,
                                           vp, sz, vp]
        lib.axonn_fc_dgrad_epi.restype = ctypes.c_int
        lib.axonn_epi_bwd.argtypes = [vp, i64, vp, i64, i64, i64, u32, epi, vp, sz, vp]
        lib.axonn_epi_bwd.restype = ctypes.c_int
        lib.axonn_epi_workspace_size.argtypes = [i64, i64, ctypes.POINTER(sz)]
        lib.axonn_epi_workspace_size.restype = ctypes.c_int
        lib.axonn_dropout.argtypes = [vp, i64, vp, i64, vp, i64, i64, i64, ctypes.c_float, vp, u32, vp]
        lib.axonn_dropout.restype = ctypes.c_int
        lib.axonn_linear_ce.argtypes = [vp, i64, vp, i64, vp, vp, i64, i64, i64, ctypes.c_float, u32,
                                        vp, vp, vp, vp, vp, i64, vp, i64, vp, sz, vp]
        lib.axonn_linear_ce.restype = ctypes.c_int
        lib.axonn_linear_ce_workspace_size.argtypes = [i64, i64, i64, u32, i32, i64, ctypes.POINTER(sz)]
        lib.axonn_linear_ce_workspace_size.restype = ctypes.c_int
        lib.axonn_fc_vgrid_static.argtypes = [ctypes.c_int, vp, vp, vp, i64, i64, i64,
                                              ctypes.POINTER(Shape), u32, vp]
        lib.axonn_fc_vgrid_static.restype = ctypes.c_int
        lib.axonn_fc_tune.argtypes = [ctypes.c_int, vp, vp, vp, i64, i64, i64, ctypes.POINTER(Shape),
                                      u32, vp, sz, vp, ctypes.POINTER(ctypes.c_int),
                                      ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                      ctypes.POINTER(ctypes.c_float)]
        lib.axonn_fc_tune.restype = ctypes.c_int
        lib.axonn_tune_cache_save.argtypes = [ctypes.c_char_p]
        lib.axonn_tune_cache_save.restype = ctypes.c_int
        lib.axonn_tune_cache_load.argtypes = [ctypes.c_char_p]
        lib.axonn_tune_cache_load.restype = ctypes.c_int
        lib.axonn_tune_cache_clear.restype = None
        lib.axonn_tune_cache_size.restype = ctypes.c_int
        lib.axonn_tune_lookup.argtypes = [ctypes.c_int, ctypes.POINTER(Shape), u32,
                                          ctypes.POINTER(ctypes.c_int)]
        lib.axonn_tune_lookup.restype = ctypes.c_int
        lib.axonn_last_choice.argtypes = [ctypes.POINTER(ctypes.c_int)] * 3
        lib.axonn_last_choice.restype = None
        for name in ("axonn_token_logprobs", "axonn_token_logprobs_bwd", "axonn_distill"):
            f = getattr(lib, name)
            f.argtypes = [ctypes.c_char_p, vp]  # the packed argument struct
            f.restype = ctypes.c_int
        lib.axonn_fc_workspace_size.argtypes = [ctypes.c_int, ctypes.POINTER(Shape), u32,
                                                ctypes.POINTER(sz)]
        lib.axonn_fc_workspace_size.restype = ctypes.c_int
        lib.axonn_block_range.argtypes = [i64, i32, i32, ctypes.POINTER(i64), ctypes.POINTER(i64)]
        lib.axonn_block_range.restype = ctypes.c_int
        lib.axonn_fc_block_extents.argtypes = [ctypes.c_int, ctypes.POINTER(Shape),
                                               ctypes.POINTER(i64), ctypes.POINTER(i64),
                                               ctypes.POINTER(i64)]
        lib.axonn_fc_block_extents.restype = ctypes.c_int
        lib.axonn_sync_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint64)]
        lib.axonn_sync_status.restype = ctypes.c_int
        lib.axonn_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
        lib.axonn_set_wait_timeout_ns.restype = None
        lib.axonn_debug_set_inject.argtypes = [ctypes.c_int]
        lib.axonn_debug_set_inject.restype = None
        lib.axonn_set_kernel_config.argtypes = [ctypes.c_int]
        lib.axonn_set_kernel_config.restype = ctypes.c_int
        lib.axonn_set_streamk.argtypes = [ctypes.c_int]
        lib.axonn_set_streamk.restype = ctypes.c_int
        lib.axonn_last_streamk_tiles.argtypes = []
        lib.axonn_last_streamk_tiles.restype = ctypes.c_int
        lib.axonn_set_pdl.argtypes = [ctypes.c_int]
        lib.axonn_set_pdl.restype = ctypes.c_int
        lib.axonn_set_l2_budget.argtypes = [ctypes.c_int64]
        lib.axonn_set_l2_budget.restype = ctypes.c_int
        lib.axonn_l2_budget.argtypes = []
        lib.axonn_l2_budget.restype = ctypes.c_int64
        lib.axonn_set_swap.argtypes = [ctypes.c_int]
        lib.axonn_set_swap.restype = ctypes.c_int
        lib.axonn_last_swap.argtypes = []
        lib.axonn_last_swap.restype = ctypes.c_int
        lib.axonn_num_kernel_configs.restype = ctypes.c_int
        lib.axonn_device_info.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
        lib.axonn_device_info.restype = ctypes.c_int
        lib.axonn_kernel_config_name.argtypes = [ctypes.c_int]
        lib.axonn_kernel_config_name.restype = ctypes.c_char_p
        lib.axonn_last_kernel_config.restype = ctypes.c_int
        lib.axonn_last_error.restype = ctypes.c_char_p
        lib.axonn_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(status: int):
    if status != OK:
        raise AxonnError(status, load().axonn_last_error().decode())


def _ptr(t) -> int:
    if t is None:
        return 0
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _ld(t, ld):
    if ld is not None:
        return int(ld)
    if t is None or isinstance(t, int):
        return 0
    if t.dim() != 2 or (t.stride(1) != 1 and t.size(1) > 1):
        raise ValueError("operands must be 2-D with unit column stride")
    return t.stride(0)


_raw_stream = None


def _current_stream() -> int:
    """The current stream's handle, without building a Stream object for each
    call (a third of a small call's host time) where torch offers that."""
    global _raw_stream
    if _raw_stream is None:
        import torch
        torch.cuda.init()
        get, device = (getattr(torch._C, n, None) for n in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
        if get is not None and device is not None:
            _raw_stream = lambda: get(device())  # noqa: E731
        else:
            _raw_stream = lambda: torch.cuda.current_stream().cuda_stream  # noqa: E731
    return _raw_stream()


_device = None


def _current_device() -> int:
    global _device
    if _device is None:
        import torch
        torch.cuda.init()
        _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return _device()


def _stream(stream) -> int:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, P, Q, C, shape, flags, ws, ldp, ldq, ldc, stream):
    lib = load()
    ws_bytes = 0
    if ws is not None and not isinstance(ws, int):
        ws_bytes = ws.numel() * ws.element_size()
    elif isinstance(ws, int):
        raise ValueError("pass the workspace as a tensor")
    st = getattr(lib, name)(_ptr(P), _ptr(Q), _ptr(C), _ld(P, ldp), _ld(Q, ldq), _ld(C, ldc),
                            ctypes.byref(shape), flags, _ptr(ws), ws_bytes, _stream(stream))
    _check(st)


def axonn_fc_fwd(X, W, Y, shape: Shape, flags: int = 0, ws=None, ldx=None, ldw=None, ldy=None,
                 stream=None):
    """Y = X . W (layer, block or virtual grid); see include/axonn_fc.h."""
    _call("axonn_fc_fwd", X, W, Y, shape, flags, ws, ldx, ldw, ldy, stream)


def axonn_fc_dgrad(dY, W, dX, shape: Shape, flags: int = 0, ws=None, lddy=None, ldw=None,
                   lddx=None, stream=None):
    """dX = dY . W^T (layer, block or virtual grid)."""
    _call("axonn_fc_dgrad", dY, W, dX, shape, flags, ws, lddy, ldw, lddx, stream)


def axonn_fc_wgrad(X, dY, dW, shape: Shape, flags: int = 0, ws=None, ldx=None, lddy=None,
                   lddw=None, stream=None):
    """dW = X^T . dY (layer, block or virtual grid)."""
    _call("axonn_fc_wgrad", X, dY, dW, shape, flags, ws, ldx, lddy, lddw, stream)


def _ptr_array(ts):
    arr = (ctypes.c_void_p * len(ts))()
    for i, t in enumerate(ts):
        arr[i] = _ptr(t)
    return arr


def axonn_shards_gather(shards, out, rows: int, cols: int, ld_shard=None, ld_out=None,
                        stream=None):
    """All-gather of row shards on one GPU: out[rows x cols] <- shards
    (shard z holds rows split_range(rows, len(shards), z))."""
    ld_s = ld_shard if ld_shard is not None else next(
        (_ld(t, None) for t in shards if t is not None and t.numel()), cols)
    _check(load().axonn_shards_gather(_ptr_array(shards), len(shards), rows, cols, ld_s, _ptr(out),
                                      _ld(out, ld_out), _stream(stream)))


def axonn_fc_wgrad_zsharded(X, dY, dW_shards, shape: Shape, flags: int = 0, ws=None, ldx=None,
                            lddy=None, ld_shard=None, stream=None):
    """Weight gradient of block (x, y) summed over the Z group and written as
    row shards (the grid's reduce-scatter) into dW_shards."""
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    ld_s = ld_shard if ld_shard is not None else next(
        (_ld(t, None) for t in dW_shards if t is not None and t.numel()), 8)
    _check(load().axonn_fc_wgrad_zsharded(_ptr(X), _ptr(dY), _ptr_array(dW_shards), _ld(X, ldx),
                                          _ld(dY, lddy), ld_s, ctypes.byref(shape), flags,
                                          _ptr(ws), ws_bytes, _stream(stream)))


def axonn_fc_vgrid_static(op, P, Q, C, shape: Shape, flags: int = 0, ldp=None, ldq=None,
                          ldc=None, stream=None):
    """Virtual-grid product with the library's fixed scratch: nothing is
    allocated and no workspace is passed (for callers that cannot allocate
    device memory).  ``op`` is 'fwd', 'dgrad' or 'wgrad'."""
    op = OPS.get(op, op)
    st = load().axonn_fc_vgrid_static(int(op), _ptr(P), _ptr(Q), _ptr(C), _ld(P, ldp), _ld(Q, ldq),
                                      _ld(C, ldc), ctypes.byref(shape), flags, _stream(stream))
    _check(st)


def axonn_goldfish_ce(logits, input_ids, labels, keep, token_loss, loss, kept, k=2, h=13,
                      dlogits=None, ld_logits=None, ld_dlogits=None, stream=None):
    """Goldfish-masked cross-entropy of bf16 logits [B*S x V] for int32
    input_ids / labels [B x S]: fills keep [B*S] (uint8), token_loss [B*S],
    loss [1], kept [1] (int32) and, if given, dlogits (bf16, the gradient of
    the mean loss)."""
    B, S = input_ids.shape
    V = logits.shape[1]
    _check(load().axonn_goldfish_ce(_ptr(logits), _ld(logits, ld_logits), _ptr(input_ids),
                                    _ptr(labels), B, S, V, int(k), int(h), _ptr(keep),
                                    _ptr(token_loss), _ptr(loss), _ptr(kept), _ptr(dlogits),
                                    _ld(dlogits, ld_dlogits) if dlogits is not None else 0,
                                    _stream(stream)))


def _host_memory(name, t):
    """A tensor that is not on the device: the kernels read and write through
    its pointer, so memory that they cannot reach is refused."""
    if not t.is_pinned():
        raise ValueError(f"{name} must be on the device, got {t.device}")


def _ws(ws):
    if ws is None:
        return None, 0
    if not ws.is_cuda:
        _host_memory("ws", ws)
    return ws.data_ptr(), ws.numel() * ws.element_size()


class _Dtypes(dict):
    """torch's dtype of a name (torch is imported at the first one asked for)."""

    def __missing__(self, name):
        import torch
        self.update(bf16=torch.bfloat16, f32=torch.float32, i32=torch.int32, u8=torch.uint8,
                    words=(torch.int64, torch.uint64))
        return self[name]


_dtypes = _Dtypes()


def _matrix(name, t, dtype, rows, cols):
    """(pointer, leading dimension) of a [rows x cols] matrix of that type, or
    (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype is not _dtypes[dtype]:
        raise ValueError(f"{name} must be {_dtypes[dtype]}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be {(rows, cols)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        _host_memory(name, t)
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld


def _vector(name, t, dtype, n):
    """Pointer of a contiguous vector of n elements of that type, or None."""
    if t is None:
        return None
    if t.dtype is not _dtypes[dtype]:
        raise ValueError(f"{name} must be {_dtypes[dtype]}, got {t.dtype}")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be contiguous of {n} elements")
    if not t.is_cuda:
        _host_memory(name, t)
    return t.data_ptr()


def _rng(rng):
    if rng is None:
        return None
    if rng.dtype not in _dtypes["words"] or rng.shape != (2,) or rng.stride(0) != 1:
        raise ValueError("rng must be two contiguous 64-bit integers on the device: seed and offset")
    if not rng.is_cuda:
        _host_memory("rng", rng)
    return rng.data_ptr()


def _act(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"activation {act!r} not in {sorted(ACTS)}")
    return code


def _layer(shape, flags, rows_name, A, rows, red, W):
    """(pointer, ld) of a product's operands: A [rows x red] (stored the other
    way round with A_T) and W [shape.K x shape.N] (with B_T likewise)."""
    a = _matrix(rows_name, A, "bf16", *((red, rows) if flags & A_T else (rows, red)))
    w = _matrix("W", W, "bf16", *((shape.N, shape.K) if flags & B_T else (shape.K, shape.N)))
    return a, w


def axonn_fc_fwd_epi(X, W, Y, shape: Shape, flags: int = 0, bias=None, act="none", pre=None,
                     residual=None, p=0.0, rng=None, stream=None):
    """Y = residual + D(act(X . W + bias)) of the whole layer; ``pre`` (bf16)
    receives X . W + bias where given.  bias is bf16, or fp32 (the tensor's
    type sets BIAS_F32); residual has Y's type.  D is dropout with probability
    p and ``rng``, two 64-bit words on the device (seed, offset)."""
    T, N = shape.T, shape.N
    if bias is not None and bias.dtype is _dtypes["f32"]:
        flags |= BIAS_F32
    out = "f32" if flags & OUT_F32 else "bf16"
    x, w = _layer(shape, flags, "X", X, T, shape.K, W)
    y = _matrix("Y", Y, out, T, N)
    e = Epilogue(_vector("bias", bias, "f32" if flags & BIAS_F32 else "bf16", N),
                 *_matrix("pre", pre, "bf16", T, N), *_matrix("residual", residual, out, T, N),
                 None, _rng(rng), _act(act), p)
    _check(load().axonn_fc_fwd_epi(x[0], w[0], y[0], x[1], w[1], y[1], ctypes.byref(shape), flags,
                                   ctypes.byref(e), _stream(stream)))


def axonn_fc_dgrad_epi(dY, W, dX, shape: Shape, flags: int = 0, pre=None, act="none", residual=None,
                       dbias=None, p=0.0, rng=None, ws=None, stream=None):
    """dX = act'(pre) D(dY . W^T) + residual, and dbias (fp32) = the column
    sums of act'(pre) D(dY . W^T): the data gradient of this layer as the
    gradient of the pre-activation before it.  dbias needs ``ws``
    (axonn_epi_workspace_size(T, K) bytes)."""
    T, K = shape.T, shape.K
    out = "f32" if flags & OUT_F32 else "bf16"
    g, w = _layer(shape, flags, "dY", dY, T, shape.N, W)
    y = _matrix("dX", dX, out, T, K)
    e = Epilogue(None, *_matrix("pre", pre, "bf16", T, K), *_matrix("residual", residual, out, T, K),
                 _vector("dbias", dbias, "f32", K), _rng(rng), _act(act), p)
    _check(load().axonn_fc_dgrad_epi(g[0], w[0], y[0], g[1], w[1], y[1], ctypes.byref(shape), flags,
                                     ctypes.byref(e), *_ws(ws), _stream(stream)))


def axonn_epi_bwd(dY, dZ, pre=None, act="none", dbias=None, p=0.0, rng=None, ws=None, stream=None):
    """dZ (bf16) = act'(pre) D(dY) and dbias (fp32) = its column sums, for
    dY [rows x cols] in bf16 or fp32 (the tensor's type sets IN_F32)."""
    rows, cols = dY.shape
    f32 = dY.dtype is _dtypes["f32"]
    e = Epilogue(None, *_matrix("pre", pre, "bf16", rows, cols), None, 0,
                 _vector("dbias", dbias, "f32", cols), _rng(rng), _act(act), p)
    _check(load().axonn_epi_bwd(*_matrix("dY", dY, "f32" if f32 else "bf16", rows, cols),
                                *_matrix("dZ", dZ, "bf16", rows, cols), rows, cols,
                                IN_F32 if f32 else 0, ctypes.byref(e), *_ws(ws), _stream(stream)))


def axonn_epi_workspace_size(rows: int, cols: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().axonn_epi_workspace_size(rows, cols, ctypes.byref(n)))
    return n.value


def axonn_dropout(X, Y, p, rng, residual=None, stream=None):
    """Y = residual + D(X), bf16 or fp32 (X's type); its backward is the same
    call on the gradient."""
    rows, cols = X.shape
    f32 = X.dtype is _dtypes["f32"]
    kind = "f32" if f32 else "bf16"
    _check(load().axonn_dropout(*_matrix("X", X, kind, rows, cols),
                                *_matrix("residual", residual, kind, rows, cols),
                                *_matrix("Y", Y, kind, rows, cols), rows, cols, p, _rng(rng),
                                IN_F32 if f32 else 0, _stream(stream)))


def axonn_linear_ce(X, W, labels, token_loss, loss, kept, ws, keep=None, lse=None, dX=None, dW=None,
                    grad_scale=1.0, flags: int = 0, stream=None):
    """Softmax cross-entropy of the logits X . W (W [K x V], or [V x K] with
    B_T) for int32 labels [T], and its gradients dX (bf16) and dW (bf16;
    fp32 with OUT_F32, added into with ACCUM_F32) where given; the logits are
    never written out.  ``ws``: axonn_linear_ce_workspace_size bytes, or less
    (smaller pieces of the vocabulary)."""
    T, K = X.shape
    V = W.shape[0 if flags & B_T else 1]
    wshape = (V, K) if flags & B_T else (K, V)
    _check(load().axonn_linear_ce(
        *_matrix("X", X, "bf16", T, K), *_matrix("W", W, "bf16", *wshape),
        _vector("labels", labels, "i32", T), _vector("keep", keep, "u8", T), T, K, V, grad_scale, flags,
        _vector("token_loss", token_loss, "f32", T), _vector("lse", lse, "f32", T),
        _vector("loss", loss, "f32", 1), _vector("kept", kept, "i32", 1), *_matrix("dX", dX, "bf16", T, K),
        *_matrix("dW", dW, "f32" if flags & (OUT_F32 | ACCUM_F32) else "bf16", *wshape),
        *_ws(ws), _stream(stream)))


def axonn_linear_ce_workspace_size(T: int, K: int, V: int, flags: int = 0, grad: bool = True,
                                   piece: int = 0) -> int:
    """Workspace bytes for pieces of ``piece`` vocabulary columns (0: pieces
    of at most 2 GiB)."""
    n = ctypes.c_size_t(0)
    _check(load().axonn_linear_ce_workspace_size(T, K, V, flags, int(grad), piece, ctypes.byref(n)))
    return n.value


# The argument structs of the operators over rows of logits, packed as C lays
# them out: one conversion for all of a call's arguments (ctypes takes a fifth
# of a microsecond for each).
_TOKEN_LOGPROBS = struct.Struct("@PqPPqqfIPPPPPqi4x")
_TOKEN_LOGPROBS_BWD = struct.Struct("@PqPPqqfIPPPPPq")
_DISTILL = struct.Struct("@PqPPqPqqfIPPPPqfi")


def _logits(logits):
    """(device, rows, columns, dtype, IN_F32 or 0) of logits, whose device must
    be the current one."""
    here = logits.get_device()
    if here < 0:
        raise ValueError(f"logits must be on the device, got {logits.device}")
    if here != _current_device():
        raise ValueError(f"logits are on device {here}, which is not the current one")
    rows, cols = logits.shape
    f32 = _dtypes["f32"]
    return (here, rows, cols, f32, IN_F32) if logits.dtype is f32 else (here, rows, cols, _dtypes["bf16"], 0)


def _refuse(name, t, dtype, shape, here):
    """Says what is wrong with a tensor beside logits on device `here`."""
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != here:
        raise ValueError(f"{name} must be on the logits' device {here}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _whole(name, t, dtype, shape, here):
    """Address of a contiguous tensor beside the logits, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != here or not t.is_contiguous():
        _refuse(name, t, dtype, shape, here)
    return t.data_ptr()


def _lse(t, T, here):
    """(address, LSE_PARTS or 0) of lse [T], or [T x 2] in parts."""
    if t is not None and len(t.shape) == 2:
        return _whole("lse", t, _dtypes["f32"], (T, 2), here), LSE_PARTS
    return _whole("lse", t, _dtypes["f32"], (T,), here), 0


def _rows(name, t, dtype, shape, here, single):
    """(address, leading dimension) of rows beside the logits, (0, 0) for None.
    The stride of a single row says nothing: it counts as `single`."""
    if t is None:
        return 0, 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != here:
        _refuse(name, t, dtype, shape, here)
    ld, inner = t.stride()
    if inner != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), ld if shape[0] > 1 else single


def _lists(index_name, index, value_name, value, T, here):
    """(k, address of the indices, of the values, leading dimension)."""
    k = (index if index is not None else value).shape[1]
    index, ld = _rows(index_name, index, _dtypes["i32"], (T, k), here, k)
    value, ld_value = _rows(value_name, value, _dtypes["f32"], (T, k), here, k)
    if index and value and ld != ld_value:
        raise ValueError(f"{index_name} and {value_name} must have the same row stride")
    return k, index, value, ld or ld_value


def axonn_token_logprobs(logits, tokens=None, logprob=None, entropy=None, lse=None, top_index=None,
                         top_logprob=None, keep=None, temperature=1.0, stream=None):
    """ln p of int32 tokens [T] under softmax(logits / temperature), logits
    [T x V] in bf16 or fp32 (the tensor's type sets IN_F32): fills, where given,
    logprob [T], entropy [T], lse [T] (or [T x 2]: the largest logit and
    lse - it / temperature), and the rows' largest logits, best first, as
    top_index (int32) and top_logprob [T x k].  Rows with keep (uint8 [T]) 0 get
    zeros and indices of -1."""
    here, T, V, kind, flags = _logits(logits)
    lse, parts = _lse(lse, T, here)
    f32, per_row, single = _dtypes["f32"], (T,), (V + 7) // 8 * 8
    k = index = value = ld_top = 0
    if top_index is not None or top_logprob is not None:
        k, index, value, ld_top = _lists("top_index", top_index, "top_logprob", top_logprob, T, here)
    _check(load().axonn_token_logprobs(_TOKEN_LOGPROBS.pack(
        *_rows("logits", logits, kind, (T, V), here, single), _whole("tokens", tokens, _dtypes["i32"], per_row, here),
        _whole("keep", keep, _dtypes["u8"], per_row, here), T, V, temperature, flags | parts,
        _whole("logprob", logprob, f32, per_row, here), _whole("entropy", entropy, f32, per_row, here),
        lse, index, value, ld_top, k), _stream(stream)))


def axonn_token_logprobs_bwd(logits, lse, dlogits, tokens=None, dlogprob=None, entropy=None, dentropy=None,
                             keep=None, temperature=1.0, stream=None):
    """dlogits (the logits' type; may be the logits) = (dlogprob (onehot(tokens)
    - p) - dentropy p (ln p + entropy)) / temperature, for lse and entropy as
    axonn_token_logprobs left them.  lse [T x 2] is right for logits of any size;
    from lse [T] rows beyond 65536 in size get NaN."""
    here, T, V, kind, flags = _logits(logits)
    lse, parts = _lse(lse, T, here)
    f32, per_row, single = _dtypes["f32"], (T,), (V + 7) // 8 * 8
    _check(load().axonn_token_logprobs_bwd(_TOKEN_LOGPROBS_BWD.pack(
        *_rows("logits", logits, kind, (T, V), here, single), _whole("tokens", tokens, _dtypes["i32"], per_row, here),
        _whole("keep", keep, _dtypes["u8"], per_row, here), T, V, temperature, flags | parts, lse,
        _whole("dlogprob", dlogprob, f32, per_row, here),
        _whole("entropy", entropy, f32, per_row, here), _whole("dentropy", dentropy, f32, per_row, here),
        *_rows("dlogits", dlogits, kind, (T, V), here, single)), _stream(stream)))


def axonn_distill(logits, top_index, top_logit, token_loss, loss, kept, dlogits=None, keep=None, temperature=1.0,
                  grad_scale=1.0, stream=None):
    """tau^2 KL of softmax(top_logit / tau) over a teacher's lists (int32
    top_index and fp32 top_logit [T x k], ended by an index outside the
    vocabulary) against softmax(logits / tau), tau the temperature: fills
    token_loss [T], loss [1], kept [1] (int32) and, if given, dlogits (the
    logits' type; may be the logits), the gradient of the mean loss times
    grad_scale."""
    here, T, V, kind, flags = _logits(logits)
    f32, i32, single = _dtypes["f32"], _dtypes["i32"], (V + 7) // 8 * 8
    k, index, value, ld_top = _lists("top_index", top_index, "top_logit", top_logit, T, here)
    _check(load().axonn_distill(_DISTILL.pack(
        *_rows("logits", logits, kind, (T, V), here, single), index, value, ld_top,
        _whole("keep", keep, _dtypes["u8"], (T,), here), T, V, temperature, flags,
        _whole("token_loss", token_loss, f32, (T,), here), _whole("loss", loss, f32, (1,), here),
        _whole("kept", kept, i32, (1,), here), *_rows("dlogits", dlogits, kind, (T, V), here, single), grad_scale, k),
        _stream(stream)))


def axonn_fc_tune(op, P, Q, C, shape: Shape, flags: int = 0, ws=None, ldp=None, ldq=None,
                  ldc=None, stream=None):
    """Time every candidate way to run this call and remember the fastest;
    returns (config, split, group_m, microseconds).  Overwrites C."""
    op = OPS.get(op, op)
    ws_bytes = ws.numel() * ws.element_size() if ws is not None else 0
    c, sp, gm, us = ctypes.c_int(), ctypes.c_int(), ctypes.c_int(), ctypes.c_float()
    _check(load().axonn_fc_tune(int(op), _ptr(P), _ptr(Q), _ptr(C), _ld(P, ldp), _ld(Q, ldq),
                                _ld(C, ldc), ctypes.byref(shape), flags, _ptr(ws), ws_bytes,
                                _stream(stream), ctypes.byref(c), ctypes.byref(sp),
                                ctypes.byref(gm), ctypes.byref(us)))
    return c.value, sp.value, gm.value, us.value


def axonn_tune_cache_save(path: str):
    _check(load().axonn_tune_cache_save(os.fsencode(path)))


def axonn_tune_cache_load(path: str):
    _check(load().axonn_tune_cache_load(os.fsencode(path)))


def axonn_tune_cache_clear():
    load().axonn_tune_cache_clear()


def axonn_tune_cache_size() -> int:
    return int(load().axonn_tune_cache_size())


def axonn_last_choice():
    """(config, split, group_m) of the last call on this thread."""
    c, s, g = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    load().axonn_last_choice(ctypes.byref(c), ctypes.byref(s), ctypes.byref(g))
    return c.value, s.value, g.value


def axonn_tune_lookup(op, shape: Shape, flags: int = 0) -> bool:
    """True when the tuning table holds an entry for this call on the
    current device."""
    op = OPS.get(op, op)
    found = ctypes.c_int(0)
    _check(load().axonn_tune_lookup(int(op), ctypes.byref(shape), flags, ctypes.byref(found)))
    return bool(found.value)


def axonn_fc_workspace_size(op, shape: Shape, flags: int = 0) -> int:
    op = OPS.get(op, op)
    n = ctypes.c_size_t(0)
    _check(load().axonn_fc_workspace_size(int(op), ctypes.byref(shape), flags, ctypes.byref(n)))
    return n.value


def axonn_block_range(D: int, G: int, b: int):
    s, e = ctypes.c_int64(0), ctypes.c_int64(0)
    _check(load().axonn_block_range(D, G, b, ctypes.byref(s), ctypes.byref(e)))
    return s.value, e.value


def axonn_fc_block_extents(op, shape: Shape):
    """((rows), (red), (cols)) of block (shape.x, shape.y, shape.z) of `op`,
    each a [start, stop) pair in the full matrices."""
    op = OPS.get(op, op)
    r, k, c = (ctypes.c_int64 * 2)(), (ctypes.c_int64 * 2)(), (ctypes.c_int64 * 2)()
    _check(load().axonn_fc_block_extents(int(op), ctypes.byref(shape), r, k, c))
    return (r[0], r[1]), (k[0], k[1]), (c[0], c[1])


def axonn_sync_status(stream=None, raise_on_error: bool = True):
    """Waits for the stream and returns (status, detail word)."""
    detail = ctypes.c_uint64(0)
    st = load().axonn_sync_status(_stream(stream), ctypes.byref(detail))
    if raise_on_error:
        _check(st)
    return st, detail.value


def axonn_set_wait_timeout_ns(ns: int):
    load().axonn_set_wait_timeout_ns(int(ns))


def axonn_debug_set_inject(mode: int):
    load().axonn_debug_set_inject(int(mode))


def axonn_set_kernel_config(config: int):
    """Force kernel configuration `config` (-1: automatic choice)."""
    _check(load().axonn_set_kernel_config(int(config)))


def axonn_set_streamk(mode: int):
    """Stream-K tail: -1 as tuned (default on), 0 off, 1 on."""
    _check(load().axonn_set_streamk(int(mode)))


def axonn_last_streamk_tiles() -> int:
    """Stream-K tiles of the last GEMM launch on this thread (0: none)."""
    return int(load().axonn_last_streamk_tiles())


def axonn_set_pdl(on: int):
    """1 (default): GEMMs are programmatic dependent launches; 0: plain launches."""
    _check(load().axonn_set_pdl(int(on)))


def axonn_set_l2_budget(nbytes: int):
    """L2 bytes a rasterisation group's kept operand panel may hold as
    evict-last lines (0: operand loads without L2 priorities)."""
    _check(load().axonn_set_l2_budget(int(nbytes)))


def axonn_l2_budget() -> int:
    return int(load().axonn_l2_budget())


def axonn_set_swap(mode: int):
    """Operand roles: -1 as tuned, 0 never exchanged, 1 exchanged (C^T = B^T.A^T)."""
    _check(load().axonn_set_swap(int(mode)))


def axonn_last_swap() -> int:
    """1 if the last call on this thread ran with exchanged operand roles."""
    return int(load().axonn_last_swap())


def axonn_device_info():
    """(SM count, resident CTA pairs) of the current device."""
    a, b = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().axonn_device_info(ctypes.byref(a), ctypes.byref(b)))
    return a.value, b.value


def axonn_num_kernel_configs() -> int:
    return int(load().axonn_num_kernel_configs())


def axonn_kernel_config_name(config: int) -> str:
    return load().axonn_kernel_config_name(int(config)).decode()


def axonn_last_kernel_config() -> int:
    return int(load().axonn_last_kernel_config())


def axonn_last_error() -> str:
    return load().axonn_last_error().decode()


def axonn_version() -> str:
    return load().axonn_version().decode()


# ---------------------------------------------------------------- helpers
def out_shape(op, T, K, N):
    """Logical output shape of an op on the full layer."""
    op = OPS.get(op, op)
    return {OP_FWD: (T, N), OP_DGRAD: (T, K), OP_WGRAD: (K, N)}[op]


def call(op, P, Q, C, shape: Shape, flags: int = 0, ws=None, stream=None):
    """Dispatch by op name ('fwd' | 'dgrad' | 'wgrad') to the entry point."""
    op = OPS.get(op, op)
    fn = {OP_FWD: axonn_fc_fwd, OP_DGRAD: axonn_fc_dgrad, OP_WGRAD: axonn_fc_wgrad}[op]
    fn(P, Q, C, shape, flags, ws, stream=stream)
