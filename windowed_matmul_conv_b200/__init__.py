"""Python binding of libwbmm.so: WBMM (Windowed Batch Matrix Multiplication)
on B200.

Each ``wbmm_*`` function has the name and meaning of the C entry point in
``include/wbmm.h`` and only marshals arguments: shapes and dtypes come from
the torch tensors, device pointers from ``data_ptr()``, the stream from
``torch.cuda.current_stream()``.  A non-zero status raises ``WbmmError``.
Plain pointers carry no sizes, so before the call the binding checks what
the library cannot: every buffer is on the current device, has the call's
dtype (fp32 for dT) and holds at least the elements the call reads or writes
(``WbmmError`` with ``WBMM_ERR_DTYPE`` or ``WBMM_ERR_INVALID_ARG``).
PyTorch is used for device memory and streams; every step of the operator
runs in the library's CUDA kernels.  Importing this package fails loudly if
the library has not been built (``python windowed_matmul_conv_b200/build.py``).

The convenience functions ``forward``, ``backward``, ``cache_matrices``,
``reparam_merge``, ``forward_cached``, ``dw3x3``, ``checkpoint``,
``checkpoint_restore``, ``backward_checkpoint``, ``scan_forward``,
``scan_forward_train``, ``scan_backward`` and ``scan_step`` allocate outputs
with torch and call the entry points above.  With ``stream`` they run as under
``torch.cuda.stream(stream)``: outputs and workspaces come from that stream's
memory, and another stream that uses the outputs waits for it first (and calls
``record_stream`` on what it may free).
"""
import ctypes
import math
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwbmm.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        "libwbmm.so is missing: build it with `python windowed_matmul_conv_b200/build.py` "
        "(nvcc, sm_100a); there is no fallback implementation")

_lib = ctypes.CDLL(LIB_PATH)

WBMM_F32, WBMM_BF16 = 0, 1
# 32-bit arrival counters at the start of a table-gradient workspace
WBMM_DT_COUNTER_WORDS = 65536
STATUS_NAMES = {0: "WBMM_OK", 1: "WBMM_ERR_INVALID_ARG", 2: "WBMM_ERR_SHAPE",
                3: "WBMM_ERR_DTYPE", 4: "WBMM_ERR_ALIGNMENT", 5: "WBMM_ERR_UNSUPPORTED",
                6: "WBMM_ERR_WORKSPACE", 7: "WBMM_ERR_CUDA", 8: "WBMM_ERR_TIMEOUT"}
EXPORTS = ("wbmm_forward", "wbmm_backward_workspace_bytes", "wbmm_backward",
           "wbmm_cache_matrices", "wbmm_reparam_merge", "wbmm_forward_cached", "wbmm_dw3x3",
           "wbmm_get_device_status", "wbmm_status_string", "wbmm_set_wait_budget",
           "wbmm_wait_selftest", "wbmm_launch_count", "wbmm_last_path",
           "wbmm_backward_dt_static", "wbmm_debug_set", "wbmm_checkpoint",
           "wbmm_checkpoint_restore", "wbmm_backward_checkpoint_workspace_bytes",
           "wbmm_backward_checkpoint", "wbmm_scan_forward", "wbmm_scan_states_bytes",
           "wbmm_scan_backward", "wbmm_scan_backward_checkpoint", "wbmm_scan_step")
# positions of a sequence that share one step in its 8-bit checkpoint
WBMM_SEQ_GROUP = 64

_vp, _i, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_lib.wbmm_forward.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]
_lib.wbmm_backward_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i]
_lib.wbmm_backward_workspace_bytes.restype = _sz
_lib.wbmm_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _sz, _i, _i, _i, _i, _i, _i, _vp]
_lib.wbmm_cache_matrices.argtypes = [_vp, _vp, _i, _i, _i, _vp]
_lib.wbmm_reparam_merge.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _vp]
_lib.wbmm_backward_dt_static.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]
_lib.wbmm_forward_cached.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _vp]
_lib.wbmm_dw3x3.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
_lib.wbmm_checkpoint.argtypes = [_vp] * 3 + [_i] * 6 + [_vp]
_lib.wbmm_checkpoint_restore.argtypes = [_vp] * 3 + [_i] * 6 + [_vp]
_lib.wbmm_backward_checkpoint_workspace_bytes.argtypes = [_i] * 6
_lib.wbmm_backward_checkpoint_workspace_bytes.restype = _sz
_lib.wbmm_backward_checkpoint.argtypes = [_vp] * 7 + [_sz] + [_i] * 6 + [_vp]
_lib.wbmm_scan_forward.argtypes = [_vp] * 11 + [_i] * 4 + [_vp]
_lib.wbmm_scan_states_bytes.argtypes = [_i] * 3
_lib.wbmm_scan_states_bytes.restype = _sz
_lib.wbmm_scan_backward.argtypes = [_vp] * 9 + [_i] * 4 + [_vp]
_lib.wbmm_scan_backward_checkpoint.argtypes = [_vp] * 11 + [_i] * 4 + [_vp]
_lib.wbmm_scan_step.argtypes = [_vp] * 5 + [_i] * 3 + [_vp]
_lib.wbmm_get_device_status.argtypes = [_vp]
_lib.wbmm_status_string.argtypes = [_i]
_lib.wbmm_status_string.restype = ctypes.c_char_p
_lib.wbmm_set_wait_budget.argtypes = [ctypes.c_ulonglong]
_lib.wbmm_set_wait_budget.restype = None
_lib.wbmm_wait_selftest.argtypes = [ctypes.c_ulonglong, _vp]
_lib.wbmm_launch_count.argtypes = []
_lib.wbmm_launch_count.restype = ctypes.c_ulonglong
_lib.wbmm_last_path.argtypes = []
_lib.wbmm_debug_set.argtypes = [_i, _i]
for _f in ("wbmm_forward", "wbmm_backward", "wbmm_backward_dt_static", "wbmm_cache_matrices",
           "wbmm_reparam_merge", "wbmm_forward_cached", "wbmm_dw3x3", "wbmm_get_device_status", "wbmm_wait_selftest", "wbmm_last_path",
           "wbmm_debug_set", "wbmm_checkpoint", "wbmm_checkpoint_restore",
           "wbmm_backward_checkpoint", "wbmm_scan_forward", "wbmm_scan_backward",
           "wbmm_scan_backward_checkpoint", "wbmm_scan_step"):
    getattr(_lib, _f).restype = _i


WBMM_ERR_INVALID_ARG, WBMM_ERR_DTYPE, WBMM_ERR_UNSUPPORTED = 1, 3, 5
_INT_MAX = 0x7fffffff


class WbmmError(RuntimeError):
    def __init__(self, status, detail=None):
        self.status = status
        msg = _lib.wbmm_status_string(status).decode()
        super().__init__(msg if detail is None else "%s: %s" % (msg, detail))


def _check(status):
    if status != 0:
        raise WbmmError(status)


_DTYPES = {torch.bfloat16: WBMM_BF16, torch.float32: WBMM_F32}


def _dt(t):
    dt = _DTYPES.get(t.dtype)
    if dt is not None:
        return dt
    raise TypeError("WBMM tensors must be bfloat16 or float32, got %s" % t.dtype)


def _p(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("WBMM tensors must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(stream, ref=None):
    """Stream handle for a call whose maps live on ``ref``'s device.  The
    library launches on the current device, so ``ref`` and the stream must
    be on it."""
    if stream is None and ref is not None:
        # the current device's current stream, without the stream object
        d = ref.get_device()
        if d == torch._C._cuda_getDevice():
            return torch._C._cuda_getCurrentRawStream(d)
    s = torch.cuda.current_stream() if stream is None else stream
    if ref is not None:
        d, cur = ref.get_device(), torch.cuda.current_device()
        if d != cur or s.device_index != d:
            raise WbmmError(WBMM_ERR_INVALID_ARG,
                            "maps on cuda:%d, stream on cuda:%d, current device cuda:%d"
                            % (d, s.device_index, cur))
    return s.cuda_stream


def _need(name, t, numel, ref, dtype=None):
    """Buffer ``t`` (optional) must sit on ``ref``'s device, have ``ref``'s
    dtype (or ``dtype``) and hold at least ``numel`` elements."""
    if t is None:
        return
    want = dtype or ref.dtype
    if t.dtype is want and t.numel() >= numel and t.get_device() == ref.get_device():
        return
    if t.get_device() != ref.get_device():
        raise WbmmError(WBMM_ERR_INVALID_ARG, "%s is on %s, the map on %s"
                        % (name, t.device, ref.device))
    if t.dtype is not want:
        raise WbmmError(WBMM_ERR_DTYPE, "%s is %s, the call needs %s" % (name, t.dtype, want))
    raise WbmmError(WBMM_ERR_INVALID_ARG, "%s holds %d elements, the call needs %d"
                    % (name, t.numel(), numel))


def _all(dtype, numel, device, *tensors):
    """True when every tensor given has the dtype, the device index and at
    least numel elements (the usual case; the caller names the offender)."""
    for t in tensors:
        if t is not None and (t.dtype is not dtype or t.numel() < numel
                              or t.get_device() != device):
            return False
    return True


def _ptrs(*tensors):
    """Addresses of tensors that are on one device (checked): CUDA, contiguous."""
    out = []
    for t in tensors:
        if t is None:
            out.append(None)
        elif t.is_cuda and t.is_contiguous():
            out.append(t.data_ptr())
        else:
            raise ValueError("WBMM tensors must be contiguous CUDA tensors")
    return out


def _tsz(w):
    return (2 * int(w) - 1) ** 2


def _ints(*sizes):
    """Refuses sizes beyond the C ABI's ints, which ctypes would cut to 32 bits."""
    for n in sizes:
        if not -_INT_MAX <= n <= _INT_MAX:
            raise WbmmError(WBMM_ERR_UNSUPPORTED, "sizes %s" % (sizes,))


def _map_shape(x):
    if x.dim() != 4:
        raise ValueError("feature maps must be [B, C, H, W]")
    if x.numel() > _INT_MAX:            # no size is larger than the product, but for empty maps
        _ints(*x.shape)
    return x.shape


def _windows(B, C, H, W, w):
    w = int(w)
    if w > _INT_MAX or w < -_INT_MAX:
        _ints(w)
    return B * C * (H // w) * (W // w) if w > 0 else 0


def _seq_shape(v):
    shape = v.shape
    if len(shape) < 2:
        raise ValueError("recurrence tensors must be [B, C, L], [B, C, H, W] or [B, C]")
    B, C = shape[0], shape[1]
    L = shape[2] if len(shape) == 3 else math.prod(shape[2:])
    if L > _INT_MAX or B > _INT_MAX or C > _INT_MAX:     # inline: the step's host time
        _ints(B, C, L)
    return B, C, L


def _need_seq(ref, B, C, L, h0, hT, lengths, states, codes=(), exps=()):
    dev, f32 = ref.get_device(), torch.float32
    if not _all(f32, B * C, dev, h0, hT):
        _need("state in", h0, B * C, ref, f32)
        _need("state out", hT, B * C, ref, f32)
    if lengths is not None:
        _need("lengths", lengths, B, ref, torch.int32)
    if states is not None:
        _need("states", states, B * C * _scan_tiles(L), ref, f32)
    if not (_all(torch.uint8, B * C * L, dev, *codes)
            and _all(torch.uint8, B * C * -(-L // WBMM_SEQ_GROUP), dev, *exps)):
        for t in codes:
            _need("codes", t, B * C * L, ref, torch.uint8)
        for t in exps:
            _need("exps", t, B * C * -(-L // WBMM_SEQ_GROUP), ref, torch.uint8)


def _scan_tiles(L):
    """Entries of the states array a row: one per 256 positions."""
    return -(-L // 256)


# --------------------------------------------------------------- entry points

def wbmm_forward(x, T, y, w, stream=None):
    B, C, H, W = _map_shape(x)
    _need("T", T, C * _tsz(w), x)
    _need("y", y, x.numel(), x)
    _check(_lib.wbmm_forward(_p(x), _p(T), _p(y), B, C, H, W, int(w), _dt(x),
                             _stream(stream, x)))


def wbmm_backward_workspace_bytes(B, C, H, W, w, dtype):
    dt = _dt(torch.empty(0, dtype=dtype))
    _ints(B, C, H, W, int(w))
    return int(_lib.wbmm_backward_workspace_bytes(B, C, H, W, int(w), dt))


def wbmm_backward(x, T, dY, dX, dT, workspace, w, stream=None):
    B, C, H, W = _map_shape(dY)
    _need("x", x, dY.numel(), dY)
    _need("T", T, C * _tsz(w), dY)
    _need("dX", dX, dY.numel(), dY)
    _need("dT", dT, C * _tsz(w), dY, torch.float32)
    if workspace is not None and workspace.get_device() != dY.get_device():
        raise WbmmError(WBMM_ERR_INVALID_ARG, "workspace is on %s, the map on %s"
                        % (workspace.device, dY.device))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.wbmm_backward(_p(x), _p(T), _p(dY), _p(dX), _p(dT), _p(workspace), ws_bytes,
                              B, C, H, W, int(w), _dt(dY), _stream(stream, dY)))


def wbmm_backward_dt_static(x, dY, dT, w, stream=None):
    """dT of wbmm_backward with the library's fixed scratch array (no allocation)."""
    B, C, H, W = _map_shape(dY)
    _need("x", x, dY.numel(), dY)
    _need("dT", dT, C * _tsz(w), dY, torch.float32)
    _check(_lib.wbmm_backward_dt_static(_p(x), _p(dY), _p(dT), B, C, H, W, int(w), _dt(dY),
                                        _stream(stream, dY)))


def wbmm_cache_matrices(T, M, w, stream=None):
    """T: [C, (2w-1)^2]; M: [C, w*w, w*w]."""
    C = int(T.shape[0])
    _ints(C)
    _need("T", T, C * _tsz(w), T)
    _need("M", M, C * int(w) ** 4, T)
    _check(_lib.wbmm_cache_matrices(_p(T), _p(M), C, int(w), _dt(T), _stream(stream, T)))


def wbmm_forward_cached(x, M, dw3x3, out, w, stream=None):
    B, C, H, W = _map_shape(x)
    _need("M", M, C * int(w) ** 4, x)
    _need("dw3x3", dw3x3, C * 9, x)
    _need("out", out, x.numel(), x)
    _check(_lib.wbmm_forward_cached(_p(x), _p(M), _p(dw3x3), _p(out), B, C, H, W, int(w),
                                    _dt(x), _stream(stream, x)))


def wbmm_dw3x3(y, K, z, stream=None):
    B, C, H, W = _map_shape(y)
    _need("K", K, C * 9, y)
    _need("z", z, y.numel(), y)
    _check(_lib.wbmm_dw3x3(_p(y), _p(K), _p(z), B, C, H, W, _dt(y), _stream(stream, y)))


def wbmm_checkpoint(x, codes, exps, w, stream=None):
    B, C, H, W = _map_shape(x)
    _need("codes", codes, x.numel(), x, torch.uint8)
    _need("exps", exps, _windows(B, C, H, W, w), x, torch.uint8)
    _check(_lib.wbmm_checkpoint(*_ptrs(x, codes, exps), B, C, H, W, int(w), _dt(x),
                                _stream(stream, x)))


def wbmm_checkpoint_restore(codes, exps, x, w, stream=None):
    B, C, H, W = _map_shape(x)
    _need("codes", codes, x.numel(), x, torch.uint8)
    _need("exps", exps, _windows(B, C, H, W, w), x, torch.uint8)
    _check(_lib.wbmm_checkpoint_restore(*_ptrs(codes, exps, x), B, C, H, W, int(w), _dt(x),
                                        _stream(stream, x)))


def wbmm_backward_checkpoint_workspace_bytes(B, C, H, W, w, dtype):
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("WBMM tensors must be bfloat16 or float32, got %s" % dtype)
    _ints(B, C, H, W, int(w))
    return int(_lib.wbmm_backward_checkpoint_workspace_bytes(B, C, H, W, int(w), dt))


def wbmm_backward_checkpoint(codes, exps, T, dY, dX, dT, workspace, w, stream=None):
    B, C, H, W = _map_shape(dY)
    _need("codes", codes, dY.numel(), dY, torch.uint8)
    _need("exps", exps, _windows(B, C, H, W, w), dY, torch.uint8)
    _need("T", T, C * _tsz(w), dY)
    _need("dX", dX, dY.numel(), dY)
    _need("dT", dT, C * _tsz(w), dY, torch.float32)
    if workspace is not None and workspace.get_device() != dY.get_device():
        raise WbmmError(WBMM_ERR_INVALID_ARG, "workspace is on %s, the map on %s"
                        % (workspace.device, dY.device))
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(_lib.wbmm_backward_checkpoint(_p(codes), _p(exps), _p(T), _p(dY), _p(dX), _p(dT),
                                         _p(workspace), ws_bytes, B, C, H, W, int(w), _dt(dY),
                                         _stream(stream, dY)))


def wbmm_scan_forward(v, g, h0, lengths, y, hT, states, v_codes, v_exps, g_codes, g_exps,
                      stream=None):
    """v, g, y: [B, C, L] or a map [B, C, H, W] (L = H*W); the rest may be None."""
    B, C, L = _seq_shape(v)
    if not _all(v.dtype, B * C * L, v.get_device(), g, y):
        _need("g", g, B * C * L, v)
        _need("y", y, B * C * L, v)
    _need_seq(v, B, C, L, h0, hT, lengths, states, (v_codes, g_codes), (v_exps, g_exps))
    _check(_lib.wbmm_scan_forward(
        *_ptrs(v, g, h0, lengths, y, hT, states, v_codes, v_exps, g_codes, g_exps), B, C, L,
        _dt(v), _stream(stream, v)))


def wbmm_scan_states_bytes(B, C, L):
    _ints(B, C, L)
    return int(_lib.wbmm_scan_states_bytes(int(B), int(C), int(L)))


def wbmm_scan_backward(v, g, states, lengths, dY, dhT, dv, dg, dh0, stream=None):
    B, C, L = _seq_shape(dY)
    if not _all(dY.dtype, B * C * L, dY.get_device(), v, g, dv, dg):
        for name, t in (("v", v), ("g", g), ("dv", dv), ("dg", dg)):
            _need(name, t, B * C * L, dY)
    _need_seq(dY, B, C, L, dhT, dh0, lengths, states)
    _check(_lib.wbmm_scan_backward(*_ptrs(v, g, states, lengths, dY, dhT, dv, dg, dh0), B, C, L,
                                   _dt(dY), _stream(stream, dY)))


def wbmm_scan_backward_checkpoint(v_codes, v_exps, g_codes, g_exps, states, lengths, dY, dhT, dv,
                                  dg, dh0, stream=None):
    B, C, L = _seq_shape(dY)
    if not _all(dY.dtype, B * C * L, dY.get_device(), dv, dg):
        _need("dv", dv, B * C * L, dY)
        _need("dg", dg, B * C * L, dY)
    _need_seq(dY, B, C, L, dhT, dh0, lengths, states, (v_codes, g_codes), (v_exps, g_exps))
    _check(_lib.wbmm_scan_backward_checkpoint(
        *_ptrs(v_codes, v_exps, g_codes, g_exps, states, lengths, dY, dhT, dv, dg, dh0), B, C, L,
        _dt(dY), _stream(stream, dY)))


def wbmm_scan_step(v, g, h, y, h_next, stream=None):
    """v, g, y: [B, C]; h, h_next: [B, C] fp32 (may be one buffer)."""
    B, C, L = _seq_shape(v)
    if L != 1:
        raise ValueError("a step takes one position: [B, C]")
    dev = v.get_device()
    if not (_all(v.dtype, B * C, dev, g, y) and _all(torch.float32, B * C, dev, h, h_next)):
        _need("g", g, B * C, v)
        _need("y", y, B * C, v)
        _need("h", h, B * C, v, torch.float32)
        _need("h_next", h_next, B * C, v, torch.float32)
    _check(_lib.wbmm_scan_step(*_ptrs(v, g, h, y, h_next), B, C, _dt(v), _stream(stream, v)))


def wbmm_get_device_status(stream=None):
    """Synchronises the stream; returns the status code (0, or 8 after a timeout)."""
    return int(_lib.wbmm_get_device_status(_stream(stream)))


def wbmm_status_string(status):
    return _lib.wbmm_status_string(int(status)).decode()


def wbmm_set_wait_budget(cycles):
    _lib.wbmm_set_wait_budget(int(cycles))


def wbmm_wait_selftest(cycles, stream=None):
    _check(_lib.wbmm_wait_selftest(int(cycles), _stream(stream)))


def wbmm_launch_count():
    return int(_lib.wbmm_launch_count())


def wbmm_last_path():
    return int(_lib.wbmm_last_path())


# test-only settings of wbmm_debug_set (include/wbmm.h)
WBMM_DEBUG_SKIP_LOAD_WINDOW_MAJOR, WBMM_DEBUG_SKIP_LOAD_TABLE_GRAD, WBMM_DEBUG_RING_CAP = 1, 2, 3


def wbmm_debug_set(what, value):
    _check(_lib.wbmm_debug_set(int(what), int(value)))


# ------------------------------------------------------------ conveniences

def _on(stream, ref, call, *args, **kw):
    """A convenience call on a given stream.  What it allocates has to come from
    that stream's memory: the current stream's may still be in use there, and a
    workspace freed to it would be handed out while the kernels run."""
    _p(ref)                     # refused as by a call without a stream
    _stream(stream, ref)
    with torch.cuda.stream(stream):
        return call(*args, **kw)


def forward(x, T, w, stream=None):
    if stream is not None:
        return _on(stream, x, forward, x, T, w)
    y = torch.empty_like(x)
    wbmm_forward(x, T, y, w)
    return y


def backward(x, T, dY, w, need_dx=True, need_dt=True, stream=None):
    if stream is not None:
        return _on(stream, dY, backward, x, T, dY, w, need_dx, need_dt)
    B, C, H, W = _map_shape(dY)
    dX = torch.empty_like(dY) if need_dx else None
    dT = torch.empty((C, (2 * w - 1) ** 2), dtype=torch.float32, device=dY.device) if need_dt else None
    ws = None
    if need_dt:
        nbytes = wbmm_backward_workspace_bytes(B, C, H, W, w, dY.dtype)
        # zero-filled: the table gradient's arrival counters start at zero
        ws = torch.zeros(max(1, nbytes // 4), dtype=torch.float32, device=dY.device)
    wbmm_backward(x, T, dY, dX, dT, ws, w)
    return dX, dT


def wbmm_reparam_merge(Tw, Tk, M, w, k, stream=None):
    """Tw: [C, (2w-1)^2]; Tk: [C, (2k-1)^2]; M: [C, w*w, w*w]."""
    C = int(Tw.shape[0])
    _ints(C)
    _need("Tw", Tw, C * _tsz(w), Tw)
    _need("Tk", Tk, C * _tsz(k), Tw)
    _need("M", M, C * int(w) ** 4, Tw)
    _check(_lib.wbmm_reparam_merge(_p(Tw), _p(Tk), _p(M), C, int(w), int(k), _dt(Tw),
                                   _stream(stream, Tw)))


def reparam_merge(Tw, Tk, w, k, stream=None):
    """Inference matrix [C, w*w, w*w] of a w-window branch (table Tw) plus a
    k-window branch (table Tk), k dividing w; feed it to forward_cached."""
    if stream is not None:
        return _on(stream, Tw, reparam_merge, Tw, Tk, w, k)
    M = torch.empty((Tw.shape[0], w * w, w * w), dtype=Tw.dtype, device=Tw.device)
    wbmm_reparam_merge(Tw, Tk, M, w, k)
    return M


def cache_matrices(T, w, stream=None):
    if stream is not None:
        return _on(stream, T, cache_matrices, T, w)
    M = torch.empty((T.shape[0], w * w, w * w), dtype=T.dtype, device=T.device)
    wbmm_cache_matrices(T, M, w)
    return M


def forward_cached(x, M, w, dw=None, stream=None):
    if stream is not None:
        return _on(stream, x, forward_cached, x, M, w, dw)
    out = torch.empty_like(x)
    wbmm_forward_cached(x, M, dw, out, w)
    return out


def dw3x3(y, K, stream=None):
    if stream is not None:
        return _on(stream, y, dw3x3, y, K)
    z = torch.empty_like(y)
    wbmm_dw3x3(y, K, z)
    return z


# The following allocate their outputs, so they check the caller's buffers only
# and pass the new ones' addresses as they are.

def checkpoint(x, w, stream=None):
    """8-bit form of a map: codes [C, B*nh*nw, w*w] and exponent bytes
    [C, B*nh*nw], one power-of-two step per window."""
    if stream is not None:
        return _on(stream, x, checkpoint, x, w)
    B, C, H, W = _map_shape(x)
    px, = _ptrs(x)
    n = _windows(B, C, H, W, w) // max(1, C)
    codes = x.new_empty((C, n, x.numel() // max(1, C * n)), dtype=torch.uint8)
    exps = x.new_empty((C, n), dtype=torch.uint8)
    # a map without a whole window has no groups to point to; its shape is refused
    pc, pe = (codes.data_ptr(), exps.data_ptr()) if n else (px, px)
    _check(_lib.wbmm_checkpoint(px, pc, pe, B, C, H, W, int(w), _dt(x),
                                _stream(None, x)))
    return codes, exps


def checkpoint_restore(codes, exps, shape, w, dtype, stream=None):
    """The map of the given shape and dtype that checkpoint() stored."""
    if stream is not None:
        return _on(stream, codes, checkpoint_restore, codes, exps, shape, w, dtype)
    B, C, H, W = shape
    n = B * C * H * W
    if n > _INT_MAX:
        _ints(B, C, H, W)
    x = codes.new_empty(shape, dtype=dtype)
    _need("codes", codes, n, x, torch.uint8)
    _need("exps", exps, _windows(B, C, H, W, w), x, torch.uint8)
    pc, pe = _ptrs(codes, exps)
    _check(_lib.wbmm_checkpoint_restore(pc, pe, x.data_ptr(), B, C, H, W, int(w), _dt(x),
                                        _stream(None, x)))
    return x


def backward_checkpoint(codes, exps, T, dY, w, need_dx=True, need_dt=True, stream=None):
    """backward() with the forward's input as checkpoint() keeps it."""
    if stream is not None:
        return _on(stream, dY, backward_checkpoint, codes, exps, T, dY, w, need_dx, need_dt)
    B, C, H, W = _map_shape(dY)
    dX = torch.empty_like(dY) if need_dx else None
    dT = dY.new_empty((C, (2 * w - 1) ** 2), dtype=torch.float32) if need_dt else None
    ws = None
    if need_dt:
        nbytes = wbmm_backward_checkpoint_workspace_bytes(B, C, H, W, w, dY.dtype)
        ws = dY.new_empty(nbytes, dtype=torch.uint8)
    wbmm_backward_checkpoint(codes, exps, T, dY, dX, dT, ws, w)
    return dX, dT


class ScanSaved(NamedTuple):
    """What scan_forward_train keeps for scan_backward: v and g themselves, or
    their 8-bit codes with exponent bytes, and the states at every 256th
    position."""
    v: torch.Tensor
    g: torch.Tensor
    v_exps: Optional[torch.Tensor]
    g_exps: Optional[torch.Tensor]
    states: torch.Tensor
    lengths: Optional[torch.Tensor]


def _scan_inputs(v, g, h0, lengths):
    """Sizes of a forward call and the addresses of its checked inputs."""
    B, C, L = _seq_shape(v)
    if not _all(v.dtype, B * C * L, v.get_device(), g):
        _need("g", g, B * C * L, v)
    if h0 is not None:
        _need("h0", h0, B * C, v, torch.float32)
    if lengths is not None:
        _need("lengths", lengths, B, v, torch.int32)
    return B, C, L, _ptrs(v, g, h0, lengths)


def scan_forward(v, g, h0=None, lengths=None, stream=None):
    """y and the last state [B, C] fp32 of the gated recurrence over [B, C, L]."""
    if stream is not None:
        return _on(stream, v, scan_forward, v, g, h0, lengths)
    B, C, L, inputs = _scan_inputs(v, g, h0, lengths)
    y, hT = torch.empty_like(v), v.new_empty((B, C), dtype=torch.float32)
    _check(_lib.wbmm_scan_forward(*inputs, y.data_ptr(), hT.data_ptr(), None, None, None, None,
                                  None, B, C, L, _dt(v), _stream(None, v)))
    return y, hT


def scan_forward_train(v, g, h0=None, lengths=None, checkpoint=False, stream=None):
    """scan_forward that also returns what scan_backward needs; with
    `checkpoint` v and g are kept in 8 bits."""
    if stream is not None:
        return _on(stream, v, scan_forward_train, v, g, h0, lengths, checkpoint)
    B, C, L, inputs = _scan_inputs(v, g, h0, lengths)
    y, hT = torch.empty_like(v), v.new_empty((B, C), dtype=torch.float32)
    states = v.new_empty((B, C, _scan_tiles(L)), dtype=torch.float32)
    if checkpoint:
        groups = (B, C, -(-L // WBMM_SEQ_GROUP))
        vc, ve = torch.empty_like(v, dtype=torch.uint8), v.new_empty(groups, dtype=torch.uint8)
        gc, ge = torch.empty_like(v, dtype=torch.uint8), v.new_empty(groups, dtype=torch.uint8)
        kept = vc.data_ptr(), ve.data_ptr(), gc.data_ptr(), ge.data_ptr()
        saved = ScanSaved(vc, gc, ve, ge, states, lengths)
    else:
        kept = None, None, None, None
        saved = ScanSaved(v, g, None, None, states, lengths)
    _check(_lib.wbmm_scan_forward(*inputs, y.data_ptr(), hT.data_ptr(), states.data_ptr(), *kept,
                                  B, C, L, _dt(v), _stream(None, v)))
    return y, hT, saved


def scan_backward(saved, dY, dhT=None, stream=None):
    """dv, dg and dh0 [B, C] fp32 from scan_forward_train's `saved`."""
    if stream is not None:
        return _on(stream, dY, scan_backward, saved, dY, dhT)
    v, g, v_exps, g_exps, states, lengths = saved
    if v.numel() != dY.numel() or v.shape[:2] != dY.shape[:2]:
        raise WbmmError(WBMM_ERR_INVALID_ARG, "dY is %s, the forward call's maps were %s"
                        % (tuple(dY.shape), tuple(v.shape)))
    B, C, L = _seq_shape(dY)
    plain = v_exps is None
    if not _all(dY.dtype if plain else torch.uint8, B * C * L, dY.get_device(), v, g):
        _need("v", v, B * C * L, dY, None if plain else torch.uint8)
        _need("g", g, B * C * L, dY, None if plain else torch.uint8)
    _need_seq(dY, B, C, L, dhT, None, lengths, states, (), () if plain else (v_exps, g_exps))
    dv, dg = torch.empty_like(dY), torch.empty_like(dY)
    dh0 = dY.new_empty((B, C), dtype=torch.float32)
    outputs = dv.data_ptr(), dg.data_ptr(), dh0.data_ptr(), B, C, L, _dt(dY), _stream(None, dY)
    if plain:
        _check(_lib.wbmm_scan_backward(*_ptrs(v, g, states, lengths, dY, dhT), *outputs))
    else:
        _check(_lib.wbmm_scan_backward_checkpoint(
            *_ptrs(v, v_exps, g, g_exps, states, lengths, dY, dhT), *outputs))
    return dv, dg, dh0


def scan_step(v, g, h, stream=None):
    """One position for every row: y [B, C] and the next state [B, C] fp32."""
    if stream is not None:
        return _on(stream, v, scan_step, v, g, h)
    B, C, L = _seq_shape(v)
    if L != 1:
        raise ValueError("a step takes one position: [B, C]")
    if not (_all(v.dtype, B * C, v.get_device(), g)
            and _all(torch.float32, B * C, v.get_device(), h)):
        _need("g", g, B * C, v)
        _need("h", h, B * C, v, torch.float32)
    pv, pg, ph = _ptrs(v, g, h)
    y, h_next = torch.empty_like(v), torch.empty_like(h)
    _check(_lib.wbmm_scan_step(pv, pg, ph, y.data_ptr(), h_next.data_ptr(), B, C, _dt(v),
                               _stream(None, v)))
    return y, h_next
