"""ctypes binding over libsx_scan.so (C ABI in include/sx_scan.h).

Argument marshalling only: shapes, strides, pointers, the workspace and the
current torch stream go to the C library, whose HIP kernels do every step of
the scan. There is no CPU fallback: without the built library every call
raises.
"""

from __future__ import annotations

import ctypes
import functools
import math
import os
import warnings

import torch
import torch.autograd.forward_ad as forward_ad

HERE = os.path.dirname(os.path.abspath(__file__))
# SX_SCAN_LIB selects another build of the same library (the host-sanitized one the
# boundary tests run under); by default the in-tree libsx_scan.so.
LIB_PATH = os.environ.get("SX_SCAN_LIB") or os.path.join(HERE, "libsx_scan.so")

SX_OK = 0
SX_E_DIM_001 = 1
SX_E_DIM_002 = 2
SX_E_DIM_003 = 3
SX_E_UNSUPPORTED = 4
SX_E_ALIAS = 5
SX_E_WORKSPACE = 6
SX_E_DEVICE = 7
SX_STATE_SCALAR = -(2 ** 31)
SX_F32 = 0
SX_BF16 = 1

BODIES = {"tanh_affine": 0, "norm_cap": 1, "max_plus": 2}
_DTYPES = {torch.float32: SX_F32, torch.bfloat16: SX_BF16}
_STATUS_NAMES = {0: "OK", 1: "E-DIM-001", 2: "E-DIM-002", 3: "E-DIM-003", 4: "E-UNSUPPORTED",
                 5: "E-ALIAS", 6: "E-WORKSPACE", 7: "E-DEVICE"}


class SxError(RuntimeError):
    """A call the library (or this binding, before calling it) refused."""

    def __init__(self, code: int, message: str):
        super().__init__(message)
        self.code = code
        self.name = _STATUS_NAMES.get(code, "E-UNKNOWN")


_lib = None

_i64p = ctypes.POINTER(ctypes.c_int64)


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libsx_scan.so once and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m scan_primitives_amd.build_lib` "
                           "(there is no CPU fallback)")
    lib = ctypes.CDLL(path)
    c_int, c_size, vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    lib.sx_element_scan.restype = c_int
    lib.sx_element_scan.argtypes = [c_int, c_int, _i64p, c_int, c_int, c_int,
                                    vp, _i64p, vp, ctypes.c_int64, _i64p, vp, ctypes.c_int64, _i64p,
                                    vp, vp, c_size, vp]
    lib.sx_element_scan_workspace_bytes.restype = c_size
    lib.sx_element_scan_workspace_bytes.argtypes = [c_int, c_int, _i64p, c_int, c_int]
    lib.sx_matrix_scan.restype = c_int
    lib.sx_matrix_scan.argtypes = [c_int, c_int, _i64p, _i64p, vp, c_int, _i64p, _i64p, vp,
                                   c_int, c_int, c_int, c_int, vp, vp, c_size, vp]
    lib.sx_matrix_scan_noalloc.restype = c_int
    lib.sx_matrix_scan_noalloc.argtypes = [c_int, c_int, _i64p, _i64p, vp, c_int, _i64p, _i64p, vp,
                                           c_int, c_int, c_int, c_int, vp, vp]
    lib.sx_matrix_scan_workspace_bytes.restype = c_size
    lib.sx_matrix_scan_workspace_bytes.argtypes = [c_int, _i64p, c_int, _i64p, c_int]
    lib.sx_matrix_scan_out_shape.restype = c_int
    lib.sx_matrix_scan_out_shape.argtypes = [c_int, _i64p, c_int, _i64p, _i64p]
    lib.sx_element_scan_backward.restype = c_int
    lib.sx_element_scan_backward.argtypes = [c_int, c_int, _i64p, c_int, c_int, c_int, vp, vp, ctypes.c_int64, _i64p,
                                             vp, ctypes.c_int64, _i64p, vp, vp, vp, vp, vp, vp, c_size, vp]
    lib.sx_element_scan_backward_workspace_bytes.restype = c_size
    lib.sx_element_scan_backward_workspace_bytes.argtypes = [c_int, c_int, _i64p, c_int, c_int, ctypes.c_int64,
                                                             ctypes.c_int64]
    lib.sx_matrix_scan_backward.restype = c_int
    lib.sx_matrix_scan_backward.argtypes = [c_int, c_int, _i64p, _i64p, vp, c_int, _i64p, vp, _i64p, vp,
                                            c_int, c_int, c_int, vp, vp, vp, c_size, vp]
    lib.sx_matrix_scan_backward_workspace_bytes.restype = c_size
    lib.sx_matrix_scan_backward_workspace_bytes.argtypes = [c_int, _i64p, c_int, _i64p, c_int, c_int]
    lib.sx_table_scan.restype = c_int
    lib.sx_table_scan.argtypes = [c_int, c_int, vp, c_int, _i64p, _i64p, vp, c_int, ctypes.c_int32, vp, vp]
    lib.sx_linear_scan.restype = c_int
    lib.sx_linear_scan.argtypes = [c_int, c_int, _i64p, _i64p, vp, c_int, _i64p, _i64p, vp,
                                   c_int, c_int, c_int, vp, vp]
    lib.sx_linear_scan_out_shape.restype = c_int
    lib.sx_linear_scan_out_shape.argtypes = [c_int, _i64p, c_int, _i64p, _i64p]
    c_i64, c_f = ctypes.c_int64, ctypes.c_float
    tensor = [_i64p, _i64p, vp]  # shape, strides, data
    lib.sx_decay_attention.restype = c_int
    lib.sx_decay_attention.argtypes = [c_int, *tensor, *tensor, *tensor, c_int, *tensor, vp, vp, c_f, vp, vp, vp,
                                       c_size, vp]
    lib.sx_decay_attention_workspace_bytes.restype = c_size
    lib.sx_decay_attention_workspace_bytes.argtypes = [c_int, _i64p, _i64p, c_i64]
    lib.sx_decay_attention_backward.restype = c_int
    lib.sx_decay_attention_backward.argtypes = [c_int, *tensor, *tensor, *tensor, c_int, *tensor, _i64p, vp, vp, vp,
                                                vp, c_f, vp, vp, vp, vp, vp, vp, c_size, vp]
    lib.sx_decay_attention_backward_workspace_bytes.restype = c_size
    lib.sx_decay_attention_backward_workspace_bytes.argtypes = [c_int, _i64p, _i64p, _i64p, c_i64]
    lib.sx_decay_attention_step.restype = c_int
    lib.sx_decay_attention_step.argtypes = [c_int, *tensor, *tensor, *tensor, c_int, *tensor, c_i64, _i64p, vp, vp,
                                            c_f, vp, vp]
    lib.sx_head_norm_rotate.restype = c_int
    lib.sx_head_norm_rotate.argtypes = [c_int, *tensor, *tensor, c_int, _i64p, vp, c_i64, vp, vp, vp, c_f, c_int, vp,
                                        vp, vp]
    lib.sx_head_norm_rotate_backward.restype = c_int
    lib.sx_head_norm_rotate_backward.argtypes = [c_int, *tensor, *tensor, c_int, _i64p, vp, c_i64, vp, _i64p, vp,
                                                 _i64p, vp, vp, vp, c_f, c_int, vp, vp, vp, vp, vp, c_size, vp]
    lib.sx_head_norm_rotate_backward_workspace_bytes.restype = c_size
    lib.sx_head_norm_rotate_backward_workspace_bytes.argtypes = [_i64p, _i64p]
    lib.sx_matrix_scan_workspace_status.restype = c_int
    lib.sx_matrix_scan_workspace_status.argtypes = [vp, c_size, vp]
    lib.sx_set_lookback_spin_limit.restype = None
    lib.sx_set_lookback_spin_limit.argtypes = [ctypes.c_uint32]
    lib.sx_status_name.restype = ctypes.c_char_p
    lib.sx_status_name.argtypes = [c_int]
    lib.sx_last_error.restype = ctypes.c_char_p
    lib.sx_last_error.argtypes = []
    lib.sx_version.restype = ctypes.c_char_p
    lib.sx_version.argtypes = []
    _lib = lib
    return lib


def i64_array(values) -> ctypes.Array:
    values = list(values)
    return (ctypes.c_int64 * max(len(values), 1))(*values)


def _check(status: int) -> None:
    if status != SX_OK:
        msg = load_library().sx_last_error().decode()
        raise SxError(status, msg or _STATUS_NAMES.get(status, str(status)))


def _stream_handle(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# Matrix-scan workspaces. The library needs each one zero-filled once and then
# leaves it ready for the next call, so no call clears anything. Eager calls get
# one per (device, stream), zero-filled when allocated. Calls captured into a
# graph get one per capture (keyed by the HIP capture id), allocated and
# zero-filled inside that capture: every graph then starts from a zeroed
# workspace of its own in its first replay, and no captured workspace is handed
# to an eager call or to another graph.
_matrix_workspaces: dict = {}
_hip_runtime = None


def _capture_id(stream_handle: int):
    """The id of the capture running on the stream, or None."""
    global _hip_runtime
    if _hip_runtime is None:
        # the HIP runtime torch has loaded (the same soname the library links)
        hip = ctypes.CDLL("libamdhip64.so.7")
        hip.hipStreamGetCaptureInfo.restype = ctypes.c_int
        hip.hipStreamGetCaptureInfo.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int),
                                                ctypes.POINTER(ctypes.c_ulonglong)]
        _hip_runtime = hip
    status, cid = ctypes.c_int(0), ctypes.c_ulonglong(0)
    err = _hip_runtime.hipStreamGetCaptureInfo(stream_handle, ctypes.byref(status), ctypes.byref(cid))
    if err != 0:
        raise SxError(SX_E_DEVICE, f"hipStreamGetCaptureInfo failed with HIP error {err}")
    return int(cid.value) if status.value == 1 else None  # 1: hipStreamCaptureStatusActive


def _matrix_workspace(nbytes: int, device: torch.device):
    if nbytes == 0:
        return None
    handle = torch.cuda.current_stream(device).cuda_stream
    cid = _capture_id(handle) if torch.cuda.is_current_stream_capturing() else None
    key = (device.index, handle, cid)
    entry = _matrix_workspaces.get(key)
    if entry is not None and entry.numel() >= nbytes:
        return entry
    size = (nbytes + (1 << 20) - 1) >> 20 << 20
    if entry is not None:
        size = max(size, entry.numel())
    ws = torch.zeros(size, dtype=torch.uint8, device=device)
    _matrix_workspaces[key] = ws
    return ws


def matrix_scan_status(device=None) -> None:
    """Raise ``SxError`` (E-DEVICE) if a matrix-scan look-back gave up on one of
    this device's eager workspaces since the last check, and clear what it
    found. Waits for the streams those workspaces belong to."""
    lib = load_library()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    for (index, handle, cid), ws in list(_matrix_workspaces.items()):
        if index != dev.index or cid is not None:
            continue
        with torch.cuda.device(dev):
            _check(lib.sx_matrix_scan_workspace_status(ws.data_ptr(), ws.numel(), handle))


def set_lookback_spin_limit(limit: int) -> None:
    """Bound on the polls a matrix-scan look-back makes before it gives up and
    records it (0 restores the default). A diagnostic for the give-up report."""
    load_library().sx_set_lookback_spin_limit(int(limit))


def _require_no_tangent(*tensors) -> None:
    """Forward-mode derivatives are not carried: a tensor with a tangent is refused, not taken without it."""
    if forward_ad._current_level < 0:  # outside of every dual_level() no tensor has one
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
            raise SxError(SX_E_UNSUPPORTED, "forward-mode differentiation (a tensor with a tangent) is not supported")


def _signed(*tensors):
    """The tensors with lazily negated views (the imaginary part of a conjugate) as tensors of the values they have."""
    return [t.resolve_neg() if isinstance(t, torch.Tensor) and t.is_neg() else t for t in tensors]


def _require_device_tensor(name: str, t) -> None:
    if not isinstance(t, torch.Tensor):
        raise SxError(SX_E_DIM_003, f"{name}: a tensor was expected, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise SxError(SX_E_UNSUPPORTED, f"{name}: the HIP library takes device tensors, got {t.device}")


def element_scan(body: str, initial: torch.Tensor, sequences, axis: int = 0, state_axis=None,
                 reverse: bool = False) -> torch.Tensor:
    """Element scan on the GPU: ``"tanh_affine"``, ``"norm_cap"`` or ``"max_plus"``.

    ``sequences`` is ``[x, decay]`` or ``[x, cost]`` (page order). ``state_axis``
    is ``None`` for a scalar state or ``-1`` for a vector state along the last
    axis. Returns a new f32 tensor of the sequences' shape. When autograd
    records (an input requires grad), the gradient runs through
    ``element_scan_backward``.
    """
    seqs = list(sequences)
    _require_no_tangent(initial, *seqs)
    initial, *seqs = _signed(initial, *seqs)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in [initial] + seqs):
        if len(seqs) != 2:
            raise SxError(SX_E_DIM_001, f"element-scan: the {body} body takes two sequences, got {len(seqs)}")
        return _ElementScanFunction.apply(body, axis, state_axis, reverse, initial, seqs[0], seqs[1])
    return _element_scan_forward(body, initial, seqs, axis, state_axis, reverse)


def _element_scan_forward(body, initial, sequences, axis, state_axis, reverse) -> torch.Tensor:
    if body not in BODIES:
        raise SxError(SX_E_UNSUPPORTED, f"element-scan: unknown body {body!r}")
    seqs = list(sequences)
    if len(seqs) != 2:
        raise SxError(SX_E_DIM_001, f"element-scan: the {body} body takes two sequences, got {len(seqs)}")
    x, s = seqs
    for name, t in (("initial", initial), ("x", x), ("sequence 2", s)):
        _require_device_tensor(name, t)
        if t.dtype != torch.float32:
            raise SxError(SX_E_DIM_002, f"element-scan: {name} is {t.dtype}, sequences and initial are f32")
    if not (x.device == s.device == initial.device):
        raise SxError(SX_E_UNSUPPORTED, "element-scan: operands on different devices")
    rank = x.dim()
    vec = state_axis is not None
    if vec:
        if rank < 2 or initial.dim() < 1:
            raise SxError(SX_E_DIM_001, "element-scan: a vector state needs sequences of rank >= 2")
        n = initial.shape[-1]
        out_shape = tuple(x.shape[:-1]) + (n,)
        if tuple(s.shape[:-1]) != tuple(x.shape[:-1]):
            raise SxError(SX_E_DIM_001, f"element-scan: sequences {tuple(x.shape)} and {tuple(s.shape)} "
                                        "differ outside the state axis")
        x_width, s_width = x.shape[-1], s.shape[-1]
        sa = state_axis
    else:
        out_shape = tuple(x.shape)
        if tuple(s.shape) != out_shape:
            raise SxError(SX_E_DIM_001, f"element-scan: sequences {tuple(x.shape)} and {tuple(s.shape)} differ")
        x_width = s_width = out_shape[-1] if rank else 1
        sa = SX_STATE_SCALAR
    ax = axis + rank if axis < 0 else axis
    if 0 <= ax < rank:
        expect_init = out_shape[:ax] + out_shape[ax + 1:]
        if tuple(initial.shape) != expect_init:
            raise SxError(SX_E_DIM_001, f"element-scan: initial {tuple(initial.shape)} f32 does not match the "
                                        f"sequence shape {out_shape} without axis {axis}")
    lib = load_library()
    out = torch.empty(out_shape, dtype=torch.float32, device=x.device)
    shape_a = i64_array(out_shape)
    ws_bytes = lib.sx_element_scan_workspace_bytes(BODIES[body], rank, shape_a, axis, sa)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device) if ws_bytes else None
    with torch.cuda.device(x.device):
        status = lib.sx_element_scan(
            BODIES[body], rank, shape_a, axis, sa, 1 if reverse else 0,
            initial.data_ptr(), i64_array(initial.stride()),
            x.data_ptr(), x_width, i64_array(x.stride()),
            s.data_ptr(), s_width, i64_array(s.stride()),
            out.data_ptr(), ws.data_ptr() if ws is not None else None, ws_bytes,
            _stream_handle(x.device))
    _check(status)
    return out


def element_scan_backward(body: str, initial: torch.Tensor, sequences, h: torch.Tensor, g: torch.Tensor,
                          axis: int = 0, state_axis=None, reverse: bool = False):
    """Gradients ``(grad_initial, [grad_x, grad_s])`` of a loss through
    ``h = element_scan(body, initial, sequences, axis, state_axis, reverse)``,
    given that call's result ``h`` and the loss's gradient ``g`` with respect
    to it. Each gradient has its tensor's shape; all are f32.
    """
    if body not in BODIES:
        raise SxError(SX_E_UNSUPPORTED, f"element-scan gradient: unknown body {body!r}")
    seqs = list(sequences)
    if len(seqs) != 2:
        raise SxError(SX_E_DIM_001, f"element-scan gradient: the {body} body takes two sequences, got {len(seqs)}")
    x, s = seqs
    _require_no_tangent(initial, x, s, h, g)
    initial, x, s, h, g = _signed(initial, x, s, h, g)
    for name, t in (("initial", initial), ("x", x), ("sequence 2", s), ("h", h), ("g", g)):
        _require_device_tensor(name, t)
        if t.dtype != torch.float32:
            raise SxError(SX_E_DIM_002, f"element-scan gradient: {name} is {t.dtype}; element scans are f32")
    if tuple(g.shape) != tuple(h.shape):
        raise SxError(SX_E_DIM_001, f"element-scan gradient: g {tuple(g.shape)} and h {tuple(h.shape)} differ")
    rank = h.dim()
    vec = state_axis is not None
    x_width = x.shape[-1] if vec else (h.shape[-1] if rank else 1)
    s_width = s.shape[-1] if vec else (h.shape[-1] if rank else 1)
    sa = state_axis if vec else SX_STATE_SCALAR
    initial, h, g = initial.contiguous(), h.contiguous(), g.contiguous()
    lib = load_library()
    shape_a = i64_array(h.shape)
    ws_bytes = lib.sx_element_scan_backward_workspace_bytes(BODIES[body], rank, shape_a, axis, sa, x_width, s_width)
    ws = torch.empty(ws_bytes, dtype=torch.uint8, device=h.device) if ws_bytes else None
    gi, gx, gs = torch.empty_like(initial), torch.empty(tuple(x.shape), dtype=torch.float32, device=h.device), \
        torch.empty(tuple(s.shape), dtype=torch.float32, device=h.device)
    with torch.cuda.device(h.device):
        status = lib.sx_element_scan_backward(
            BODIES[body], rank, shape_a, axis, sa, 1 if reverse else 0, initial.data_ptr(),
            x.data_ptr(), x_width, i64_array(x.stride()), s.data_ptr(), s_width, i64_array(s.stride()),
            h.data_ptr(), g.data_ptr(), gi.data_ptr(), gx.data_ptr(), gs.data_ptr(),
            ws.data_ptr() if ws is not None else None, ws_bytes, _stream_handle(h.device))
    _check(status)
    return gi, [gx, gs]


class _ElementScanFunction(torch.autograd.Function):
    """element_scan with its gradient from the library: saves the inputs and the result."""

    @staticmethod
    def forward(ctx, body, axis, state_axis, reverse, initial, x, s):
        h = _element_scan_forward(body, initial, [x, s], axis, state_axis, reverse)
        ctx.save_for_backward(initial, x, s, h)
        ctx.args = (body, axis, state_axis, reverse)
        return h

    @staticmethod
    def backward(ctx, g):
        initial, x, s, h = ctx.saved_tensors
        body, axis, state_axis, reverse = ctx.args
        gi, (gx, gs) = element_scan_backward(body, initial, [x, s], h, g, axis=axis, state_axis=state_axis,
                                             reverse=reverse)
        return None, None, None, None, gi, gx, gs


def matrix_scan(a: torch.Tensor, b: torch.Tensor, axis: int = 0, reverse: bool = False,
                out_dtype=None, projective: bool = False) -> torch.Tensor:
    """Matrix scan on the GPU: ``h[t] = a[t] @ h[t-1] + b[t]`` along ``axis``.

    ``a`` is ``[..., n, n]`` and ``b`` ``[..., n, m]`` of one dtype (f32 or
    bf16); the leading dims broadcast. The result has the broadcast leading
    shape plus ``[n, m]`` and ``b``'s dtype unless ``out_dtype`` says
    otherwise. Computation is f32. When autograd records (an input requires
    grad), the gradient runs through ``matrix_scan_backward``.
    """
    _require_no_tangent(a, b)
    a, b = _signed(a, b)
    if torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in (a, b)):
        return _MatrixScanFunction.apply(a, b, axis, reverse, out_dtype, projective)
    return _matrix_scan_forward(a, b, axis, reverse, out_dtype, projective)


def _matrix_scan_forward(a, b, axis, reverse, out_dtype, projective) -> torch.Tensor:
    _require_device_tensor("a", a)
    _require_device_tensor("b", b)
    if a.dtype != b.dtype or a.dtype not in _DTYPES:
        raise SxError(SX_E_DIM_002, f"matrix-scan: a is {a.dtype} and b is {b.dtype}; one float dtype "
                                    "(f32 or bf16) is required")
    if a.device != b.device:
        raise SxError(SX_E_UNSUPPORTED, "matrix-scan: operands on different devices")
    out_dtype = b.dtype if out_dtype is None else out_dtype
    if out_dtype not in _DTYPES:
        raise SxError(SX_E_DIM_002, f"matrix-scan: out dtype {out_dtype} is not f32 or bf16")
    lib = load_library()
    # The library reads the two matrix dims row-major; other layouts are copied to that one here.
    if a.dim() >= 2 and not _matrix_dims_contiguous(a):
        a = a.contiguous()
    if b.dim() >= 2 and not _matrix_dims_contiguous(b):
        b = b.contiguous()
    a_shape, b_shape = i64_array(a.shape), i64_array(b.shape)
    oshape = i64_array([0] * 10)
    r = lib.sx_matrix_scan_out_shape(a.dim(), a_shape, b.dim(), b_shape, oshape)
    if r < 0:
        # let the library produce the precise status and message
        _check(lib.sx_matrix_scan(_DTYPES[a.dtype], a.dim(), a_shape, None, None, b.dim(), b_shape, None, None,
                                  axis, 0, 0, _DTYPES[out_dtype], None, None, 0, None))
        raise SxError(SX_E_DIM_001, "matrix-scan: shapes do not fit")
    out = torch.empty(tuple(oshape[:r]), dtype=out_dtype, device=a.device)
    ws_bytes = lib.sx_matrix_scan_workspace_bytes(a.dim(), a_shape, b.dim(), b_shape, axis)
    ws = _matrix_workspace(ws_bytes, a.device)
    with torch.cuda.device(a.device):
        status = lib.sx_matrix_scan(
            _DTYPES[a.dtype], a.dim(), a_shape, i64_array(a.stride()), a.data_ptr(),
            b.dim(), b_shape, i64_array(b.stride()), b.data_ptr(),
            axis, 1 if reverse else 0, 1 if projective else 0, _DTYPES[out_dtype], out.data_ptr(),
            ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
            _stream_handle(a.device))
    _check(status)
    return out


def linear_scan(a, b, axis: int = 0, reverse: bool = False, out_dtype=None) -> torch.Tensor:
    """Linear scan on the GPU: ``h[t] = a[t] * h[t-1] + b[t]`` along ``axis`` from ``h = 0``.

    Matrix-scan over one-by-one matrices. ``a`` and ``b`` are tensors of one
    float dtype (f32 or bf16) or numbers, broadcast to one shape (at least one
    of them a tensor of rank >= 1); a number takes the tensor's dtype. The
    result has the broadcast shape and that dtype unless ``out_dtype`` says
    otherwise. Computation is f32.
    """
    _require_no_tangent(a, b)
    a, b = _signed(a, b)
    ta = a if isinstance(a, torch.Tensor) else None
    tb = b if isinstance(b, torch.Tensor) else None
    if ta is None and tb is None:
        raise SxError(SX_E_DIM_001, "linear-scan: a and b are both numbers; there is no axis to scan along")
    ref = tb if tb is not None else ta
    _require_device_tensor("a" if ref is ta else "b", ref)
    # A number becomes a rank-0 tensor on the device (a fill kernel, no host copy).
    if ta is None:
        ta = torch.full((), float(a), dtype=ref.dtype, device=ref.device)
    if tb is None:
        tb = torch.full((), float(b), dtype=ref.dtype, device=ref.device)
    _require_device_tensor("a", ta)
    _require_device_tensor("b", tb)
    if ta.dtype != tb.dtype or ta.dtype not in _DTYPES:
        raise SxError(SX_E_DIM_002, f"linear-scan: a is {ta.dtype} and b is {tb.dtype}; one float dtype "
                                    "(f32 or bf16) is required")
    if ta.device != tb.device:
        raise SxError(SX_E_UNSUPPORTED, "linear-scan: operands on different devices")
    out_dtype = tb.dtype if out_dtype is None else out_dtype
    if out_dtype not in _DTYPES:
        raise SxError(SX_E_DIM_002, f"linear-scan: out dtype {out_dtype} is not f32 or bf16")
    lib = load_library()
    a_shape, b_shape = i64_array(ta.shape), i64_array(tb.shape)
    oshape = i64_array([0] * 8)
    r = lib.sx_linear_scan_out_shape(ta.dim(), a_shape, tb.dim(), b_shape, oshape)
    if r < 0:
        # let the library produce the precise status and message
        _check(lib.sx_linear_scan(_DTYPES[ta.dtype], ta.dim(), a_shape, None, None, tb.dim(), b_shape, None, None,
                                  axis, 0, _DTYPES[out_dtype], None, None))
        raise SxError(SX_E_DIM_001, "linear-scan: shapes do not fit")
    out = torch.empty(tuple(oshape[:r]), dtype=out_dtype, device=ref.device)
    with torch.cuda.device(ref.device):
        status = lib.sx_linear_scan(
            _DTYPES[ta.dtype], ta.dim(), a_shape, i64_array(ta.stride()), ta.data_ptr(),
            tb.dim(), b_shape, i64_array(tb.stride()), tb.data_ptr(),
            axis, 1 if reverse else 0, _DTYPES[out_dtype], out.data_ptr(), _stream_handle(ref.device))
    _check(status)
    return out


def table_scan(table: torch.Tensor, symbols: torch.Tensor, axis: int = -1, start: int = 0) -> torch.Tensor:
    """Deterministic automaton on the GPU: along ``axis``, reading a symbol
    moves the state to ``table[previous, symbol]``, starting at ``start``. ``table`` is
    ``[states, symbols]``, both int32; returns every state (int32, symbols'
    shape). Out-of-range symbols and reached entries are clamped into range."""
    _require_device_tensor("table", table)
    _require_device_tensor("symbols", symbols)
    if table.dtype != torch.int32 or symbols.dtype != torch.int32:
        raise SxError(SX_E_DIM_002, f"table-scan: table is {table.dtype} and symbols {symbols.dtype}; both must be "
                                    ":i32")
    if table.dim() != 2:
        raise SxError(SX_E_DIM_001, f"table-scan: the table must be [states symbols], got {tuple(table.shape)}")
    if table.device != symbols.device:
        raise SxError(SX_E_UNSUPPORTED, "table-scan: operands on different devices")
    table = table.contiguous()
    lib = load_library()
    out = torch.empty(tuple(symbols.shape), dtype=torch.int32, device=symbols.device)
    with torch.cuda.device(symbols.device):
        status = lib.sx_table_scan(int(table.shape[0]), int(table.shape[1]), table.data_ptr(), symbols.dim(),
                                   i64_array(symbols.shape), i64_array(symbols.stride()), symbols.data_ptr(),
                                   axis, int(start), out.data_ptr(), _stream_handle(symbols.device))
    _check(status)
    return out


def cumsum(x: torch.Tensor, axis: int = 0, reverse: bool = False, out_dtype=None) -> torch.Tensor:
    """Running sum along ``axis`` (from the end when ``reverse``): linear-scan with ``a = 1``."""
    return linear_scan(1.0, x, axis=axis, reverse=reverse, out_dtype=out_dtype)


def matrix_scan_backward(a: torch.Tensor, b_shape, h: torch.Tensor, g: torch.Tensor, axis: int = 0,
                         reverse: bool = False, grad_dtype=None):
    """Gradients ``(grad_a, grad_b)`` of a loss through ``h = matrix_scan(a, b, axis, reverse)``.

    ``h`` is that call's result and ``g`` the loss's gradient with respect to
    it; ``a``, ``h`` and ``g`` share one dtype (f32 or bf16). ``grad_a`` and
    ``grad_b`` have the shapes of ``a`` and ``b`` (summed over broadcast dims)
    and ``grad_dtype`` (default: a's dtype). The adjoint is computed in f32.
    """
    _require_no_tangent(a, h, g)
    a, h, g = _signed(a, h, g)
    for name, t in (("a", a), ("h", h), ("g", g)):
        _require_device_tensor(name, t)
    if not (a.dtype == h.dtype == g.dtype) or a.dtype not in _DTYPES:
        raise SxError(SX_E_DIM_002, f"matrix-scan gradient: a is {a.dtype}, h {h.dtype} and g {g.dtype}; one float "
                                    "dtype (f32 or bf16) is required")
    if not (a.device == h.device == g.device):
        raise SxError(SX_E_UNSUPPORTED, "matrix-scan gradient: operands on different devices")
    grad_dtype = a.dtype if grad_dtype is None else grad_dtype
    if grad_dtype not in _DTYPES:
        raise SxError(SX_E_DIM_002, f"matrix-scan gradient: grad dtype {grad_dtype} is not f32 or bf16")
    b_shape = tuple(int(d) for d in b_shape)
    if tuple(g.shape) != tuple(h.shape):
        raise SxError(SX_E_DIM_001, f"matrix-scan gradient: g {tuple(g.shape)} and h {tuple(h.shape)} differ")
    lib = load_library()
    if a.dim() >= 2 and not _matrix_dims_contiguous(a):
        a = a.contiguous()
    if g.dim() >= 2 and not _matrix_dims_contiguous(g):
        g = g.contiguous()
    h = h.contiguous()
    a_shape, bs = i64_array(a.shape), i64_array(b_shape)
    ws_bytes = lib.sx_matrix_scan_backward_workspace_bytes(a.dim(), a_shape, len(b_shape), bs, axis,
                                                           _DTYPES[grad_dtype])
    ws = _matrix_workspace(ws_bytes, a.device)
    grad_a = torch.empty(tuple(a.shape), dtype=grad_dtype, device=a.device)
    grad_b = torch.empty(b_shape, dtype=grad_dtype, device=a.device)
    with torch.cuda.device(a.device):
        status = lib.sx_matrix_scan_backward(
            _DTYPES[a.dtype], a.dim(), a_shape, i64_array(a.stride()), a.data_ptr(),
            len(b_shape), bs, h.data_ptr(), i64_array(g.stride()), g.data_ptr(),
            axis, 1 if reverse else 0, _DTYPES[grad_dtype], grad_a.data_ptr(), grad_b.data_ptr(),
            ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
            _stream_handle(a.device))
    _check(status)
    return grad_a, grad_b


class _MatrixScanFunction(torch.autograd.Function):
    """matrix_scan with its gradient from the library: saves a and the result."""

    @staticmethod
    def forward(ctx, a, b, axis, reverse, out_dtype, projective):
        h = _matrix_scan_forward(a, b, axis, reverse, out_dtype, projective)
        ctx.save_for_backward(a, h)
        ctx.b_shape, ctx.b_dtype, ctx.axis, ctx.reverse = tuple(b.shape), b.dtype, axis, reverse
        ctx.projective = projective
        return h

    @staticmethod
    def backward(ctx, g):
        if ctx.projective:  # "Tensor operations", matrix-scan: the :projective result has no gradient
            raise SxError(SX_E_UNSUPPORTED, "matrix-scan: :projective true has no gradient; differentiating "
                                            "through it is an error")
        a, h = ctx.saved_tensors
        g = g.to(h.dtype)
        # The gradient scan takes a, h and g of one dtype. With an out_dtype other than the
        # operands' one, widen to f32 (exact): a for bf16 operands with an f32 result; h and g
        # for f32 operands with a bf16 result (grad_a then uses the result as rounded to bf16,
        # a relative change of at most 2^-9 per element). Gradients take the operands' dtype.
        if a.dtype != h.dtype:
            if h.dtype == torch.float32:
                a = a.float()
            else:
                h, g = h.float(), g.float()
        grad_a, grad_b = matrix_scan_backward(a, ctx.b_shape, h, g, axis=ctx.axis, reverse=ctx.reverse,
                                              grad_dtype=ctx.b_dtype)
        return grad_a, grad_b, None, None, None, None


def _matrix_dims_contiguous(t: torch.Tensor) -> bool:
    rows, cols = t.shape[-2], t.shape[-1]
    st = t.stride()
    return (cols <= 1 or st[-1] == 1) and (rows <= 1 or cols == 0 or st[-2] == cols)


# ---------------------------------------------------------------- linear attention
#
# A single token's call takes the GPU a few microseconds, so what the binding
# does on the host counts. Calls whose tensors are as the library takes them go
# the short way (csrc/py_marshal.cpp), which answers None to any other; those go
# the long way below, which checks everything by name, converts, records for
# autograd and switches devices.

MARSHAL_PATH = os.path.join(HERE, "_sx_marshal.so")


class _LongWay:
    """In the place of the short way where that is not built or does not load: every call goes the long one."""

    def _none(*args):
        return None

    decay_attention = decay_attention_backward = decay_attention_step = _none
    head_norm_rotate = head_norm_rotate_backward = _none


_marshal = None


def _load_marshal():
    """The short way, bound to the loaded library."""
    global _marshal
    from importlib import machinery, util

    lib = load_library()
    loader = machinery.ExtensionFileLoader("_sx_marshal", MARSHAL_PATH)
    try:
        module = util.module_from_spec(util.spec_from_loader("_sx_marshal", loader))
        loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"{MARSHAL_PATH} is not built or does not load ({e}): linear-attention calls cost more on the "
                      "host; run `python -m scan_primitives_amd.build_lib`", RuntimeWarning, stacklevel=3)
        _marshal = _LongWay()
        return _marshal
    names = ("sx_decay_attention", "sx_decay_attention_workspace_bytes", "sx_decay_attention_backward",
             "sx_decay_attention_backward_workspace_bytes", "sx_decay_attention_step", "sx_head_norm_rotate",
             "sx_head_norm_rotate_backward", "sx_head_norm_rotate_backward_workspace_bytes")
    module.bind(tuple(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in names),
                torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
    _marshal = module
    return module


def _done(answer):
    """The results of the short way; its status raises."""
    if type(answer) is int:
        _check(answer)
    return answer


@functools.lru_cache(maxsize=4096)
def _i64(values: tuple) -> ctypes.Array:
    """The values as an array the library reads (never one it writes)."""
    return i64_array(values)


def _device_index(op: str, names, tensors, optional=()) -> int:
    """The index of the one device all tensors are on. `optional` (name, tensor) pairs may be None."""
    index = -1
    for name, t in zip(names, tensors):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            _require_device_tensor(f"{op}: {name}", t)
        at = t.get_device()
        if index >= 0 and at != index:
            raise SxError(SX_E_UNSUPPORTED, f"{op}: operands on different devices")
        index = at
    for name, t in optional:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            _require_device_tensor(f"{op}: {name}", t)
        if t.get_device() != index:
            raise SxError(SX_E_UNSUPPORTED, f"{op}: operands on different devices")
    return index


def _require_dtype(op: str, names, tensors) -> int:
    """One float dtype (f32 or bf16) for all; its code."""
    first = tensors[0].dtype
    code = _DTYPES.get(first)
    if code is not None:
        for t in tensors:
            if t.dtype is not first:
                code = None
    if code is None:
        said = ", ".join(f"{name} is {t.dtype}" for name, t in zip(names, tensors))
        raise SxError(SX_E_DIM_002, f"{op}: {said}; one float dtype (f32 or bf16) is required")
    return code


def _require(op: str, name: str, t, dtype, shape) -> None:
    """An optional operand of a fixed dtype and shape."""
    if t is None:
        return
    if t.dtype is not dtype:
        raise SxError(SX_E_DIM_002, f"{op}: {name} is {t.dtype}, {dtype} is required")
    if shape is not None and t.shape != shape:
        raise SxError(SX_E_DIM_001, f"{op}: {name} is {tuple(t.shape)}, {tuple(shape)} is required")


def _args(t: torch.Tensor):
    return _i64(t.shape), _i64(t.stride()), t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _contiguous(t):
    return None if t is None else t.contiguous()


def _records(*tensors) -> bool:
    """Whether autograd has to see the call."""
    if torch.is_grad_enabled():
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.requires_grad:
                return True
    return False


def _enqueue(index: int, entry, *args) -> None:
    """Call a library entry with the current stream of device `index` as its last argument."""
    if torch.cuda.current_device() == index:
        _check(entry(*args, _raw_stream(index)))
    else:
        with torch.cuda.device(index):
            _check(entry(*args, _raw_stream(index)))


def _raw_stream(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _decay_operands(op, q, k, v, log_decay, token_dims, more, optional):
    """Checks what the C library cannot see (types, devices, optional operands); the dtype code, H and the device."""
    index = _device_index(op, ("q", "k", "v", "log_decay", *(n for n, _ in more)),
                          (q, k, v, log_decay, *(t for _, t in more)), optional)
    code = _require_dtype(op, ("q", "k", "v"), (q, k, v))
    rank = 2 + token_dims
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() != rank:
            raise SxError(SX_E_DIM_001, f"{op}: {name} {tuple(t.shape)} must have {rank} dims")
    if log_decay.dtype is not torch.float32:
        raise SxError(SX_E_DIM_002, f"{op}: log_decay is {log_decay.dtype}, torch.float32 is required")
    if log_decay.dim() not in (1, 1 + token_dims):
        raise SxError(SX_E_DIM_001, f"{op}: log_decay {tuple(log_decay.shape)} must be [heads] or have a value a token")
    return code, log_decay.shape[-1], index


@functools.lru_cache(maxsize=1024)
def _decay_workspace_bytes(code, q_shape, v_shape, heads):
    return load_library().sx_decay_attention_workspace_bytes(code, _i64(q_shape), _i64(v_shape), heads)


@functools.lru_cache(maxsize=1024)
def _decay_backward_workspace_bytes(code, q_shape, k_shape, v_shape, heads):
    return load_library().sx_decay_attention_backward_workspace_bytes(code, _i64(q_shape), _i64(k_shape),
                                                                      _i64(v_shape), heads)


def decay_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, initial=None,
                    lengths=None, scale: float = 1.0, return_state: bool = False):
    """Linear attention with a decay for each head, on the GPU:
    ``S[t] = exp(log_decay[t]) S[t-1] + k[t] v[t]^T`` and ``out[t] = scale * S[t]^T q[t]``.

    ``q`` and ``k`` are ``[B, T, heads, dk]`` and ``v`` ``[B, T, heads, dv]``, of one
    dtype (f32 or bf16) and any strides; ``log_decay`` is f32, ``[H]`` or
    ``[B, T, H]`` (``-inf`` cuts off what came before). The heads of q, k and v
    each divide H, and are shared by H / heads heads. ``initial`` is the state
    before the first token (f32 ``[B, H, dk, dv]``, zero when None); tokens of
    row b from ``lengths[b]`` (int32 ``[B]``) on do not exist. Returns out
    ``[B, T, H, dv]``, and the last state too when ``return_state``. When autograd
    records, the gradient runs through ``decay_attention_backward``.
    """
    got = (_marshal or _load_marshal()).decay_attention(q, k, v, log_decay, initial, lengths, scale, return_state)
    if got is not None:
        return _done(got) if return_state else _done(got)[0]
    _require_no_tangent(q, k, v, log_decay, initial)
    q, k, v, log_decay, initial = _signed(q, k, v, log_decay, initial)
    if _records(q, k, v, log_decay, initial):
        out, state = _DecayAttentionFunction.apply(q, k, v, log_decay, initial, lengths, scale, return_state)
    else:
        out, state = _decay_attention_forward(q, k, v, log_decay, initial, lengths, scale, return_state)
    return (out, state) if return_state else out


def _decay_attention_forward(q, k, v, log_decay, initial, lengths, scale, return_state):
    op = "decay-attention"
    code, heads, index = _decay_operands(op, q, k, v, log_decay, 2, (), (("initial", initial), ("lengths", lengths)))
    b, t, _, dk = q.shape
    dv = v.shape[-1]
    _require(op, "initial", initial, torch.float32, (b, heads, dk, dv))
    _require(op, "lengths", lengths, torch.int32, (b,))
    initial, lengths = _contiguous(initial), _contiguous(lengths)
    dev = q.device
    out = torch.empty((b, t, heads, dv), dtype=q.dtype, device=dev)
    state = torch.empty((b, heads, dk, dv), dtype=torch.float32, device=dev) if return_state else None
    nbytes = _decay_workspace_bytes(code, q.shape, v.shape, heads)
    ws = _workspace(nbytes, dev)
    _enqueue(index, load_library().sx_decay_attention, code, *_args(q), *_args(k), *_args(v), log_decay.dim(),
             *_args(log_decay), _ptr(initial), _ptr(lengths), float(scale), out.data_ptr(), _ptr(state), _ptr(ws),
             nbytes)
    return out, state


def decay_attention_backward(q, k, v, log_decay, grad_out, initial=None, lengths=None, scale: float = 1.0,
                             grad_state=None):
    """Gradients ``(grad_q, grad_k, grad_v, grad_log_decay, grad_initial)`` of a loss through
    ``decay_attention(q, k, v, log_decay, initial, lengths, scale)``.

    ``grad_out`` is the loss's gradient with respect to out (its shape, q's
    dtype), ``grad_state`` the one with respect to the last state (f32, or None).
    Each gradient has its operand's shape and dtype; ``grad_initial`` is the
    gradient of the state before the first token, also when that was zero.
    """
    got = (_marshal or _load_marshal()).decay_attention_backward(q, k, v, log_decay, grad_out, initial, lengths, scale,
                                                                 grad_state)
    if got is not None:
        return _done(got)
    _require_no_tangent(q, k, v, log_decay, grad_out, initial, grad_state)
    q, k, v, log_decay, grad_out, initial, grad_state = _signed(q, k, v, log_decay, grad_out, initial, grad_state)
    op = "decay-attention gradient"
    code, heads, index = _decay_operands(op, q, k, v, log_decay, 2, (("grad_out", grad_out),),
                                         (("initial", initial), ("lengths", lengths), ("grad_state", grad_state)))
    b, t, _, dk = q.shape
    dv = v.shape[-1]
    state_shape = (b, heads, dk, dv)
    _require(op, "initial", initial, torch.float32, state_shape)
    _require(op, "lengths", lengths, torch.int32, (b,))
    _require(op, "grad_out", grad_out, q.dtype, (b, t, heads, dv))
    _require(op, "grad_state", grad_state, torch.float32, state_shape)
    initial, lengths, grad_state = _contiguous(initial), _contiguous(lengths), _contiguous(grad_state)
    dev = q.device
    gq, gk, gv = (torch.empty(x.shape, dtype=x.dtype, device=dev) for x in (q, k, v))
    gg = torch.empty(log_decay.shape, dtype=torch.float32, device=dev)
    gi = torch.empty(state_shape, dtype=torch.float32, device=dev)
    nbytes = _decay_backward_workspace_bytes(code, q.shape, k.shape, v.shape, heads)
    ws = _workspace(nbytes, dev)
    _enqueue(index, load_library().sx_decay_attention_backward, code, *_args(q), *_args(k), *_args(v),
             log_decay.dim(), *_args(log_decay), _i64(grad_out.stride()), grad_out.data_ptr(), _ptr(grad_state),
             _ptr(initial), _ptr(lengths), float(scale), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(), gg.data_ptr(),
             gi.data_ptr(), _ptr(ws), nbytes)
    return gq, gk, gv, gg, gi


class _DecayAttentionFunction(torch.autograd.Function):
    """decay_attention with its gradient from the library: saves the inputs."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, initial, lengths, scale, return_state):
        out, state = _decay_attention_forward(q, k, v, log_decay, initial, lengths, scale, return_state)
        ctx.save_for_backward(q, k, v, log_decay, initial, lengths)
        ctx.scale = scale
        ctx.set_materialize_grads(False)
        return out, state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out, grad_state):
        q, k, v, log_decay, initial, lengths = ctx.saved_tensors
        if grad_out is None:
            grad_out = torch.zeros((1, 1, 1, 1), dtype=q.dtype, device=q.device).expand(
                q.shape[0], q.shape[1], log_decay.shape[-1], v.shape[-1])
        gq, gk, gv, gg, gi = decay_attention_backward(q, k, v, log_decay, grad_out, initial=initial, lengths=lengths,
                                                      scale=ctx.scale, grad_state=grad_state)
        return gq, gk, gv, gg, gi if initial is not None else None, None, None, None


def decay_attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                         state: torch.Tensor, slots=None, scale: float = 1.0) -> torch.Tensor:
    """One token of every request of a batch: ``S = exp(log_decay) S + k v^T``, ``out = scale * S^T q``.

    ``q`` and ``k`` are ``[B, heads, dk]``, ``v`` ``[B, heads, dv]``, ``log_decay``
    ``[H]`` or ``[B, H]``. ``state`` (f32 ``[pool, H, dk, dv]``) is updated in
    place; row b uses state ``slots[b]`` (int32 ``[B]``; state b when None). A row
    whose slot lies outside the pool is idle: zero out, no state changed; two
    rows of one slot race. Returns out ``[B, H, dv]``. No gradient is recorded,
    so a ``state`` that autograd records is refused; one that it has saved is
    marked as modified in place.
    """
    got = (_marshal or _load_marshal()).decay_attention_step(q, k, v, log_decay, state, slots, scale)
    if got is not None:
        return _done(got)[0]
    _require_no_tangent(q, k, v, log_decay, state)
    q, k, v, log_decay = _signed(q, k, v, log_decay)
    op = "decay-attention step"
    code, heads, index = _decay_operands(op, q, k, v, log_decay, 1, (("state", state),), (("slots", slots),))
    if state.is_neg():
        raise SxError(SX_E_UNSUPPORTED, f"{op}: state is a lazily negated view, which cannot be written in place")
    if _records(state):
        raise SxError(SX_E_UNSUPPORTED, f"{op}: state requires grad, and a step records none; detach it, or call the "
                                        "step under torch.no_grad()")
    b, _, dk = q.shape
    dv = v.shape[-1]
    if state.dim() != 4 or state.shape[1:] != (heads, dk, dv):
        raise SxError(SX_E_DIM_001, f"{op}: state is {tuple(state.shape)}, [states, {heads}, {dk}, {dv}] is required")
    _require(op, "state", state, torch.float32, None)
    _require(op, "slots", slots, torch.int32, (b,))
    slots = _contiguous(slots)
    out = torch.empty((b, heads, dv), dtype=q.dtype, device=q.device)
    _enqueue(index, load_library().sx_decay_attention_step, code, *_args(q), *_args(k), *_args(v), log_decay.dim(),
             *_args(log_decay), state.shape[0], _i64(state.stride()), state.data_ptr(), _ptr(slots), float(scale),
             out.data_ptr())
    torch.autograd.graph.increment_version(state)
    return out


def rotation_turns(rotated: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """Turns (of 2 pi) a position of each pair of ``rotated`` components: ``base^(-2 i / rotated) / (2 pi)``,
    f64 ``[rotated / 2]``, for ``head_norm_rotate``."""
    if rotated < 0 or rotated % 2 != 0:
        raise SxError(SX_E_DIM_001, f"rotation_turns: {rotated} components do not make pairs")
    i = torch.arange(rotated // 2, dtype=torch.float64, device=device)
    return float(base) ** (-2.0 * i / max(rotated, 1)) / (2.0 * math.pi)


def _rotate_operands(op, q, k, positions, turns, q_weight, k_weight, more=()):
    index = _device_index(op, ("q", "k", "positions", "turns", *(n for n, _ in more)),
                          (q, k, positions, turns, *(t for _, t in more)),
                          (("q_weight", q_weight), ("k_weight", k_weight)))
    code = _require_dtype(op, ("q", "k"), (q, k))
    for name, t in (("q", q), ("k", k)):
        if t.dim() != 4:
            raise SxError(SX_E_DIM_001, f"{op}: {name} {tuple(t.shape)} must be [batch, tokens, heads, width]")
    b, t, _, d = q.shape
    if positions.dtype is not torch.int64 and positions.dtype is not torch.int32:
        raise SxError(SX_E_DIM_002, f"{op}: positions are {positions.dtype}, int32 or int64 is required")
    if positions.shape == (t,):
        positions = positions[None].expand(b, t)
    _require(op, "positions", positions, positions.dtype, (b, t))
    if turns.dim() != 1:
        raise SxError(SX_E_DIM_001, f"{op}: turns {tuple(turns.shape)} must have one dim")
    _require(op, "turns", turns, torch.float64, None)
    _require(op, "q_weight", q_weight, torch.float32, (d,))
    _require(op, "k_weight", k_weight, torch.float32, (d,))
    return code, index, positions, turns.contiguous(), _contiguous(q_weight), _contiguous(k_weight)


@functools.lru_cache(maxsize=1024)
def _rotate_workspace_bytes(q_shape, k_shape):
    return load_library().sx_head_norm_rotate_backward_workspace_bytes(_i64(q_shape), _i64(k_shape))


def head_norm_rotate(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, turns: torch.Tensor, q_weight=None,
                     k_weight=None, eps: float = 1e-6, neighbours: bool = False):
    """The root-mean-square norm of each head of ``q`` and ``k`` and their rotation by position, in one pass.

    ``q`` and ``k`` are ``[B, T, heads, d]`` (f32 or bf16, any strides),
    ``positions`` int32 or int64 ``[B, T]`` or ``[T]``, ``turns`` f64 (see
    ``rotation_turns``): the first ``2 * len(turns)`` components turn in pairs
    ``(i, i + len(turns))``, or ``(2 i, 2 i + 1)`` when ``neighbours``. The weights
    are f32 ``[d]`` (ones when None). Returns the two results, contiguous, in q's
    dtype. When autograd records, the gradient runs through
    ``head_norm_rotate_backward``.
    """
    got = (_marshal or _load_marshal()).head_norm_rotate(q, k, positions, turns, q_weight, k_weight, eps, neighbours)
    if got is not None:
        return _done(got)
    _require_no_tangent(q, k, q_weight, k_weight)
    q, k, turns, q_weight, k_weight = _signed(q, k, turns, q_weight, k_weight)
    if _records(q, k, q_weight, k_weight):
        return _HeadNormRotateFunction.apply(q, k, positions, turns, q_weight, k_weight, eps, neighbours)
    return _head_norm_rotate_forward(q, k, positions, turns, q_weight, k_weight, eps, neighbours)


def _head_norm_rotate_forward(q, k, positions, turns, q_weight, k_weight, eps, neighbours):
    op = "head-norm-rotate"
    code, index, positions, turns, q_weight, k_weight = _rotate_operands(op, q, k, positions, turns, q_weight, k_weight)
    dev = q.device
    oq, ok = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=k.dtype, device=dev)
    _enqueue(index, load_library().sx_head_norm_rotate, code, *_args(q), *_args(k),
             1 if positions.dtype is torch.int64 else 0, _i64(positions.stride()), positions.data_ptr(),
             2 * turns.shape[0], turns.data_ptr(), _ptr(q_weight), _ptr(k_weight), float(eps), 1 if neighbours else 0,
             oq.data_ptr(), ok.data_ptr())
    return oq, ok


def head_norm_rotate_backward(q, k, positions, turns, grad_out_q, grad_out_k, q_weight=None, k_weight=None,
                              eps: float = 1e-6, neighbours: bool = False):
    """Gradients ``(grad_q, grad_k, grad_q_weight, grad_k_weight)`` of a loss through
    ``head_norm_rotate(q, k, positions, turns, q_weight, k_weight, eps, neighbours)``, given its gradients with
    respect to the two results (their shapes, q's dtype). A weight that is None has None for its gradient."""
    got = (_marshal or _load_marshal()).head_norm_rotate_backward(q, k, positions, turns, grad_out_q, grad_out_k,
                                                                  q_weight, k_weight, eps, neighbours)
    if got is not None:
        return _done(got)
    _require_no_tangent(q, k, grad_out_q, grad_out_k, q_weight, k_weight)
    q, k, turns, grad_out_q, grad_out_k, q_weight, k_weight = _signed(q, k, turns, grad_out_q, grad_out_k, q_weight,
                                                                      k_weight)
    op = "head-norm-rotate gradient"
    code, index, positions, turns, q_weight, k_weight = _rotate_operands(
        op, q, k, positions, turns, q_weight, k_weight, (("grad_out_q", grad_out_q), ("grad_out_k", grad_out_k)))
    _require(op, "grad_out_q", grad_out_q, q.dtype, q.shape)
    _require(op, "grad_out_k", grad_out_k, k.dtype, k.shape)
    dev = q.device
    gq, gk = torch.empty(q.shape, dtype=q.dtype, device=dev), torch.empty(k.shape, dtype=k.dtype, device=dev)
    gqw, gkw = (None if w is None else torch.empty(w.shape, dtype=w.dtype, device=dev) for w in (q_weight, k_weight))
    nbytes = 0 if gqw is None and gkw is None else _rotate_workspace_bytes(q.shape, k.shape)
    ws = _workspace(nbytes, dev)
    _enqueue(index, load_library().sx_head_norm_rotate_backward, code, *_args(q), *_args(k),
             1 if positions.dtype is torch.int64 else 0, _i64(positions.stride()), positions.data_ptr(),
             2 * turns.shape[0], turns.data_ptr(), _i64(grad_out_q.stride()), grad_out_q.data_ptr(),
             _i64(grad_out_k.stride()), grad_out_k.data_ptr(), _ptr(q_weight), _ptr(k_weight), float(eps),
             1 if neighbours else 0, gq.data_ptr(), gk.data_ptr(), _ptr(gqw), _ptr(gkw), _ptr(ws), nbytes)
    return gq, gk, gqw, gkw


class _HeadNormRotateFunction(torch.autograd.Function):
    """head_norm_rotate with its gradient from the library: saves the inputs."""

    @staticmethod
    def forward(ctx, q, k, positions, turns, q_weight, k_weight, eps, neighbours):
        ctx.save_for_backward(q, k, positions, turns, q_weight, k_weight)
        ctx.eps, ctx.neighbours = eps, neighbours
        return _head_norm_rotate_forward(q, k, positions, turns, q_weight, k_weight, eps, neighbours)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_out_q, grad_out_k):
        q, k, positions, turns, q_weight, k_weight = ctx.saved_tensors
        gq, gk, gqw, gkw = head_norm_rotate_backward(q, k, positions, turns, grad_out_q, grad_out_k, q_weight=q_weight,
                                                     k_weight=k_weight, eps=ctx.eps, neighbours=ctx.neighbours)
        return gq, gk, None, None, gqw, gkw, None, None
