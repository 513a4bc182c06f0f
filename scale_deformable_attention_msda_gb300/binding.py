"""Thin Python binding of libmsda's C ABI (include/msda.h), same names.

Argument marshalling only: every step of the operator runs in libmsda's CUDA
kernels. Tensors must be CUDA, contiguous and of one float dtype; the calls are
enqueued on the current torch CUDA stream and return without synchronising.
There is no CPU path: if libmsda.so is missing or the tensors are not on a GPU,
the call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch
from torch.autograd import forward_ad

from . import build as _build

MSDA_F32, MSDA_BF16, MSDA_F16, MSDA_F64 = 0, 1, 2, 3
MSDA_ACC_NATIVE, MSDA_ACC_FP32_BUFFER, MSDA_ACC_AUTO, MSDA_ACC_FP16_BUFFER = 0, 1, 2, 3
_DTYPES = {torch.float32: MSDA_F32, torch.bfloat16: MSDA_BF16, torch.float16: MSDA_F16,
           torch.float64: MSDA_F64}
STATUS = {0: "MSDA_OK", 1: "MSDA_ERR_NULL", 2: "MSDA_ERR_SHAPE", 3: "MSDA_ERR_DTYPE",
          4: "MSDA_ERR_ALIGN", 5: "MSDA_ERR_WORKSPACE", 6: "MSDA_ERR_CUDA",
          7: "MSDA_ERR_DEVICE_BOUNDS", 8: "MSDA_ERR_DEVICE_WAIT"}
MSDA_ERR_DEVICE_BOUNDS, MSDA_ERR_DEVICE_WAIT = 7, 8
EXPORTED = ("msda_forward", "msda_backward_workspace_bytes", "msda_backward",
            "msda_backward_zero", "msda_backward_accumulate", "msda_backward_finish",
            "msda_backward_static_workspace", "msda_forward_softmax", "msda_backward_softmax",
            "msda_debug_corners", "msda_checked_build", "msda_device_check",
            "msda_debug_bounds_self_test", "msda_set_sample_split", "msda_status_string",
            "msda_version", "msda_layer_norm_forward", "msda_layer_norm_backward_workspace_bytes",
            "msda_layer_norm_backward", "msda_grad_norm_workspace_bytes", "msda_grad_norm",
            "msda_clip_grad_norm", "msda_attention_forward_workspace_bytes",
            "msda_attention_backward_workspace_bytes", "msda_attention_forward",
            "msda_attention_backward", "msda_dropout", "msda_dropout_next")


class msda_dims_t(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("B", "S", "Q", "M", "D", "L", "K")]


class msda_norm_dims_t(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("C", ctypes.c_int64)]


class msda_grad_list_t(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("grads", ctypes.c_void_p), ("outs", ctypes.c_void_p),
                ("sizes", ctypes.c_void_p), ("dtypes", ctypes.c_void_p),
                ("out_dtypes", ctypes.c_void_p)]


class msda_attention_dims_t(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "Q", "S", "M", "N", "D")] +
                [(n, ctypes.c_int64 * 3) for n in ("q_stride", "k_stride", "v_stride")] +
                [("mask_stride", ctypes.c_int64 * 4)])


class MSDAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} "
                         f"({lib().msda_status_string(status).decode()})")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIBRARY


def load(path: str | None = None):
    """Open libmsda.so and declare its entry points (no CUDA call is made)."""
    path = path or library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libmsda.so not found at {path}; build it with "
                           "`python -c 'import __graft_entry__ as g; g.build()'`")
    so = ctypes.CDLL(path)
    vp, i32p = ctypes.c_void_p, ctypes.c_void_p
    dims = ctypes.POINTER(msda_dims_t)
    so.msda_forward.argtypes = [vp, vp, vp, vp, vp, i32p, vp, dims, ctypes.c_int, vp]
    so.msda_forward.restype = ctypes.c_int
    so.msda_backward_workspace_bytes.argtypes = [dims, ctypes.c_int, ctypes.c_int]
    so.msda_backward_workspace_bytes.restype = ctypes.c_size_t
    so.msda_backward.argtypes = [vp, vp, vp, vp, vp, i32p, vp, vp, vp, vp, vp, ctypes.c_size_t,
                                 ctypes.c_int, dims, ctypes.c_int, vp]
    so.msda_backward.restype = ctypes.c_int
    so.msda_forward_softmax.argtypes = so.msda_forward.argtypes
    so.msda_forward_softmax.restype = ctypes.c_int
    so.msda_backward_softmax.argtypes = so.msda_backward.argtypes
    so.msda_backward_softmax.restype = ctypes.c_int
    so.msda_backward_accumulate.argtypes = so.msda_backward.argtypes
    so.msda_backward_accumulate.restype = ctypes.c_int
    so.msda_backward_zero.argtypes = [vp, vp, ctypes.c_size_t, ctypes.c_int, dims, ctypes.c_int, vp]
    so.msda_backward_zero.restype = ctypes.c_int
    so.msda_backward_finish.argtypes = [vp, ctypes.c_size_t, vp, ctypes.c_int, dims, ctypes.c_int,
                                        vp]
    so.msda_backward_finish.restype = ctypes.c_int
    so.msda_backward_static_workspace.argtypes = [vp, vp, vp, vp, vp, i32p, vp, vp, vp, vp, dims,
                                                  ctypes.c_int, vp]
    so.msda_backward_static_workspace.restype = ctypes.c_int
    so.msda_debug_corners.argtypes = [vp, vp, vp, vp, dims, ctypes.c_int, vp]
    so.msda_debug_corners.restype = ctypes.c_int
    so.msda_checked_build.argtypes = []
    so.msda_checked_build.restype = ctypes.c_int
    so.msda_device_check.argtypes = [vp]
    so.msda_device_check.restype = ctypes.c_int
    so.msda_debug_bounds_self_test.argtypes = [vp]
    so.msda_debug_bounds_self_test.restype = ctypes.c_int
    so.msda_set_sample_split.argtypes = [ctypes.c_int]
    so.msda_set_sample_split.restype = ctypes.c_int
    so.msda_status_string.argtypes = [ctypes.c_int]
    so.msda_status_string.restype = ctypes.c_char_p
    norm_dims = ctypes.POINTER(msda_norm_dims_t)
    so.msda_layer_norm_forward.argtypes = [vp] * 8 + [ctypes.c_double, norm_dims, ctypes.c_int,
                                                      ctypes.c_int, vp]
    so.msda_layer_norm_forward.restype = ctypes.c_int
    so.msda_layer_norm_backward_workspace_bytes.argtypes = [norm_dims, ctypes.c_int]
    so.msda_layer_norm_backward_workspace_bytes.restype = ctypes.c_size_t
    so.msda_layer_norm_backward.argtypes = [vp] * 11 + [ctypes.c_size_t, norm_dims, ctypes.c_int,
                                                        ctypes.c_int, vp]
    so.msda_layer_norm_backward.restype = ctypes.c_int
    grad_list = ctypes.POINTER(msda_grad_list_t)
    so.msda_grad_norm_workspace_bytes.argtypes = [grad_list]
    so.msda_grad_norm_workspace_bytes.restype = ctypes.c_size_t
    so.msda_grad_norm.argtypes = [grad_list, ctypes.c_int, vp, vp, ctypes.c_size_t, vp]
    so.msda_grad_norm.restype = ctypes.c_int
    so.msda_clip_grad_norm.argtypes = [grad_list, ctypes.c_int, ctypes.c_double, vp, vp,
                                       ctypes.c_size_t, vp]
    so.msda_clip_grad_norm.restype = ctypes.c_int
    attention_dims = ctypes.POINTER(msda_attention_dims_t)
    for name in ("msda_attention_forward_workspace_bytes", "msda_attention_backward_workspace_bytes"):
        getattr(so, name).argtypes = [attention_dims, ctypes.c_int, ctypes.c_int]
        getattr(so, name).restype = ctypes.c_size_t
    so.msda_attention_forward.argtypes = [vp] * 7 + [ctypes.c_double, vp, ctypes.c_size_t,
                                                     attention_dims, ctypes.c_int, vp]
    so.msda_attention_forward.restype = ctypes.c_int
    so.msda_attention_backward.argtypes = [vp] * 11 + [ctypes.c_double, vp, ctypes.c_size_t,
                                                       attention_dims, ctypes.c_int, vp]
    so.msda_attention_backward.restype = ctypes.c_int
    so.msda_dropout.argtypes = [vp, vp, vp, ctypes.c_int64, ctypes.c_double, vp, ctypes.c_int, vp]
    so.msda_dropout.restype = ctypes.c_int
    so.msda_dropout_next.argtypes = [vp, vp, vp]
    so.msda_dropout_next.restype = ctypes.c_int
    so.msda_version.argtypes = []
    so.msda_version.restype = ctypes.c_int
    return so


def use_library(path: str | None = None):
    """Make every call of this module go to the library at `path` (default:
    libmsda.so), e.g. the range-checked build at build.CHECKED_LIBRARY;
    returns its handle."""
    global _lib
    with _lock:
        _lib = load(path)
    return _lib


def lib():
    global _lib
    if _lib is None:
        with _lock:
            if _lib is None:
                _lib = load()
    return _lib


# ------------------------------------------------------------- marshalling

def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check_cuda(*tensors):
    for t in tensors:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libmsda runs on CUDA tensors only (no CPU path)")
        if not t.is_contiguous():
            raise ValueError("libmsda needs contiguous tensors")


def dims_of(value, spatial_shapes, sampling_locations) -> msda_dims_t:
    B, S, M, D = value.shape
    _, Q, M2, L, K, two = sampling_locations.shape
    if M2 != M or two != 2 or tuple(spatial_shapes.shape) != (L, 2):
        raise ValueError("inconsistent operand shapes")
    return msda_dims_t(B, S, Q, M, D, L, K)


def _dtype(t) -> int:
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}") from None


def _call(name, status):
    if status != 0:
        raise MSDAError(status, name)


def msda_forward(value, spatial_shapes, level_start_index, sampling_locations,
                 attention_weights, query_order=None, out=None, stream=None, softmax=False):
    """out (B, Q, M*D) of value's dtype; see msda_forward in include/msda.h.
    softmax=True: attention_weights are logits (msda_forward_softmax)."""
    d = dims_of(value, spatial_shapes, sampling_locations)
    if out is None:
        out = torch.empty((d.B, d.Q, d.M * d.D), dtype=value.dtype, device=value.device)
    _check_cuda(value, spatial_shapes, level_start_index, sampling_locations,
                attention_weights, query_order, out)
    name = "msda_forward_softmax" if softmax else "msda_forward"
    _call(name, getattr(lib(), name)(
        _ptr(value), _ptr(spatial_shapes), _ptr(level_start_index), _ptr(sampling_locations),
        _ptr(attention_weights), _ptr(query_order), _ptr(out), ctypes.byref(d), _dtype(value),
        _stream(stream)))
    return out


def msda_backward_workspace_bytes(dims: msda_dims_t, dtype, accum: int) -> int:
    dt = dtype if isinstance(dtype, int) else _DTYPES[dtype]
    return int(lib().msda_backward_workspace_bytes(ctypes.byref(dims), dt, accum))


def msda_backward(value, spatial_shapes, level_start_index, sampling_locations,
                  attention_weights, grad_out, accum: int = MSDA_ACC_FP32_BUFFER,
                  query_order=None, grad_value=None, grad_sampling_locations=None,
                  grad_attention_weights=None, workspace=None, stream=None, softmax=False):
    """(grad_value, grad_sampling_locations, grad_attention_weights); with
    softmax=True the weights are logits and the third output is their
    gradient (msda_backward_softmax)."""
    d = dims_of(value, spatial_shapes, sampling_locations)
    dev, dt = value.device, value.dtype
    if grad_value is None:
        grad_value = torch.empty_like(value)
    if grad_sampling_locations is None:
        grad_sampling_locations = torch.empty_like(sampling_locations)
    if grad_attention_weights is None:
        grad_attention_weights = torch.empty_like(attention_weights)
    need = msda_backward_workspace_bytes(d, dt, accum)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check_cuda(value, spatial_shapes, level_start_index, sampling_locations, attention_weights,
                grad_out, query_order, grad_value, grad_sampling_locations,
                grad_attention_weights, workspace)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    name = "msda_backward_softmax" if softmax else "msda_backward"
    _call(name, getattr(lib(), name)(
        _ptr(value), _ptr(spatial_shapes), _ptr(level_start_index), _ptr(sampling_locations),
        _ptr(attention_weights), _ptr(query_order), _ptr(grad_out), _ptr(grad_value),
        _ptr(grad_sampling_locations), _ptr(grad_attention_weights), _ptr(workspace),
        ctypes.c_size_t(ws_bytes), accum, ctypes.byref(d), _dtype(value), _stream(stream)))
    return grad_value, grad_sampling_locations, grad_attention_weights


class BackwardBuffers:
    """Outputs and workspace of one backward shape, allocated once and reused
    (the benchmark and the split-step API use this to avoid per-call allocation)."""

    def __init__(self, value, sampling_locations, attention_weights, accum=MSDA_ACC_FP32_BUFFER):
        self.dims = msda_dims_t(*[int(v) for v in value.shape[:2]], int(sampling_locations.shape[1]),
                                *[int(v) for v in value.shape[2:]],
                                *[int(v) for v in sampling_locations.shape[3:5]])
        self.accum = accum
        self.grad_value = torch.empty_like(value)
        self.grad_sampling_locations = torch.empty_like(sampling_locations)
        self.grad_attention_weights = torch.empty_like(attention_weights)
        need = msda_backward_workspace_bytes(self.dims, value.dtype, accum)
        self.workspace = (torch.empty(need, dtype=torch.uint8, device=value.device)
                          if need > 0 else None)
        self.workspace_bytes = need


def msda_backward_zero(buf: BackwardBuffers, dtype, stream=None):
    _call("msda_backward_zero", lib().msda_backward_zero(
        _ptr(buf.grad_value), _ptr(buf.workspace), ctypes.c_size_t(buf.workspace_bytes),
        buf.accum, ctypes.byref(buf.dims), _DTYPES[dtype], _stream(stream)))


def msda_backward_accumulate(value, spatial_shapes, level_start_index, sampling_locations,
                             attention_weights, grad_out, buf: BackwardBuffers,
                             query_order=None, stream=None):
    _check_cuda(value, spatial_shapes, level_start_index, sampling_locations, attention_weights,
                grad_out, query_order)
    _call("msda_backward_accumulate", lib().msda_backward_accumulate(
        _ptr(value), _ptr(spatial_shapes), _ptr(level_start_index), _ptr(sampling_locations),
        _ptr(attention_weights), _ptr(query_order), _ptr(grad_out), _ptr(buf.grad_value),
        _ptr(buf.grad_sampling_locations), _ptr(buf.grad_attention_weights),
        _ptr(buf.workspace), ctypes.c_size_t(buf.workspace_bytes), buf.accum,
        ctypes.byref(buf.dims), _dtype(value), _stream(stream)))


def msda_backward_finish(buf: BackwardBuffers, dtype, stream=None):
    _call("msda_backward_finish", lib().msda_backward_finish(
        _ptr(buf.workspace), ctypes.c_size_t(buf.workspace_bytes), _ptr(buf.grad_value),
        buf.accum, ctypes.byref(buf.dims), _DTYPES[dtype], _stream(stream)))


def msda_device_check(stream=None) -> int:
    """Synchronize `stream`, then read and clear the fault word: returns MSDA_OK (0),
    MSDA_ERR_DEVICE_BOUNDS (7, range-checked build) or MSDA_ERR_DEVICE_WAIT (8: a wait inside
    an attention kernel ran out). Raises on a CUDA failure."""
    st = int(lib().msda_device_check(_stream(stream)))
    if st not in (0, MSDA_ERR_DEVICE_BOUNDS, MSDA_ERR_DEVICE_WAIT):
        raise MSDAError(st, "msda_device_check")
    return st


def msda_set_sample_split(log2_groups: int = -1):
    """Process-wide sample split of the 16-bit and fp32 kernels: -1 (the
    default) chooses it per launch from the problem size, 0..3 force 2^s lane
    groups per query-head (clamped per launch). For tests and tuning."""
    _call("msda_set_sample_split", lib().msda_set_sample_split(int(log2_groups)))


def msda_debug_bounds_self_test(stream=None):
    """Enqueue one range check that must fail (no memory access): the next
    msda_device_check of the checked build returns MSDA_ERR_DEVICE_BOUNDS."""
    _call("msda_debug_bounds_self_test", lib().msda_debug_bounds_self_test(_stream(stream)))


def msda_debug_corners(spatial_shapes, level_start_index, sampling_locations, S: int,
                       stream=None):
    """int32 (B,Q,M,L,K,4) corner rows, -1 outside the map."""
    B, Q, M, L, K, _ = sampling_locations.shape
    d = msda_dims_t(B, S, Q, M, 8, L, K)
    rows = torch.empty((B, Q, M, L, K, 4), dtype=torch.int32, device=sampling_locations.device)
    _check_cuda(spatial_shapes, level_start_index, sampling_locations, rows)
    _call("msda_debug_corners", lib().msda_debug_corners(
        _ptr(spatial_shapes), _ptr(level_start_index), _ptr(sampling_locations), _ptr(rows),
        ctypes.byref(d), _dtype(sampling_locations), _stream(stream)))
    return rows


class MSDAFunction(torch.autograd.Function):
    """Autograd wrapper: forward and backward both run libmsda kernels.
    With softmax=True the weights are logits (the fused-softmax variant)."""

    @staticmethod
    def forward(ctx, value, spatial_shapes, level_start_index, sampling_locations,
                attention_weights, accum=MSDA_ACC_FP32_BUFFER, softmax=False):
        ctx.save_for_backward(value, spatial_shapes, level_start_index, sampling_locations,
                              attention_weights)
        ctx.accum = accum
        ctx.softmax = softmax
        return msda_forward(value, spatial_shapes, level_start_index, sampling_locations,
                            attention_weights, softmax=softmax)

    @staticmethod
    def backward(ctx, grad_out):
        value, shapes, starts, loc, attn = ctx.saved_tensors
        gv, gl, ga = msda_backward(value, shapes, starts, loc, attn, grad_out.contiguous(),
                                   accum=ctx.accum, softmax=ctx.softmax)
        return gv, None, None, gl, ga, None, None


def multi_scale_deformable_attention(value, spatial_shapes, level_start_index,
                                     sampling_locations, attention_weights,
                                     accum=MSDA_ACC_FP32_BUFFER, softmax=False):
    """Differentiable MSDA: value (B,S,M,D), locations (B,Q,M,L,K,2), weights
    (B,Q,M,L,K) or (B,Q,M,L*K) -> (B,Q,M*D). softmax=True: the weights are
    logits normalised over L*K inside the kernels."""
    B, Q, M, L, K, _ = sampling_locations.shape
    attn = attention_weights.reshape(B, Q, M, L, K).contiguous()
    return MSDAFunction.apply(value.contiguous(), spatial_shapes, level_start_index,
                              sampling_locations.contiguous(), attn, accum, softmax)


# ------------------------------------------------------- layer norm, residual

def _at(t):
    return None if t is None else t.data_ptr()


# handle of a device's current stream by its index, without building a Stream object
_current_stream = torch._C._cuda_getCurrentRawStream


@contextlib.contextmanager
def _on(device, stream):
    """Make `device` current, and `stream` (None: its current stream), so that what is
    allocated belongs to the stream the kernels run on."""
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device):
        if stream is None:
            yield
        else:
            with torch.cuda.stream(stream):
                yield


def _check_like(name, t, shape, dtype, device):
    if t is None:
        return
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x is on {device}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} is not contiguous: libmsda needs contiguous tensors")


def _unlike(t, shape, dtype, index):
    """Whether _check_like would raise for t, a tensor, beside one on CUDA device `index`."""
    return not (t.dtype is dtype and t.get_device() == index and t.shape == shape and
                t.is_contiguous())


@functools.lru_cache(maxsize=256)
def _norm_dims(numel, C):
    return ctypes.byref(msda_norm_dims_t(numel // C if C else 0, C))


@functools.lru_cache(maxsize=256)
def _norm_workspace(numel, C, dtype):
    return int(lib().msda_layer_norm_backward_workspace_bytes(_norm_dims(numel, C), dtype))


_PROXY = torch._C._TorchDispatchModeKey.PROXY


def _refuse_recording(name):
    """Raise while torch records operations by dispatch (make_fx): a launch on addresses is
    not among them, and its record would return the output's allocation."""
    if torch._C._len_torch_dispatch_stack() and torch._C._get_dispatch_mode(_PROXY) is not None:
        raise RuntimeError(f"{name} cannot be recorded: it launches on addresses, which torch does not see")


def _refuse_modes(name, tensors):
    """As _refuse_recording, for a call that has no autograd function either: while
    torch.jit.trace runs, and of tensors that carry a forward-mode tangent."""
    _refuse_recording(name)
    if torch._C._get_tracing_state() is not None:
        raise RuntimeError(f"{name} cannot be recorded: it launches on addresses, which torch does not see")
    if forward_ad._current_level >= 0:
        for t in tensors:
            if t is not None and forward_ad.unpack_dual(t).tangent is not None:
                raise RuntimeError(f"{name} has no forward-mode derivative: a tangent would be dropped")


def _param_dtype(x, weight, bias, given=None):
    params = weight if weight is not None else bias
    pdt = params.dtype if params is not None else given if given is not None else x.dtype
    if pdt is not x.dtype and not (pdt is torch.float32 and x.dtype in (torch.bfloat16, torch.float16)):
        raise ValueError(f"parameters of {pdt} with data of {x.dtype}: give the data's type, or "
                         "float32 with 16-bit data")
    return pdt


def _norm_operands(x, weight, bias, pdt, residual, also=()):
    """Raise unless x is a contiguous CUDA tensor with a channel dimension, the residual and
    `also` (pairs of name and tensor) are like it or None, and weight and bias hold a value
    of type pdt for each channel. Returns x's device index."""
    index, shape, dtype = x.get_device(), x.shape, x.dtype
    if not x.is_cuda:
        raise ValueError("libmsda runs on CUDA tensors only (no CPU path)")
    if not shape:
        raise ValueError("x needs a channel dimension")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if not x.is_contiguous():
        _check_like("x", x, shape, dtype, x.device)
    if residual is not None and _unlike(residual, shape, dtype, index):
        _check_like("residual", residual, shape, dtype, x.device)
    for name, t in also:
        if t is not None and _unlike(t, shape, dtype, index):
            _check_like(name, t, shape, dtype, x.device)
    channels = shape[-1:]
    if weight is not None and _unlike(weight, channels, pdt, index):
        _check_like("weight", weight, channels, pdt, x.device)
    if bias is not None and _unlike(bias, channels, pdt, index):
        _check_like("bias", bias, channels, pdt, x.device)
    return index


def _apart(outs, ins):
    """Refuse an output the caller gave that shares memory with an input or another output."""
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in outs + ins
             if t is not None]
    n = len([t for t in outs if t is not None])
    for i, (lo, hi) in enumerate(spans[:n]):
        for lo2, hi2 in spans[i + 1:]:
            if lo < hi2 and lo2 < hi:
                raise ValueError("an output overlaps an input or another output")


def _stats_dtype(x):
    return torch.float64 if x.dtype is torch.float64 else torch.float32


def _norm_forward(x, weight, bias, residual, eps, return_sum, stats, out, pdt, index):
    """The launch, on the current device and stream, of operands already checked. `stats`:
    None, or True for (mean, rstd) as one tensor of two halves."""
    if out is None:
        out = torch.empty_like(x)
    total = torch.empty_like(x) if return_sum else None
    mean = rstd = None
    numel, C = int(x.numel()), int(x.shape[-1])      # a trace makes tensors of sizes
    if stats:
        rows = numel // C if C else 0
        stats = torch.empty(2 * rows, dtype=_stats_dtype(x), device=x.device)
        mean = stats.data_ptr()
        rstd = mean + rows * stats.element_size()
    status = lib().msda_layer_norm_forward(
        x.data_ptr(), None if residual is None else residual.data_ptr(),
        None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(),
        out.data_ptr(), None if total is None else total.data_ptr(), mean, rstd, eps,
        _norm_dims(numel, C), _DTYPES[x.dtype], _DTYPES[pdt], _current_stream(index))
    if status:
        raise MSDAError(status, "msda_layer_norm_forward")
    return out, total, stats


def _norm_backward(grad_out, x, mean, rstd, weight, residual, grad_sum, pdt, want):
    """The launch, on the current device and stream, of operands already checked; mean and
    rstd are addresses."""
    dims, dt = _norm_dims(x.numel(), x.shape[-1]), _DTYPES[x.dtype]
    grad_x = torch.empty_like(x) if want[0] else None
    grad_weight = grad_bias = workspace = None
    need = 0
    if want[1] or want[2]:
        C, device = x.shape[-1], x.device
        grad_weight, grad_bias = [
            None if not w else torch.empty(C, dtype=pdt, device=device) if weight is None
            else torch.empty_like(weight) for w in want[1:]]
        need = _norm_workspace(x.numel(), C, dt)
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    status = lib().msda_layer_norm_backward(
        grad_out.data_ptr(), _at(grad_sum), x.data_ptr(), _at(residual), _at(weight),
        mean, rstd, _at(grad_x), _at(grad_weight), _at(grad_bias),
        _at(workspace), need, dims, dt, _DTYPES[pdt], _current_stream(x.get_device()))
    if status:
        raise MSDAError(status, "msda_layer_norm_backward")
    return grad_x, grad_weight, grad_bias


def _elsewhere(index, stream=None):
    """Whether the launch needs another device or stream than the current ones."""
    return stream is not None or torch._C._cuda_getDevice() != index


def msda_layer_norm_forward(x, weight=None, bias=None, residual=None, eps: float = 1e-5,
                            return_sum: bool = False, stats: bool = True, out=None, stream=None):
    """(out, sum, mean, rstd) of the rows of x + residual over x's last dimension; sum is
    None unless return_sum, mean and rstd are None unless stats (the backward needs them).
    See msda_layer_norm_forward in include/msda.h."""
    _refuse_modes("msda_layer_norm_forward", (x, weight, bias, residual))
    pdt = _param_dtype(x, weight, bias)
    index = _norm_operands(x, weight, bias, pdt, residual, (("out", out),))
    if out is not None:
        _apart([out], [x, residual, weight, bias])
    given = out
    args = (x, weight, bias, residual, eps, return_sum, stats, out, pdt, index)
    if _elsewhere(index, stream):
        with _on(x.device, stream):
            out, total, both = _norm_forward(*args)
    else:
        out, total, both = _norm_forward(*args)
    if given is not None and not out.is_inference():
        torch.autograd.graph.increment_version(out)
    if not stats:
        return out, total, None, None
    mean, rstd = both.view(2, *x.shape[:-1])
    return out, total, mean, rstd


def msda_layer_norm_backward(grad_out, x, mean, rstd, weight=None, residual=None, grad_sum=None,
                             param_dtype=None, want=(True, True, True), stream=None):
    """(grad_x, grad_weight, grad_bias), None where `want` says so; grad_x is the gradient of
    x and of residual alike. param_dtype: the parameters' type where weight is None. See
    msda_layer_norm_backward in include/msda.h."""
    _refuse_modes("msda_layer_norm_backward", (grad_out, x, mean, rstd, weight, residual, grad_sum))
    pdt = _param_dtype(x, weight, None, param_dtype)
    index = _norm_operands(x, weight, None, pdt, residual, (("grad_out", grad_out), ("grad_sum", grad_sum)))
    shape, sdt = x.shape[:-1], _stats_dtype(x)
    if _unlike(mean, shape, sdt, index) or _unlike(rstd, shape, sdt, index):
        _check_like("mean", mean, shape, sdt, x.device)
        _check_like("rstd", rstd, shape, sdt, x.device)
    args = (grad_out, x, mean.data_ptr(), rstd.data_ptr(), weight, residual, grad_sum, pdt, want)
    if _elsewhere(index, stream):
        with _on(x.device, stream):
            return _norm_backward(*args)
    return _norm_backward(*args)


def _norm_gradients(ctx, grad_out, grad_sum):
    """What LayerNormFunction.backward returns."""
    _refuse_recording("layer_norm's backward")
    need_x, need_res, need_w, need_b, _, _ = ctx.needs_input_grad
    if grad_sum is not None:
        grad_sum = grad_sum.contiguous()
    if grad_out is None:                 # the normalised rows were not used
        gx = gw = gb = None
        if need_x or need_res:
            gx = grad_sum
    else:
        x, residual, weight, stats = ctx.saved_tensors
        mean = stats.data_ptr()
        args = (grad_out.contiguous(), x, mean, mean + stats.numel() // 2 * stats.element_size(),
                weight, residual, grad_sum, ctx.param_dtype, (need_x or need_res, need_w, need_b))
        if _elsewhere(x.get_device()):
            with _on(x.device, None):
                gx, gw, gb = _norm_backward(*args)
        else:
            gx, gw, gb = _norm_backward(*args)
    return gx if need_x else None, gx if need_res else None, gw, gb, None, None


class LayerNormFunction(torch.autograd.Function):
    """Autograd wrapper of the two calls above (first derivatives only)."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps, return_sum):
        pdt = ctx.param_dtype = _param_dtype(x, weight, bias)
        index = _norm_operands(x, weight, bias, pdt, residual)
        args = (x, weight, bias, residual, eps, return_sum, True, None, pdt, index)
        if _elsewhere(index):
            with _on(x.device, None):
                out, total, stats = _norm_forward(*args)
        else:
            out, total, stats = _norm_forward(*args)
        ctx.save_for_backward(x, residual, weight, stats)
        ctx.set_materialize_grads(False)
        return (out, total) if return_sum else out

    @staticmethod
    def backward(ctx, grad_out, grad_sum=None):
        if torch.is_grad_enabled():      # create_graph: second derivatives are an error, if asked for
            return LayerNormFunction.backward_once(ctx, grad_out, grad_sum)
        return _norm_gradients(ctx, grad_out, grad_sum)

    backward_once = staticmethod(torch.autograd.function.once_differentiable(_norm_gradients))


def _through_autograd():
    """Whether torch must see an operation although no gradient is wanted: while
    torch.jit.trace runs, whose record of a launch on addresses would be the output's
    allocation alone, and inside a forward-mode level, whose tangents it would drop (the
    autograd function has no jvp and says so)."""
    return torch._C._get_tracing_state() is not None or forward_ad._current_level >= 0


def layer_norm(x, weight=None, bias=None, residual=None, eps: float = 1e-5, return_sum: bool = False):
    """Differentiable layer norm over x's last dimension, of x + residual where a residual is
    given (same shape as x; the sum is not rounded before it is normalised). weight and bias
    (C,) of x's type, or float32 with 16-bit x. return_sum: (normalised, x + residual)."""
    if return_sum and residual is None:
        raise ValueError("return_sum needs a residual")
    _refuse_recording("layer_norm")
    x = x.contiguous()
    grad = x.requires_grad
    if residual is not None:
        residual = residual.contiguous()
        grad = grad or residual.requires_grad
    if weight is not None:
        weight = weight.contiguous()
        grad = grad or weight.requires_grad
    if bias is not None:
        bias = bias.contiguous()
        grad = grad or bias.requires_grad
    if (grad and torch.is_grad_enabled()) or _through_autograd():
        return LayerNormFunction.apply(x, residual, weight, bias, eps, return_sum)
    pdt = _param_dtype(x, weight, bias)
    index = _norm_operands(x, weight, bias, pdt, residual)
    args = (x, weight, bias, residual, eps, return_sum, False, None, pdt, index)
    if _elsewhere(index):
        with _on(x.device, None):
            out, total, _ = _norm_forward(*args)
    else:
        out, total, _ = _norm_forward(*args)
    return (out, total) if return_sum else out


# ------------------------------------------------------ gradient norm, clipping

def _dense(t):
    """Whether t's entries fill one span of memory, each place once."""
    if t.is_contiguous():
        return True
    expected = 1
    for stride, size in sorted((st, n) for st, n in zip(t.stride(), t.shape) if n != 1):
        if stride != expected:
            return False
        expected *= size
    return True


def _span(t):
    at = t.data_ptr()
    return at, at + t.numel() * t.element_size()


class GradientBuffers:
    """A list of gradient tensors, checked once, for msda_grad_norm and
    msda_clip_grad_norm: what a training loop whose gradients keep their memory (zeroed in
    place, views of a flat buffer, or captured in a graph) holds across its steps.

    grads: CUDA tensors of one device, of any of the four types, each dense (contiguous, or
    e.g. channels-last), none sharing memory with another. out: None to clip in place, or as
    many tensors that receive the clipped gradients, of the same shapes and of the
    gradients' types, or float32 for 16-bit gradients."""

    def __init__(self, grads, out=None):
        grads = list(grads)
        outs = grads if out is None else list(out)
        if len(outs) != len(grads):
            raise ValueError(f"{len(outs)} outputs for {len(grads)} gradients")
        device = grads[0].device if grads else None
        for g, o in zip(grads, outs):
            if not g.is_cuda:
                raise ValueError("libmsda runs on CUDA tensors only (no CPU path)")
            if g.layout != torch.strided:
                raise ValueError("a gradient is sparse: give dense gradients")
            if g.dtype not in _DTYPES:
                raise ValueError(f"unsupported dtype {g.dtype}")
            if g.device != device or o.device != device:
                raise ValueError(f"tensors on {device}, {g.device} and {o.device}: give one device's")
            if not _dense(g):
                raise ValueError("a gradient is not dense: libmsda needs its entries in one span")
            if o is not g:
                if o.shape != g.shape or (o.stride() != g.stride() and not
                                          (o.is_contiguous() and g.is_contiguous())):
                    raise ValueError("an output's shape or strides differ from its gradient's")
                if o.dtype != g.dtype and not (o.dtype == torch.float32 and
                                               g.dtype in (torch.bfloat16, torch.float16)):
                    raise ValueError(f"an output of {o.dtype} for a gradient of {g.dtype}: give the "
                                     "gradient's type, or float32 for a 16-bit gradient")
        self.device = device
        self.in_place = out is None
        # aliases: what the caller does to its own tensor objects does not reach them
        self._grads = [g.detach() for g in grads]
        self._outs = self._grads if out is None else [o.detach() for o in outs]
        self._all = self._grads if out is None else self._grads + self._outs
        self._counted = [o for o in self._outs if not o.is_inference()]
        self.norm_dtype = (torch.float64 if any(g.dtype is torch.float64 for g in grads)
                           else torch.float32)
        n = len(grads)
        self._sizes = (ctypes.c_int64 * n)(*[g.numel() for g in grads])
        self._dtypes = (ctypes.c_int32 * n)(*[_DTYPES[g.dtype] for g in grads])
        self._out_dtypes = (ctypes.c_int32 * n)(*[_DTYPES[o.dtype] for o in outs])
        self._read_addresses()
        self._watch()

    def _read_addresses(self):
        spans = sorted(_span(t) for t in self._all if t.numel())
        for (_, end), (begin, _) in zip(spans, spans[1:]):
            if begin < end:
                raise ValueError("two of the tensors share memory")
        for t in self._all:
            held = t.untyped_storage().nbytes() - t.storage_offset() * t.element_size()
            if held < t.numel() * t.element_size():
                raise ValueError("a tensor's storage was resized to less than the tensor")
        addresses = list(map(torch.Tensor.data_ptr, self._all))
        n = len(self._grads)
        self._at = (ctypes.c_void_p * n)(*addresses[:n])
        self._out_at = self._at if self.in_place else (ctypes.c_void_p * n)(*addresses[n:])
        self._list = msda_grad_list_t(n, *[ctypes.addressof(a) for a in (
            self._at, self._out_at, self._sizes, self._dtypes, self._out_dtypes)])
        self._ref = ctypes.byref(self._list)
        self.workspace_bytes = int(lib().msda_grad_norm_workspace_bytes(self._ref))

    def _watch(self):
        storages = [t.untyped_storage() for t in self._all]
        self._storages = list({s._cdata: s for s in storages}.values())
        self._memory = self._read_memory()

    def _read_memory(self):
        """Where the tensors' storages lie and how large they are. The aliases change in
        nothing else, and a storage freed and made anew may have its address again, and be
        smaller."""
        return (list(map(torch.UntypedStorage.data_ptr, self._storages)),
                list(map(torch.UntypedStorage.nbytes, self._storages)))

    def _prepare(self):
        memory = self._read_memory()
        if memory != self._memory:
            self._read_addresses()
            self._memory = memory


class _OneCall(GradientBuffers):
    """A list given to a call: read by that call alone."""

    def _watch(self):
        pass

    def _prepare(self):
        pass


def _norm_kind(norm_type):
    norm_type = float(norm_type)
    if norm_type == 2.0:
        return 0
    if norm_type == float("inf"):
        return 1
    raise ValueError(f"norm_type {norm_type}: 2 and inf are supported")


def _grad_call(buf, kind, max_norm, stream):
    buf._prepare()
    norm = torch.empty((), dtype=buf.norm_dtype, device=buf.device)
    workspace = torch.empty(buf.workspace_bytes, dtype=torch.uint8, device=buf.device)
    s = _current_stream(norm.get_device())
    if max_norm is None:
        _call("msda_grad_norm", lib().msda_grad_norm(
            buf._ref, kind, norm.data_ptr(), workspace.data_ptr(), buf.workspace_bytes, s))
    else:
        _call("msda_clip_grad_norm", lib().msda_clip_grad_norm(
            buf._ref, kind, max_norm, norm.data_ptr(), workspace.data_ptr(), buf.workspace_bytes, s))
        torch.autograd.graph.increment_version(buf._counted)
    return norm


def _grad_norm(grads, norm_type, max_norm, stream):
    kind = _norm_kind(norm_type)
    name = "msda_grad_norm" if max_norm is None else "msda_clip_grad_norm"
    if isinstance(grads, GradientBuffers):
        _refuse_modes(name, ())          # aliases without tangents
        buf = grads
    else:
        grads = list(grads)
        _refuse_modes(name, grads)
        buf = _OneCall(grads)
    if buf.device is None:               # an empty list
        return torch.zeros(())
    if stream is not None or torch._C._cuda_getDevice() != buf.device.index:
        with _on(buf.device, stream):
            return _grad_call(buf, kind, max_norm, stream)
    return _grad_call(buf, kind, max_norm, stream)


def msda_grad_norm(grads, norm_type: float = 2.0, stream=None):
    """The norm of all entries of `grads` (GradientBuffers, or a list of tensors): a 0-d
    float32 tensor on their device (float64 where one of them is). norm_type 2 or inf. See
    msda_grad_norm in include/msda.h."""
    return _grad_norm(grads, norm_type, None, stream)


def msda_clip_grad_norm(grads, max_norm: float, norm_type: float = 2.0, stream=None):
    """The norm, as msda_grad_norm; and the gradients times min(1, max_norm / (norm + 1e-6)),
    in place or in the buffers' outputs. Nothing waits for the device."""
    return _grad_norm(grads, norm_type, float(max_norm), stream)


def clip_grad_norm_(parameters, max_norm: float, norm_type: float = 2.0,
                    error_if_nonfinite: bool = False):
    """Clip the gradients of `parameters` (a tensor or an iterable of them; those without a
    gradient are passed over) to a joint norm of max_norm, in place; returns the norm they
    had. error_if_nonfinite: raise where that is not finite (waits for the device; the
    gradients are then left as they were)."""
    if isinstance(parameters, torch.Tensor):
        parameters = [parameters]
    grads = [p.grad for p in parameters if p.grad is not None]
    _refuse_modes("clip_grad_norm_", grads)
    buf = _OneCall(grads)
    if error_if_nonfinite:
        norm = msda_grad_norm(buf, norm_type)
        if not torch.isfinite(norm):
            raise RuntimeError(f"the norm of the gradients is {float(norm)}: not clipped")
    return msda_clip_grad_norm(buf, max_norm, norm_type)


# ------------------------------------------------------------------ attention

_ATTENTION_DTYPES = (torch.float32, torch.bfloat16, torch.float16)


def _attention_check(q, k, v, mask):
    """Raise unless the shapes, types and strides of q, k, v and the mask fit each other."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError("libmsda runs on CUDA tensors only (no CPU path)")
        if t.dim() != 4:
            raise ValueError(f"{name} needs four dimensions (batch, position, head, channel), "
                             f"has shape {tuple(t.shape)}")
        if t.dtype != q.dtype:
            raise ValueError(f"{name} is {t.dtype}, q is {q.dtype}")
    if q.dtype not in _ATTENTION_DTYPES:
        raise ValueError(f"unsupported dtype {q.dtype}: float32, bfloat16 and float16 are supported")
    B, Q, M, D = q.shape
    S, N = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != D or v.shape != k.shape:
        raise ValueError(f"q {tuple(q.shape)}, k {tuple(k.shape)} and v {tuple(v.shape)} do not fit")
    if N < 1 or M < N or M % N:
        raise ValueError(f"{M} query heads for {N} key heads: give a multiple")
    if not 8 <= D <= 128 or D % 8:
        raise ValueError(f"{D} channels a head: multiples of 8 from 8 to 128 are supported")
    if mask is not None:
        if mask.dtype is not torch.bool:
            raise ValueError(f"the mask is {mask.dtype}: give torch.bool, true where a query may attend")
        try:
            mask.expand(B, M, Q, S)
        except RuntimeError:
            raise ValueError(f"a mask of shape {tuple(mask.shape)} does not broadcast to "
                             f"{(B, M, Q, S)}") from None


class _AttentionPlan:
    """What one set of shapes, strides and types needs: the C dims, the workspaces' bytes,
    and which of q, k and v have to be copied first (channels not contiguous, or rows not on
    16-byte boundaries)."""

    def __init__(self, q, k, v, mask):
        _attention_check(q, k, v, mask)
        B, Q, M, D = q.shape
        S, N = k.shape[1], k.shape[2]
        e = q.element_size()
        self.copies = [t.stride(3) != 1 or any(n > 1 and (st <= 0 or st * e % 16)
                                               for st, n in zip(t.stride()[:3], t.shape))
                       for t in (q, k, v)]
        self.copy = any(self.copies)
        self.dtype = _DTYPES[q.dtype]
        self.out_shape, self.stats_shape = (B, Q, M * D), (B, M, Q)
        self.default_scale = D ** -0.5
        strides = [(ctypes.c_int64 * 3)(*t.stride()[:3]) for t in (q, k, v)]
        mask_strides = (0, 0, 0, 0)
        if mask is not None:
            mask_strides = [st if n > 1 else 0
                            for st, n in zip(mask.expand(B, M, Q, S).stride(), (B, M, Q, S))]
        self.dims = msda_attention_dims_t(B, Q, S, M, N, D, *strides, (ctypes.c_int64 * 4)(*mask_strides))
        self.ref = ctypes.byref(self.dims)
        so = lib()
        self.forward_bytes = int(so.msda_attention_forward_workspace_bytes(
            self.ref, self.dtype, mask is not None))
        self.backward_bytes = int(so.msda_attention_backward_workspace_bytes(
            self.ref, self.dtype, mask is not None))


_attention_plans = {}


def _plan_of(q, k, v, mask):
    """(the plan of these operands' shapes, strides and types, their device's index)"""
    key = (q.shape, k.shape, v.shape, q.stride(), k.stride(), v.stride(), q.dtype, k.dtype, v.dtype,
           None if mask is None else (mask.shape, mask.stride(), mask.dtype))
    index = q.get_device()
    if index < 0 or k.get_device() != index or v.get_device() != index or (
            mask is not None and mask.get_device() != index):
        _attention_check(q, k, v, mask)
        raise ValueError("q, k, v and the mask are on "
                         f"{[str(t.device) for t in (q, k, v, mask) if t is not None]}: give one device's")
    plan = _attention_plans.get(key)
    if plan is None:
        plan = _AttentionPlan(q, k, v, mask)
        if len(_attention_plans) >= 256:
            _attention_plans.clear()
        _attention_plans[key] = plan
    return plan, index


def _scale_of(scale, plan):
    if scale is None:
        return plan.default_scale
    scale = float(scale)
    if not 0.0 <= scale <= 2.3e38:
        raise ValueError(f"scale {scale}: give a number from zero to 2.3e38")
    return scale


def _ready(q, k, v, mask, plan):
    """q, k and v, or copies that the kernels can read, and their plan. On the device and
    stream of the launch."""
    copies = plan.copies if plan.copy else (False, False, False)
    made = [t.clone(memory_format=torch.contiguous_format) if c or t.data_ptr() % 16 else t
            for t, c in zip((q, k, v), copies)]
    if made[0] is q and made[1] is k and made[2] is v:
        return q, k, v, plan
    return (*made, _plan_of(*made, mask)[0])


def _attend(q, k, v, mask, plan, index, scale, lse, rest, out):
    """The launch, on the current device and stream, of operands already checked. rest: also
    what out's rounding left (16-bit types)."""
    if plan.copy or (q.data_ptr() | k.data_ptr() | v.data_ptr()) % 16:
        q, k, v, plan = _ready(q, k, v, mask, plan)
    device = q.device
    if out is None:
        out = torch.empty(plan.out_shape, dtype=q.dtype, device=device)
    lse = torch.empty(plan.stats_shape, dtype=torch.float32, device=device) if lse else None
    rest = torch.empty_like(out) if rest and q.dtype is not torch.float32 else None
    need = plan.forward_bytes
    workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    status = lib().msda_attention_forward(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), None if mask is None else mask.data_ptr(),
        out.data_ptr(), None if rest is None else rest.data_ptr(), None if lse is None else lse.data_ptr(),
        scale, None if workspace is None else workspace.data_ptr(), need, plan.ref, plan.dtype,
        _current_stream(index))
    if status:
        raise MSDAError(status, "msda_attention_forward")
    return out, lse, rest


def _attend_backward(grad_out, q, k, v, out, rest, lse, mask, plan, index, scale, want):
    """The launch, on the current device and stream, of operands already checked."""
    if plan.copy or (q.data_ptr() | k.data_ptr() | v.data_ptr()) % 16:
        q, k, v, plan = _ready(q, k, v, mask, plan)
    grad_out, out, rest = _at16(grad_out), _at16(out), None if rest is None else _at16(rest)
    dtype, device = q.dtype, q.device
    gq = torch.empty(q.shape, dtype=dtype, device=device) if want[0] else None
    gk = gv = None
    if want[1] or want[2]:
        gk, gv = [torch.empty(k.shape, dtype=dtype, device=device) for _ in range(2)]
    need = plan.backward_bytes
    workspace = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    status = lib().msda_attention_backward(
        grad_out.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(mask), out.data_ptr(),
        _at(rest), lse.data_ptr(), _at(gq), _at(gk), _at(gv), scale, _at(workspace), need, plan.ref,
        plan.dtype, _current_stream(index))
    if status:
        raise MSDAError(status, "msda_attention_backward")
    return gq, gk if want[1] else None, gv if want[2] else None


def _at16(t):
    """t, contiguous, or a copy that starts on a 16-byte boundary."""
    return t if t.data_ptr() % 16 == 0 else t.clone()


def msda_attention_forward(q, k, v, mask=None, scale=None, lse: bool = True, out=None, stream=None,
                           rest: bool = False):
    """(out (B, Q, M*D), lse (B, M, Q)) of q (B, Q, M, D) over k, v (B, S, N, D); lse is None
    unless `lse` (the backward needs it). rest: a third tensor, what out's rounding to 16 bits
    left (None for float32), for gradients as good as from an out of twice the digits. mask: bool, broadcasts to (B, M, Q, S), true where a
    query may attend. scale: D ** -0.5 unless given. See msda_attention_forward in
    include/msda.h."""
    _refuse_modes("msda_attention_forward", (q, k, v))
    plan, index = _plan_of(q, k, v, mask)
    scale = _scale_of(scale, plan)
    if out is not None:
        _check_like("out", out, plan.out_shape, q.dtype, q.device)
        if out.data_ptr() % 16:
            raise ValueError("out does not start on a 16-byte boundary")
        for t in (q, k, v, mask):        # spans of strided tensors
            if t is not None and t.numel() and out.numel():
                last = sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
                if (t.data_ptr() < out.data_ptr() + out.numel() * out.element_size()
                        and out.data_ptr() < t.data_ptr() + (last + 1) * t.element_size()):
                    raise ValueError("an output overlaps an input or another output")
    given = out
    args = (q, k, v, mask, plan, index, scale, lse, rest, out)
    if _elsewhere(index, stream):
        with _on(q.device, stream):
            out, stats, left = _attend(*args)
    else:
        out, stats, left = _attend(*args)
    if given is not None and not out.is_inference():
        torch.autograd.graph.increment_version(out)
    return (out, stats, left) if rest else (out, stats)


def msda_attention_backward(grad_out, q, k, v, out, lse, mask=None, scale=None,
                            want=(True, True, True), stream=None, rest=None):
    """(grad_q, grad_k, grad_v) of q's, k's and v's shapes, contiguous, None where `want` says
    so; out, lse and rest (if it was asked for) are the forward's. See msda_attention_backward in include/msda.h."""
    _refuse_modes("msda_attention_backward", (grad_out, q, k, v, out, lse, rest))
    plan, index = _plan_of(q, k, v, mask)
    scale = _scale_of(scale, plan)
    for name, t in (("grad_out", grad_out), ("out", out), ("rest", rest)):
        _check_like(name, t, plan.out_shape, q.dtype, q.device)
    _check_like("lse", lse, plan.stats_shape, torch.float32, q.device)
    args = (grad_out, q, k, v, out, rest, lse, mask, plan, index, scale, want)
    if _elsewhere(index, stream):
        with _on(q.device, stream):
            return _attend_backward(*args)
    return _attend_backward(*args)


def _attention_gradients(ctx, grad_out):
    """What AttentionFunction.backward returns."""
    _refuse_recording("attention's backward")
    q, k, v, mask, out, lse, rest = ctx.saved_tensors
    plan, index = _plan_of(q, k, v, mask)
    args = (grad_out.contiguous(), q, k, v, out, rest, lse, mask, plan, index, ctx.scale,
            ctx.needs_input_grad[:3])
    if _elsewhere(index):
        with _on(q.device, None):
            grads = _attend_backward(*args)
    else:
        grads = _attend_backward(*args)
    return (*grads, None, None)


class AttentionFunction(torch.autograd.Function):
    """Autograd wrapper of the two calls above (first derivatives only)."""

    @staticmethod
    def forward(ctx, q, k, v, mask, scale):
        plan, index = _plan_of(q, k, v, mask)
        ctx.scale = _scale_of(scale, plan)
        args = (q, k, v, mask, plan, index, ctx.scale, True, True, None)
        if _elsewhere(index):
            with _on(q.device, None):
                out, lse, rest = _attend(*args)
        else:
            out, lse, rest = _attend(*args)
        ctx.save_for_backward(q, k, v, mask, out, lse, rest)
        return out

    @staticmethod
    def backward(ctx, grad_out):
        if torch.is_grad_enabled():      # create_graph: second derivatives are an error, if asked for
            return AttentionFunction.backward_once(ctx, grad_out)
        return _attention_gradients(ctx, grad_out)

    backward_once = staticmethod(torch.autograd.function.once_differentiable(_attention_gradients))


def attention(q, k, v, mask=None, scale=None):
    """Differentiable attention: q (B, Q, M, D) over k, v (B, S, N, D) -> (B, Q, M*D), query
    head m reading key head m / (M / N). mask: bool, broadcasts to (B, M, Q, S), true where a
    query may attend; a query with no key gets zeros. scale: D ** -0.5 unless given. D is a
    multiple of 8 up to 128; float32, bfloat16 or float16. q, k and v may be strided, as parts
    of one projection are."""
    _refuse_recording("attention")
    if (torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad)
            or _through_autograd()):
        return AttentionFunction.apply(q, k, v, mask, scale)
    plan, index = _plan_of(q, k, v, mask)
    args = (q, k, v, mask, plan, index, _scale_of(scale, plan), False, False, None)
    if _elsewhere(index):
        with _on(q.device, None):
            return _attend(*args)[0]
    return _attend(*args)[0]


# -------------------------------------------------------------------- dropout

def _drop_operands(x, p, counter, residual):
    index, dtype = x.get_device(), x.dtype
    if index < 0:
        raise ValueError("libmsda runs on CUDA tensors only (no CPU path)")
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"a probability of {p}: give one from 0 to 1")
    if not x.is_contiguous():
        _check_like("x", x, x.shape, dtype, x.device)
    if residual is not None and _unlike(residual, x.shape, dtype, index):
        _check_like("residual", residual, x.shape, dtype, x.device)
    if _unlike(counter, (2,), torch.int64, index):
        _check_like("counter", counter, (2,), torch.int64, x.device)
    return index


def _drop(x, p, counter, residual, out):
    """The launch, on the current device and stream, of operands already checked."""
    if out is None:
        out = torch.empty_like(x)
    status = lib().msda_dropout(x.data_ptr(), _at(residual), out.data_ptr(), int(x.numel()), p,
                                counter.data_ptr(), _DTYPES[x.dtype], _current_stream(x.get_device()))
    if status:
        raise MSDAError(status, "msda_dropout")
    return out


def msda_dropout(x, p, counter, residual=None, out=None, stream=None):
    """residual + x with each entry kept with probability 1 - p and scaled by 1 / (1 - p), in
    steps of 2^-16. counter: two int64 on x's device, the generator's seed and the draw's
    number. out may be x or residual. See msda_dropout in include/msda.h."""
    _refuse_modes("msda_dropout", (x, residual))
    p = float(p)
    _drop_operands(x, p, counter, residual)
    given = out
    if out is not None:
        _check_like("out", out, x.shape, x.dtype, x.device)
        _apart([out], [t for t in (x, residual) if t is not None and t.data_ptr() != out.data_ptr()] + [counter])
    if _elsewhere(x.get_device(), stream):
        with _on(x.device, stream):
            out = _drop(x, p, counter, residual, out)
    else:
        out = _drop(x, p, counter, residual, out)
    if given is not None and not out.is_inference():
        torch.autograd.graph.increment_version(out)
    return out


def dropout_next(state, stream=None):
    """The generator's next draw: a new tensor of `state`'s seed and number (two int64 on the
    device), whose number is then advanced by one, on the device (a captured call draws anew
    each time it is replayed)."""
    _refuse_modes("dropout_next", ())
    if not state.is_cuda:
        raise ValueError("libmsda runs on CUDA tensors only (no CPU path)")
    _check_like("state", state, (2,), torch.int64, state.device)
    with _on(state.device, stream):
        drawn = torch.empty_like(state)
        _call("msda_dropout_next", lib().msda_dropout_next(
            state.data_ptr(), drawn.data_ptr(), _current_stream(state.get_device())))
    if not state.is_inference():
        torch.autograd.graph.increment_version(state)
    return drawn


def _drop_gradient(ctx, grad_out):
    """What DropoutFunction.backward returns."""
    _refuse_recording("dropout's backward")
    counter, = ctx.saved_tensors
    gx = None
    if ctx.needs_input_grad[0]:
        grad = grad_out.contiguous()
        if _elsewhere(grad.get_device()):
            with _on(grad.device, None):
                gx = _drop(grad, ctx.p, counter, None, None)
        else:
            gx = _drop(grad, ctx.p, counter, None, None)
    return gx, grad_out if ctx.needs_input_grad[1] else None, None, None


class DropoutFunction(torch.autograd.Function):
    """Autograd wrapper: the backward draws the same mask again (first derivatives only)."""

    @staticmethod
    def forward(ctx, x, residual, p, counter):
        _drop_operands(x, p, counter, residual)
        ctx.p = p
        ctx.save_for_backward(counter)
        if _elsewhere(x.get_device()):
            with _on(x.device, None):
                return _drop(x, p, counter, residual, None)
        return _drop(x, p, counter, residual, None)

    @staticmethod
    def backward(ctx, grad_out):
        if torch.is_grad_enabled():      # create_graph: second derivatives are an error, if asked for
            return DropoutFunction.backward_once(ctx, grad_out)
        return _drop_gradient(ctx, grad_out)

    backward_once = staticmethod(torch.autograd.function.once_differentiable(_drop_gradient))


def dropout(x, p, counter, residual=None):
    """Differentiable dropout, and the residual stream it is added to: residual + x with each
    entry kept with probability 1 - p and scaled by 1 / (1 - p). counter: two int64 on x's
    device, the seed and the draw's number (dropout_next gives one); the same counter draws
    the same mask, and the mask is not stored."""
    _refuse_recording("dropout")
    p = float(p)
    x = x.contiguous()
    if residual is not None:
        residual = residual.contiguous()
    if (torch.is_grad_enabled() and (x.requires_grad or residual is not None and residual.requires_grad)
            or _through_autograd()):
        return DropoutFunction.apply(x, residual, p, counter)
    _drop_operands(x, p, counter, residual)
    if _elsewhere(x.get_device()):
        with _on(x.device, None):
            return _drop(x, p, counter, residual, None)
    return _drop(x, p, counter, residual, None)
