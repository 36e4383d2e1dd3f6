"""Python binding of libmamba2, the GB300 (sm_103a) Mamba2 recurrent hot path.

Argument marshalling only: every step runs in the CUDA kernels behind the C ABI
declared in ``include/mamba2.h``. Tensors are torch CUDA tensors (device memory
and streams come from PyTorch); batch metadata (``cu_seqlens``, ``slots``,
``fresh``) are host sequences. There is no fallback: importing the package
without the built library raises.

Entry points (same names as the C ABI without the ``mamba2_`` prefix):
``causal_conv1d``, ``ssd_scan`` (+ ``ssd_scan_workspace_bytes``),
``gated_rmsnorm``, ``decode_step``, ``decode_step_device``, ``prefill_host`` (+
``prefill_host_workspace_bytes``), ``padded_spans``, ``pack_rows``, ``unpack_rows``,
``in_proj``, ``out_proj``, ``state_bytes_per_layer``; and the Mamba-3 SISO forward
``mamba3_siso_varlen_forward`` (C name unchanged). The operators of the recurrent block
(``include/block.h``): ``add_rmsnorm``, ``linear`` and ``gated_recurrence``, each with its
``_backward``, and ``gated_recurrence_step`` / ``gated_recurrence_step_device``;
``selective_scan_gb300.recurrent_block`` runs them together. ``selective_scan_gb300.padded`` holds the padded-batch
layer view built on them (attention mask in, HF-style cache out).
"""
from __future__ import annotations

import array
import contextlib
import ctypes
from pathlib import Path
from typing import Optional, Sequence

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libmamba2.so"

F32, BF16, E4M3 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3}
# tokens between two checkpoints of the gated recurrence, and of the chunks whose checkpoints a run has whole
RECURRENCE_STEP, RECURRENCE_CHUNK = 16, 128
(OK, ERR_INVALID_ARGUMENT, ERR_SLOT_OUT_OF_RANGE, ERR_SLOT_SHARED, ERR_RUNS_DONT_COVER_ROWS,
 ERR_NOT_IMPLEMENTED, ERR_CUDA, ERR_WORKSPACE_TOO_SMALL) = range(8)
MAX_SEQS = 1024
MAX_BLOCK_SIZE = 0x7fff0000  # most rows and columns of the recurrent block's operators


class Mamba2Error(RuntimeError):
    """A non-OK status from libmamba2; ``.status`` holds the code."""

    def __init__(self, status: int, op: str, detail: str = ""):
        msg = f"{op}: {_lib().mamba2_status_string(status).decode()}"
        if detail:
            msg += f" ({detail})"
        super().__init__(msg)
        self.status = status


class RecurrentBatch(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int32),
                ("cu_seqlens", ctypes.POINTER(ctypes.c_int32)),
                ("slots", ctypes.POINTER(ctypes.c_int32)),
                ("fresh", ctypes.POINTER(ctypes.c_uint8))]


class Dims(ctypes.Structure):
    _fields_ = [("heads", ctypes.c_int32), ("headdim", ctypes.c_int32), ("d_state", ctypes.c_int32),
                ("ngroups", ctypes.c_int32), ("conv_kernel", ctypes.c_int32)]


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not LIB_PATH.exists():
            raise ImportError(f"{LIB_PATH} is not built; run selective_scan_gb300/build.py (nvcc, sm_103a)")
        lib = ctypes.CDLL(str(LIB_PATH))
        p, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        rb, dims = ctypes.POINTER(RecurrentBatch), ctypes.POINTER(Dims)
        lib.mamba2_causal_conv1d.argtypes = [p, p, p, p, p, i32, i32, i32, i32, ctypes.c_int, rb, p]
        lib.mamba2_ssd_scan_workspace_bytes.argtypes = [dims, i32, rb]
        lib.mamba2_ssd_scan_workspace_bytes.restype = sz
        lib.mamba2_ssd_scan.argtypes = [p, p, p, p, p, p, p, i32, i32, dims, ctypes.c_int, rb, p, sz, p]
        lib.mamba2_gated_rmsnorm.argtypes = [p, p, p, p, i32, i32, i32, f32, ctypes.c_int, p]
        lib.mamba2_decode_step.argtypes = [p, p, p, p, p, p, p, p, p, p, i32, f32, p, p, i32, dims,
                                           ctypes.c_int, rb, p]
        lib.mamba2_decode_step_device.argtypes = [p, p, p, p, p, p, p, p, p, p, i32, f32, p, p, i32, dims,
                                                  ctypes.c_int, p, p, p, i32, p, p]
        lib.mamba2_in_proj.argtypes = [p, p, p, p, p, i32, i32, dims, ctypes.c_int, p]
        lib.mamba2_out_proj.argtypes = [p, p, p, i32, i32, i32, ctypes.c_int, p]
        lib.mamba2_padded_spans.argtypes = [p, i32, i32, p, p]
        lib.mamba2_pack_rows.argtypes = [p, p, i32, i32, i32, p, p, p]
        lib.mamba2_unpack_rows.argtypes = [p, p, i32, i32, i32, p, p, p]
        lib.mamba2_state_bytes_per_layer.argtypes = [dims, ctypes.c_int]
        lib.mamba2_state_bytes_per_layer.restype = ctypes.c_int64
        lib.mamba2_status_string.argtypes = [ctypes.c_int]
        lib.mamba2_status_string.restype = ctypes.c_char_p
        lib.mamba2_last_cuda_error.restype = ctypes.c_char_p
        lib.mamba2_device_timeouts.restype = ctypes.c_uint
        lib.mamba2_selftest_bounded_wait.argtypes = [p, p]
        lib.mamba2_selftest_bounded_wait.restype = ctypes.c_int
        lib.mamba2_prefill_host_workspace_bytes.argtypes = [dims, ctypes.c_int, rb, i32]
        lib.mamba2_prefill_host_workspace_bytes.restype = sz
        lib.mamba2_prefill_host.argtypes = [p, p, p, p, p, p, p, p, p, p, i32, f32, p, p, i32, dims, ctypes.c_int,
                                            rb, i32, p, sz, p]
        lib.mamba3_siso_varlen_forward.argtypes = [p] * 16 + [p, i32, i32, i32, i32, i32, i32, p]
        i64, act = ctypes.c_int64, ctypes.c_int
        lib.mamba2_gated_recurrence_checkpoints.argtypes = [p, i32]
        lib.mamba2_gated_recurrence_checkpoints.restype = i64
        lib.mamba2_gated_recurrence_workspace_bytes.argtypes = [p, i32, i32, i32]
        lib.mamba2_gated_recurrence_workspace_bytes.restype = sz
        lib.mamba2_gated_recurrence.argtypes = [p] * 6 + [i32, i32, i32, i64, i64, i64, act, rb, p, sz, p]
        lib.mamba2_gated_recurrence_step.argtypes = [p] * 5 + [i32, i32, i64, i64, i64, act, rb, p]
        lib.mamba2_gated_recurrence_step_device.argtypes = [p] * 5 + [i32, i32, i64, i64, i64, act, p, p, p, i32, p, p]
        lib.mamba2_gated_recurrence_backward.argtypes = [p] * 10 + [i32, i32, i64, i64, i64, i64, i64, act, p, i32, p,
                                                                    sz, p]
        lib.mamba2_add_rmsnorm.argtypes = [p] * 6 + [i32, i32, f32, act, act, act, p]
        lib.mamba2_add_rmsnorm_backward_workspace_bytes.argtypes = [i32, i32]
        lib.mamba2_add_rmsnorm_backward_workspace_bytes.restype = sz
        lib.mamba2_add_rmsnorm_backward.argtypes = [p] * 7 + [i32, i32, f32, act, act, p, sz, p]
        lib.mamba2_linear.argtypes = [p] * 8 + [i32, i32, i32, i64, i64, i64, act, act, act, p]
        lib.mamba2_linear_backward_workspace_bytes.argtypes = [i32, i32, i32]
        lib.mamba2_linear_backward_workspace_bytes.restype = sz
        lib.mamba2_linear_backward.argtypes = [p] * 7 + [i32, i32, i32, i64, act, p, sz, p]
        for name in ("mamba2_gated_recurrence", "mamba2_gated_recurrence_step", "mamba2_gated_recurrence_step_device",
                     "mamba2_gated_recurrence_backward", "mamba2_add_rmsnorm", "mamba2_add_rmsnorm_backward",
                     "mamba2_linear", "mamba2_linear_backward"):
            getattr(lib, name).restype = ctypes.c_int
        for name in ("mamba2_causal_conv1d", "mamba2_ssd_scan", "mamba2_gated_rmsnorm", "mamba2_decode_step",
                     "mamba2_decode_step_device", "mamba2_prefill_host", "mamba2_padded_spans", "mamba2_pack_rows",
                     "mamba2_unpack_rows", "mamba2_in_proj", "mamba2_out_proj", "mamba3_siso_varlen_forward"):
            getattr(lib, name).restype = ctypes.c_int
        _LIB = lib
    return _LIB


def library():
    """The loaded ctypes library (raises ImportError if it is not built)."""
    return _lib()


# --------------------------------------------------------------------------
# marshalling
# --------------------------------------------------------------------------

def _dt(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported activation dtype {t.dtype}")


def _alike(first, others, f32=()):
    """Shapes and types of an operator's tensors: ``others`` (name, tensor) are like ``first``; ``f32`` (name, tensor,
    shape) are fp32 of that shape; None passes. One pass without calls when all is well (it is part of every call)."""
    shape, dtype = first.shape, first.dtype
    for name, t in others:
        if t is not None and (t.shape != shape or t.dtype != dtype):
            _same(name, t, shape, dtype)
    for name, t, want in f32:
        if t is not None and (t.shape != want or t.dtype != _float32()):
            _same(name, t, want, _float32())


def _float32():
    global _float32
    import torch
    f = torch.float32
    _float32 = lambda: f  # noqa: E731
    return f


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _rows(t):
    """(pointer, row stride) of a matrix whose columns are adjacent: a contiguous one or a column range of one."""
    (rows, cols), (ld, one) = t.shape, t.stride()
    if cols > 1 and one != 1:
        raise ValueError("expected a matrix with adjacent columns")
    if rows <= 1:
        return t.data_ptr(), cols
    if ld < cols:
        raise ValueError("rows overlap")
    return t.data_ptr(), ld


def _type(t) -> int:
    import torch
    return E4M3 if t.dtype == torch.float8_e4m3fn else _dt(t)


def _same(name, t, shape, dtype=None):
    """Raises ValueError unless the tensor (None passes) has this shape, and this type where one is given."""
    if t is not None and (t.shape != shape or (dtype is not None and t.dtype != dtype)):
        raise ValueError(f"{name}: expected shape {tuple(shape)}" + (f" of {dtype}" if dtype is not None else "") +
                         f", got {tuple(t.shape)} of {t.dtype}")


def _on(stream):
    """Makes a stream (torch's, a raw handle, or another's by its ``cuda_stream``) torch's current one; None leaves the
    one that is. Handle 0 is the legacy default stream (of which ExternalStream would make a new stream)."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def _workspace(need: int, workspace, device, stream):
    """(pointer, bytes, tensor) of the caller's workspace, or of one made here; keep the tensor until the call returns.
    Its memory comes from `stream`'s own: what another stream has freed may still be in use there, and what is freed
    here goes to `stream`'s next work."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        import torch
        with _on(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace


def _current_stream() -> int:
    """The current device's current stream, without the Stream object that torch.cuda.current_stream makes (most of
    a small call's host time)."""
    global _current_stream
    import torch
    raw, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
    if raw is None or device is None:
        def current():
            return torch.cuda.current_stream().cuda_stream
    else:
        def current():
            return raw(device())
    torch.cuda.init()
    _current_stream = current
    return current()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _int32s(values):
    """A ctypes array of these ints (of one 0 if there are none). By way of array.array where it takes them: 64 in a
    third of the time."""
    if not isinstance(values, (bytes, bytearray)):
        try:
            a = array.array("i", values)
            return (ctypes.c_int32 * len(a)).from_buffer(a) if a else (ctypes.c_int32 * 1)()
        except (TypeError, OverflowError):  # floats and the like, and what c_int32 wraps
            pass
    return (ctypes.c_int32 * max(1, len(values)))(*map(int, values))


class Batch:
    """A RecurrentBatch marshalled once (host arrays kept alive); pass it as
    ``batch=`` to reuse it across calls instead of cu_seqlens/slots/fresh."""

    def __init__(self, cu_seqlens: Optional[Sequence[int]], slots: Sequence[int], fresh: Sequence[int]):
        n = len(slots)
        if cu_seqlens is not None and n > 0 and len(cu_seqlens) <= n:
            raise ValueError(f"cu_seqlens: {n} runs have {n + 1} boundaries, got {len(cu_seqlens)}")
        self.slots = _int32s(slots)
        flags = bytearray(map(bool, fresh)).ljust(max(n, 1), b"\0")
        if len(flags) > max(n, 1):
            raise IndexError("fresh: more entries than slots")
        self.fresh = (ctypes.c_uint8 * len(flags)).from_buffer(flags)
        self.cu = None if cu_seqlens is None else _int32s(cu_seqlens)
        self.rb = RecurrentBatch(n, self.cu, self.slots, self.fresh)  # (arrays pass as the pointers)

    def ref(self):
        return ctypes.byref(self.rb)


_Batch = Batch


def _batch(cu_seqlens, slots, fresh, batch):
    return batch if batch is not None else Batch(cu_seqlens, slots, fresh)


def _dims(d) -> Dims:
    if isinstance(d, Dims):
        return d
    return Dims(int(d.heads), int(d.headdim), int(d.d_state), int(d.ngroups), int(d.conv_kernel))


def _check(st: int, op: str):
    if st != OK:
        detail = _lib().mamba2_last_cuda_error().decode() if st == ERR_CUDA else ""
        raise Mamba2Error(st, op, detail)


# --------------------------------------------------------------------------
# entry points
# --------------------------------------------------------------------------

def causal_conv1d(dst, x, weight, bias, conv_state, cu_seqlens=None, slots=None, fresh=None, stream=None,
                  check=True, batch=None) -> int:
    """``mamba2_causal_conv1d``: dst = silu(depthwise causal conv) per run; conv_state updated."""
    rows, conv_dim = x.shape
    b = _batch(cu_seqlens, slots, fresh, batch)
    st = _lib().mamba2_causal_conv1d(_ptr(dst), _ptr(x), _ptr(weight), _ptr(bias), _ptr(conv_state),
                                     conv_state.shape[0], rows, conv_dim, weight.shape[1], _dt(x), b.ref(),
                                     _stream(stream))
    if check:
        _check(st, "mamba2_causal_conv1d")
    return st


def ssd_scan_workspace_bytes(dims, rows, cu_seqlens=None, slots=None, fresh=None, batch=None) -> int:
    """``mamba2_ssd_scan_workspace_bytes`` for this batch on the current device."""
    b = _batch(cu_seqlens, slots, fresh, batch)
    d = _dims(dims)
    return int(_lib().mamba2_ssd_scan_workspace_bytes(ctypes.byref(d), int(rows), b.ref()))


def ssd_scan(dst, xbc, dt, A_log, dt_bias, D, ssm_state, dims, cu_seqlens=None, slots=None, fresh=None,
             workspace=None, stream=None, check=True, batch=None) -> int:
    """``mamba2_ssd_scan``: chunked selective scan; ssm_state updated at the slots.

    ``workspace`` is a device tensor of at least ``ssd_scan_workspace_bytes`` bytes
    (allocated here with torch when None and needed).
    """
    rows = xbc.shape[0]
    d = _dims(dims)
    b = _batch(cu_seqlens, slots, fresh, batch)
    need = int(_lib().mamba2_ssd_scan_workspace_bytes(ctypes.byref(d), rows, b.ref())) if workspace is None else 0
    ws_ptr, ws_bytes, _keep = _workspace(need, workspace, xbc.device, stream)
    st = _lib().mamba2_ssd_scan(_ptr(dst), _ptr(xbc), _ptr(dt), _ptr(A_log), _ptr(dt_bias), _ptr(D),
                                _ptr(ssm_state), ssm_state.shape[0], rows, ctypes.byref(d), _dt(xbc), b.ref(),
                                ws_ptr, ws_bytes, _stream(stream))
    if check:
        _check(st, "mamba2_ssd_scan")
    return st


def gated_rmsnorm(dst, x, z, weight, groups, eps, stream=None, check=True) -> int:
    """``mamba2_gated_rmsnorm``: dst = rmsnorm(x * silu(z)) * weight per group."""
    rows, dim = x.shape
    st = _lib().mamba2_gated_rmsnorm(_ptr(dst), _ptr(x), _ptr(z), _ptr(weight), rows, dim, int(groups),
                                     float(eps), _dt(x), _stream(stream))
    if check:
        _check(st, "mamba2_gated_rmsnorm")
    return st


def decode_step(dst, xBC, z, dt, conv_w, conv_b, A_log, dt_bias, D, norm_w, norm_groups, eps,
                conv_state, ssm_state, dims, slots=None, fresh=None, cu_seqlens=None, stream=None, check=True,
                batch=None) -> int:
    """``mamba2_decode_step``: fused conv -> scan -> gated norm for one token per sequence."""
    d = _dims(dims)
    b = _batch(cu_seqlens, slots, fresh, batch)
    st = _lib().mamba2_decode_step(_ptr(dst), _ptr(xBC), _ptr(z), _ptr(dt), _ptr(conv_w), _ptr(conv_b),
                                   _ptr(A_log), _ptr(dt_bias), _ptr(D), _ptr(norm_w), int(norm_groups),
                                   float(eps), _ptr(conv_state), _ptr(ssm_state), ssm_state.shape[0],
                                   ctypes.byref(d), _dt(xBC), b.ref(), _stream(stream))
    if check:
        _check(st, "mamba2_decode_step")
    return st


def decode_step_device(dst, xBC, z, dt, conv_w, conv_b, A_log, dt_bias, D, norm_w, norm_groups, eps,
                       conv_state, ssm_state, dims, slots_dev, fresh_dev, num_seqs_dev, status_dev,
                       stream=None, check=True) -> int:
    """``mamba2_decode_step_device``: the fused decode step with its batch in device memory.

    ``slots_dev`` (int32), ``fresh_dev`` (uint8) are device tensors of the capacity
    (their length); ``num_seqs_dev`` and ``status_dev`` are one-element int32 device
    tensors. The batch is checked on the device: ``status_dev`` holds the outcome once
    the stream has passed the call. The return value covers the host checks only.
    """
    d = _dims(dims)
    st = _lib().mamba2_decode_step_device(_ptr(dst), _ptr(xBC), _ptr(z), _ptr(dt), _ptr(conv_w), _ptr(conv_b),
                                          _ptr(A_log), _ptr(dt_bias), _ptr(D), _ptr(norm_w), int(norm_groups),
                                          float(eps), _ptr(conv_state), _ptr(ssm_state), ssm_state.shape[0],
                                          ctypes.byref(d), _dt(xBC), _ptr(slots_dev), _ptr(fresh_dev),
                                          _ptr(num_seqs_dev), int(slots_dev.shape[0]), _ptr(status_dev),
                                          _stream(stream))
    if check:
        _check(st, "mamba2_decode_step_device")
    return st


def in_proj(z, xBC, dt, hidden, w_in, dims, stream=None, check=True) -> int:
    """``mamba2_in_proj``: hidden . w_in^T split into z, xBC, dt (tcgen05 GEMM, bf16)."""
    d = _dims(dims)
    st = _lib().mamba2_in_proj(_ptr(z), _ptr(xBC), _ptr(dt), _ptr(hidden), _ptr(w_in), hidden.shape[0],
                               hidden.shape[1], ctypes.byref(d), _dt(hidden), _stream(stream))
    if check:
        _check(st, "mamba2_in_proj")
    return st


def out_proj(out, x, w_out, stream=None, check=True) -> int:
    """``mamba2_out_proj``: out = x . w_out^T (tcgen05 GEMM, bf16)."""
    st = _lib().mamba2_out_proj(_ptr(out), _ptr(x), _ptr(w_out), x.shape[0], x.shape[1], w_out.shape[0], _dt(x),
                                _stream(stream))
    if check:
        _check(st, "mamba2_out_proj")
    return st


def padded_spans(mask):
    """``mamba2_padded_spans``: (cu_seqlens, first) lists of a [batch, seqlen] host mask
    (nonzero = token); raises Mamba2Error when a row's tokens are not one span."""
    import torch
    m = mask.to(torch.uint8).contiguous()
    batch, seqlen = int(m.shape[0]), int(m.shape[1])
    cu = (ctypes.c_int32 * (batch + 1))()
    first = (ctypes.c_int32 * max(batch, 1))()
    st = _lib().mamba2_padded_spans(m.data_ptr() if m.numel() else None, batch, seqlen, cu, first)
    _check(st, "mamba2_padded_spans")
    return list(cu), list(first)[:batch]


def _pack(fn, name, dst, src, batch, seqlen, width_bytes, cu_seqlens, first, stream, check):
    cu = (ctypes.c_int32 * (len(cu_seqlens)))(*[int(v) for v in cu_seqlens])
    fi = (ctypes.c_int32 * max(len(first), 1))(*[int(v) for v in first])
    st = fn(_ptr(dst), _ptr(src), int(batch), int(seqlen), int(width_bytes), cu, fi, _stream(stream))
    if check:
        _check(st, name)
    return st


def pack_rows(dst, src, cu_seqlens, first, stream=None, check=True) -> int:
    """``mamba2_pack_rows``: padded ``src`` [batch, seqlen, ...] -> packed ``dst`` [rows, ...]."""
    width = src[0, 0].numel() * src.element_size() if src.numel() else dst.shape[-1] * dst.element_size()
    return _pack(_lib().mamba2_pack_rows, "mamba2_pack_rows", dst, src, src.shape[0], src.shape[1], width,
                 cu_seqlens, first, stream, check)


def unpack_rows(dst, src, cu_seqlens, first, stream=None, check=True) -> int:
    """``mamba2_unpack_rows``: packed ``src`` [rows, ...] -> padded ``dst`` [batch, seqlen, ...], zeros at padding."""
    width = dst[0, 0].numel() * dst.element_size() if dst.numel() else src.shape[-1] * src.element_size()
    return _pack(_lib().mamba2_unpack_rows, "mamba2_unpack_rows", dst, src, dst.shape[0], dst.shape[1], width,
                 cu_seqlens, first, stream, check)


def prefill_host_workspace_bytes(dims, act: int, piece_rows: int, cu_seqlens=None, slots=None, fresh=None,
                                 batch=None) -> int:
    """``mamba2_prefill_host_workspace_bytes`` for this batch and piece size."""
    b = _batch(cu_seqlens, slots, fresh, batch)
    d = _dims(dims)
    return int(_lib().mamba2_prefill_host_workspace_bytes(ctypes.byref(d), int(act), b.ref(), int(piece_rows)))


def prefill_host(out_host, xBC_host, z_host, dt_host, conv_w, conv_b, A_log, dt_bias, D, norm_w, norm_groups, eps,
                 conv_state, ssm_state, dims, cu_seqlens=None, slots=None, fresh=None, piece_rows=8192,
                 workspace=None, stream=None, check=True, batch=None) -> int:
    """``mamba2_prefill_host``: conv -> scan -> gated norm from host tensors, streamed in pieces.

    ``out_host``, ``xBC_host``, ``z_host``, ``dt_host`` are CPU tensors (pinned for
    overlap); the weights and pools are device tensors. ``workspace`` is a device
    tensor of at least ``prefill_host_workspace_bytes`` bytes (allocated here with
    torch when None). Asynchronous: synchronise the stream before reading ``out_host``.
    """
    d = _dims(dims)
    b = _batch(cu_seqlens, slots, fresh, batch)
    act = _dt(xBC_host)
    need = 0
    if workspace is None:
        need = max(1, int(_lib().mamba2_prefill_host_workspace_bytes(ctypes.byref(d), act, b.ref(), int(piece_rows))))
    ws_ptr, ws_bytes, _keep = _workspace(need, workspace, ssm_state.device, stream)
    st = _lib().mamba2_prefill_host(_ptr(out_host), _ptr(xBC_host), _ptr(z_host), _ptr(dt_host), _ptr(conv_w),
                                    _ptr(conv_b), _ptr(A_log), _ptr(dt_bias), _ptr(D), _ptr(norm_w), int(norm_groups),
                                    float(eps), _ptr(conv_state), _ptr(ssm_state), ssm_state.shape[0], ctypes.byref(d),
                                    act, b.ref(), int(piece_rows), ws_ptr, ws_bytes, _stream(stream))
    if check:
        _check(st, "mamba2_prefill_host")
    return st


def mamba3_siso_varlen_forward(out, final_angle, final_ssm, final_k, final_v, q, k, v, adt, dt, trap, q_bias,
                               k_bias, angles, d, z, cu_seqlens, stream=None, check=True) -> int:
    """``mamba3_siso_varlen_forward`` (include/mamba3.h): the Mamba-3 SISO forward over a
    packed batch. q, k [rows, d_state]; v, z, out [rows, heads, headdim]; adt, dt, trap
    [rows, heads]; angles [rows, rot_dim]; biases [heads, d_state]; d [heads]; the final
    states [num_seqs, heads, ...]; cu_seqlens a host sequence."""
    cu = list(cu_seqlens)
    n = len(cu) - 1
    rows, heads, headdim = v.shape
    arr = (ctypes.c_int32 * max(1, len(cu)))(*cu)
    st = _lib().mamba3_siso_varlen_forward(
        _ptr(out), _ptr(final_angle), _ptr(final_ssm), _ptr(final_k), _ptr(final_v), _ptr(q), _ptr(k), _ptr(v),
        _ptr(adt), _ptr(dt), _ptr(trap), _ptr(q_bias), _ptr(k_bias), _ptr(angles), _ptr(d), _ptr(z), arr, n,
        int(rows), int(heads), int(headdim), int(q.shape[1]), int(angles.shape[1]), _stream(stream))
    if check:
        _check(st, "mamba3_siso_varlen_forward")
    return st


def _cu(cu_seqlens):
    return cu_seqlens if isinstance(cu_seqlens, ctypes.Array) else _int32s(cu_seqlens)


def gated_recurrence_checkpoints(cu_seqlens) -> int:
    """``mamba2_gated_recurrence_checkpoints``: rows of the ``checkpoints`` of a batch with these runs."""
    cu = _cu(cu_seqlens)
    n = int(_lib().mamba2_gated_recurrence_checkpoints(cu, len(cu) - 1))
    if n < 0:
        raise Mamba2Error(ERR_RUNS_DONT_COVER_ROWS, "mamba2_gated_recurrence_checkpoints")
    return n


def gated_recurrence_workspace_bytes(cu_seqlens, dim, backward=False) -> int:
    """``mamba2_gated_recurrence_workspace_bytes`` of the forward or backward call."""
    cu = _cu(cu_seqlens)
    return int(_lib().mamba2_gated_recurrence_workspace_bytes(cu, len(cu) - 1, int(dim), 1 if backward else 0))


def gated_recurrence(y, x, gate, lower, state, cu_seqlens=None, slots=None, fresh=None, checkpoints=None,
                     workspace=None, stream=None, check=True, batch=None) -> int:
    """``mamba2_gated_recurrence``: h_t = f_t h_{t-1} + (1 - f_t) x_t over packed runs, f from ``gate`` and the
    lower bounds; ``state`` updated at the slots. x, gate and y may be column ranges of wider matrices.
    ``checkpoints`` [gated_recurrence_checkpoints(cu_seqlens), dim] f32 is for the backward pass."""
    rows, dim = x.shape
    b = _batch(cu_seqlens, slots, fresh, batch)
    _alike(x, (("gate", gate), ("y", y)), (("lower", lower, (dim,)), ("state", state, (state.shape[0], dim))))
    if checkpoints is not None and b.cu is not None:
        _same("checkpoints", checkpoints, (gated_recurrence_checkpoints(b.cu), dim), _float32())
    need = gated_recurrence_workspace_bytes(b.cu, dim) if workspace is None and b.cu is not None else 0
    ws, ws_bytes, _keep = _workspace(need, workspace, x.device, stream)
    (yp, ly), (xp, lx), (gp, lg) = _rows(y), _rows(x), _rows(gate)
    st = _lib().mamba2_gated_recurrence(yp, _ptr(checkpoints), xp, gp, _ptr(lower), _ptr(state), state.shape[0], rows,
                                        dim, ly, lx, lg, _dt(x), b.ref(), ws, ws_bytes, _stream(stream))
    if check:
        _check(st, "mamba2_gated_recurrence")
    return st


def gated_recurrence_step(y, x, gate, lower, state, slots=None, fresh=None, cu_seqlens=None, stream=None, check=True,
                          batch=None) -> int:
    """``mamba2_gated_recurrence_step``: one token per sequence."""
    import torch
    b = _batch(cu_seqlens, slots, fresh, batch)
    dim = x.shape[1]
    _same("x", x, (b.rb.num_seqs, dim))
    _same("gate", gate, x.shape, x.dtype)
    _same("y", y, x.shape, x.dtype)
    _same("lower", lower, (dim,), torch.float32)
    _same("state", state, (state.shape[0], dim), torch.float32)
    (yp, ly), (xp, lx), (gp, lg) = _rows(y), _rows(x), _rows(gate)
    st = _lib().mamba2_gated_recurrence_step(yp, xp, gp, _ptr(lower), _ptr(state), state.shape[0], dim, ly, lx, lg,
                                             _dt(x), b.ref(), _stream(stream))
    if check:
        _check(st, "mamba2_gated_recurrence_step")
    return st


def gated_recurrence_step_device(y, x, gate, lower, state, slots_dev, fresh_dev, num_seqs_dev, status_dev, stream=None,
                                 check=True) -> int:
    """``mamba2_gated_recurrence_step_device``: the step with its batch in device memory, as ``decode_step_device``
    takes it (``fresh_dev`` may be None: no sequence is fresh)."""
    import torch
    cap, dim, num_slots, i32 = slots_dev.shape[0], x.shape[1], state.shape[0], torch.int32
    _alike(x, (("gate", gate), ("y", y)), (("lower", lower, (dim,)), ("state", state, (num_slots, dim))))
    if (x.shape[0] != cap or slots_dev.dtype != i32 or num_seqs_dev.dtype != i32 or status_dev.dtype != i32 or
            num_seqs_dev.numel() != 1 or status_dev.numel() != 1 or slots_dev.dim() != 1 or
            (fresh_dev is not None and (fresh_dev.dtype != torch.uint8 or fresh_dev.shape[0] != cap))):
        _same("x", x, (cap, dim))
        _same("slots_dev", slots_dev, (cap,), i32)
        _same("fresh_dev", fresh_dev, (cap,), torch.uint8)
        _same("num_seqs_dev", num_seqs_dev, (1,), i32)
        _same("status_dev", status_dev, (1,), i32)
    (yp, ly), (xp, lx), (gp, lg) = _rows(y), _rows(x), _rows(gate)
    st = _lib().mamba2_gated_recurrence_step_device(yp, xp, gp, _ptr(lower), _ptr(state), num_slots, dim, ly, lx,
                                                    lg, _dt(x), _ptr(slots_dev), _ptr(fresh_dev), _ptr(num_seqs_dev),
                                                    cap, _ptr(status_dev), _stream(stream))
    if check:
        _check(st, "mamba2_gated_recurrence_step_device")
    return st


def gated_recurrence_backward(dx, dgate, dlower, dstate, dy, dstate_end, x, gate, lower, checkpoints, cu_seqlens,
                              workspace=None, stream=None, check=True) -> int:
    """``mamba2_gated_recurrence_backward``: gradients of x, gate, lower and the initial states (``dlower``, ``dstate``
    and ``dstate_end`` may be None) from the forward call's checkpoints."""
    import torch
    rows, dim = x.shape
    cu = _cu(cu_seqlens)
    n = len(cu) - 1
    for name, t in (("gate", gate), ("dy", dy), ("dx", dx), ("dgate", dgate)):
        _same(name, t, x.shape, x.dtype)
    for name, t in (("lower", lower), ("dlower", dlower)):
        _same(name, t, (dim,), torch.float32)
    for name, t in (("dstate", dstate), ("dstate_end", dstate_end)):
        _same(name, t, (n, dim), torch.float32)
    _same("checkpoints", checkpoints, (gated_recurrence_checkpoints(cu), dim), torch.float32)
    need = gated_recurrence_workspace_bytes(cu, dim, True) if workspace is None else 0
    ws, ws_bytes, _keep = _workspace(need, workspace, x.device, stream)
    (dxp, ldx), (dgp, ldg), (dyp, ldy), (xp, lx), (gp, lg) = _rows(dx), _rows(dgate), _rows(dy), _rows(x), _rows(gate)
    st = _lib().mamba2_gated_recurrence_backward(dxp, dgp, _ptr(dlower), _ptr(dstate), dyp, _ptr(dstate_end), xp, gp,
                                                 _ptr(lower), _ptr(checkpoints), rows, dim, ldx, ldg, ldy, lx, lg,
                                                 _dt(x), cu, n, ws, ws_bytes, _stream(stream))
    if check:
        _check(st, "mamba2_gated_recurrence_backward")
    return st


def add_rmsnorm(out, x, weight, eps, residual=None, sum=None, scale=None, stream=None, check=True) -> int:
    """``mamba2_add_rmsnorm``: s = x + residual, out = s / rms(s) * weight; ``sum`` gets s (it may be ``residual``).
    An e4m3 ``out`` takes a ``scale`` per row: out * scale is the normed row."""
    rows, dim = x.shape
    wide = residual if residual is not None else sum
    stype = _dt(wide) if wide is not None else _dt(x)
    if out.shape != x.shape:
        _same("out", out, x.shape)
    if wide is not None:
        _same("sum", wide, x.shape)
    _alike(wide if wide is not None else x, (("sum", sum),), (("weight", weight, (dim,)), ("scale", scale, (rows,))))
    st = _lib().mamba2_add_rmsnorm(_ptr(out), _ptr(scale), _ptr(sum), _ptr(x), _ptr(residual), _ptr(weight), rows, dim,
                                   float(eps), _dt(x), stype, _type(out), _stream(stream))
    if check:
        _check(st, "mamba2_add_rmsnorm")
    return st


def add_rmsnorm_backward(dx, dresidual, dweight, dy, dsum, sum, weight, eps, workspace=None, stream=None,
                         check=True) -> int:
    """``mamba2_add_rmsnorm_backward``: from ``sum`` and the gradients of both outputs (``dsum`` may be None) to those
    of x, the residual and the weight (each may be None). ``dresidual`` may be ``dsum`` itself."""
    import torch
    rows, dim = sum.shape
    _same("dy", dy, sum.shape)
    _same("dx", dx, sum.shape, dy.dtype)
    _same("dresidual", dresidual, sum.shape, sum.dtype)
    _same("dsum", dsum, sum.shape, sum.dtype)
    _same("weight", weight, (dim,), torch.float32)
    _same("dweight", dweight, (dim,), torch.float32)
    need = 0
    if workspace is None and dweight is not None:
        need = int(_lib().mamba2_add_rmsnorm_backward_workspace_bytes(rows, dim))
    ws, ws_bytes, _keep = _workspace(need, workspace, sum.device, stream)
    st = _lib().mamba2_add_rmsnorm_backward(_ptr(dx), _ptr(dresidual), _ptr(dweight), _ptr(dy), _ptr(dsum), _ptr(sum),
                                            _ptr(weight), rows, dim, float(eps), _dt(dy), _dt(sum), ws, ws_bytes,
                                            _stream(stream))
    if check:
        _check(st, "mamba2_add_rmsnorm_backward")
    return st


def linear(out, x, w, x_scale=None, w_scale=None, bias=None, residual=None, activation="none", pre=None, stream=None,
           check=True) -> int:
    """``mamba2_linear``: out = activation(x . w^T * scales + bias) + residual from bf16 or e4m3 operands. x, out and
    residual may be column ranges of wider matrices; ``pre`` gets the pre-activation for the backward pass."""
    (rows, k), n = x.shape, w.shape[0]
    if out.shape != (rows, n) or w.shape != (n, k) or w.dtype != x.dtype:
        _same("w", w, (n, k), x.dtype)
        _same("out", out, (rows, n))
    _alike(out, (("residual", residual),), (("x_scale", x_scale, (rows,)), ("w_scale", w_scale, (n,)), ("bias", bias, (n,))))
    if pre is not None:
        import torch
        _same("pre", pre, (rows, n), torch.bfloat16)
    (op, lo), (xp, lx) = _rows(out), _rows(x)
    rp, lr = _rows(residual) if residual is not None else (None, 0)
    st = _lib().mamba2_linear(op, _ptr(pre), xp, _ptr(x_scale), _ptr(w), _ptr(w_scale), _ptr(bias), rp, rows, k, n, lo,
                              lx, lr, _type(x), _dt(out), ACTIVATIONS[activation], _stream(stream))
    if check:
        _check(st, "mamba2_linear")
    return st


def linear_backward(dx, dw, dbias, dy, x, w, activation="none", pre=None, workspace=None, stream=None,
                    check=True) -> int:
    """``mamba2_linear_backward``: gradients of x, w and bias (each may be None) from dy and the forward's ``pre``."""
    import torch
    (rows, k), n = x.shape, w.shape[0]
    bf16 = torch.bfloat16
    _same("x", x, (rows, k), bf16)
    _same("w", w, (n, k), bf16)
    _same("dy", dy, (rows, n), bf16)
    _same("pre", pre, (rows, n), bf16)
    _same("dx", dx, (rows, k), bf16)
    _same("dw", dw, (n, k), bf16)
    _same("dbias", dbias, (n,), torch.float32)
    need = int(_lib().mamba2_linear_backward_workspace_bytes(rows, k, n)) if workspace is None else 0
    ws, ws_bytes, _keep = _workspace(need, workspace, x.device, stream)
    xp, lx = _rows(x)
    st = _lib().mamba2_linear_backward(_ptr(dx), _ptr(dw), _ptr(dbias), _ptr(dy), _ptr(pre), xp, _ptr(w), rows, k, n,
                                       lx, ACTIVATIONS[activation], ws, ws_bytes, _stream(stream))
    if check:
        _check(st, "mamba2_linear_backward")
    return st


def state_bytes_per_layer(dims, conv_dtype: int = BF16) -> int:
    """``mamba2_state_bytes_per_layer``: fp32 SSM state + conv history per sequence per layer."""
    d = _dims(dims)
    return int(_lib().mamba2_state_bytes_per_layer(ctypes.byref(d), int(conv_dtype)))


def status_string(status: int) -> str:
    return _lib().mamba2_status_string(int(status)).decode()
