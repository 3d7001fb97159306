"""Residual vector quantisation (RVQ) encode and decode on one GB300 GPU.

A thin ctypes binding over the C ABI of include/rvq.h (librvq.so, built for
sm_103a by residual_vector_quantisation_gb300.build).  The functions below
carry the C names and only marshal arguments: torch tensors become device
pointers and the current CUDA stream.  Every step of encode and decode runs in
the library's CUDA kernels; there is no CPU path.  Loading fails loudly when
the library has not been built.

    from residual_vector_quantisation_gb300 import RVQ
    rvq = RVQ(w_in, codebook, w_out, b_in=None, b_out=None)   # cuda float32 tensors
    codes = rvq.encode(x)            # [N][n_q] int32
    y = rvq.decode(codes)            # [N][D] float32
    codes, x_hat = rvq.reconstruct(x)
"""

from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from . import build as _build

__all__ = [
    "RVQError", "load_library", "library_path", "rvq_dims", "rvq_weights",
    "rvq_dims_supported", "rvq_tables_bytes", "rvq_prepare", "rvq_encode_scratch_bytes",
    "rvq_encode_min_scratch_bytes", "rvq_encode", "rvq_decode", "rvq_reconstruct",
    "rvq_status_string", "rvq_version", "rvq_encode_static", "RVQ_STATIC_SCRATCH_BYTES", "RVQ",
    "EXPORTED_SYMBOLS", "rvq_pipeline_workspace_bytes", "rvq_pipeline_create", "rvq_pipeline_destroy",
    "rvq_pipeline_reconstruct", "RVQPipeline", "rvq_set_stream_max_frames", "rvq_stream_plan",
    "rvq_read_status", "rvq_read_error_count", "rvq_pipeline_set_cancel", "RVQ_CANCEL_FN",
    "rvq_norm_dims", "rvq_layer_norm", "rvq_layer_norm_workspace_bytes", "rvq_layer_norm_backward",
    "rvq_distill_dims", "rvq_distill", "rvq_distill_backward", "rvq_beam_dims", "rvq_beam_workspace_bytes",
    "rvq_beam_select", "rvq_beam_state", "rvq_beam_states", "rvq_beam_reorder", "RVQ_BEAM_LOGITS", "RVQ_BEAM_RAW",
    "RVQ_BEAM_MAX_STATES", "DTYPES", "layer_norm", "distill_loss", "distill_loss_and_grad", "BeamSearch",
    "rvq_dropout_mask", "rvq_dropout_dims", "rvq_dropout", "dropout", "rvq_rms_8bit", "rvq_rms_norm",
    "rvq_rms_norm_workspace_bytes", "rvq_rms_norm_backward", "RVQ_SCALE_F32", "RVQ_SCALE_E8M0", "rms_norm",
    "rms_norm_8bit", "rvq_log_probs_dims", "rvq_log_probs", "rvq_log_probs_backward", "log_probs", "LogProbs",
]

RVQ_OK = 0
STATUS_NAMES = {0: "RVQ_OK", -1: "RVQ_ERR_INVALID_ARG", -2: "RVQ_ERR_UNSUPPORTED",
                -3: "RVQ_ERR_WORKSPACE", -4: "RVQ_ERR_CUDA", -5: "RVQ_ERR_TIMEOUT",
                -6: "RVQ_ERR_CANCELLED", -7: "RVQ_ERR_INTERNAL"}
RVQ_ERR_TIMEOUT = -5
RVQ_ERR_CANCELLED = -6
RVQ_ERR_INTERNAL = -7

EXPORTED_SYMBOLS = [
    "rvq_dims_supported", "rvq_tables_bytes", "rvq_prepare", "rvq_encode_scratch_bytes",
    "rvq_encode_min_scratch_bytes", "rvq_encode", "rvq_decode", "rvq_reconstruct",
    "rvq_status_string", "rvq_version", "rvq_encode_static", "rvq_pipeline_workspace_bytes",
    "rvq_pipeline_create", "rvq_pipeline_destroy", "rvq_pipeline_reconstruct", "rvq_set_stream_max_frames",
    "rvq_stream_plan", "rvq_read_status", "rvq_read_error_count", "rvq_pipeline_set_cancel",
    "rvq_layer_norm", "rvq_layer_norm_workspace_bytes", "rvq_layer_norm_backward", "rvq_distill",
    "rvq_distill_backward", "rvq_beam_workspace_bytes", "rvq_beam_select", "rvq_beam_reorder",
    "rvq_dropout", "rvq_rms_norm", "rvq_rms_norm_workspace_bytes", "rvq_rms_norm_backward",
    "rvq_log_probs", "rvq_log_probs_backward",
]

# int (*rvq_cancel_fn)(void *user)
RVQ_CANCEL_FN = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_void_p)

RVQ_STATIC_SCRATCH_BYTES = 16 << 20  # include/rvq.h


class RVQError(RuntimeError):
    def __init__(self, func: str, status: int):
        self.status = status
        super().__init__(f"{func} returned {STATUS_NAMES.get(status, status)}")


RVQ_METRIC_L2 = 0       # include/rvq.h
RVQ_METRIC_COSINE = 1
METRICS = {"l2": RVQ_METRIC_L2, "cosine": RVQ_METRIC_COSINE}
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}  # RVQ_DTYPE_*
RVQ_BEAM_LOGITS = 0
RVQ_BEAM_RAW = 1
RVQ_BEAM_MAX_STATES = 32
RVQ_SCALE_F32 = 0
RVQ_SCALE_E8M0 = 1
SCALES = {torch.float32: RVQ_SCALE_F32, torch.float8_e8m0fnu: RVQ_SCALE_E8M0}


class rvq_dims(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int32), ("d", ctypes.c_int32), ("K", ctypes.c_int32), ("Q", ctypes.c_int32),
                ("metric", ctypes.c_int32), ("D_in", ctypes.c_int32), ("D_out", ctypes.c_int32)]


class rvq_weights(ctypes.Structure):
    _fields_ = [("w_in", ctypes.c_void_p), ("b_in", ctypes.c_void_p), ("codebook", ctypes.c_void_p),
                ("w_out", ctypes.c_void_p), ("b_out", ctypes.c_void_p), ("fc_w", ctypes.c_void_p),
                ("fc_b", ctypes.c_void_p), ("fc2_w", ctypes.c_void_p), ("fc2_b", ctypes.c_void_p)]


class rvq_norm_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("param_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class rvq_distill_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int32), ("top", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("top_dtype", ctypes.c_int32), ("temperature", ctypes.c_float)]


class rvq_dropout_mask(ctypes.Structure):
    """What stays in a dropout (see rvq.h): p, seed, offset, and step: None, or a tensor of one int64 on the GPU, which
    the mask keeps alive."""

    _fields_ = [("p", ctypes.c_float), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64), ("step", ctypes.c_void_p)]

    def __init__(self, p: float, seed: int, offset: int = 0, step: Optional[torch.Tensor] = None):
        if not (0 <= seed < 1 << 64 and 0 <= offset < 1 << 64):
            raise ValueError("seed and offset must be numbers of 64 bits, not negative")
        if step is not None and not (step.is_cuda and step.dtype is torch.int64 and step.numel() == 1):
            raise ValueError("step must be one int64 on the GPU")
        super().__init__(p, seed, offset, None if step is None else step.data_ptr())
        self.tensor = step

    def copy(self) -> "rvq_dropout_mask":
        """The same mask, with the same step; changes of one's fields do not reach the other."""
        other = rvq_dropout_mask.from_buffer_copy(self)
        other.tensor = self.tensor
        return other


class rvq_dropout_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("width", ctypes.c_int64), ("dtype", ctypes.c_int32)]


class rvq_rms_8bit(ctypes.Structure):
    _fields_ = [("values", ctypes.c_void_p), ("stride", ctypes.c_int64), ("scales", ctypes.c_void_p),
                ("block", ctypes.c_int32), ("scale_type", ctypes.c_int32)]


class rvq_log_probs_dims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int32), ("top", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("temperature", ctypes.c_float)]


class rvq_beam_dims(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int64), ("beams", ctypes.c_int32), ("vocab", ctypes.c_int32),
                ("select", ctypes.c_int32), ("mode", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class rvq_beam_state(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("layers", ctypes.c_int64),
                ("row_bytes", ctypes.c_int64), ("src_layer_stride", ctypes.c_int64),
                ("src_group_stride", ctypes.c_int64), ("src_beam_stride", ctypes.c_int64),
                ("dst_layer_stride", ctypes.c_int64), ("dst_group_stride", ctypes.c_int64),
                ("dst_beam_stride", ctypes.c_int64)]


_lib = None


def library_path() -> str:
    return _build.LIB


def load_library(path: Optional[str] = None):
    """Load librvq.so.  Raises if it has not been built (no fallback exists)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or _build.LIB
    if not os.path.exists(p):
        raise RuntimeError(f"RVQ CUDA library not built ({p} missing); run "
                           "`python -m residual_vector_quantisation_gb300.build` first")
    lib = ctypes.CDLL(p)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "rvq_dims_supported": ([rvq_dims], ctypes.c_int),
        "rvq_tables_bytes": ([rvq_dims], sz),
        "rvq_prepare": ([rvq_dims, ctypes.POINTER(rvq_weights), vp, sz, vp], ctypes.c_int),
        "rvq_encode_scratch_bytes": ([rvq_dims, i64, i32], sz),
        "rvq_encode_min_scratch_bytes": ([rvq_dims, i32], sz),
        "rvq_encode": ([rvq_dims, vp, vp, i64, i32, vp, vp, sz, vp], ctypes.c_int),
        "rvq_decode": ([rvq_dims, vp, vp, i64, i32, vp, vp, vp], ctypes.c_int),
        "rvq_reconstruct": ([rvq_dims, vp, vp, i64, i32, vp, vp, vp, sz, vp], ctypes.c_int),
        "rvq_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "rvq_version": ([], ctypes.c_char_p),
        "rvq_encode_static": ([rvq_dims, vp, vp, i64, i32, vp, vp], ctypes.c_int),
        "rvq_pipeline_workspace_bytes": ([rvq_dims, i32, i64], sz),
        "rvq_pipeline_create": ([rvq_dims, i32, i64, vp, sz, ctypes.POINTER(vp)], ctypes.c_int),
        "rvq_pipeline_destroy": ([vp], ctypes.c_int),
        "rvq_pipeline_reconstruct": ([vp, vp, vp, i64, vp, vp], ctypes.c_int),
        "rvq_set_stream_max_frames": ([i64], i64),
        "rvq_stream_plan": ([rvq_dims, i32, i64, ctypes.POINTER(i64)], ctypes.c_int),
        "rvq_read_status": ([vp, vp], ctypes.c_int),
        "rvq_read_error_count": ([vp, ctypes.POINTER(i64), vp], ctypes.c_int),
        "rvq_pipeline_set_cancel": ([vp, RVQ_CANCEL_FN, vp], ctypes.c_int),
        "rvq_layer_norm": ([rvq_norm_dims, vp, i64, vp, vp, vp, i64, vp, vp, vp], ctypes.c_int),
        "rvq_layer_norm_workspace_bytes": ([i64, i32], sz),
        "rvq_layer_norm_backward": ([rvq_norm_dims, vp, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, vp, sz, vp],
                                    ctypes.c_int),
        "rvq_distill": ([rvq_distill_dims, vp, i64, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp], ctypes.c_int),
        "rvq_distill_backward": ([rvq_distill_dims, vp, vp, i64, vp, vp, vp, vp, vp, vp, i64, vp], ctypes.c_int),
        "rvq_dropout": ([rvq_dropout_dims, vp, i64, vp, i64, ctypes.POINTER(rvq_dropout_mask), vp, i64, vp],
                        ctypes.c_int),
        "rvq_rms_norm": ([rvq_norm_dims, vp, i64, vp, i64, ctypes.POINTER(rvq_dropout_mask), vp, vp, i64, vp, i64, vp,
                          ctypes.POINTER(rvq_rms_8bit), vp], ctypes.c_int),
        "rvq_rms_norm_workspace_bytes": ([i64, i32], sz),
        "rvq_rms_norm_backward": ([rvq_norm_dims, vp, i64, vp, i64, vp, i64, ctypes.POINTER(rvq_dropout_mask), vp, vp,
                                   vp, i64, vp, i64, vp, vp, sz, vp], ctypes.c_int),
        "rvq_log_probs": ([rvq_log_probs_dims, vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp], ctypes.c_int),
        "rvq_log_probs_backward": ([rvq_log_probs_dims, vp, vp, vp, vp, i64, vp, vp, vp, vp, i64, vp], ctypes.c_int),
        "rvq_beam_workspace_bytes": ([rvq_beam_dims], sz),
        "rvq_beam_select": ([rvq_beam_dims, vp, i64, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "rvq_beam_reorder": ([rvq_beam_dims, vp, ctypes.POINTER(rvq_beam_state), i32, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


# ---------------------------------------------------------------------------
# argument marshalling
# ---------------------------------------------------------------------------

def _ptr(t: Optional[torch.Tensor], on: Optional[int] = None) -> Optional[int]:
    """Address of a contiguous CUDA tensor (on GPU `on`, where that is given; None: null)."""
    if t is None:
        return None
    if t.get_device() != on if on is not None else not t.is_cuda:
        raise ValueError("RVQ buffers must be CUDA tensors, those of one call on one device")
    if not t.is_contiguous():
        raise ValueError("RVQ buffers must be contiguous")
    return t.data_ptr()


def _enqueue(name: str, on: int, stream, *args) -> None:
    """Calls entry point `name` for tensors on GPU `on` (the first one's; the others have been compared with it),
    whichever device is current: with the stream given, which has to be one of that GPU's, or with its current one."""
    cuda = torch._C
    if stream is None and on >= 0 and cuda._cuda_getDevice() == on:  # the usual call
        status = getattr(load_library(), name)(*args, cuda._cuda_getCurrentRawStream(on))
    else:
        status = _status(name, on, stream, *args)
    if status != RVQ_OK:
        raise RVQError(name, status)


def _status(name: str, on: int, stream, *args) -> int:
    """What entry point `name` returns."""
    if on < 0:
        raise ValueError(f"{name}: the tensors must be CUDA tensors")
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(on)
    else:
        handle = stream.cuda_stream
        if getattr(stream, "device_index", on) != on:  # (other libraries' streams need not say)
            raise ValueError(f"{name}: the stream must be one of cuda:{on}")
    call = getattr(load_library(), name)
    if torch._C._cuda_getDevice() == on:
        return call(*args, handle)
    with torch.cuda.device(on):
        return call(*args, handle)


def _used_on(stream, *tensors) -> None:
    """Tells torch's allocator that work on `stream` uses these tensors: their memory is given to nobody else before
    that work has ended, whenever they are dropped."""
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)


def _run_on(stream, device, call, touched):
    """call() with `stream` current (None: as it is), so that what it allocates is that stream's: a block that another
    stream freed may still be in use there.  touched(): the other tensors that its work uses."""
    if stream is None:
        return call()
    if hasattr(stream, "cuda_stream") and not isinstance(stream, torch.cuda.Stream):  # another library's
        stream = torch.cuda.ExternalStream(stream.cuda_stream, device)
    with torch.cuda.stream(stream):
        out = call()
    _used_on(stream, *touched())
    _used_on(torch.cuda.current_stream(device), *(out if isinstance(out, tuple) else (out,)))
    return out


def _check(name: str, status: int):
    if status != RVQ_OK:
        raise RVQError(name, status)


def _dims(D: int, d: int, K: int, Q: int, metric: int = RVQ_METRIC_L2, D_in: int = 0, D_out: int = 0) -> rvq_dims:
    return rvq_dims(int(D), int(d), int(K), int(Q), int(metric), int(D_in), int(D_out))


def rvq_dims_supported(dims: rvq_dims) -> int:
    return load_library().rvq_dims_supported(dims)


def rvq_tables_bytes(dims: rvq_dims) -> int:
    return load_library().rvq_tables_bytes(dims)


def rvq_encode_scratch_bytes(dims: rvq_dims, n_frames: int, n_q: int) -> int:
    return load_library().rvq_encode_scratch_bytes(dims, int(n_frames), int(n_q))


def rvq_encode_min_scratch_bytes(dims: rvq_dims, n_q: int) -> int:
    return load_library().rvq_encode_min_scratch_bytes(dims, int(n_q))


def rvq_prepare(dims: rvq_dims, w_in, codebook, w_out, b_in, b_out, tables: torch.Tensor, stream=None,
                fc_w=None, fc_b=None, fc2_w=None, fc2_b=None) -> None:
    on = tables.get_device()
    w = rvq_weights(*(_ptr(t, on) for t in (w_in, b_in, codebook, w_out, b_out, fc_w, fc_b, fc2_w, fc2_b)))
    _enqueue("rvq_prepare", on, stream, dims, ctypes.byref(w), _ptr(tables, on), tables.numel() * tables.element_size())


def rvq_encode(dims: rvq_dims, tables, x, n_q: int, codes, scratch, stream=None) -> None:
    on = tables.get_device()
    n = x.shape[0]
    _enqueue("rvq_encode", on, stream, dims, _ptr(tables, on), _ptr(x, on), n, int(n_q), _ptr(codes, on),
             _ptr(scratch, on), scratch.numel() * scratch.element_size())


def rvq_decode(dims: rvq_dims, tables, codes, n_q: int, y, bad_codes=None, stream=None) -> None:
    on = tables.get_device()
    n = codes.shape[0]
    _enqueue("rvq_decode", on, stream, dims, _ptr(tables, on), _ptr(codes, on), n, int(n_q), _ptr(y, on),
             _ptr(bad_codes, on))


def rvq_reconstruct(dims: rvq_dims, tables, x, n_q: int, codes, x_hat, scratch, stream=None) -> None:
    on = tables.get_device()
    n = x.shape[0]
    _enqueue("rvq_reconstruct", on, stream, dims, _ptr(tables, on), _ptr(x, on), n, int(n_q), _ptr(codes, on),
             _ptr(x_hat, on), _ptr(scratch, on), scratch.numel() * scratch.element_size())


def rvq_encode_static(dims: rvq_dims, tables, x, n_q: int, codes, stream=None) -> None:
    """Encode with the library's own fixed scratch (no scratch argument; see rvq.h)."""
    on = tables.get_device()
    n = x.shape[0]
    _enqueue("rvq_encode_static", on, stream, dims, _ptr(tables, on), _ptr(x, on), n, int(n_q), _ptr(codes, on))


def rvq_pipeline_workspace_bytes(dims: rvq_dims, n_q: int, chunk_frames: int) -> int:
    return load_library().rvq_pipeline_workspace_bytes(dims, int(n_q), int(chunk_frames))


def rvq_pipeline_create(dims: rvq_dims, n_q: int, chunk_frames: int, workspace: torch.Tensor) -> ctypes.c_void_p:
    out = ctypes.c_void_p()
    _check("rvq_pipeline_create", load_library().rvq_pipeline_create(
        dims, int(n_q), int(chunk_frames), _ptr(workspace), workspace.numel() * workspace.element_size(),
        ctypes.byref(out)))
    return out


def rvq_pipeline_destroy(pipeline) -> None:
    _check("rvq_pipeline_destroy", load_library().rvq_pipeline_destroy(pipeline))


def _host_ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if t.is_cuda or not t.is_contiguous():
        raise ValueError("host buffers must be contiguous CPU tensors")
    return ctypes.c_void_p(t.data_ptr())


def rvq_pipeline_reconstruct(pipeline, tables, x_host, codes_host, x_hat_host=None) -> None:
    _check("rvq_pipeline_reconstruct", load_library().rvq_pipeline_reconstruct(
        pipeline, _ptr(tables), _host_ptr(x_host), x_host.shape[0], _host_ptr(codes_host), _host_ptr(x_hat_host)))


def rvq_read_status(scratch: Optional[torch.Tensor] = None, stream=None) -> int:
    """Synchronise `stream` and return the status (an rvq_status value, not
    raised) that the encode last enqueued with `scratch` left in its status
    word; scratch=None reads the library's own scratch (rvq_encode_static)."""
    on = torch.cuda.current_device() if scratch is None else scratch.get_device()
    return int(_status("rvq_read_status", on, stream, _ptr(scratch, on)))


def rvq_read_error_count(bad_codes: torch.Tensor, stream=None) -> int:
    """Synchronise `stream` and return rvq_decode's bad-code counter."""
    out = ctypes.c_int64(0)
    on = bad_codes.get_device()
    _enqueue("rvq_read_error_count", on, stream, _ptr(bad_codes, on), ctypes.byref(out))
    return int(out.value)


def rvq_pipeline_set_cancel(pipeline, fn, user=None) -> None:
    """fn: an RVQ_CANCEL_FN (the caller keeps it alive) or None to remove."""
    _check("rvq_pipeline_set_cancel", load_library().rvq_pipeline_set_cancel(
        pipeline, fn if fn is not None else RVQ_CANCEL_FN(), user))


def rvq_status_string(status: int) -> str:
    return load_library().rvq_status_string(int(status)).decode()


def rvq_version() -> str:
    return load_library().rvq_version().decode()


def rvq_set_stream_max_frames(max_frames: int) -> int:
    """Threshold (frames per call) of the small-batch kernel; returns the previous one."""
    return int(load_library().rvq_set_stream_max_frames(int(max_frames)))


def rvq_stream_plan(dims: rvq_dims, n_q: int, n_frames: int) -> dict:
    """How one call of n_frames frames would run on the current device."""
    out = (ctypes.c_int64 * 6)()
    _check("rvq_stream_plan", load_library().rvq_stream_plan(dims, int(n_q), int(n_frames), out))
    keys = ("stream", "cluster_ctas", "group_frames", "groups_per_cluster", "clusters", "slice_buffers")
    return {k: int(v) for k, v in zip(keys, out)}


# ---------------------------------------------------------------------------
# operators of a code predictor (norms, dropout, log probabilities, distillation loss, beam step)
# ---------------------------------------------------------------------------

def _at(t: Optional[torch.Tensor], on: int, dtype, shape, name: str):
    """Address of a contiguous tensor of this dtype and shape on GPU `on` (None: null)."""
    if t is None:
        return None
    if t.dtype is dtype and t.shape == shape and t.get_device() == on and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous tensor of {dtype} and shape {tuple(shape)} on cuda:{on}")


def _rows_at(t: torch.Tensor, on: int, dtype, shape, name: str):
    """Address and row stride of a 2-d tensor on GPU `on` whose rows are contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != on:
        raise ValueError(f"{name} must be a tensor of {dtype} and shape {tuple(shape)} on cuda:{on}")
    stride, one = t.stride()
    if one != 1 and shape[1] > 1 and shape[0] > 0:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), stride


def _workspace(t: Optional[torch.Tensor], on: int):
    """Address and bytes of a workspace."""
    if t is None:
        return None, 0
    if t.get_device() != on or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{on}")
    return t.data_ptr(), t.nbytes


def _shape2(t: torch.Tensor, name: str):
    if t.dim() != 2 or t.dtype not in DTYPES:
        raise ValueError(f"{name} must be a 2-d tensor of float32, bfloat16 or float16")
    return t.shape


def rvq_layer_norm_workspace_bytes(rows: int, width: int) -> int:
    return load_library().rvq_layer_norm_workspace_bytes(int(rows), int(width))


def rvq_layer_norm(x, weight, bias, eps: float, y, mean=None, rstd=None, stream=None) -> None:
    """Layer norm of the rows of x [rows][width] into y (see rvq.h); mean and rstd [rows] are optional outputs."""
    on = x.get_device()
    shape, dtype = _shape2(x, "x"), x.dtype
    rows, width = shape
    p = weight if weight is not None else bias
    pd = torch.float32 if p is None else p.dtype
    xp, xs = _rows_at(x, on, dtype, shape, "x")
    yp, ys = _rows_at(y, on, dtype, shape, "y")
    _enqueue("rvq_layer_norm", on, stream, rvq_norm_dims(rows, width, DTYPES[dtype], DTYPES.get(pd, -1), eps), xp, xs,
             _at(weight, on, pd, (width,), "weight"), _at(bias, on, pd, (width,), "bias"), yp, ys,
             _at(mean, on, torch.float32, (rows,), "mean"), _at(rstd, on, torch.float32, (rows,), "rstd"))


def rvq_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, workspace, stream=None) -> None:
    """Gradients of rvq_layer_norm; dx, dweight and dbias may each be None (not computed)."""
    on = x.get_device()
    shape, dtype = _shape2(x, "x"), x.dtype
    rows, width = shape
    p = weight if weight is not None else dweight if dweight is not None else dbias
    pd = torch.float32 if p is None else p.dtype
    dyp, dys = _rows_at(dy, on, dtype, shape, "dy")
    xp, xs = _rows_at(x, on, dtype, shape, "x")
    dxp, dxs = (None, 0) if dx is None else _rows_at(dx, on, dtype, shape, "dx")
    if mean is None or rstd is None:
        raise ValueError("rvq_layer_norm_backward needs the forward pass's mean and rstd")
    _enqueue("rvq_layer_norm_backward", on, stream, rvq_norm_dims(rows, width, DTYPES[dtype], DTYPES.get(pd, -1), 0.0),
             dyp, dys, xp, xs, _at(weight, on, pd, (width,), "weight"), _at(mean, on, torch.float32, (rows,), "mean"),
             _at(rstd, on, torch.float32, (rows,), "rstd"), dxp, dxs, _at(dweight, on, pd, (width,), "dweight"),
             _at(dbias, on, pd, (width,), "dbias"), *_workspace(workspace, on))


def _rows_or_none(t: Optional[torch.Tensor], on: int, dtype, shape, name: str):
    return (None, 0) if t is None else _rows_at(t, on, dtype, shape, name)


def _mask_on(mask: Optional[rvq_dropout_mask], on: int):
    """A pointer to the mask, whose step has to be on GPU `on` (None: null)."""
    if mask is None:
        return None
    if mask.tensor is not None and mask.tensor.get_device() != on:
        raise ValueError(f"the mask's step must be on cuda:{on}")
    return ctypes.byref(mask)


def rvq_dropout(x, mask: rvq_dropout_mask, y, residual=None, stream=None) -> None:
    """Dropout of x [rows][width] into y, plus residual (see rvq.h); on the gradient of y, its backward pass."""
    on = x.get_device()
    shape, dtype = _shape2(x, "x"), x.dtype
    _enqueue("rvq_dropout", on, stream, rvq_dropout_dims(*shape, DTYPES[dtype]), *_rows_at(x, on, dtype, shape, "x"),
             *_rows_or_none(residual, on, dtype, shape, "residual"), _mask_on(mask, on),
             *_rows_at(y, on, dtype, shape, "y"))


def rvq_rms_norm_workspace_bytes(rows: int, width: int) -> int:
    return load_library().rvq_rms_norm_workspace_bytes(int(rows), int(width))


def rvq_rms_norm(x, weight, eps: float, y, rstd=None, residual=None, mask: Optional[rvq_dropout_mask] = None,
                 total=None, q=None, scales=None, block: int = 0, stream=None) -> None:
    """Root-mean-square norm of the rows of residual + drop(x) [rows][width] into y (see rvq.h).  Optional outputs:
    rstd [rows], total (the sum), q (float8_e4m3fn) with scales [rows][ceil(width / block)] (block 0: [rows][1];
    float32, or float8_e8m0fnu for powers of two); y may be None."""
    on = x.get_device()
    shape, dtype = _shape2(x, "x"), x.dtype
    rows, width = shape
    pd = torch.float32 if weight is None else weight.dtype
    eight = None
    if (q is None) != (scales is None):
        raise ValueError("q and scales go together")
    if q is not None:
        if scales.dtype not in SCALES:
            raise ValueError("scales must be float32 or float8_e8m0fnu")
        qp, qs = _rows_at(q, on, torch.float8_e4m3fn, shape, "q")
        count = 1 if block <= 0 else -(-width // block)
        eight = rvq_rms_8bit(qp, qs, _at(scales, on, scales.dtype, (rows, count), "scales"), block, SCALES[scales.dtype])
    _enqueue("rvq_rms_norm", on, stream, rvq_norm_dims(rows, width, DTYPES[dtype], DTYPES.get(pd, -1), eps),
             *_rows_at(x, on, dtype, shape, "x"), *_rows_or_none(residual, on, dtype, shape, "residual"),
             _mask_on(mask, on), _at(weight, on, pd, (width,), "weight"),
             *_rows_or_none(total, on, dtype, shape, "total"), *_rows_or_none(y, on, dtype, shape, "y"),
             _at(rstd, on, torch.float32, (rows,), "rstd"), None if eight is None else ctypes.byref(eight))


def rvq_rms_norm_backward(dy, total, weight, rstd, dresidual, dweight, workspace, dtotal=None,
                          mask: Optional[rvq_dropout_mask] = None, dx=None, stream=None) -> None:
    """Gradients of rvq_rms_norm from its total (x, where it had neither residual nor mask), mask and rstd; dresidual,
    dweight and dx may each be None (not computed)."""
    on = total.get_device()
    shape, dtype = _shape2(total, "total"), total.dtype
    rows, width = shape
    p = weight if weight is not None else dweight
    pd = torch.float32 if p is None else p.dtype
    if rstd is None:
        raise ValueError("rvq_rms_norm_backward needs the forward pass's rstd")
    _enqueue("rvq_rms_norm_backward", on, stream, rvq_norm_dims(rows, width, DTYPES[dtype], DTYPES.get(pd, -1), 0.0),
             *_rows_at(dy, on, dtype, shape, "dy"), *_rows_or_none(dtotal, on, dtype, shape, "dtotal"),
             *_rows_at(total, on, dtype, shape, "total"), _mask_on(mask, on), _at(weight, on, pd, (width,), "weight"),
             _at(rstd, on, torch.float32, (rows,), "rstd"), *_rows_or_none(dresidual, on, dtype, shape, "dresidual"),
             *_rows_or_none(dx, on, dtype, shape, "dx"), _at(dweight, on, pd, (width,), "dweight"),
             *_workspace(workspace, on))


def rvq_log_probs(logits, codes, temperature: float, log_probs=None, entropy=None, lse=None, stats=None,
                  top_log_probs=None, top_codes=None, bad_codes=None, stream=None) -> None:
    """Log probabilities [rows] of codes [rows] (int32, -1: none) under logits [rows][vocab] (see rvq.h), and what else
    has a place to go: entropy and lse [rows], stats [rows][2], top_log_probs and top_codes [rows][top]."""
    on = logits.get_device()
    rows, vocab = shape = _shape2(logits, "logits")
    top = 0 if top_codes is None else top_codes.shape[-1]
    one, best, f32 = (rows,), (rows, top), torch.float32
    _enqueue("rvq_log_probs", on, stream, rvq_log_probs_dims(rows, vocab, top, DTYPES[logits.dtype], temperature),
             *_rows_at(logits, on, logits.dtype, shape, "logits"), _at(codes, on, torch.int32, one, "codes"),
             _at(log_probs, on, f32, one, "log_probs"), _at(entropy, on, f32, one, "entropy"),
             _at(lse, on, f32, one, "lse"), _at(stats, on, f32, (rows, 2), "stats"),
             _at(top_log_probs, on, f32, best, "top_log_probs"), _at(top_codes, on, torch.int32, best, "top_codes"),
             _at(bad_codes, on, torch.int64, (1,), "bad_codes"))


def rvq_log_probs_backward(grad_log_probs, grad_entropy, grad_lse, logits, codes, temperature: float, stats, entropy,
                           dlogits, stream=None) -> None:
    """dlogits from the gradients [rows] of rvq_log_probs' log_probs, entropy and lse (None: zero), with its stats and
    entropy."""
    on = logits.get_device()
    rows, vocab = shape = _shape2(logits, "logits")
    one, f32 = (rows,), torch.float32
    _enqueue("rvq_log_probs_backward", on, stream, rvq_log_probs_dims(rows, vocab, 0, DTYPES[logits.dtype], temperature),
             _at(grad_log_probs, on, f32, one, "grad_log_probs"), _at(grad_entropy, on, f32, one, "grad_entropy"),
             _at(grad_lse, on, f32, one, "grad_lse"), *_rows_at(logits, on, logits.dtype, shape, "logits"),
             _at(codes, on, torch.int32, one, "codes"), _at(stats, on, f32, (rows, 2), "stats"),
             _at(entropy, on, f32, one, "entropy"), *_rows_at(dlogits, on, logits.dtype, shape, "dlogits"))


def _distill_args(logits, top_logits, top_codes, teacher_lse, weights, temperature):
    on = logits.get_device()
    rows, vocab = shape = _shape2(logits, "logits")
    entries = _shape2(top_logits, "top_logits")
    if entries[0] != rows:
        raise ValueError("top_logits must have the logits' rows")
    dims = rvq_distill_dims(rows, vocab, entries[1], DTYPES[logits.dtype], DTYPES[top_logits.dtype], temperature)
    zp, zs = _rows_at(logits, on, logits.dtype, shape, "logits")
    return dims, on, (rows,), zp, zs, (_at(top_logits, on, top_logits.dtype, entries, "top_logits"),
                                       _at(top_codes, on, torch.int32, entries, "top_codes"),
                                       _at(teacher_lse, on, torch.float32, (rows,), "teacher_lse"),
                                       _at(weights, on, torch.float32, (rows,), "weights"))


def rvq_distill(logits, top_logits, top_codes, teacher_lse, weights, temperature: float, loss, lse=None, dlogits=None,
                bad_codes=None, stream=None) -> None:
    """Distillation loss [rows] of logits [rows][vocab] from the teacher's entries [rows][top] (see rvq.h); with
    dlogits, the gradient in the same pass; with lse [rows][2], what rvq_distill_backward needs."""
    dims, on, rows, zp, zs, teacher = _distill_args(logits, top_logits, top_codes, teacher_lse, weights, temperature)
    dp, ds = (None, 0) if dlogits is None else _rows_at(dlogits, on, logits.dtype, logits.shape, "dlogits")
    _enqueue("rvq_distill", on, stream, dims, zp, zs, *teacher, _at(loss, on, torch.float32, rows, "loss"),
             None if lse is None else _at(lse, on, torch.float32, rows + (2,), "lse"), dp, ds,
             None if bad_codes is None else _at(bad_codes, on, torch.int64, bad_codes.shape, "bad_codes"))


def rvq_distill_backward(grad_loss, logits, top_logits, top_codes, teacher_lse, weights, temperature: float, lse,
                         dlogits, stream=None) -> None:
    """dlogits = grad_loss[row] * d loss[row] / d logits, with rvq_distill's lse; grad_loss None: ones."""
    dims, on, rows, zp, zs, teacher = _distill_args(logits, top_logits, top_codes, teacher_lse, weights, temperature)
    dp, ds = _rows_at(dlogits, on, logits.dtype, logits.shape, "dlogits")
    _enqueue("rvq_distill_backward", on, stream, dims, _at(grad_loss, on, torch.float32, rows, "grad_loss"), zp, zs,
             *teacher, _at(lse, on, torch.float32, rows + (2,), "lse"), dp, ds)


def rvq_beam_workspace_bytes(dims: rvq_beam_dims) -> int:
    return load_library().rvq_beam_workspace_bytes(dims)


def rvq_beam_select(dims: rvq_beam_dims, logits, scores, finished, end_code: int, out_scores, parents, codes,
                    out_finished, workspace, stream=None) -> None:
    """One selection step (see rvq.h): logits [groups][beams][vocab] (or [groups * beams][vocab]), scores and finished
    [groups][beams]; outputs [groups][select].  finished, out_finished: bool or uint8 tensors, or None."""
    groups, beams, vocab = dims.groups, dims.beams, dims.vocab
    on = logits.get_device()
    if DTYPES.get(logits.dtype) != dims.dtype:
        raise ValueError("logits must have the dtype in dims")
    if logits.dim() == 3:
        stride = logits.stride(0 if beams == 1 else 1)  # (an axis of size one may have any)
        if logits.shape != (groups, beams, vocab) or (groups > 1 and logits.stride(0) != beams * stride):
            raise ValueError(f"logits must be {(groups, beams, vocab)} with evenly spaced rows")
    else:
        if logits.shape != (groups * beams, vocab):
            raise ValueError(f"logits must be {(groups, beams, vocab)} or {(groups * beams, vocab)}")
        stride = logits.stride(0)
    if vocab > 1 and logits.stride(-1) != 1:
        raise ValueError("logits must have contiguous rows")
    held, kept = (groups, beams), (groups, dims.select)
    for t in (finished, out_finished):
        if t is not None and t.dtype is not torch.bool and t.dtype is not torch.uint8:
            raise ValueError("finished and out_finished must be bool or uint8")
    _enqueue("rvq_beam_select", on, stream, dims, logits.data_ptr(), stride,
             _at(scores, on, torch.float32, held, "scores"),
             None if finished is None else _at(finished, on, finished.dtype, held, "finished"), end_code,
             _at(out_scores, on, torch.float32, kept, "out_scores"), _at(parents, on, torch.int32, kept, "parents"),
             _at(codes, on, torch.int32, kept, "codes"),
             None if out_finished is None else _at(out_finished, on, out_finished.dtype, kept, "out_finished"),
             *_workspace(workspace, on))


def rvq_beam_states(pairs, layered: bool = False):
    """The (source, destination) tensors that rvq_beam_reorder moves, described once for any number of calls:
    [groups][beams][...] and [groups][select][...], with a leading layer axis where `layered`.  The axes after the
    beams' must be contiguous; slices of them (the filled part of a cache) are taken as they are.  A tensor paired
    with itself is reordered in place.  Returns an array for rvq_beam_reorder; it keeps the tensors alive."""
    pairs = list(pairs)
    out = (rvq_beam_state * len(pairs))()
    lead = 3 if layered else 2
    for s, (src, dst) in zip(out, pairs):
        if not (src.is_cuda and dst.is_cuda) or src.dtype != dst.dtype or src.dim() < lead or src.dim() != dst.dim():
            raise ValueError("a state and its destination must be CUDA tensors of one dtype with the same axes")
        if src.shape[lead:] != dst.shape[lead:] or src.shape[:lead - 1] != dst.shape[:lead - 1]:
            raise ValueError("a state and its destination differ in more than the number of beams")
        size = src.element_size()
        row = size
        for t in (src, dst) if src.numel() else ():
            row = size
            for n, step in zip(reversed(t.shape[lead:]), reversed(t.stride()[lead:])):
                if n != 1 and step * size != row:
                    raise ValueError("the axes of a state after the beams' must be contiguous")
                row *= n
        a, b = ([st * size for st in t.stride()[:lead]] for t in (src, dst))
        s.src, s.dst, s.row_bytes = src.data_ptr(), dst.data_ptr(), row if src.numel() else 0
        s.layers = src.shape[0] if layered else 1
        s.src_layer_stride, s.dst_layer_stride = (a[0], b[0]) if layered else (0, 0)
        s.src_group_stride, s.src_beam_stride = a[-2:]
        s.dst_group_stride, s.dst_beam_stride = b[-2:]
    out.shapes = [(src.shape[lead - 2:lead], dst.shape[lead - 2:lead]) for src, dst in pairs]
    out.tensors = pairs
    on = {t.get_device() for pair in pairs for t in pair}
    if len(on) > 1:
        raise ValueError("states must all be on one device")
    out.device = on.pop() if on else None
    return out


def rvq_beam_reorder(dims: rvq_beam_dims, parents, states, stream=None) -> None:
    """Every state's rows follow parents [groups][select]; `states` from rvq_beam_states."""
    want = (dims.groups, dims.beams), (dims.groups, dims.select)
    for shapes in states.shapes:
        if shapes != want:
            raise ValueError(f"states must have {want[0]} and {want[1]} groups and beams")
    on = parents.get_device()
    if states.device != on and states.device is not None:
        raise ValueError(f"states must be on cuda:{on}, with their parents")
    _enqueue("rvq_beam_reorder", on, stream, dims, _at(parents, on, torch.int32, want[1], "parents"), states, len(states))


# ---------------------------------------------------------------------------
# convenience object: owns the tables and a scratch buffer (torch allocations)
# ---------------------------------------------------------------------------

class RVQ:
    """Prepared RVQ weights on one CUDA device.

    w_in [Q][d][D], codebook [Q][K][d], w_out [Q][D][d], b_in [Q][d] or None,
    b_out [Q][D] or None; float32 tensors (moved to `device` if needed).
    metric: "l2" (squared L2) or "cosine" (both sides L2-normalised before the
    argmin, as RVQ_METRIC_COSINE in include/rvq.h).
    fc_w [D][D_in], fc_b [D] (optional): a Linear layer applied to each frame
    before the quantizer; fc2_w [D_out][D], fc2_b [D_out] (optional): one
    applied to the decoded sum.  Both are folded into the tables.

    The calls run on the current stream, or on `stream`, where their inputs
    have to be ready.  The object owns a scratch buffer; one object serves one
    stream at a time.
    """

    def __init__(self, w_in, codebook, w_out, b_in=None, b_out=None, device=None, stream=None,
                 metric: str = "l2", fc_w=None, fc_b=None, fc2_w=None, fc2_b=None):
        device = torch.device(device) if device is not None else (w_in.device if w_in.is_cuda else torch.device("cuda"))
        f = lambda t: None if t is None else t.to(device=device, dtype=torch.float32).contiguous()
        w_in, codebook, w_out, b_in, b_out = map(f, (w_in, codebook, w_out, b_in, b_out))
        fc_w, fc_b, fc2_w, fc2_b = map(f, (fc_w, fc_b, fc2_w, fc2_b))
        Q, d, D = w_in.shape
        K = codebook.shape[1]
        self.D, self.d, self.K, self.Q = D, d, K, Q
        self.D_in = fc_w.shape[1] if fc_w is not None else D
        self.D_out = fc2_w.shape[0] if fc2_w is not None else D
        self.device = device
        self.metric = metric
        self.dims = _dims(D, d, K, Q, METRICS[metric], self.D_in, self.D_out)
        status = rvq_dims_supported(self.dims)
        _check("rvq_dims_supported", status)
        nbytes = rvq_tables_bytes(self.dims)
        self.tables = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.tables.device  # with its index: a "cuda" of later calls may be another one
        with torch.cuda.device(device):
            rvq_prepare(self.dims, w_in, codebook, w_out, b_in, b_out, self.tables, stream, fc_w, fc_b, fc2_w, fc2_b)
        self._scratch = None

    def scratch_for(self, n_frames: int, n_q: int) -> torch.Tensor:
        need = max(rvq_encode_scratch_bytes(self.dims, n_frames, n_q), 16)
        if self._scratch is None or self._scratch.numel() < need:
            self._scratch = torch.empty(need, dtype=torch.uint8, device=self.device)
        return self._scratch

    def _frames(self, x):
        if x.dim() != 2 or x.shape[1] != self.D_in:
            raise ValueError(f"x must be [N][{self.D_in}]")
        return x.to(device=self.device, dtype=torch.float32).contiguous()

    def encode(self, x, n_q: Optional[int] = None, codes=None, stream=None):
        def call():
            depth, frames = self.Q if n_q is None else int(n_q), self._frames(x)
            out = codes
            if out is None:
                out = torch.empty((frames.shape[0], depth), dtype=torch.int32, device=self.device)
            rvq_encode(self.dims, self.tables, frames, depth, out, self.scratch_for(frames.shape[0], depth), stream)
            return out

        return _run_on(stream, self.device, call, lambda: (x, codes, self.tables, self._scratch))

    def decode(self, codes, n_q: Optional[int] = None, y=None, bad_codes=None, stream=None):
        def call():
            c = codes.to(device=self.device, dtype=torch.int32).contiguous()
            out = y
            if out is None:
                out = torch.empty((c.shape[0], self.D_out), dtype=torch.float32, device=self.device)
            rvq_decode(self.dims, self.tables, c, c.shape[1] if n_q is None else int(n_q), out, bad_codes, stream)
            return out

        return _run_on(stream, self.device, call, lambda: (codes, y, bad_codes, self.tables))

    def reconstruct(self, x, n_q: Optional[int] = None, codes=None, x_hat=None, stream=None):
        def call():
            depth, frames = self.Q if n_q is None else int(n_q), self._frames(x)
            n = frames.shape[0]
            c, y = codes, x_hat
            if c is None:
                c = torch.empty((n, depth), dtype=torch.int32, device=self.device)
            if y is None:
                y = torch.empty((n, self.D_out), dtype=torch.float32, device=self.device)
            rvq_reconstruct(self.dims, self.tables, frames, depth, c, y, self.scratch_for(n, depth), stream)
            return c, y

        return _run_on(stream, self.device, call, lambda: (x, codes, x_hat, self.tables, self._scratch))


class RVQPipeline:
    """Encode + decode of frames held in host memory, copies overlapped with compute.

    Wraps rvq_pipeline_*: the device workspace is a torch allocation owned by
    this object.  Pinned host tensors give full copy bandwidth.
    """

    def __init__(self, rvq: "RVQ", n_q: Optional[int] = None, chunk_frames: int = 38912):
        self.rvq = rvq
        self.n_q = rvq.Q if n_q is None else int(n_q)
        nbytes = rvq_pipeline_workspace_bytes(rvq.dims, self.n_q, chunk_frames)
        if nbytes == 0:
            raise ValueError("unsupported pipeline arguments")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=rvq.device)
        with torch.cuda.device(rvq.device):
            self.handle = rvq_pipeline_create(rvq.dims, self.n_q, chunk_frames, self.workspace)

    def reconstruct(self, x_host: torch.Tensor, codes_host: Optional[torch.Tensor] = None,
                    x_hat_host: Optional[torch.Tensor] = None, want_x_hat: bool = True):
        n = x_host.shape[0]
        if codes_host is None:
            codes_host = torch.empty((n, self.n_q), dtype=torch.int32, pin_memory=True)
        if x_hat_host is None and want_x_hat:
            x_hat_host = torch.empty((n, self.rvq.D_out), dtype=torch.float32, pin_memory=True)
        with torch.cuda.device(self.rvq.device):
            rvq_pipeline_reconstruct(self.handle, self.rvq.tables, x_host, codes_host, x_hat_host)
        return codes_host, x_hat_host

    def set_cancel(self, should_stop=None):
        """should_stop() -> bool is polled before each chunk; None removes it."""
        self._cancel = None if should_stop is None else RVQ_CANCEL_FN(lambda _user: 1 if should_stop() else 0)
        rvq_pipeline_set_cancel(self.handle, self._cancel)

    def close(self):
        if getattr(self, "handle", None) is not None:
            rvq_pipeline_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


from .predictor import (BeamSearch, LogProbs, distill_loss, distill_loss_and_grad, dropout, layer_norm,  # noqa: E402
                        log_probs, rms_norm, rms_norm_8bit)
