"""Python binding for libstreamkl (fused attention KL divergence, sm_103a).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libstreamkl.so``.  PyTorch supplies device memory and streams.
There is no CPU fallback: if the library is missing or the device is not a
GB300 (sm_103a), calls raise.

Functions mirror the C ABI in ``include/streamkl.h`` and keep its names.
"""

import contextlib
import ctypes
import functools
import os

import torch

__all__ = [
    "StreamKLError", "lib", "library_path",
    "streamkl_fwd", "streamkl_fwd_splitk", "streamkl_fwd_splitk_workspace_bytes",
    "streamkl_suggest_splits", "streamkl_fwd_splitk_noalloc", "streamkl_bwd", "streamkl_status_string",
    "streamkl_fwd_scaled", "streamkl_fwd_splitk_scaled", "streamkl_bwd_scaled",
    "streamkl_fwd_gqa", "streamkl_fwd_splitk_gqa", "streamkl_bwd_gqa", "streamkl_bwd_both",
    "streamkl_bwd_workspace_bytes", "streamkl_bwd_gqa_ws",
    "AttnSide", "streamkl_fwd_mod", "streamkl_fwd_mod_workspace_bytes", "streamkl_bwd_mod",
    "streamkl_bwd_mod_workspace_bytes",
    "status_string", "STREAMKL_STATIC_WORKSPACE_BYTES",
    "streamkl_get_device_status", "streamkl_probe_ex2", "streamkl_selftest_wait_timeout",
    "streamkl_selftest_turn_timeout",
    "STREAMKL_OK", "STREAMKL_INVALID_ARG", "STREAMKL_UNSUPPORTED", "STREAMKL_CUDA_ERROR",
    "STREAMKL_DEVICE_TIMEOUT", "STREAMKL_DEBUG_BOUNDS", "STREAMKL_GRAD_P2", "STREAMKL_GRAD_P1",
]

STREAMKL_OK = 0
STREAMKL_INVALID_ARG = 1
STREAMKL_UNSUPPORTED = 2
STREAMKL_CUDA_ERROR = 3
STREAMKL_DEVICE_TIMEOUT = 4
STREAMKL_DEBUG_BOUNDS = 5
STREAMKL_GRAD_P2 = 0
STREAMKL_GRAD_P1 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libstreamkl.so")
_lib = None

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_SZ = ctypes.c_size_t

_LL = ctypes.c_longlong


class _View(ctypes.Structure):
    _fields_ = [("data", _P), ("stride_b", _LL), ("stride_h", _LL), ("stride_n", _LL)]


class _Side(ctypes.Structure):
    _fields_ = [("q", _View), ("k", _View), ("d", _I), ("HK", _I), ("scale", ctypes.c_double),
                ("softcap", _F), ("slopes", _P),
                ("table", _P), ("num_buckets", _I), ("max_distance", _I), ("bidirectional", _I)]


class _Visible(ctypes.Structure):
    _fields_ = [("causal", _I), ("prefix", _P), ("doc_q", _P), ("doc_k", _P)]


_SP, _VP, _VISP = ctypes.POINTER(_Side), ctypes.POINTER(_View), ctypes.POINTER(_Visible)

_SIGS = {
    "streamkl_fwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P]),
    "streamkl_fwd_splitk": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I, _P, _SZ,
                                 _P, _P, _P, _P]),
    "streamkl_fwd_splitk_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "streamkl_fwd_splitk_noalloc": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _I,
                                         _P, _P, _P, _P]),
    "streamkl_suggest_splits": (_I, [_I, _I, _I, _I, _I]),
    "streamkl_bwd": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _I, _P, _P, _P, _P, _I, _I,
                          _P, _P, _P]),
    "streamkl_fwd_scaled": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _P, _P]),
    "streamkl_fwd_splitk_scaled": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _I, _I, _P, _SZ,
                                        _P, _P, _P, _P]),
    "streamkl_bwd_scaled": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _P, _P, _I,
                                 _I, _P, _P, _P]),
    "streamkl_fwd_gqa": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _P, _P]),
    "streamkl_fwd_splitk_gqa": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _I, _P, _SZ,
                                     _P, _P, _P, _P]),
    "streamkl_bwd_gqa": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _P, _P, _I,
                              _I, _P, _P, _P]),
    "streamkl_bwd_both": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _P, _P, _I,
                               _P, _P, _P, _P, _P]),
    "streamkl_bwd_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "streamkl_bwd_gqa_ws": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _P, _P, _P, _I,
                                 _I, _P, _P, _P, _SZ, _P]),
    "streamkl_fwd_mod_workspace_bytes": (_SZ, [_SP, _SP, _VISP, _I, _I, _I, _I, _I]),
    "streamkl_fwd_mod": (_I, [_SP, _SP, _VISP, _I, _I, _I, _I, _I, _P, _SZ, _P, _P, _P, _P]),
    "streamkl_bwd_mod_workspace_bytes": (_SZ, [_SP, _SP, _VISP, _I, _I, _I, _I, _I, _I, _I]),
    "streamkl_bwd_mod": (_I, [_SP, _SP, _VISP, _I, _I, _I, _I, _P, _P, _P, _P, _I, _I, _VP, _VP, _P, _P, _SZ, _P]),
    "streamkl_status_string": (ctypes.c_char_p, [_I]),
    "streamkl_get_device_status": (_I, []),
    "streamkl_probe_ex2": (_I, [_P, _I, _I, _P]),
    "streamkl_selftest_wait_timeout": (_I, [_I, _P]),
    "streamkl_selftest_turn_timeout": (_I, [_I, _P, _P]),
}


class StreamKLError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def lib():
    """The loaded ``libstreamkl.so`` (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(library_path):
            raise RuntimeError(f"{library_path} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        handle = ctypes.CDLL(library_path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def status_string(status):
    return lib().streamkl_status_string(int(status)).decode()


streamkl_status_string = status_string


def _check(status, where):
    if status != STREAMKL_OK:
        raise StreamKLError(status, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dims(q1, k1, q2, k2):
    for name, t in (("q1", q1), ("k1", k1), ("q2", q2), ("k2", k2)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA bf16 tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
    B, H, NQ, d1 = q1.shape
    NK = k1.shape[2]
    d2 = q2.shape[3]
    if tuple(k1.shape) != (B, H, NK, d1) or tuple(q2.shape) != (B, H, NQ, d2) or \
            tuple(k2.shape) != (B, H, NK, d2):
        raise ValueError("inconsistent shapes: want q1 [B,H,NQ,d1], k1 [B,H,NK,d1], "
                         "q2 [B,H,NQ,d2], k2 [B,H,NK,d2]")
    return B, H, NQ, NK, d1, d2


def _dims_gqa(q1, k1, q2, k2):
    """Like _dims, with k1 and k2 allowed their own head counts (grouped key
    heads; the library checks that each divides the query head count)."""
    for name, t in (("q1", q1), ("k1", k1), ("q2", q2), ("k2", k2)):
        if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA bf16 tensor")
        if t.dim() != 4 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
    B, H, NQ, d1 = q1.shape
    HK1, NK = k1.shape[1], k1.shape[2]
    HK2, d2 = k2.shape[1], q2.shape[3]
    if tuple(k1.shape) != (B, HK1, NK, d1) or tuple(q2.shape) != (B, H, NQ, d2) or \
            tuple(k2.shape) != (B, HK2, NK, d2):
        raise ValueError("inconsistent shapes: want q1 [B,H,NQ,d1], k1 [B,HK1,NK,d1], "
                         "q2 [B,H,NQ,d2], k2 [B,HK2,NK,d2]")
    return B, H, HK1, HK2, NQ, NK, d1, d2


def _out(t, shape, device, name):
    if t is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous() \
            or t.device != device:
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {tuple(shape)} on {device}")
    return t


_here = contextlib.nullcontext()


def _making(stream):
    """Where a call's own tensors are made: on the stream that it runs on.  Memory of the
    current stream may still be in use there, by work that `stream` does not wait for."""
    return _here if stream is None else torch.cuda.stream(stream)


def _handed_over(stream, device, *pairs):
    """Tensors made by this call for the caller (old one None), who goes on on the current stream."""
    if stream is not None:
        here = torch.cuda.current_stream(device)
        for old, new in pairs:
            if old is None and new is not None:
                new.record_stream(here)


def _on_its_stream(fn):
    """fn (its last parameter is `stream`) as a whole on the stream it is handed, where one is."""
    at = fn.__code__.co_argcount - 1

    @functools.wraps(fn)
    def call(*args, **kw):
        stream = args[at] if len(args) > at else kw.get("stream")
        if stream is None:
            return fn(*args, **kw)
        here = torch.cuda.current_stream()
        on = stream
        if hasattr(stream, "cuda_stream") and not isinstance(stream, torch.Stream):  # another library's
            on = torch.cuda.ExternalStream(stream.cuda_stream)
        with _making(on):
            out = fn(*args, **kw)
        for t in out:
            t.record_stream(here)
        return out
    return call


@_on_its_stream
def streamkl_fwd(q1, k1, q2, k2, scale, causal, kl=None, lse1=None, lse2=None, stream=None):
    """Per-row KL(P1 || P2), LSE1, LSE2 (fp32 [B, H, NQ]); see include/streamkl.h."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                              B, H, NQ, NK, d1, d2, float(scale), int(bool(causal)),
                              kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd")
    return kl, lse1, lse2


def streamkl_fwd_splitk_workspace_bytes(B, H, NQ, num_splits):
    return int(lib().streamkl_fwd_splitk_workspace_bytes(B, H, NQ, num_splits))


def streamkl_suggest_splits(B, H, NQ, NK, causal):
    return int(lib().streamkl_suggest_splits(B, H, NQ, NK, int(bool(causal))))


@_on_its_stream
def streamkl_fwd_splitk(q1, k1, q2, k2, scale, causal, num_splits, workspace=None,
                        kl=None, lse1=None, lse2=None, stream=None):
    """Key-split forward plus merge; ``workspace`` is a caller-owned byte buffer."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    need = streamkl_fwd_splitk_workspace_bytes(B, H, NQ, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q1.device)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd_splitk(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                     B, H, NQ, NK, d1, d2, float(scale), int(bool(causal)),
                                     int(num_splits), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(),
                                     kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd_splitk")
    return kl, lse1, lse2


# Size in bytes of the library's fixed key-split workspace (see the header).
STREAMKL_STATIC_WORKSPACE_BYTES = 32 << 20


@_on_its_stream
def streamkl_fwd_splitk_noalloc(q1, k1, q2, k2, scale, causal, num_splits, kl=None, lse1=None,
                                lse2=None, stream=None):
    """Key-split forward that allocates no device memory inside the library.

    For callers that cannot provide scratch memory (for example code running
    under an allocator that owns all device memory): the per-split partials
    live in a fixed array of STREAMKL_STATIC_WORKSPACE_BYTES inside the
    library.  Calls overlapping on the GPU race on that array; the first call
    on a device should precede any stream capture there.  Pass preallocated
    ``kl``/``lse1``/``lse2`` to keep this wrapper allocation-free as well.
    """
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd_splitk_noalloc(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                             B, H, NQ, NK, d1, d2, float(scale), int(bool(causal)),
                                             int(num_splits), kl.data_ptr(), lse1.data_ptr(),
                                             lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd_splitk_noalloc")
    return kl, lse1, lse2


@_on_its_stream
def streamkl_bwd(q1, k1, q2, k2, scale, causal, kl, lse1, lse2, dkl, mode=STREAMKL_GRAD_P2,
                 deterministic=False, dq=None, dk=None, stream=None):
    """(dQ, dK) fp32 for the side ``mode`` selects; see include/streamkl.h."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    dg = d2 if mode == STREAMKL_GRAD_P2 else d1
    for name, t in (("kl", kl), ("lse1", lse1), ("lse2", lse2), ("dkl", dkl)):
        _out(t, (B, H, NQ), q1.device, name)
    dq = _out(dq, (B, H, NQ, dg), q1.device, "dq")
    dk = _out(dk, (B, H, NK, dg), q1.device, "dk")
    _check(lib().streamkl_bwd(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                              B, H, NQ, NK, d1, d2, float(scale), int(bool(causal)),
                              kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), dkl.data_ptr(),
                              int(mode), int(bool(deterministic)), dq.data_ptr(), dk.data_ptr(),
                              _stream(stream)),
           "streamkl_bwd")
    return dq, dk


@_on_its_stream
def streamkl_fwd_scaled(q1, k1, q2, k2, scale1, scale2, causal, kl=None, lse1=None, lse2=None, stream=None):
    """streamkl_fwd with S1 = scale1 Q1 K1^T and S2 = scale2 Q2 K2^T."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd_scaled(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                     B, H, NQ, NK, d1, d2, float(scale1), float(scale2), int(bool(causal)),
                                     kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd_scaled")
    return kl, lse1, lse2


@_on_its_stream
def streamkl_fwd_splitk_scaled(q1, k1, q2, k2, scale1, scale2, causal, num_splits, workspace=None,
                               kl=None, lse1=None, lse2=None, stream=None):
    """streamkl_fwd_splitk with a softmax scale per side."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    need = streamkl_fwd_splitk_workspace_bytes(B, H, NQ, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q1.device)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd_splitk_scaled(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                            B, H, NQ, NK, d1, d2, float(scale1), float(scale2),
                                            int(bool(causal)), int(num_splits), workspace.data_ptr(),
                                            workspace.numel() * workspace.element_size(),
                                            kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd_splitk_scaled")
    return kl, lse1, lse2


@_on_its_stream
def streamkl_bwd_scaled(q1, k1, q2, k2, scale1, scale2, causal, kl, lse1, lse2, dkl, mode=STREAMKL_GRAD_P2,
                        deterministic=False, dq=None, dk=None, stream=None):
    """streamkl_bwd with a softmax scale per side (kl/lse from streamkl_fwd_scaled)."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    dg = d2 if mode == STREAMKL_GRAD_P2 else d1
    for name, t in (("kl", kl), ("lse1", lse1), ("lse2", lse2), ("dkl", dkl)):
        _out(t, (B, H, NQ), q1.device, name)
    dq = _out(dq, (B, H, NQ, dg), q1.device, "dq")
    dk = _out(dk, (B, H, NK, dg), q1.device, "dk")
    _check(lib().streamkl_bwd_scaled(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                     B, H, NQ, NK, d1, d2, float(scale1), float(scale2), int(bool(causal)),
                                     kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), dkl.data_ptr(),
                                     int(mode), int(bool(deterministic)), dq.data_ptr(), dk.data_ptr(),
                                     _stream(stream)),
           "streamkl_bwd_scaled")
    return dq, dk


@_on_its_stream
def streamkl_fwd_gqa(q1, k1, q2, k2, scale1, scale2, causal, kl=None, lse1=None, lse2=None, stream=None):
    """streamkl_fwd_scaled with grouped key heads: k1 [B, HK1, NK, d1] and
    k2 [B, HK2, NK, d2], query head h reading key head h // (H // HK)."""
    B, H, HK1, HK2, NQ, NK, d1, d2 = _dims_gqa(q1, k1, q2, k2)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd_gqa(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                  B, H, HK1, HK2, NQ, NK, d1, d2, float(scale1), float(scale2), int(bool(causal)),
                                  kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd_gqa")
    return kl, lse1, lse2


@_on_its_stream
def streamkl_fwd_splitk_gqa(q1, k1, q2, k2, scale1, scale2, causal, num_splits, workspace=None,
                            kl=None, lse1=None, lse2=None, stream=None):
    """streamkl_fwd_splitk_scaled with grouped key heads."""
    B, H, HK1, HK2, NQ, NK, d1, d2 = _dims_gqa(q1, k1, q2, k2)
    need = streamkl_fwd_splitk_workspace_bytes(B, H, NQ, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q1.device)
    kl = _out(kl, (B, H, NQ), q1.device, "kl")
    lse1 = _out(lse1, (B, H, NQ), q1.device, "lse1")
    lse2 = _out(lse2, (B, H, NQ), q1.device, "lse2")
    _check(lib().streamkl_fwd_splitk_gqa(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                         B, H, HK1, HK2, NQ, NK, d1, d2, float(scale1), float(scale2),
                                         int(bool(causal)), int(num_splits), workspace.data_ptr(),
                                         workspace.numel() * workspace.element_size(),
                                         kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), _stream(stream)),
           "streamkl_fwd_splitk_gqa")
    return kl, lse1, lse2


@_on_its_stream
def streamkl_bwd_gqa(q1, k1, q2, k2, scale1, scale2, causal, kl, lse1, lse2, dkl, mode=STREAMKL_GRAD_P2,
                     deterministic=False, dq=None, dk=None, stream=None):
    """streamkl_bwd_scaled with grouped key heads: dq [B, H, NQ, dg] per query
    head, dk [B, HK_g, NK, dg] per key head of the gradient side (summed over
    the query heads that read it)."""
    B, H, HK1, HK2, NQ, NK, d1, d2 = _dims_gqa(q1, k1, q2, k2)
    dg, hkg = (d2, HK2) if mode == STREAMKL_GRAD_P2 else (d1, HK1)
    for name, t in (("kl", kl), ("lse1", lse1), ("lse2", lse2), ("dkl", dkl)):
        _out(t, (B, H, NQ), q1.device, name)
    dq = _out(dq, (B, H, NQ, dg), q1.device, "dq")
    dk = _out(dk, (B, hkg, NK, dg), q1.device, "dk")
    _check(lib().streamkl_bwd_gqa(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                  B, H, HK1, HK2, NQ, NK, d1, d2, float(scale1), float(scale2), int(bool(causal)),
                                  kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), dkl.data_ptr(),
                                  int(mode), int(bool(deterministic)), dq.data_ptr(), dk.data_ptr(),
                                  _stream(stream)),
           "streamkl_bwd_gqa")
    return dq, dk


def streamkl_bwd_workspace_bytes(B, H, HK1, HK2, NK, d1, d2, mode=STREAMKL_GRAD_P2, deterministic=True):
    """Scratch bytes streamkl_bwd_gqa_ws needs (see the header)."""
    return int(lib().streamkl_bwd_workspace_bytes(B, H, HK1, HK2, NK, d1, d2, int(mode), int(bool(deterministic))))


@_on_its_stream
def streamkl_bwd_gqa_ws(q1, k1, q2, k2, scale1, scale2, causal, kl, lse1, lse2, dkl, workspace,
                        mode=STREAMKL_GRAD_P2, deterministic=True, dq=None, dk=None, stream=None):
    """streamkl_bwd_gqa with the deterministic mode's scratch in `workspace`
    (a CUDA tensor of at least streamkl_bwd_workspace_bytes bytes, or None
    when that is 0)."""
    B, H, HK1, HK2, NQ, NK, d1, d2 = _dims_gqa(q1, k1, q2, k2)
    dg, hkg = (d2, HK2) if mode == STREAMKL_GRAD_P2 else (d1, HK1)
    for name, t in (("kl", kl), ("lse1", lse1), ("lse2", lse2), ("dkl", dkl)):
        _out(t, (B, H, NQ), q1.device, name)
    dq = _out(dq, (B, H, NQ, dg), q1.device, "dq")
    dk = _out(dk, (B, hkg, NK, dg), q1.device, "dk")
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().streamkl_bwd_gqa_ws(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                     B, H, HK1, HK2, NQ, NK, d1, d2, float(scale1), float(scale2),
                                     int(bool(causal)), kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(),
                                     dkl.data_ptr(), int(mode), int(bool(deterministic)), dq.data_ptr(),
                                     dk.data_ptr(), ws_ptr, ws_bytes, _stream(stream)),
           "streamkl_bwd_gqa_ws")
    return dq, dk


@_on_its_stream
def streamkl_bwd_both(q1, k1, q2, k2, scale1, scale2, causal, kl, lse1, lse2, dkl, deterministic=False,
                      dq1=None, dk1=None, dq2=None, dk2=None, stream=None):
    """(dQ1, dK1, dQ2, dK2) fp32: the gradients of sum(dkl * KL) on both sides."""
    B, H, NQ, NK, d1, d2 = _dims(q1, k1, q2, k2)
    for name, t in (("kl", kl), ("lse1", lse1), ("lse2", lse2), ("dkl", dkl)):
        _out(t, (B, H, NQ), q1.device, name)
    dq1 = _out(dq1, (B, H, NQ, d1), q1.device, "dq1")
    dk1 = _out(dk1, (B, H, NK, d1), q1.device, "dk1")
    dq2 = _out(dq2, (B, H, NQ, d2), q1.device, "dq2")
    dk2 = _out(dk2, (B, H, NK, d2), q1.device, "dk2")
    _check(lib().streamkl_bwd_both(q1.data_ptr(), k1.data_ptr(), q2.data_ptr(), k2.data_ptr(),
                                   B, H, NQ, NK, d1, d2, float(scale1), float(scale2), int(bool(causal)),
                                   kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(), dkl.data_ptr(),
                                   int(bool(deterministic)), dq1.data_ptr(), dk1.data_ptr(), dq2.data_ptr(),
                                   dk2.data_ptr(), _stream(stream)),
           "streamkl_bwd_both")
    return dq1, dk1, dq2, dk2


def _view(t):
    b, h, n, _ = t.stride()
    return _View(t.data_ptr(), b, h, n)


class AttnSide:
    """One attention distribution over modified scores (see the header):
    q [B, H, NQ, d] and k [B, HK, NK, d] bf16 (any strides that are multiples
    of 8 with a dense last dimension, a transposed [B, N, H, d] for one),
    scale, an optional softcap, and either slopes [H] or a learned table
    [H, num_buckets] (fp32, contiguous) with max_distance and bidirectional.

    Holds references to its tensors, no copies; may be used for any number of
    calls while they keep their memory.
    """

    def __init__(self, q, k, scale, softcap=0.0, slopes=None, table=None, max_distance=128, bidirectional=False):
        for t in (q, k):
            if not isinstance(t, torch.Tensor) or t.dtype != torch.bfloat16 or not t.is_cuda:
                raise TypeError("q and k must be CUDA bf16 tensors")
            if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
                raise ValueError("q and k must be [B, heads, N, d] tensors whose last dimension is dense")
        B, H, NQ, d = q.shape
        Bk, HK, NK, dk = k.shape
        device = q.device
        if Bk != B or dk != d:
            raise ValueError("inconsistent shapes: want q [B,H,NQ,d] and k [B,HK,NK,d]")
        if k.device != device:
            raise ValueError("q and k must be on the same device")
        if slopes is not None or table is not None:
            for name, t in (("slopes", slopes), ("table", table)):
                if t is not None and (not isinstance(t, torch.Tensor) or t.dtype != torch.float32 or
                                      t.device != device or not t.is_contiguous()):
                    raise TypeError(f"{name} must be a contiguous fp32 tensor on {device}")
            if slopes is not None and tuple(slopes.shape) != (H,):
                raise ValueError(f"slopes must have one value for each of the {H} heads")
            if table is not None and (table.dim() != 2 or table.shape[0] != H):
                raise ValueError(f"table must have one row for each of the {H} heads")
        self.q, self.k, self.slopes, self.table = q, k, slopes, table
        self.device, self.rows, self.keys = device, (B, H, NQ), NK
        self.num_buckets = 0 if table is None else table.shape[1]
        self._c = _Side(_view(q), _view(k), d, HK, float(scale), float(softcap),
                        None if slopes is None else slopes.data_ptr(), None if table is None else table.data_ptr(),
                        self.num_buckets, int(max_distance), int(bool(bidirectional)))


def _mod_call(p1, p2, causal, prefix, doc_q, doc_k):
    """(B, H, NQ, NK, streamkl_visible) of a call, its shapes and devices checked."""
    B, H, NQ = p1.rows
    NK = p1.keys
    if p2.rows != p1.rows or p2.keys != NK:
        raise ValueError("both sides must have the same B, H, NQ and NK")
    if p2.device != p1.device:
        raise ValueError("both sides must be on the same device")
    if prefix is None and doc_q is None and doc_k is None:
        return B, H, NQ, NK, _Visible(1 if causal else 0)
    for name, t, shape in (("prefix", prefix, (B,)), ("doc_q", doc_q, (B, NQ)), ("doc_k", doc_k, (B, NK))):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.device != p1.device or \
                not t.is_contiguous() or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on {p1.device}")
    return B, H, NQ, NK, _Visible(1 if causal else 0, *(None if t is None else t.data_ptr()
                                                        for t in (prefix, doc_q, doc_k)))


def _mod_workspace(workspace, need, device, stream):
    """(address, bytes, tensor to keep) of the workspace; torch's own when the caller gives none."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        with _making(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _mod_rows(given, names, shape, device, stream):
    """Per-row outputs, those given checked; the others made here."""
    if given[0] is given[1] is given[2] is None and stream is None:
        return [torch.empty(shape, dtype=torch.float32, device=device) for _ in names]
    with _making(stream):
        out = [_out(t, shape, device, name) for t, name in zip(given, names)]
    _handed_over(stream, device, *zip(given, out))
    return out


# The current stream's handle without a Stream object around it, where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _mod_stream(stream, device):
    if stream is None and _raw_stream is not None:
        return _raw_stream(device.index)
    return _stream(stream)


def _check_stream(stream, device):
    if stream is not None and stream.device != device:
        raise ValueError(f"stream must be one of {device}")


def _on_device(fn):
    """Runs fn with the first side's device current (the library launches there)."""
    @functools.wraps(fn)
    def wrapped(p1, *a, **k):
        if p1.device.index == torch.cuda.current_device():
            return fn(p1, *a, **k)
        with torch.cuda.device(p1.device):
            return fn(p1, *a, **k)
    return wrapped


def _grad_out(t, shape, device, name):
    if t is None:
        return torch.empty(shape, dtype=torch.bfloat16, device=device)
    if t.dtype != torch.bfloat16 or tuple(t.shape) != tuple(shape) or t.device != device or \
            (t.shape[3] > 1 and t.stride(3) != 1):
        raise ValueError(f"{name} must be a bf16 tensor of shape {tuple(shape)} on {device} with a dense last dimension")
    return t


@_on_device
def streamkl_fwd_mod_workspace_bytes(p1, p2, causal=False, prefix=None, doc_q=None, doc_k=None, num_splits=0):
    """Workspace bytes streamkl_fwd_mod needs for these arguments."""
    B, H, NQ, NK, vis = _mod_call(p1, p2, causal, prefix, doc_q, doc_k)
    return int(lib().streamkl_fwd_mod_workspace_bytes(p1._c, p2._c, vis, B, H, NQ, NK, int(num_splits)))


@_on_device
def streamkl_fwd_mod(p1, p2, causal=False, prefix=None, doc_q=None, doc_k=None, num_splits=0, workspace=None, kl=None,
                     lse1=None, lse2=None, stream=None):
    """Per-row KL(P1 || P2), LSE1, LSE2 (fp32 [B, H, NQ]) of two AttnSides,
    over the keys that causal, prefix [B] (int32, with causal) and the
    document ids doc_q [B, NQ], doc_k [B, NK] (int32, negative: padding) leave
    visible; rows that see none get KL 0 and LSE -inf.  num_splits 0: the
    library's choice."""
    B, H, NQ, NK, vis = _mod_call(p1, p2, causal, prefix, doc_q, doc_k)
    dev, num_splits, c = p1.device, int(num_splits), lib()
    if stream is not None:
        _check_stream(stream, dev)
    need = c.streamkl_fwd_mod_workspace_bytes(p1._c, p2._c, vis, B, H, NQ, NK, num_splits)
    ws, ws_bytes, keep = _mod_workspace(workspace, need, dev, stream)
    kl, lse1, lse2 = _mod_rows((kl, lse1, lse2), ("kl", "lse1", "lse2"), (B, H, NQ), dev, stream)
    _check(c.streamkl_fwd_mod(p1._c, p2._c, vis, B, H, NQ, NK, num_splits, ws, ws_bytes, kl.data_ptr(),
                              lse1.data_ptr(), lse2.data_ptr(), _mod_stream(stream, dev)),
           "streamkl_fwd_mod")
    return kl, lse1, lse2


@_on_device
def streamkl_bwd_mod_workspace_bytes(p1, p2, mode=STREAMKL_GRAD_P2, causal=False, prefix=None, doc_q=None, doc_k=None,
                                     deterministic=False, table_grad=True):
    """Workspace bytes streamkl_bwd_mod needs for these arguments."""
    B, H, NQ, NK, vis = _mod_call(p1, p2, causal, prefix, doc_q, doc_k)
    return int(lib().streamkl_bwd_mod_workspace_bytes(p1._c, p2._c, vis, B, H, NQ, NK, int(mode),
                                                      int(bool(deterministic)), int(bool(table_grad))))


@_on_device
def streamkl_bwd_mod(p1, p2, kl, lse1, lse2, dkl, mode=STREAMKL_GRAD_P2, causal=False, prefix=None, doc_q=None,
                     doc_k=None, deterministic=False, table_grad=True, dq=None, dk=None, dtable=None, workspace=None,
                     stream=None):
    """(dq, dk, dtable) for the side `mode` selects: bf16 gradients of its q
    and k (each score's gradient is rounded to bf16 before its products, their
    sums once more), and fp32 of its table (None when it has none or table_grad
    is False).  kl, lse1, lse2 come from streamkl_fwd_mod over the same
    arguments."""
    B, H, NQ, NK, vis = _mod_call(p1, p2, causal, prefix, doc_q, doc_k)
    g = p2 if mode == STREAMKL_GRAD_P2 else p1
    dev, c = g.device, lib()
    if stream is not None:
        _check_stream(stream, dev)
    for name, t in (("kl", kl), ("lse1", lse1), ("lse2", lse2), ("dkl", dkl)):
        if t is None:
            raise ValueError(f"{name} is missing")
        _out(t, (B, H, NQ), dev, name)
    if dtable is not None and g.table is None:
        raise ValueError("dtable given for a side without a table")
    want_table = g.table is not None and (table_grad or dtable is not None)
    det = int(bool(deterministic))
    need = c.streamkl_bwd_mod_workspace_bytes(p1._c, p2._c, vis, B, H, NQ, NK, int(mode), det, int(want_table))
    ws, ws_bytes, keep = _mod_workspace(workspace, need, dev, stream)
    given = (dq, dk, dtable)
    with _making(stream):
        dq = _grad_out(dq, g.q.shape, dev, "dq")
        dk = _grad_out(dk, g.k.shape, dev, "dk")
        if want_table:
            dtable = _out(dtable, (H, g.num_buckets), dev, "dtable")
    _handed_over(stream, dev, *zip(given, (dq, dk, dtable)))
    _check(c.streamkl_bwd_mod(p1._c, p2._c, vis, B, H, NQ, NK, kl.data_ptr(), lse1.data_ptr(), lse2.data_ptr(),
                              dkl.data_ptr(), int(mode), det, _view(dq), _view(dk),
                              dtable.data_ptr() if want_table else None, ws, ws_bytes, _mod_stream(stream, dev)),
           "streamkl_bwd_mod")
    return dq, dk, dtable if want_table else None


def streamkl_get_device_status():
    return int(lib().streamkl_get_device_status())


def streamkl_probe_ex2(out, blocks, iters, stream=None):
    _check(lib().streamkl_probe_ex2(out.data_ptr(), int(blocks), int(iters), _stream(stream)),
           "streamkl_probe_ex2")


def streamkl_selftest_wait_timeout(limit_us, stream=None):
    """Runs a kernel whose barrier wait must time out (see the header)."""
    _check(lib().streamkl_selftest_wait_timeout(int(limit_us), _stream(stream)),
           "streamkl_selftest_wait_timeout")


def streamkl_selftest_turn_timeout(limit_us, words, stream=None):
    """Runs a kernel whose turn wait must time out (see the header); `words`
    is a CUDA int32 tensor of at least 5 elements."""
    _check(lib().streamkl_selftest_turn_timeout(int(limit_us), words.data_ptr(), _stream(stream)),
           "streamkl_selftest_turn_timeout")
