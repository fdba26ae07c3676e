"""ctypes binding of libgdn.so (see include/gdn.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, and their ``data_ptr()`` and the current CUDA stream are handed to
the C entry points.  All computation happens in the library's CUDA kernels.
PyTorch is used for device memory and streams.  If the shared library is
missing, every call raises ``GdnError``: there is no fallback.
"""
import contextlib
import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_PKG, "libgdn.so")

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_TIMEOUT = 0, 1, 2, 3, 4
GDN_F32, GDN_BF16 = 0, 1
_DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_CODES = {torch.int8: 0, torch.float8_e4m3fn: 1}   # gdn_code values
# gdn_prefill_kernel values
PREFILL_KERNELS = {"auto": 0, "simt": 1, "tc": 2}


class GdnError(RuntimeError):
    """A non-OK status from libgdn.so, or the library could not be loaded."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


_lib = None


class PipelineOptions(ctypes.Structure):
    """gdn_pipeline_options: chain_ctas (0 = automatic), wait_limit_cycles (0 = 2^32)."""
    _fields_ = [("chain_ctas", ctypes.c_int), ("wait_limit_cycles", ctypes.c_longlong)]


def library():
    """Loads libgdn.so once (no build step at run time; see ``build.py``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIBRARY_PATH):
            raise GdnError(f"libgdn.so not found at {LIBRARY_PATH}; build it with "
                           "`python -m linear_attention_recurrence_07_b200.build`")
        lib = ctypes.CDLL(LIBRARY_PATH)
        vp, fp, I = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        lib.gdn_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp,
                                      I, I, I, I, I, I, I, I, vp]
        lib.gdn_chunk_fwd.restype = I
        lib.gdn_decode_step.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp,
                                        I, I, I, I, I, I, vp]
        lib.gdn_decode_step.restype = I
        lib.gdn_chunk_fwd_varlen.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, vp,
                                             I, I, I, I, I, I, I, I, vp]
        lib.gdn_chunk_fwd_varlen.restype = I
        lib.gdn_chunk_fwd_split_workspace.argtypes = [I, I, I, I, I, I]
        lib.gdn_chunk_fwd_split_workspace.restype = ctypes.c_size_t
        lib.gdn_chunk_fwd_split.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp,
                                            I, I, I, I, I, I, I, I, I, vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_fwd_split.restype = I
        lib.gdn_chunk_fwd_split_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp,
                                                    I, I, I, I, I, I, I, I, I, vp]
        lib.gdn_chunk_fwd_split_noalloc.restype = I
        lib.gdn_decode_tokens.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, fp,
                                          I, I, I, I, I, I, I, vp]
        lib.gdn_decode_tokens.restype = I
        lib.gdn_decode_step_slots.argtypes = [vp, vp, vp, fp, fp, fp, vp, vp,
                                              I, I, I, I, I, I, I, vp]
        lib.gdn_decode_step_slots.restype = I
        lib.gdn_bwd_workspace.argtypes = [I, I, I, I, I]
        lib.gdn_bwd_workspace.restype = ctypes.c_size_t
        lib.gdn_bwd.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp, fp, fp, fp, fp, fp, fp,
                                I, I, I, I, I, I, I, vp, ctypes.c_size_t, vp]
        lib.gdn_bwd.restype = I
        lib.gdn_bwd_chunk_workspace.argtypes = [I, I, I, I, I]
        lib.gdn_bwd_chunk_workspace.restype = ctypes.c_size_t
        lib.gdn_bwd_chunk.argtypes = lib.gdn_bwd.argtypes
        lib.gdn_bwd_chunk.restype = I
        lib.gdn_chunk_fwd_pipelined_workspace.argtypes = [I, I, I, I, I]
        lib.gdn_chunk_fwd_pipelined_workspace.restype = ctypes.c_size_t
        lib.gdn_chunk_fwd_pipelined.argtypes = [vp, vp, vp, fp, fp, fp, vp, fp,
                                                I, I, I, I, I, I, I, I,
                                                ctypes.POINTER(PipelineOptions), vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_fwd_pipelined.restype = I
        sz = ctypes.c_size_t
        lib.gdn_decay_fwd_workspace.argtypes = [I, I, I, I, I, I]
        lib.gdn_decay_fwd_workspace.restype = sz
        lib.gdn_decay_bwd_workspace.argtypes = [I, I, I, I, I, I, I]
        lib.gdn_decay_bwd_workspace.restype = sz
        for name, args in (
                ("gdn_decay_fwd", [vp] * 7 + [I] * 7 + [vp, sz, vp]),
                ("gdn_decay_fwd_varlen", [vp] * 8 + [I] * 7 + [vp]),
                ("gdn_decay_decode_step", [vp] * 7 + [I] * 6 + [vp]),
                ("gdn_decay_decode_step_slots", [vp] * 7 + [I] * 7 + [vp]),
                ("gdn_decay_bwd", [vp] * 11 + [I] * 7 + [vp, sz, vp]),
                ("gdn_decode_tree", [vp] * 9 + [I] * 8 + [vp]),
                ("gdn_tree_commit", [vp] * 8 + [I] * 8 + [vp]),
                ("gdn_decay_decode_tree", [vp] * 8 + [I] * 8 + [vp]),
                ("gdn_decay_tree_commit", [vp] * 7 + [I] * 8 + [vp]),
                ("gdn_state_store", [vp] * 5 + [I] * 7 + [vp]),
                ("gdn_state_load", [vp] * 5 + [I] * 7 + [vp])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = I
        lib.gdn_set_decay_wait_limit.argtypes = [ctypes.c_longlong]
        lib.gdn_set_decay_wait_limit.restype = I
        lib.gdn_get_decay_wait_limit.argtypes = []
        lib.gdn_get_decay_wait_limit.restype = ctypes.c_longlong
        lib.gdn_device_status.argtypes = [vp]
        lib.gdn_device_status.restype = I
        lib.gdn_status_string.argtypes = [I]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_last_cuda_error.argtypes = []
        lib.gdn_last_cuda_error.restype = I
        lib.gdn_version.argtypes = []
        lib.gdn_version.restype = I
        lib.gdn_set_prefill_kernel.argtypes = [I]
        lib.gdn_set_prefill_kernel.restype = I
        lib.gdn_get_prefill_kernel.argtypes = []
        lib.gdn_get_prefill_kernel.restype = I
        lib.gdn_prefill_kernel_for.argtypes = [I, I, I]
        lib.gdn_prefill_kernel_for.restype = I
        _lib = lib
    return _lib


def _call(dev, fn, *args):
    """Runs the C entry point with ``dev`` as the current CUDA device (the library
    looks up per-device state, such as static scratch, on the current device)."""
    if torch.cuda.current_device() == dev.index:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _check(status, what):
    if status != GDN_OK:
        lib = library()
        name = lib.gdn_status_string(status).decode()
        extra = ""
        if status == GDN_ERR_CUDA:
            extra = f" (cudaError {lib.gdn_last_cuda_error()})"
        raise GdnError(f"{what} failed: {name}{extra}", status)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without making a Stream object (3 us of a decode call's 13).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device):
    if stream is None:
        if _raw_stream is not None and device.index is not None:
            return _raw_stream(device.index)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def _expect_cuda(q):
    if q.dtype not in _DTYPES:
        raise GdnError(f"unsupported dtype {q.dtype}")
    if q.device.type != "cuda":
        raise GdnError(f"tensors must be on a CUDA device, got {q.device}")


def _expect(t, name, shape, dtype, device):
    if t is not None and t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous():
        return
    if t is None:
        raise GdnError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise GdnError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise GdnError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise GdnError(f"{name}: expected device {device}, got {t.device}")
    if not t.is_contiguous():
        raise GdnError(f"{name} must be contiguous")


def gdn_chunk_fwd(q, k, v, alpha, beta, S0, o, S_final, chunk=64, stream=None):
    """Prefill of T tokens (C entry point ``gdn_chunk_fwd``); writes o and S_final.

    q, k [B, T, Hqk, dk] and v, o [B, T, Hv, dv] (float32 or bfloat16, all the
    same); alpha, beta [B, T, Hv] float32; S0, S_final [B, Hv, dk, dv] float32
    or None.  Asynchronous on ``stream`` (default: the current stream)."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, T, Hv, dv), q.dtype),
                               ("o", o, (B, T, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, T, Hv), torch.float32),
                               ("beta", beta, (B, T, Hv), torch.float32)):
        _expect(t, name, shape, dt, dev)
    for name, t in (("S0", S0), ("S_final", S_final)):
        if t is not None:
            _expect(t, name, (B, Hv, dk, dv), torch.float32, dev)
    _check(_call(dev, library().gdn_chunk_fwd, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                                   _ptr(o), _ptr(S_final), B, T, Hqk, Hv, dk, dv, chunk,
                                   _DTYPES[q.dtype], _stream_handle(stream, dev)),
           "gdn_chunk_fwd")


def gdn_decode_step(q, k, v, alpha, beta, S, o, S_new, stream=None):
    """One decode token (C entry point ``gdn_decode_step``); writes o and S_new
    (S_new may be S itself).  q, k [B, Hqk, dk]; v, o [B, Hv, dv]; alpha, beta
    [B, Hv] float32; S, S_new [B, Hv, dk, dv] float32."""
    B, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, Hv, dv), q.dtype),
                               ("o", o, (B, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, Hv), torch.float32),
                               ("beta", beta, (B, Hv), torch.float32),
                               ("S", S, (B, Hv, dk, dv), torch.float32),
                               ("S_new", S_new, (B, Hv, dk, dv), torch.float32)):
        _expect(t, name, shape, dt, dev)
    _check(_call(dev, library().gdn_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S),
                                     _ptr(o), _ptr(S_new), B, Hqk, Hv, dk, dv,
                                     _DTYPES[q.dtype], _stream_handle(stream, dev)),
           "gdn_decode_step")


def set_prefill_kernel(name):
    """Selects the kernel of every later prefill call of this thread (C entry point
    ``gdn_set_prefill_kernel``, a per-thread setting): one of ``PREFILL_KERNELS``."""
    if name not in PREFILL_KERNELS:
        raise GdnError(f"unknown prefill kernel {name!r}; one of {sorted(PREFILL_KERNELS)}")
    _check(library().gdn_set_prefill_kernel(PREFILL_KERNELS[name]), "gdn_set_prefill_kernel")


def get_prefill_kernel():
    """The current prefill kernel choice, as a key of ``PREFILL_KERNELS``."""
    code = library().gdn_get_prefill_kernel()
    return {v: k for k, v in PREFILL_KERNELS.items()}[code]


def prefill_kernel_for(B, Hv, dtype):
    """The kernel a prefill of B sequences x Hv V heads in ``dtype`` (a torch dtype)
    runs under the current choice (C entry point ``gdn_prefill_kernel_for``)."""
    code = library().gdn_prefill_kernel_for(B, Hv, _DTYPES[dtype])
    if code < 0:
        raise GdnError(f"no prefill kernel takes B={B}, Hv={Hv}, {dtype} under the current choice",
                       GDN_ERR_UNSUPPORTED)
    return {v: k for k, v in PREFILL_KERNELS.items()}[code]


@contextlib.contextmanager
def prefill_kernel(name):
    """Context manager: ``name`` is the prefill kernel inside the block, the previous
    choice is restored after it."""
    prev = get_prefill_kernel()
    set_prefill_kernel(name)
    try:
        yield
    finally:
        set_prefill_kernel(prev)


def split_workspace_bytes(B, T, Hv, segments=0, dk=128, dv=128):
    """Device scratch bytes gdn_chunk_fwd_split needs (C entry point
    ``gdn_chunk_fwd_split_workspace``); 0 when no split happens."""
    return library().gdn_chunk_fwd_split_workspace(B, T, Hv, dk, dv, segments)


def gdn_chunk_fwd_split(q, k, v, alpha, beta, S0, o, S_final, segments=0, workspace=None,
                        chunk=64, stream=None):
    """Segment-parallel prefill (C entry point ``gdn_chunk_fwd_split``): the same
    arguments and results as gdn_chunk_fwd.  ``workspace`` is a uint8 CUDA tensor of
    at least split_workspace_bytes(...) bytes; None allocates one for this call."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, T, Hv, dv), q.dtype),
                               ("o", o, (B, T, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, T, Hv), torch.float32),
                               ("beta", beta, (B, T, Hv), torch.float32)):
        _expect(t, name, shape, dt, dev)
    for name, t in (("S0", S0), ("S_final", S_final)):
        if t is not None:
            _expect(t, name, (B, Hv, dk, dv), torch.float32, dev)
    if workspace is None:
        need = split_workspace_bytes(B, T, Hv, segments, dk, dv)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8:
        raise GdnError("workspace must be a uint8 tensor on the inputs' device")
    _check(_call(dev, library().gdn_chunk_fwd_split, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                         _ptr(S0), _ptr(o), _ptr(S_final), B, T, Hqk, Hv, dk, dv,
                                         chunk, segments, _DTYPES[q.dtype], _ptr(workspace),
                                         workspace.numel(), _stream_handle(stream, dev)),
           "gdn_chunk_fwd_split")


def bwd_workspace_bytes(B, T, Hv, dk=128, dv=128):
    """Device scratch bytes gdn_bwd needs (C entry point ``gdn_bwd_workspace``)."""
    return library().gdn_bwd_workspace(B, T, Hv, dk, dv)


def bwd_chunk_workspace_bytes(B, T, Hv, dk=128, dv=128):
    """Device scratch bytes gdn_bwd_chunk needs (C entry point ``gdn_bwd_chunk_workspace``)."""
    return library().gdn_bwd_chunk_workspace(B, T, Hv, dk, dv)


def _run_bwd(entry, ws_bytes, q, k, v, alpha, beta, S0, dO, dS_final, dq, dk, dv, dalpha, dbeta, dS0,
             workspace, stream):
    B, T, Hqk, dkk = q.shape
    Hv, dvv = v.shape[2], v.shape[3]
    dev = q.device
    _expect_cuda(q)
    f32 = torch.float32
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, T, Hv, dvv), q.dtype),
                               ("dO", dO, (B, T, Hv, dvv), q.dtype),
                               ("alpha", alpha, (B, T, Hv), f32), ("beta", beta, (B, T, Hv), f32),
                               ("dq", dq, q.shape, f32), ("dk", dk, q.shape, f32),
                               ("dv", dv, (B, T, Hv, dvv), f32), ("dalpha", dalpha, (B, T, Hv), f32),
                               ("dbeta", dbeta, (B, T, Hv), f32), ("dS0", dS0, (B, Hv, dkk, dvv), f32)):
        _expect(t, name, shape, dt, dev)
    for name, t in (("S0", S0), ("dS_final", dS_final)):
        if t is not None:
            _expect(t, name, (B, Hv, dkk, dvv), f32, dev)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes(B, T, Hv, dkk, dvv), 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8:
        raise GdnError("workspace must be a uint8 tensor on the inputs' device")
    _check(_call(dev, getattr(library(), entry), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0),
                 _ptr(dO), _ptr(dS_final), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dalpha), _ptr(dbeta),
                 _ptr(dS0), B, T, Hqk, Hv, dkk, dvv, _DTYPES[q.dtype], _ptr(workspace),
                 workspace.numel(), _stream_handle(stream, dev)),
           entry)


def gdn_bwd(q, k, v, alpha, beta, S0, dO, dS_final, dq, dk, dv, dalpha, dbeta, dS0,
            workspace=None, stream=None):
    """Gradients of sum <dO, o> + <dS_final, S_final> (C entry point ``gdn_bwd``).

    q, k, v, dO: the forward's dtype; alpha, beta, S0, dS_final fp32 (S0 and
    dS_final may be None).  Outputs (fp32, overwritten): dq, dk like q; dv like v;
    dalpha, dbeta like alpha; dS0 [B, Hv, dk, dv].  ``workspace``: uint8 CUDA
    tensor of at least bwd_workspace_bytes(...) bytes; None allocates one."""
    _run_bwd("gdn_bwd", bwd_workspace_bytes, q, k, v, alpha, beta, S0, dO, dS_final, dq, dk, dv,
             dalpha, dbeta, dS0, workspace, stream)


def gdn_bwd_chunk(q, k, v, alpha, beta, S0, dO, dS_final, dq, dk, dv, dalpha, dbeta, dS0,
                  workspace=None, stream=None):
    """The gradients of gdn_bwd in the chunkwise form on tensor cores (C entry point
    ``gdn_bwd_chunk``); bf16 q, k, v, dO, the same arguments; ``workspace`` of at
    least bwd_chunk_workspace_bytes(...) bytes, None allocates one."""
    _run_bwd("gdn_bwd_chunk", bwd_chunk_workspace_bytes, q, k, v, alpha, beta, S0, dO, dS_final, dq, dk,
             dv, dalpha, dbeta, dS0, workspace, stream)


def gdn_chunk_fwd_split_noalloc(q, k, v, alpha, beta, S0, o, S_final, segments=0, chunk=64,
                                stream=None):
    """gdn_chunk_fwd_split with the library's static scratch (C entry point
    ``gdn_chunk_fwd_split_noalloc``); the same arguments without a workspace."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, T, Hv, dv), q.dtype),
                               ("o", o, (B, T, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, T, Hv), torch.float32),
                               ("beta", beta, (B, T, Hv), torch.float32)):
        _expect(t, name, shape, dt, dev)
    for name, t in (("S0", S0), ("S_final", S_final)):
        if t is not None:
            _expect(t, name, (B, Hv, dk, dv), torch.float32, dev)
    _check(_call(dev, library().gdn_chunk_fwd_split_noalloc, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                                 _ptr(S0), _ptr(o), _ptr(S_final), B, T, Hqk, Hv,
                                                 dk, dv, chunk, segments, _DTYPES[q.dtype],
                                                 _stream_handle(stream, dev)),
           "gdn_chunk_fwd_split_noalloc")


def gdn_chunk_fwd_varlen(q, k, v, alpha, beta, S0, o, S_final, cu_seqlens, chunk=64,
                         stream=None):
    """Prefill of N packed sequences (C entry point ``gdn_chunk_fwd_varlen``).  q, k
    [T_total, Hqk, dk] and v, o [T_total, Hv, dv] (float32 or bfloat16); alpha,
    beta [T_total, Hv] float32; cu_seqlens [N + 1] int32; S0, S_final
    [N, Hv, dk, dv] float32 or None."""
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    N = cu_seqlens.shape[0] - 1
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (T, Hv, dv), q.dtype),
                               ("o", o, (T, Hv, dv), q.dtype),
                               ("alpha", alpha, (T, Hv), torch.float32),
                               ("beta", beta, (T, Hv), torch.float32),
                               ("cu_seqlens", cu_seqlens, (N + 1,), torch.int32)):
        _expect(t, name, shape, dt, dev)
    for name, t in (("S0", S0), ("S_final", S_final)):
        if t is not None:
            _expect(t, name, (N, Hv, dk, dv), torch.float32, dev)
    _check(_call(dev, library().gdn_chunk_fwd_varlen, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                          _ptr(S0), _ptr(o), _ptr(S_final), _ptr(cu_seqlens),
                                          N, T, Hqk, Hv, dk, dv, chunk, _DTYPES[q.dtype],
                                          _stream_handle(stream, dev)),
           "gdn_chunk_fwd_varlen")


def gdn_decode_tokens(q, k, v, alpha, beta, S, o, S_new, S_steps=None, stream=None):
    """n decode tokens per sequence (C entry point ``gdn_decode_tokens``); writes o,
    S_new (may be S itself) and, if given, S_steps.  q, k [B, n, Hqk, dk]; v, o
    [B, n, Hv, dv]; alpha, beta [B, n, Hv] float32; S, S_new [B, Hv, dk, dv]
    float32; S_steps [B, n, Hv, dk, dv] float32 or None."""
    B, n, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, n, Hv, dv), q.dtype),
                               ("o", o, (B, n, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, n, Hv), torch.float32),
                               ("beta", beta, (B, n, Hv), torch.float32),
                               ("S", S, (B, Hv, dk, dv), torch.float32),
                               ("S_new", S_new, (B, Hv, dk, dv), torch.float32)):
        _expect(t, name, shape, dt, dev)
    if S_steps is not None:
        _expect(S_steps, "S_steps", (B, n, Hv, dk, dv), torch.float32, dev)
    _check(_call(dev, library().gdn_decode_tokens, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S),
                                       _ptr(o), _ptr(S_new), _ptr(S_steps), B, n, Hqk, Hv, dk, dv,
                                       _DTYPES[q.dtype], _stream_handle(stream, dev)),
           "gdn_decode_tokens")


def gdn_decode_step_slots(q, k, v, alpha, beta, state_pool, slots, o, stream=None):
    """One decode token per sequence with states in a pool (C entry point
    ``gdn_decode_step_slots``): state_pool[slots[b]] is updated in place.  q, k
    [B, Hqk, dk]; v, o [B, Hv, dv]; alpha, beta [B, Hv] float32; state_pool
    [n_slots, Hv, dk, dv] float32; slots [B] int32."""
    B, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    n_slots = state_pool.shape[0]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, Hv, dv), q.dtype),
                               ("o", o, (B, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, Hv), torch.float32),
                               ("beta", beta, (B, Hv), torch.float32),
                               ("state_pool", state_pool, (n_slots, Hv, dk, dv), torch.float32),
                               ("slots", slots, (B,), torch.int32)):
        _expect(t, name, shape, dt, dev)
    _check(_call(dev, library().gdn_decode_step_slots, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta),
                                           _ptr(state_pool), _ptr(slots), _ptr(o), B, n_slots,
                                           Hqk, Hv, dk, dv, _DTYPES[q.dtype],
                                           _stream_handle(stream, dev)),
           "gdn_decode_step_slots")


def pipelined_workspace_bytes(B, Hqk, Hv, dk=128, dv=128):
    """Device scratch bytes gdn_chunk_fwd_pipelined needs on the current device (C
    entry point ``gdn_chunk_fwd_pipelined_workspace``)."""
    return library().gdn_chunk_fwd_pipelined_workspace(B, Hqk, Hv, dk, dv)


def gdn_chunk_fwd_pipelined(q, k, v, alpha, beta, S0, o, S_final, chain_ctas=0,
                            wait_limit_cycles=0, workspace=None, chunk=64, stream=None):
    """Prefill with the chunks' WY preparation streamed from SMs of its own (C entry
    point ``gdn_chunk_fwd_pipelined``): the same arguments and results as
    gdn_chunk_fwd.  ``workspace`` is a uint8 CUDA tensor of at least
    pipelined_workspace_bytes(...) bytes; None allocates one for this call."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    dev = q.device
    _expect_cuda(q)
    for name, t, shape, dt in (("k", k, q.shape, q.dtype), ("v", v, (B, T, Hv, dv), q.dtype),
                               ("o", o, (B, T, Hv, dv), q.dtype),
                               ("alpha", alpha, (B, T, Hv), torch.float32),
                               ("beta", beta, (B, T, Hv), torch.float32)):
        _expect(t, name, shape, dt, dev)
    for name, t in (("S0", S0), ("S_final", S_final)):
        if t is not None:
            _expect(t, name, (B, Hv, dk, dv), torch.float32, dev)
    if workspace is None:
        with torch.cuda.device(dev):
            need = pipelined_workspace_bytes(B, Hqk, Hv, dk, dv)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8:
        raise GdnError("workspace must be a uint8 tensor on the inputs' device")
    opts = PipelineOptions(int(chain_ctas), int(wait_limit_cycles))
    _check(_call(dev, library().gdn_chunk_fwd_pipelined, _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
                 _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_final), B, T, Hqk, Hv, dk, dv, chunk,
                 _DTYPES[q.dtype], ctypes.byref(opts), _ptr(workspace), workspace.numel(),
                 _stream_handle(stream, dev)),
           "gdn_chunk_fwd_pipelined")


def _workspace(workspace, nbytes, dev, stream):
    """The caller's workspace checked, or one for this call: memory of ``stream``, which the
    allocator hands out again in that stream's order only."""
    if workspace is None:
        if nbytes == 0:
            return None
        if stream is None:
            return torch.empty(nbytes, dtype=torch.uint8, device=dev)
        with torch.cuda.stream(stream):
            return torch.empty(nbytes, dtype=torch.uint8, device=dev)
    elif workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise GdnError("workspace must be a contiguous uint8 tensor on the inputs' device")
    return workspace


def _shape(t, name, dims):
    if t is None:
        raise GdnError(f"{name} is required")
    shape = t.shape
    if len(shape) != dims:
        raise GdnError(f"{name}: expected {dims} dimensions, got shape {tuple(shape)}")
    return shape


def _pointers(dev, *expected):
    """Data pointers of (name, tensor, shape, dtype) entries, each checked as _expect does; a
    name ending in "?" may be None.  (The checks are most of a small call's time on the host.)"""
    index, out = dev.index, []
    for name, t, shape, dtype in expected:
        if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
            if t is None and name[-1] == "?":
                out.append(None)
                continue
            _expect(t, name.rstrip("?"), shape, dtype, dev)
        out.append(t.data_ptr())
    return out


def _dtype_code(q):
    code = _DTYPES.get(q.dtype)
    if code is None or not q.is_cuda:
        _expect_cuda(q)
    return code


def decay_fwd_workspace_bytes(B, T, Hv, dtype, dk=128, dv=128):
    """Device scratch bytes gdn_decay_fwd needs on the current device (C entry point
    ``gdn_decay_fwd_workspace``); 0 when it cuts no sequence into segments."""
    return library().gdn_decay_fwd_workspace(B, T, Hv, dk, dv, _DTYPES[dtype])


def decay_bwd_workspace_bytes(B, T, Hqk, Hv, dtype, dk=128, dv=128):
    """Device scratch bytes gdn_decay_bwd needs on the current device (C entry point
    ``gdn_decay_bwd_workspace``)."""
    return library().gdn_decay_bwd_workspace(B, T, Hqk, Hv, dk, dv, _DTYPES[dtype])


def gdn_decay_fwd(q, k, v, decay, S0, o, S_final, workspace=None, stream=None):
    """Prefill of linear attention with a constant decay per head (C entry point
    ``gdn_decay_fwd``); writes o and S_final.

    q, k [B, T, Hqk, dk] and v, o [B, T, Hv, dv] (float32 or bfloat16); decay [Hv]
    float32; S0, S_final [B, Hv, dk, dv] float32 or None (S_final may be S0).
    ``workspace``: uint8 CUDA tensor of decay_fwd_workspace_bytes(...) bytes; None
    allocates one for this call."""
    qk = B, T, Hqk, dk = _shape(q, "q", 4)
    _, _, Hv, dv = _shape(v, "v", 4)
    dev, dt, code = q.device, q.dtype, _dtype_code(q)
    rows, state = (B, T, Hv, dv), (B, Hv, dk, dv)
    ptrs = _pointers(dev, ("q", q, qk, dt), ("k", k, qk, dt), ("v", v, rows, dt), ("decay", decay, (Hv,), torch.float32),
                     ("S0?", S0, state, torch.float32), ("o", o, rows, dt), ("S_final?", S_final, state, torch.float32))
    need = _call(dev, library().gdn_decay_fwd_workspace, B, T, Hv, dk, dv, code)
    workspace = _workspace(workspace, need, dev, stream)
    _check(_call(dev, library().gdn_decay_fwd, *ptrs, B, T, Hqk, Hv, dk, dv, code, _ptr(workspace),
                 0 if workspace is None else workspace.numel(), _stream_handle(stream, dev)),
           "gdn_decay_fwd")


def gdn_decay_fwd_varlen(q, k, v, decay, S0, o, S_final, cu_seqlens, stream=None):
    """gdn_decay_fwd of N packed sequences (C entry point ``gdn_decay_fwd_varlen``).
    q, k [T_total, Hqk, dk]; v, o [T_total, Hv, dv]; decay [Hv]; cu_seqlens [N + 1]
    int32; S0, S_final [N, Hv, dk, dv] float32 or None."""
    qk = T, Hqk, dk = _shape(q, "q", 3)
    _, Hv, dv = _shape(v, "v", 3)
    N = _shape(cu_seqlens, "cu_seqlens", 1)[0] - 1
    if N < 0:
        raise GdnError("cu_seqlens: at least one entry is required")
    dev, dt, code = q.device, q.dtype, _dtype_code(q)
    rows, state = (T, Hv, dv), (N, Hv, dk, dv)
    ptrs = _pointers(dev, ("q", q, qk, dt), ("k", k, qk, dt), ("v", v, rows, dt), ("decay", decay, (Hv,), torch.float32),
                     ("S0?", S0, state, torch.float32), ("o", o, rows, dt), ("S_final?", S_final, state, torch.float32),
                     ("cu_seqlens", cu_seqlens, (N + 1,), torch.int32))
    _check(_call(dev, library().gdn_decay_fwd_varlen, *ptrs, N, T, Hqk, Hv, dk, dv, code, _stream_handle(stream, dev)),
           "gdn_decay_fwd_varlen")


def gdn_decay_decode_step(q, k, v, decay, S, o, S_new, stream=None):
    """One decode token with a constant decay per head (C entry point
    ``gdn_decay_decode_step``); writes o and S_new (which may be S).  q, k
    [B, Hqk, dk]; v, o [B, Hv, dv]; decay [Hv]; S, S_new [B, Hv, dk, dv] float32."""
    qk = B, Hqk, dk = _shape(q, "q", 3)
    _, Hv, dv = _shape(v, "v", 3)
    dev, dt, code = q.device, q.dtype, _dtype_code(q)
    rows, state = (B, Hv, dv), (B, Hv, dk, dv)
    ptrs = _pointers(dev, ("q", q, qk, dt), ("k", k, qk, dt), ("v", v, rows, dt), ("decay", decay, (Hv,), torch.float32),
                     ("S", S, state, torch.float32), ("o", o, rows, dt), ("S_new", S_new, state, torch.float32))
    _check(_call(dev, library().gdn_decay_decode_step, *ptrs, B, Hqk, Hv, dk, dv, code, _stream_handle(stream, dev)),
           "gdn_decay_decode_step")


def gdn_decay_decode_step_slots(q, k, v, decay, state_pool, slots, o, stream=None):
    """gdn_decay_decode_step with states in a pool, updated in place (C entry point
    ``gdn_decay_decode_step_slots``): state_pool [n_slots, Hv, dk, dv] float32;
    slots [B] int32, out of range = padding."""
    qk = B, Hqk, dk = _shape(q, "q", 3)
    _, Hv, dv = _shape(v, "v", 3)
    n_slots = _shape(state_pool, "state_pool", 4)[0]
    dev, dt, code = q.device, q.dtype, _dtype_code(q)
    rows = (B, Hv, dv)
    ptrs = _pointers(dev, ("q", q, qk, dt), ("k", k, qk, dt), ("v", v, rows, dt), ("decay", decay, (Hv,), torch.float32),
                     ("state_pool", state_pool, (n_slots, Hv, dk, dv), torch.float32),
                     ("slots", slots, (B,), torch.int32), ("o", o, rows, dt))
    _check(_call(dev, library().gdn_decay_decode_step_slots, *ptrs, B, n_slots, Hqk, Hv, dk, dv, code,
                 _stream_handle(stream, dev)),
           "gdn_decay_decode_step_slots")


def gdn_decay_bwd(q, k, v, decay, S0, dO, dS_final, dq, dk, dv, dS0, workspace=None, stream=None):
    """Gradients of sum <dO, o> + <dS_final, S_final> through gdn_decay_fwd (C entry
    point ``gdn_decay_bwd``).  q, k, v, dO of one dtype (float32 or bfloat16); S0,
    dS_final float32 or None.  Outputs (overwritten): dq, dk, dv like q, k, v, in their
    dtype; dS0 [B, Hv, dk, dv] float32 or None.  ``workspace``: uint8 CUDA tensor of
    decay_bwd_workspace_bytes(...) bytes; None allocates one."""
    qk = B, T, Hqk, dkk = _shape(q, "q", 4)
    _, _, Hv, dvv = _shape(v, "v", 4)
    dev, dt, code = q.device, q.dtype, _dtype_code(q)
    rows, state = (B, T, Hv, dvv), (B, Hv, dkk, dvv)
    ptrs = _pointers(dev, ("q", q, qk, dt), ("k", k, qk, dt), ("v", v, rows, dt), ("decay", decay, (Hv,), torch.float32),
                     ("S0?", S0, state, torch.float32), ("dO", dO, rows, dt),
                     ("dS_final?", dS_final, state, torch.float32), ("dq", dq, qk, dt), ("dk", dk, qk, dt),
                     ("dv", dv, rows, dt), ("dS0?", dS0, state, torch.float32))
    need = _call(dev, library().gdn_decay_bwd_workspace, B, T, Hqk, Hv, dkk, dvv, code)
    workspace = _workspace(workspace, need, dev, stream)
    _check(_call(dev, library().gdn_decay_bwd, *ptrs, B, T, Hqk, Hv, dkk, dvv, code, _ptr(workspace),
                 0 if workspace is None else workspace.numel(), _stream_handle(stream, dev)),
           "gdn_decay_bwd")


@contextlib.contextmanager
def decay_wait_limit(microseconds):
    """Context manager: how long a wait inside this thread's bf16 decay prefill and
    gradient kernels may take before it gives up (C entry point
    ``gdn_set_decay_wait_limit``; 0 = the default of two seconds); the previous limit is
    restored after the block."""
    lib = library()
    prev = lib.gdn_get_decay_wait_limit()
    _check(lib.gdn_set_decay_wait_limit(int(microseconds)), "gdn_set_decay_wait_limit")
    try:
        yield
    finally:
        lib.gdn_set_decay_wait_limit(prev)


def _tree_call(what, q, k, v, gates, parents, accepted, state_pool, slots, o, stream):
    """The four tree entry points: q and o, or accepted; gates (alpha, beta) or (decay,)."""
    qk = B, n, Hqk, dk = _shape(k, "k", 4)
    _, _, Hv, dv = _shape(v, "v", 4)
    n_slots = _shape(state_pool, "state_pool", 4)[0]
    dev, dt, code = k.device, k.dtype, _dtype_code(k)
    rows = (B, n, Hv, dv)
    names = ("decay",) if len(gates) == 1 else ("alpha", "beta")
    gate = (Hv,) if len(gates) == 1 else (B, n, Hv)
    expected = [] if accepted is not None else [("q", q, qk, dt)]
    expected += [("k", k, qk, dt), ("v", v, rows, dt)]
    expected += [(name, t, gate, torch.float32) for name, t in zip(names, gates)]
    expected.append(("parents", parents, (B, n), torch.int32))
    if accepted is not None:
        expected.append(("accepted", accepted, (B,), torch.int32))
    expected += [("state_pool", state_pool, (n_slots, Hv, dk, dv), torch.float32), ("slots?", slots, (B,), torch.int32)]
    if accepted is None:
        expected.append(("o", o, rows, dt))
    _check(_call(dev, getattr(library(), what), *_pointers(dev, *expected), B, n, n_slots, Hqk, Hv, dk, dv, code,
                 _stream_handle(stream, dev)), what)


def gdn_decode_tree(q, k, v, alpha, beta, parents, state_pool, slots, o, stream=None):
    """Outputs of trees of drafted tokens (C entry point ``gdn_decode_tree``): node i
    of sequence b continues node parents[b, i] < i, or the state state_pool[slots[b]]
    where that is -1; any other parent marks padding, whose o rows stay as they were.

    q, k [B, n, Hqk, dk]; v, o [B, n, Hv, dv]; alpha, beta [B, n, Hv] float32;
    parents [B, n] int32; state_pool [n_slots, Hv, dk, dv] float32 (not changed);
    slots [B] int32 or None (sequence b uses row b).  n <= 64."""
    _tree_call("gdn_decode_tree", q, k, v, (alpha, beta), parents, None, state_pool, slots, o, stream)


def gdn_tree_commit(k, v, alpha, beta, parents, accepted, state_pool, slots, stream=None):
    """Moves state_pool[slots[b]] to the state after node accepted[b] of its tree, in
    place (C entry point ``gdn_tree_commit``); accepted [B] int32, out of range =
    nothing accepted.  Other arguments as gdn_decode_tree."""
    if accepted is None:
        raise GdnError("accepted is required")
    _tree_call("gdn_tree_commit", None, k, v, (alpha, beta), parents, accepted, state_pool, slots, None, stream)


def gdn_decay_decode_tree(q, k, v, decay, parents, state_pool, slots, o, stream=None):
    """gdn_decode_tree for the constant-decay rule (C entry point
    ``gdn_decay_decode_tree``): decay [Hv] float32 in place of the gates."""
    _tree_call("gdn_decay_decode_tree", q, k, v, (decay,), parents, None, state_pool, slots, o, stream)


def gdn_decay_tree_commit(k, v, decay, parents, accepted, state_pool, slots, stream=None):
    """gdn_tree_commit for the constant-decay rule (C entry point
    ``gdn_decay_tree_commit``)."""
    if accepted is None:
        raise GdnError("accepted is required")
    _tree_call("gdn_decay_tree_commit", None, k, v, (decay,), parents, accepted, state_pool, slots, None, stream)


def _cache_args(state_pool, slots, codes, scales, cache_slots):
    """Pointers of state_pool, slots, codes, scales, cache_slots, and the sizes."""
    pool = n_slots, Hv, dk, dv = _shape(state_pool, "state_pool", 4)
    n_cache = _shape(codes, "codes", 4)[0]
    N = _shape(slots, "slots", 1)[0]
    dev, code = state_pool.device, _CODES.get(codes.dtype)
    if not state_pool.is_cuda:
        raise GdnError(f"tensors must be on a CUDA device, got {dev}")
    if code is None:
        raise GdnError(f"codes: expected torch.int8 or torch.float8_e4m3fn, got {codes.dtype}")
    ptrs = _pointers(dev, ("state_pool", state_pool, pool, torch.float32), ("slots", slots, (N,), torch.int32),
                     ("codes", codes, (n_cache, Hv, dk, dv), codes.dtype),
                     ("scales", scales, (n_cache, Hv, dk), torch.float32), ("cache_slots", cache_slots, (N,), torch.int32))
    return ptrs, (N, n_slots, n_cache, Hv, dk, dv, code)


def gdn_state_store(state_pool, slots, codes, scales, cache_slots, stream=None):
    """Snapshots of pool states as 8-bit codes with one scale per key row (C entry
    point ``gdn_state_store``): row cache_slots[i] of the cache gets
    state_pool[slots[i]].  state_pool [n_slots, Hv, dk, dv] float32; codes
    [n_cache, Hv, dk, dv] int8 or float8_e4m3fn; scales [n_cache, Hv, dk] float32;
    slots, cache_slots [N] int32, out of range = skipped."""
    ptrs, sizes = _cache_args(state_pool, slots, codes, scales, cache_slots)
    dev = state_pool.device
    _check(_call(dev, library().gdn_state_store, *ptrs, *sizes, _stream_handle(stream, dev)), "gdn_state_store")


def gdn_state_load(codes, scales, cache_slots, state_pool, slots, stream=None):
    """Brings snapshots back (C entry point ``gdn_state_load``): state_pool[slots[i]] =
    codes * scales of cache row cache_slots[i].  Arguments as gdn_state_store."""
    (pool, slot, code, scale, cache_slot), sizes = _cache_args(state_pool, slots, codes, scales, cache_slots)
    dev = state_pool.device
    _check(_call(dev, library().gdn_state_load, code, scale, cache_slot, pool, slot, *sizes, _stream_handle(stream, dev)),
           "gdn_state_load")


def device_status(stream=None, device=None):
    """Waits for ``stream`` and returns (and clears) the library's device error
    state as a status name: "GDN_OK", or "GDN_ERR_TIMEOUT" if a bounded wait inside
    a kernel gave up (C entry point ``gdn_device_status``)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    code = _call(dev, library().gdn_device_status, _stream_handle(stream, dev))
    return library().gdn_status_string(code).decode()


def chunk_fwd(q, k, v, alpha, beta, S0=None, chunk=64, stream=None):
    """Allocating convenience wrapper: returns (o, S_final)."""
    B, T, Hqk, dk = q.shape
    Hv, dv = v.shape[2], v.shape[3]
    o = torch.empty((B, T, Hv, dv), dtype=q.dtype, device=q.device)
    S_final = torch.empty((B, Hv, dk, dv), dtype=torch.float32, device=q.device)
    gdn_chunk_fwd(q, k, v, alpha, beta, S0, o, S_final, chunk=chunk, stream=stream)
    return o, S_final


def decode_step(q, k, v, alpha, beta, S, stream=None):
    """In-place decode convenience wrapper: updates S and returns o."""
    B, Hv, dv = v.shape
    o = torch.empty((B, Hv, dv), dtype=q.dtype, device=q.device)
    gdn_decode_step(q, k, v, alpha, beta, S, o, S, stream=stream)
    return o
