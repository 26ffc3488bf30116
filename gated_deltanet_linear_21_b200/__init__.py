"""Gated DeltaNet token mixer forward pass for NVIDIA B200 (sm_100a).

A thin ctypes binding over ``libgdn.so`` (declared in ``include/gdn.h``):
argument marshalling only -- every step of the computation runs in the CUDA
kernels of the library. PyTorch provides device memory and streams. There is
no CPU fallback: if the library is missing the import of an op fails loudly.

    o, state_out = prefill(q, k, v, g, beta, state_in=None, cu_seqlens=None)
    o = decode(q, k, v, g, beta, state)          # state updated in place

    o, state_out = linear_prefill(q, k, v, g, state_in=None, cu_seqlens=None)   # without the delta term
    o = linear_decode(q, k, v, g, state)

    codes, exps = state_pool(n_slots, Hv, dv, dk)  # states of many sequences, in 8 bits
    state_store(state, codes, exps, slots)
    state = state_load(codes, exps, slots)

q, k and v may be bf16, f16 or fp32 (all three the same); g, beta and the
prefill states are fp32.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

__all__ = ["prefill", "prefill_noalloc", "decode", "prefill_workspace_bytes", "prefill_plan", "device_error",
           "wait_selftest",
           "linear_prefill", "linear_prefill_workspace_bytes", "linear_decode",
           "state_pool", "state_store", "state_load",
           "GdnError",
           "lib", "debug_lib", "library_path", "debug_library_path", "GDN_BF16", "GDN_F32", "GDN_F16"]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "libgdn.so")
debug_library_path = os.path.join(_PKG, "libgdn_debug.so")   # GDN_DEBUG build: device-side index checks

(GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_DEVICE_TIMEOUT,
 GDN_ERR_DEVICE_CHECK) = range(6)
GDN_BF16, GDN_F32, GDN_F16 = 0, 1, 2
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED",
                3: "GDN_ERR_CUDA", 4: "GDN_ERR_DEVICE_TIMEOUT", 5: "GDN_ERR_DEVICE_CHECK"}


class GdnPlan(ctypes.Structure):
    """struct gdn_plan: the tensor-core prefill's launch plan (0 = the library's choice)."""
    _fields_ = [("dvp", ctypes.c_int), ("n_chain_ctas", ctypes.c_int)]


def _plan_arg(plan):
    """A (dvp, n_chain_ctas) pair (None or 0 per field: the library's choice) as a
    gdn_plan pointer, or None."""
    if plan is None:
        return None
    dvp, nc = plan
    return ctypes.byref(GdnPlan(int(dvp or 0), int(nc or 0)))


class GdnError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


_lock = threading.Lock()
_lib = None

_vp, _fp, _i32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
_i, _i64, _f, _sz = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t

SIGNATURES = {
    "gdn_version": (_i, []),
    "gdn_last_error": (ctypes.c_char_p, []),
    "gdn_prefill_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "gdn_prefill": (_i, [_vp, _vp, _vp, _fp, _fp, _fp, _i32p, _i, _i64, _i, _i, _i, _i, _f, _i, _i,
                         _vp, _fp, _vp, _sz, _vp]),
    "gdn_decode": (_i, [_vp, _vp, _vp, _fp, _fp, _fp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "gdn_decode_bf16_state": (_i, [_vp, _vp, _vp, _fp, _fp, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "gdn_prefill_noalloc": (_i, [_vp, _vp, _vp, _fp, _fp, _fp, _i32p, _i, _i64, _i, _i, _i, _i, _f, _i, _i,
                                 _vp, _fp, _vp]),
    "gdn_device_error": (_i, [_vp]),
    "gdn_wait_selftest": (_i, [_i, _vp]),
    "gdn_prefill_ex": (_i, [_vp, _vp, _vp, _fp, _fp, _fp, _i32p, _i, _i64, _i, _i, _i, _i, _f, _i, _i,
                            _vp, _fp, _vp, _sz, _vp, _vp]),
    "gdn_prefill_plan": (_i, [_i, _i64, _i, _i, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "gdn_debug_checks": (_i, []),
    "gdn_linear_prefill_workspace_bytes": (_sz, [_i, _i64, _i, _i, _i, _i]),
    "gdn_linear_prefill": (_i, [_vp, _vp, _vp, _fp, _i, _fp, _i32p, _i, _i64, _i, _i, _i, _i, _f, _i,
                                _vp, _fp, _vp, _sz, _vp]),
    "gdn_linear_decode": (_i, [_vp, _vp, _vp, _fp, _i, _fp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "gdn_linear_decode_bf16_state": (_i, [_vp, _vp, _vp, _fp, _i, _vp, _i, _i, _i, _i, _i, _f, _i, _vp, _vp]),
    "gdn_state_store": (_i, [_vp, _i, _i32p, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp]),
    "gdn_state_load": (_i, [_vp, _vp, _i32p, _i, _i, _i, _i, _i, _i, _vp, _i, _vp]),
}


def _open(path):
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing: build it with "
            "`python -m gated_deltanet_linear_21_b200.build` (there is no CPU fallback)")
    handle = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = res, args
    return handle


def lib():
    """Load libgdn.so (built in-tree); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is None:
            _lib = _open(library_path)
    return _lib


_debug_lib = None


def debug_lib():
    """Load libgdn_debug.so, the GDN_DEBUG build (same C ABI, device-side index
    checks reported as GDN_ERR_DEVICE_CHECK by its gdn_device_error); a ctypes
    handle for direct calls. The Python wrappers above always use libgdn.so."""
    global _debug_lib
    with _lock:
        if _debug_lib is None:
            _debug_lib = _open(debug_library_path)
    return _debug_lib


def _check(status: int):
    if status != GDN_OK:
        raise GdnError(status, lib().gdn_last_error().decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return GDN_BF16
    if t.dtype == torch.float16:
        return GDN_F16
    if t.dtype == torch.float32:
        return GDN_F32
    raise TypeError(f"q, k, v must be bf16, f16 or fp32, got {t.dtype}")


def _torch_dtype_code(dtype) -> int:
    return {torch.bfloat16: GDN_BF16, torch.float16: GDN_F16, torch.float32: GDN_F32}[dtype]


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _prefill_args(q, k, v, g, beta, state_in, cu_seqlens, o, state_out):
    """Checks and default outputs shared by the prefill entry points."""
    _dev(q, "q"); _dev(k, "k", q.dtype); _dev(v, "v", q.dtype)
    _dev(g, "g", torch.float32); _dev(beta, "beta", torch.float32)
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k must be [T, Hqk, dk] and v [T, Hv, dv]")
    T, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    _shape(k, "k", (T, Hqk, dk)); _shape(v, "v", (T, Hv, dv))
    _shape(g, "g", (T, Hv)); _shape(beta, "beta", (T, Hv))
    if cu_seqlens is None:
        cu_seqlens = torch.tensor([0, T], dtype=torch.int32, device=q.device)
    _dev(cu_seqlens, "cu_seqlens", torch.int32)
    N = cu_seqlens.numel() - 1
    if state_in is not None:
        _dev(state_in, "state_in", torch.float32)
        _shape(state_in, "state_in", (N, Hv, dv, dk))
    if o is None:
        o = torch.empty(T, Hv, dv, dtype=q.dtype, device=q.device)
    _dev(o, "o", q.dtype); _shape(o, "o", (T, Hv, dv))
    if state_out is None:
        state_out = torch.empty(N, Hv, dv, dk, dtype=torch.float32, device=q.device)
    _dev(state_out, "state_out", torch.float32); _shape(state_out, "state_out", (N, Hv, dv, dk))
    return T, Hqk, dk, Hv, dv, N, cu_seqlens, o, state_out


def _dev(t, name, dtype=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    return t


def _stream_handle(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def prefill_workspace_bytes(n_seqs, Hv, dk, dv, dtype=torch.bfloat16) -> int:
    return int(lib().gdn_prefill_workspace_bytes(n_seqs, Hv, dk, dv, _torch_dtype_code(dtype)))


def prefill_plan(n_seqs, total_T, Hv, dk=128, dv=128, dtype=torch.bfloat16, sm_count=0, requested=None):
    """(dvp, n_chain_ctas, rounds): the launch plan the tensor-core prefill would
    use for this problem, given a `requested` (dvp, n_chain_ctas) plan or None;
    host only. sm_count=0 asks the current device."""
    out = [ctypes.c_int(0) for _ in range(3)]
    _check(lib().gdn_prefill_plan(int(n_seqs), int(total_T), int(Hv), int(dk), int(dv), _torch_dtype_code(dtype),
                                  int(sm_count), _plan_arg(requested), *[ctypes.byref(x) for x in out]))
    return tuple(x.value for x in out)


def prefill(q, k, v, g, beta, state_in=None, cu_seqlens=None, *, scale=None, chunk=0,
            o=None, state_out=None, workspace=None, plan=None, stream=None):
    """Chunked prefill over packed sequences.

    q, k [T, Hqk, dk]; v [T, Hv, dv] (bf16, f16 or fp32, same dtype); g, beta
    [T, Hv] fp32; state_in [N, Hv, dv, dk] fp32 or None; cu_seqlens [N+1] int32
    (None = one sequence of T tokens). `plan` = (dvp, n_chain_ctas) for the
    tensor-core kernel (gdn_prefill_ex; None or 0: the library's choice).
    Returns (o [T, Hv, dv], state_out [N, Hv, dv, dk]).
    """
    T, Hqk, dk, Hv, dv, N, cu_seqlens, o, state_out = _prefill_args(q, k, v, g, beta, state_in, cu_seqlens,
                                                                    o, state_out)
    need = prefill_workspace_bytes(N, Hv, dk, dv, q.dtype)
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().gdn_prefill_ex(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        state_in.data_ptr() if state_in is not None else None, cu_seqlens.data_ptr(),
        N, T, Hqk, Hv, dk, dv, float(scale or 0.0), int(chunk), _dtype_code(q),
        o.data_ptr(), state_out.data_ptr(), ws_ptr, ws_bytes, _plan_arg(plan), _stream_handle(stream)))
    return o, state_out


def prefill_noalloc(q, k, v, g, beta, state_in=None, cu_seqlens=None, *, scale=None, o=None,
                    state_out=None, stream=None):
    """gdn_prefill_noalloc: the prefill with the library's built-in scratch
    instead of a workspace (for callers that cannot allocate device memory).
    Outputs are allocated here only if not given."""
    T, Hqk, dk, Hv, dv, N, cu_seqlens, o, state_out = _prefill_args(q, k, v, g, beta, state_in, cu_seqlens,
                                                                    o, state_out)
    _check(lib().gdn_prefill_noalloc(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
        state_in.data_ptr() if state_in is not None else None, cu_seqlens.data_ptr(),
        N, T, Hqk, Hv, dk, dv, float(scale or 0.0), 0, _dtype_code(q),
        o.data_ptr(), state_out.data_ptr(), _stream_handle(stream)))
    return o, state_out


def decode(q, k, v, g, beta, state, *, scale=None, o=None, stream=None):
    """One decode step: q, k [B, Hqk, dk]; v [B, Hv, dv]; g, beta [B, Hv];
    state [B, Hv, dv, dk] updated in place -- fp32 (gdn_decode) or bf16
    (gdn_decode_bf16_state: fp32 arithmetic, stored rounded to nearest even).
    Returns o [B, Hv, dv]."""
    _dev(q, "q"); _dev(k, "k", q.dtype); _dev(v, "v", q.dtype)
    _dev(g, "g", torch.float32); _dev(beta, "beta", torch.float32)
    _dev(state, "state")
    if state.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"state must be fp32 or bf16, got {state.dtype}")
    B, Hqk, dk = q.shape
    Hv, dv = v.shape[1], v.shape[2]
    if o is None:
        o = torch.empty(B, Hv, dv, dtype=q.dtype, device=q.device)
    fn = lib().gdn_decode if state.dtype == torch.float32 else lib().gdn_decode_bf16_state
    _check(fn(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(),
        B, Hqk, Hv, dk, dv, float(scale or 0.0), _dtype_code(q), o.data_ptr(),
        _stream_handle(stream)))
    return o


def wait_selftest(max_wait_us: int = 2000, stream=None) -> None:
    """Enqueue the bounded-wait self test (gdn_wait_selftest): a following
    device_error() raises GdnError with GDN_ERR_DEVICE_TIMEOUT."""
    _check(lib().gdn_wait_selftest(int(max_wait_us), _stream_handle(stream)))


def device_error(stream=None) -> None:
    """Synchronise and raise GdnError if a bounded device wait ran out."""
    _check(lib().gdn_device_error(_stream_handle(stream)))


# ------------------------------------------------------- linear attention ---
# The checks are written so that a good call costs a few comparisons: a step of one
# token takes the GPU a few microseconds. Where one fails, _explain names the argument.
_fns = {}
_here = contextlib.nullcontext()


def _fn(name):
    f = _fns.get(name)
    if f is None:
        f = _fns[name] = getattr(lib(), name)
    return f


def _fits(t, dtype, shape, device):
    return t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()


def _explain(t, name, dtype, shape, device):
    """Raises for an argument that _fits refuses."""
    _dev(t, name, dtype)
    _shape(t, name, shape)
    raise ValueError(f"{name} must be on {device}, is on {t.device}")


def _running_on(device, stream):
    """A context in which `device` and `stream` (None: the device's current one) are
    current: what a call allocates belongs to the stream that its kernels run on, so
    the memory is not handed out again before they have run."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
        return torch.cuda.stream(stream)
    return _here if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _raw_stream(device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


def _qkv(q, k, v, rows):
    """Checks q, k [rows, Hqk, dk], v [rows, Hv, dv] of one type; (device, dtype code, Hqk, dk, Hv, dv)."""
    if not (isinstance(q, torch.Tensor) and isinstance(v, torch.Tensor) and q.is_cuda and q.is_contiguous()):
        _dev(q, "q"); _dev(v, "v")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q, k must be [{rows}, Hqk, dk] and v [{rows}, Hv, dv]")
    dtype, device = q.dtype, q.device
    n, Hqk, dk = q.shape
    _, Hv, dv = v.shape
    if not (isinstance(k, torch.Tensor) and _fits(k, dtype, q.shape, device)):
        _explain(k, "k", dtype, (n, Hqk, dk), device)
    if not _fits(v, dtype, (n, Hv, dv), device):
        _explain(v, "v", dtype, (n, Hv, dv), device)
    return device, _dtype_code(q), n, Hqk, dk, Hv, dv


def _decay(g, rows, Hv, device):
    """The token stride of log-decays [rows, Hv] or [Hv]."""
    if not isinstance(g, torch.Tensor) or g.dtype != torch.float32 or g.device != device or not g.is_contiguous():
        _dev(g, "g", torch.float32)
        raise ValueError(f"g must be on {device}, is on {g.device}")
    if g.shape == (Hv,):
        return 0
    _shape(g, "g", (rows, Hv))
    return Hv


def linear_prefill_workspace_bytes(n_seqs, total_T, Hv, dk, dv, dtype=torch.bfloat16) -> int:
    """Bytes of workspace that linear_prefill takes for n_seqs packed sequences of total_T tokens."""
    return _fn("gdn_linear_prefill_workspace_bytes")(n_seqs, total_T, Hv, dk, dv, _torch_dtype_code(dtype))


def linear_prefill(q, k, v, g, state_in=None, cu_seqlens=None, *, scale=None, o=None, state_out=None,
                   workspace=None, stream=None):
    """Decayed linear attention over packed sequences: S_t = exp(g_t) S_{t-1} +
    v_t k_t^T, o_t = scale S_t q_t (scale None, zero or negative: dk^-1/2).

    q, k [T, Hqk, dk]; v [T, Hv, dv] (bf16, f16 or fp32, same dtype); g fp32
    [T, Hv], or [Hv] for a decay fixed per value head; state_in [N, Hv, dv, dk]
    fp32 or None; cu_seqlens [N+1] int32 (None = one sequence of T tokens).
    state_out may be state_in. Returns (o [T, Hv, dv], state_out [N, Hv, dv, dk]).
    What the call allocates belongs to the stream it runs on.
    """
    device, code, T, Hqk, dk, Hv, dv = _qkv(q, k, v, "T")
    g_stride = _decay(g, T, Hv, device)
    f32 = torch.float32
    with _running_on(device, stream):
        if cu_seqlens is None:   # filled on the device: no copy from the host, which a graph could not capture
            cu_seqlens = torch.arange(0, T + 1, T, dtype=torch.int32, device=device) if T > 0 else \
                torch.zeros(2, dtype=torch.int32, device=device)
        elif not (isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dim() == 1 and cu_seqlens.numel() > 0
                  and _fits(cu_seqlens, torch.int32, cu_seqlens.shape, device)):
            _dev(cu_seqlens, "cu_seqlens", torch.int32)
            raise ValueError(f"cu_seqlens must have shape (N + 1,) on {device}, got {tuple(cu_seqlens.shape)} on "
                             f"{cu_seqlens.device}")
        N = cu_seqlens.numel() - 1
        if state_in is not None and not (isinstance(state_in, torch.Tensor)
                                         and _fits(state_in, f32, (N, Hv, dv, dk), device)):
            _explain(state_in, "state_in", f32, (N, Hv, dv, dk), device)
        if o is None:
            o = torch.empty(v.shape, dtype=q.dtype, device=device)
        elif not (isinstance(o, torch.Tensor) and _fits(o, q.dtype, v.shape, device)):
            _explain(o, "o", q.dtype, v.shape, device)
        if state_out is None:
            state_out = torch.empty((N, Hv, dv, dk), dtype=f32, device=device)
        elif not (isinstance(state_out, torch.Tensor) and _fits(state_out, f32, (N, Hv, dv, dk), device)):
            _explain(state_out, "state_out", f32, (N, Hv, dv, dk), device)
        if workspace is None:
            need = _fn("gdn_linear_prefill_workspace_bytes")(N, T, Hv, dk, dv, code)
            if need > 0:
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
        elif _dev(workspace, "workspace").device != device:
            raise ValueError(f"workspace must be on {device}, is on {workspace.device}")
        _check(_fn("gdn_linear_prefill")(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), g_stride,
            None if state_in is None else state_in.data_ptr(), cu_seqlens.data_ptr(),
            N, T, Hqk, Hv, dk, dv, scale or 0.0, code, o.data_ptr(), state_out.data_ptr(),
            None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.nbytes,
            _raw_stream(device)))
    return o, state_out


def linear_decode(q, k, v, g, state, *, scale=None, o=None, stream=None):
    """One step of decayed linear attention: q, k [B, Hqk, dk]; v [B, Hv, dv]; g
    [B, Hv] or [Hv]; state [B, Hv, dv, dk] updated in place -- fp32
    (gdn_linear_decode) or bf16 (gdn_linear_decode_bf16_state). Returns o [B, Hv, dv]."""
    device, code, B, Hqk, dk, Hv, dv = _qkv(q, k, v, "B")
    g_stride = _decay(g, B, Hv, device)
    sdt = state.dtype if isinstance(state, torch.Tensor) else None
    if sdt != torch.float32 and sdt != torch.bfloat16:
        raise TypeError(f"state must be an fp32 or bf16 tensor, got {sdt or type(state).__name__}")
    if not _fits(state, sdt, (B, Hv, dv, dk), device):
        _explain(state, "state", sdt, (B, Hv, dv, dk), device)
    with _running_on(device, stream):
        if o is None:
            o = torch.empty(v.shape, dtype=q.dtype, device=device)
        elif not (isinstance(o, torch.Tensor) and _fits(o, q.dtype, v.shape, device)):
            _explain(o, "o", q.dtype, v.shape, device)
        _check(_fn("gdn_linear_decode" if sdt == torch.float32 else "gdn_linear_decode_bf16_state")(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), g_stride, state.data_ptr(),
            B, Hqk, Hv, dk, dv, scale or 0.0, code, o.data_ptr(), _raw_stream(device)))
    return o


# ------------------------------------------------------------- state pool ---
_CODES = {torch.float8_e4m3fn: 0, torch.int8: 1}


def state_pool(n_slots, Hv, dv, dk, *, dtype=torch.float8_e4m3fn, device="cuda"):
    """(codes [n_slots, Hv, dv, dk], exps [n_slots, Hv, dv, dk / min(32, dk)]) of
    zero states: a pool for state_store and state_load, in float8_e4m3fn or int8."""
    if dtype not in _CODES:
        raise TypeError(f"codes must be float8_e4m3fn or int8, got {dtype}")
    if dk not in (16, 32, 64, 128) or dv not in (16, 32, 64, 128):
        raise ValueError(f"dk={dk}, dv={dv} (supported: 16, 32, 64, 128)")
    codes = torch.zeros(n_slots, Hv, dv, dk, dtype=torch.int8, device=device).view(dtype)
    return codes, torch.zeros(n_slots, Hv, dv, dk // min(32, dk), dtype=torch.uint8, device=device)


def _pool_args(codes, exps, slots):
    """Checks a pool and slot numbers; (device, n, n_slots, Hv, dk, dv, code)."""
    code = _CODES.get(codes.dtype) if isinstance(codes, torch.Tensor) else None
    if code is None or not codes.is_cuda or not codes.is_contiguous():
        _dev(codes, "codes")
        raise TypeError(f"codes must be float8_e4m3fn or int8, got {codes.dtype}")
    device = codes.device
    if codes.dim() != 4:
        raise ValueError(f"codes must be [n_slots, Hv, dv, dk], got {tuple(codes.shape)}")
    n_slots, Hv, dv, dk = codes.shape
    want = (n_slots, Hv, dv, dk // min(32, dk) if dk else 0)
    if not (isinstance(exps, torch.Tensor) and _fits(exps, torch.uint8, want, device)):
        _explain(exps, "exps", torch.uint8, want, device)
    if not (isinstance(slots, torch.Tensor) and slots.dim() == 1
            and _fits(slots, torch.int32, slots.shape, device)):
        _dev(slots, "slots", torch.int32)
        raise ValueError(f"slots must have shape (n,) on {device}, got {tuple(slots.shape)} on {slots.device}")
    return device, slots.shape[0], n_slots, Hv, dk, dv, code


def _pool_state(state, shape, device):
    sdt = state.dtype if isinstance(state, torch.Tensor) else None
    if sdt != torch.float32 and sdt != torch.bfloat16:
        raise TypeError(f"state must be an fp32 or bf16 tensor, got {sdt or type(state).__name__}")
    if not _fits(state, sdt, shape, device):
        _explain(state, "state", sdt, shape, device)
    return GDN_F32 if sdt == torch.float32 else GDN_BF16


def state_store(state, codes, exps, slots, *, stream=None) -> None:
    """Quantises state [n, Hv, dv, dk] (fp32 or bf16) into the slots [n] int32 of
    the pool: value = code 2^(exp - 127), one exponent byte for each 32 values
    along dk. A slot outside the pool is passed over; of several states for one
    slot the last is kept."""
    device, n, n_slots, Hv, dk, dv, code = _pool_args(codes, exps, slots)
    sdt = _pool_state(state, (n, Hv, dv, dk), device)
    with _running_on(device, stream):
        _check(_fn("gdn_state_store")(state.data_ptr(), sdt, slots.data_ptr(), n, n_slots, Hv, dk, dv, code,
                                      codes.data_ptr(), exps.data_ptr(), _raw_stream(device)))


def state_load(codes, exps, slots, *, state=None, dtype=torch.float32, stream=None):
    """Reads slots [n] int32 of the pool into state [n, Hv, dv, dk] (fp32 or bf16;
    allocated as `dtype` if not given) and returns it. A slot outside the pool
    gives a zero state."""
    device, n, n_slots, Hv, dk, dv, code = _pool_args(codes, exps, slots)
    with _running_on(device, stream):
        if state is None:
            state = torch.empty((n, Hv, dv, dk), dtype=dtype, device=device)
        sdt = _pool_state(state, (n, Hv, dv, dk), device)
        _check(_fn("gdn_state_load")(codes.data_ptr(), exps.data_ptr(), slots.data_ptr(), n, n_slots, Hv, dk, dv, code,
                                     state.data_ptr(), sdt, _raw_stream(device)))
    return state
