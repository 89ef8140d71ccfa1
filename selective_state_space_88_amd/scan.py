"""Python binding of libssscan.so (argument marshalling only; every step runs in the HIP kernels).

PyTorch supplies device memory and the stream.  Tensors are passed to the C ABI as
(pointer, dtype, shape, strides) descriptors; nothing is computed on the host and there is
no fallback: if the library is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libssscan.so")

SS_F32, SS_BF16, SS_I32 = 0, 1, 2
SS_DELTA_SOFTPLUS = 1 << 0
SS_Z_GATE_SILU = 1 << 1
SS_DETERMINISTIC = 1 << 2   # forward paths are deterministic by construction; the backward rejects it
SS_ZOH = 1 << 3
SS_TRAPEZOID = 1 << 4
SS_CONV_SILU = 1 << 0   # flag of ss_conv1d
SS_ROPE_INTERLEAVED = 1 << 0   # flags of ss_rope
SS_ROPE_INVERSE = 1 << 1
SS_NORM_GATE_FIRST = 1 << 0   # flag of ss_gatenorm_fwd and ss_gatenorm_bwd
SS_ERR_SCRATCH = -10
NOALLOC_SCRATCH_BYTES = 64 << 20   # the static scratch of ss_scan_fwd_noalloc, per device
EXPORTS = ("ss_scan_fwd", "ss_scan_fwd_state", "ss_scan_fwd_noalloc", "ss_scan_step", "ss_scan_bwd",
           "ss_conv1d", "ss_linattn_fwd", "ss_linattn_bwd", "ss_linattn_step", "ss_linattn_workspace", "ss_rope",
           "ss_addnorm_fwd", "ss_addnorm_bwd", "ss_gatenorm_fwd", "ss_gatenorm_bwd", "ss_norm_workspace",
           "ss_check", "ss_strerror", "ss_version")


class SSTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class ScanError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__("selective-scan call failed (%d): %s" % (code, msg))
        self.code = code


_lib = None


def lib() -> ctypes.CDLL:
    """Load libssscan.so (built in-tree by build.py); raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libssscan.so is not built (run selective_state_space_88_amd/build.py)")
        l = ctypes.CDLL(LIB_PATH)
        P = ctypes.POINTER(SSTensor)
        l.ss_scan_fwd.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_uint32, P, ctypes.c_void_p]
        l.ss_scan_fwd.restype = ctypes.c_int
        l.ss_scan_fwd_state.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_uint32, P, P, P, ctypes.c_void_p]
        l.ss_scan_fwd_state.restype = ctypes.c_int
        l.ss_scan_fwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_uint32, P, P, P, ctypes.c_void_p]
        l.ss_scan_fwd_noalloc.restype = ctypes.c_int
        l.ss_scan_step.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_uint32, P, P, ctypes.c_void_p]
        l.ss_scan_step.restype = ctypes.c_int
        l.ss_scan_bwd.argtypes = [P, P, P, P, P, P, P, P, ctypes.c_uint32, P, P, P, P, P, P, P, P, P,
                                  ctypes.c_void_p]
        l.ss_scan_bwd.restype = ctypes.c_int
        l.ss_conv1d.argtypes = [P, P, P, P, P, ctypes.c_uint32, P, ctypes.c_void_p]
        l.ss_conv1d.restype = ctypes.c_int
        F, U, V, I, J = ctypes.c_float, ctypes.c_uint32, ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        T = V   # a descriptor: its address, a byref() of it, or None
        for name, args, res in (
                ("ss_linattn_fwd", [T, T, T, T, F, T, T, T, T, T, V], ctypes.c_int),
                ("ss_linattn_bwd", [T, T, T, T, F, T, T, T, T, T, T, T, T, T, V], ctypes.c_int),
                ("ss_linattn_step", [T, T, T, T, F, T, T, T, V], ctypes.c_int),
                ("ss_linattn_workspace", [J] * 8 + [I, I], J),
                ("ss_rope", [T, T, T, J, T, F, U, T, T, V], ctypes.c_int),
                ("ss_addnorm_fwd", [T, T, T, F, F, T, T, V], ctypes.c_int),
                ("ss_addnorm_bwd", [T, T, T, T, F, F, T, T, T, T, V], ctypes.c_int),
                ("ss_gatenorm_fwd", [T, T, T, I, F, U, T, V], ctypes.c_int),
                ("ss_gatenorm_bwd", [T, T, T, T, I, F, U, T, T, T, T, V], ctypes.c_int),
                ("ss_norm_workspace", [J, J, J, I], J)):
            getattr(l, name).argtypes = args
            getattr(l, name).restype = res
        l.ss_check.argtypes = [ctypes.c_void_p]
        l.ss_check.restype = ctypes.c_int
        l.ss_strerror.argtypes = [ctypes.c_int]
        l.ss_strerror.restype = ctypes.c_char_p
        l.ss_version.argtypes = []
        l.ss_version.restype = ctypes.c_int
        _lib = l
    return _lib


def strerror(code: int) -> str:
    return lib().ss_strerror(code).decode()


def check(stream: Optional[int] = None) -> int:
    """ss_check: synchronise ``stream`` and return SS_OK (0), SS_ERR_HIP (-8) if enqueued work failed,
    or SS_ERR_DEADLOCK (-9) if a kernel's bounded wait between waves ran out since the last check."""
    return lib().ss_check(ctypes.c_void_p(stream or 0))


def version() -> int:
    return lib().ss_version()


def describe(t: Optional[torch.Tensor]) -> Optional[SSTensor]:
    """ss_tensor descriptor of a torch tensor (no copy).  None stays None."""
    if t is None:
        return None
    if t.dtype == torch.float32:
        code = SS_F32
    elif t.dtype == torch.bfloat16:
        code = SS_BF16
    else:
        raise TypeError("unsupported dtype %s (float32 or bfloat16)" % t.dtype)
    if t.dim() < 1 or t.dim() > 4:
        raise ValueError("tensors must have 1 to 4 dimensions")
    d = SSTensor()
    d.data = t.data_ptr() if t.numel() else 0
    d.dtype = code
    d.ndim = t.dim()
    for i, (n, s) in enumerate(zip(t.shape, t.stride())):
        d.shape[i] = n
        d.stride[i] = s
    return d


def _ref(d: Optional[SSTensor]):
    return ctypes.byref(d) if d is not None else None


def call(u, delta, A, B, C, D, z, delta_bias, flags: int, y, stream) -> int:
    """Raw call with descriptors (or None); returns the library's code."""
    return lib().ss_scan_fwd(_ref(u), _ref(delta), _ref(A), _ref(B), _ref(C), _ref(D), _ref(z),
                             _ref(delta_bias), ctypes.c_uint32(flags), _ref(y),
                             ctypes.c_void_p(stream or 0))


def call_state(u, delta, A, B, C, D, z, delta_bias, flags: int, h_init, h_final, y, stream) -> int:
    """Raw ss_scan_fwd_state call with descriptors (or None); returns the library's code."""
    return lib().ss_scan_fwd_state(_ref(u), _ref(delta), _ref(A), _ref(B), _ref(C), _ref(D), _ref(z),
                                   _ref(delta_bias), ctypes.c_uint32(flags), _ref(h_init), _ref(h_final),
                                   _ref(y), ctypes.c_void_p(stream or 0))


def call_noalloc(u, delta, A, B, C, D, z, delta_bias, flags: int, h_init, h_final, y, stream) -> int:
    """Raw ss_scan_fwd_noalloc call with descriptors (or None); returns the library's code."""
    return lib().ss_scan_fwd_noalloc(_ref(u), _ref(delta), _ref(A), _ref(B), _ref(C), _ref(D), _ref(z),
                                     _ref(delta_bias), ctypes.c_uint32(flags), _ref(h_init), _ref(h_final),
                                     _ref(y), ctypes.c_void_p(stream or 0))


def call_step(u, delta, A, B, C, D, z, delta_bias, flags: int, h, y, stream) -> int:
    """Raw ss_scan_step call with descriptors (or None); returns the library's code."""
    return lib().ss_scan_step(_ref(u), _ref(delta), _ref(A), _ref(B), _ref(C), _ref(D), _ref(z),
                              _ref(delta_bias), ctypes.c_uint32(flags), _ref(h), _ref(y),
                              ctypes.c_void_p(stream or 0))


def _check_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be GPU tensors")


def scan_fwd(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
             C: torch.Tensor, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
             delta_bias: Optional[torch.Tensor] = None, *, softplus: bool = True,
             y: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
             stream: Optional[int] = None, h_init: Optional[torch.Tensor] = None,
             h_final: Optional[torch.Tensor] = None, zoh: bool = False,
             trapezoid: bool = False, deterministic: bool = False) -> torch.Tensor:
    """Selective-scan forward on the GPU through ss_scan_fwd (see include/ss_scan.h).

    u, z: [batch, channels, L]; delta: [batch, heads, L]; A: [channels, N] (diagonal) or
    [heads] (scalar decay); B, C: [batch, groups, N, L]; D: [channels] or [heads];
    delta_bias: [heads].  Returns y [batch, channels, L] (float32 unless out_dtype/y say so).
    With h_init and/or h_final ([batch, channels, N] float32) the call goes through
    ss_scan_fwd_state: the scan starts from h_init and writes its final state to h_final.
    ``zoh`` selects the zero-order-hold input coefficient (SS_ZOH), ``trapezoid`` the
    exponential-trapezoidal rule (SS_TRAPEZOID); ``deterministic`` passes SS_DETERMINISTIC (the
    forward is bitwise reproducible either way).
    """
    _check_cuda(u, delta, A, B, C, D, z, delta_bias, h_init, h_final)
    if y is None:
        y = torch.empty(u.shape, dtype=out_dtype, device=u.device)
    flags = (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_Z_GATE_SILU if z is not None else 0) | \
        (SS_ZOH if zoh else 0) | (SS_TRAPEZOID if trapezoid else 0) | (SS_DETERMINISTIC if deterministic else 0)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    args = (describe(u), describe(delta), describe(A), describe(B), describe(C), describe(D),
            describe(z), describe(delta_bias), flags)
    if h_init is None and h_final is None:
        rc = call(*args, describe(y), stream)
    else:
        rc = call_state(*args, describe(h_init), describe(h_final), describe(y), stream)
    if rc != 0:
        raise ScanError(rc, strerror(rc))
    return y


def scan_fwd_noalloc(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                     C: torch.Tensor, y: torch.Tensor, D: Optional[torch.Tensor] = None,
                     z: Optional[torch.Tensor] = None, delta_bias: Optional[torch.Tensor] = None, *,
                     softplus: bool = True, stream: Optional[int] = None,
                     h_init: Optional[torch.Tensor] = None, h_final: Optional[torch.Tensor] = None,
                     zoh: bool = False, trapezoid: bool = False) -> torch.Tensor:
    """scan_fwd through ss_scan_fwd_noalloc: the caller passes y, and the library allocates
    nothing (its scratch -- scalar decay's operands, the states handed between sequence segments --
    is a static 64 MiB array per device; larger calls raise ScanError with code SS_ERR_SCRATCH).  Calls that overlap on one GPU race on that scratch."""
    _check_cuda(u, delta, A, B, C, D, z, delta_bias, h_init, h_final, y)
    flags = (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_Z_GATE_SILU if z is not None else 0) | \
        (SS_ZOH if zoh else 0) | (SS_TRAPEZOID if trapezoid else 0)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    rc = call_noalloc(describe(u), describe(delta), describe(A), describe(B), describe(C), describe(D),
                      describe(z), describe(delta_bias), flags, describe(h_init), describe(h_final),
                      describe(y), stream)
    if rc != 0:
        raise ScanError(rc, strerror(rc))
    return y


def fwd_launcher(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                 C: torch.Tensor, D: Optional[torch.Tensor], z: Optional[torch.Tensor],
                 delta_bias: Optional[torch.Tensor], y: torch.Tensor, *, softplus: bool = True,
                 stream: Optional[int] = None, zoh: bool = False, trapezoid: bool = False):
    """The same ss_scan_fwd call as scan_fwd, with its descriptors built once: returns a
    function of no arguments that launches the scan on these tensors (which it keeps alive) and
    raises ScanError on a failing code.  For loops that repeat one call on the same buffers,
    where per-call argument marshalling would otherwise cost more host time than the kernel."""
    _check_cuda(u, delta, A, B, C, D, z, delta_bias, y)
    flags = (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_Z_GATE_SILU if z is not None else 0) | \
        (SS_ZOH if zoh else 0) | (SS_TRAPEZOID if trapezoid else 0)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    keep = (u, delta, A, B, C, D, z, delta_bias, y)
    descs = [describe(t) for t in keep]
    refs = [_ref(d) for d in descs]
    fn = lib().ss_scan_fwd
    cflags, cstream = ctypes.c_uint32(flags), ctypes.c_void_p(stream or 0)
    args = tuple(refs[:8]) + (cflags, refs[8], cstream)

    def launch() -> None:
        rc = fn(*args)
        if rc != 0:
            raise ScanError(rc, strerror(rc))

    launch.keep = (keep, descs)   # the tensors and descriptors live as long as the launcher
    return launch


def scan_step(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
              C: torch.Tensor, D: Optional[torch.Tensor], z: Optional[torch.Tensor],
              delta_bias: Optional[torch.Tensor], h: torch.Tensor, *, softplus: bool = True,
              y: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
              stream: Optional[int] = None, zoh: bool = False, trapezoid: bool = False,
              deterministic: bool = False) -> torch.Tensor:
    """One decoding step through ss_scan_step: h (float32 [batch, channels, N]) is updated in
    place and y [batch, channels] returned.  u, z: [batch, channels]; delta: [batch, heads];
    B, C: [batch, groups, N]; A, D, delta_bias as in scan_fwd."""
    _check_cuda(u, delta, A, B, C, D, z, delta_bias, h)
    if y is None:
        y = torch.empty(u.shape, dtype=out_dtype, device=u.device)
    flags = (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_Z_GATE_SILU if z is not None else 0) | \
        (SS_ZOH if zoh else 0) | (SS_TRAPEZOID if trapezoid else 0) | (SS_DETERMINISTIC if deterministic else 0)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    rc = call_step(describe(u), describe(delta), describe(A), describe(B), describe(C), describe(D),
                   describe(z), describe(delta_bias), flags, describe(h), describe(y), stream)
    if rc != 0:
        raise ScanError(rc, strerror(rc))
    return y


def call_bwd(u, delta, A, B, C, D, z, delta_bias, flags: int, dy, du, ddelta, dA, dB, dC, dD, dz, ddelta_bias,
             stream) -> int:
    """Raw ss_scan_bwd call with descriptors (or None); returns the library's code."""
    return lib().ss_scan_bwd(_ref(u), _ref(delta), _ref(A), _ref(B), _ref(C), _ref(D), _ref(z), _ref(delta_bias),
                             ctypes.c_uint32(flags), _ref(dy), _ref(du), _ref(ddelta), _ref(dA), _ref(dB), _ref(dC),
                             _ref(dD), _ref(dz), _ref(ddelta_bias), ctypes.c_void_p(stream or 0))


def scan_bwd(u: torch.Tensor, delta: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
             D: Optional[torch.Tensor], z: Optional[torch.Tensor], delta_bias: Optional[torch.Tensor],
             dy: torch.Tensor, *, softplus: bool = True, stream: Optional[int] = None,
             deterministic: bool = False) -> dict:
    """Gradients of sum(dy * y) through ss_scan_bwd.  Returns a dict of float32 tensors du, ddelta,
    dA, dB, dC and, when the input is given, dD, dz, ddelta_bias.  ``deterministic`` passes
    SS_DETERMINISTIC, which the backward rejects (its summed gradients use atomic adds)."""
    _check_cuda(u, delta, A, B, C, D, z, delta_bias, dy)
    f = lambda t: torch.empty(t.shape, dtype=torch.float32, device=u.device)
    g = dict(du=f(u), ddelta=f(delta), dA=f(A), dB=f(B), dC=f(C), dD=None if D is None else f(D),
             dz=None if z is None else f(z), ddelta_bias=None if delta_bias is None else f(delta_bias))
    flags = (SS_DELTA_SOFTPLUS if softplus else 0) | (SS_Z_GATE_SILU if z is not None else 0) | \
        (SS_DETERMINISTIC if deterministic else 0)
    if stream is None:
        stream = torch.cuda.current_stream(u.device).cuda_stream
    rc = call_bwd(describe(u), describe(delta), describe(A), describe(B), describe(C), describe(D), describe(z),
                  describe(delta_bias), flags, describe(dy), *(describe(g[k]) for k in
                  ("du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias")), stream)
    if rc != 0:
        raise ScanError(rc, strerror(rc))
    return g


def call_conv(x, weight, bias, state_in, state_out, flags: int, out, stream) -> int:
    """Raw ss_conv1d call with descriptors (or None); returns the library's code."""
    return lib().ss_conv1d(_ref(x), _ref(weight), _ref(bias), _ref(state_in), _ref(state_out),
                           ctypes.c_uint32(flags), _ref(out), ctypes.c_void_p(stream or 0))


def conv1d(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None, *,
           state_in: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
           silu: bool = False, out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.float32,
           stream: Optional[int] = None) -> torch.Tensor:
    """Causal depthwise convolution through ss_conv1d: x [batch, channels, L], weight [channels, W]
    (float32, W <= 8), bias [channels]; state_in / state_out [batch, channels, W - 1] float32 hold
    the inputs before the sequence / receive its last W - 1 inputs.  Returns out [batch, channels, L]
    (silu applied when ``silu``)."""
    _check_cuda(x, weight, bias, state_in, state_out)
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=x.device)
    if stream is None:
        stream = torch.cuda.current_stream(x.device).cuda_stream
    rc = call_conv(describe(x), describe(weight), describe(bias), describe(state_in), describe(state_out),
                   SS_CONV_SILU if silu else 0, describe(out), stream)
    if rc != 0:
        raise ScanError(rc, strerror(rc))
    return out


# ---- linear attention, rotary positions, norms: token-major tensors [batch, L, ...] ----------

_CODES = {torch.float32: SS_F32, torch.bfloat16: SS_BF16, torch.int32: SS_I32}
# an SSTensor in one packing step, by the number of dimensions (unused entries zero)
_PACK = {n: struct.Struct("=Qii%dq%dx%dq%dx" % (n, 8 * (4 - n), n, 8 * (4 - n))).pack_into for n in range(1, 5)}
_SIZE = ctypes.sizeof(SSTensor)
# the current stream of a device as a number, without a Stream object where torch has that
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _gpu(t: torch.Tensor) -> int:
    """Index of the GPU that the call runs on: that of its first tensor."""
    index = t.get_device()
    if index < 0:
        raise ValueError("all tensors must be GPU tensors")
    return index


class _Scratch(threading.local):
    """A thread's place for the descriptors of one call: the library reads them before it returns."""

    def __init__(self):
        self.buf = ctypes.create_string_buffer(_SIZE * 16)
        self.at = ctypes.addressof(self.buf)


_scratch = _Scratch()


def _call(fn, index: int, stream: Optional[int], *args) -> None:
    """Call the library's ``fn`` on GPU ``index`` and its current stream (or ``stream``) with ``args`` in
    its order: tensors become descriptors, None and numbers go as they are."""
    buf, at, place = _scratch.buf, _scratch.at, 0
    c = []
    for t in args:
        if not isinstance(t, torch.Tensor):
            c.append(t)
            continue
        code, shape = _CODES.get(t.dtype), t.shape
        n = len(shape)
        if code is None:
            raise TypeError("unsupported dtype %s (float32, bfloat16, or int32 positions and lengths)" % t.dtype)
        if n not in _PACK:
            raise ValueError("tensors must have 1 to 4 dimensions")
        if t.get_device() != index:
            raise ValueError("all tensors must be on one GPU")
        _PACK[n](buf, place, t.data_ptr(), code, n, *shape, *t.stride())
        c.append(at + place)
        place += _SIZE
    c.append(_raw_stream(index) if stream is None else stream)
    before = torch.cuda.current_device()
    if before == index:
        rc = fn(*c)
    else:
        torch.cuda.set_device(index)
        try:
            rc = fn(*c)
        finally:
            torch.cuda.set_device(before)
    if rc != 0:
        raise ScanError(rc, strerror(rc))


def _workspace(index: int, stream: Optional[int], floats: int) -> Optional[torch.Tensor]:
    """Scratch from torch's allocator, which orders its reuse on torch's current stream and gives a
    captured graph memory of its own; on a stream passed by number the library's pool is used."""
    if floats < 0:
        raise ScanError(floats, strerror(floats))
    if floats == 0 or stream is not None:
        return None
    return torch.empty(floats, dtype=torch.float32, device=index)


def _on(index: int, floats, *args) -> int:
    """floats(*args) with GPU ``index`` current (a workspace's size goes by the device)."""
    before = torch.cuda.current_device()
    if before == index:
        return floats(*args)
    with torch.cuda.device(index):
        return floats(*args)


def linattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, *,
                scale: Optional[float] = None, lengths: Optional[torch.Tensor] = None,
                s_init: Optional[torch.Tensor] = None, s_final: Optional[torch.Tensor] = None,
                o: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> torch.Tensor:
    """Linear attention with a decay per head through ss_linattn_fwd: q [batch, L, heads_q, K], k
    [batch, L, heads_k, K], v [batch, L, heads_v, V], log_decay [heads] float32; each heads_x divides
    heads.  ``scale`` defaults to K ** -0.5.  ``lengths`` [batch] int32 for padded rows; ``s_init`` and
    ``s_final`` [batch, heads, K, V] float32 carry the state in and out.  Returns o [batch, L, heads, V]."""
    gpu = _gpu(q)
    ws = _workspace(gpu, stream, _on(gpu, _linattn_floats, q, k, v, log_decay.shape[0], 0))
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], log_decay.shape[0], v.shape[-1], dtype=q.dtype, device=gpu)
    _call((_lib or lib()).ss_linattn_fwd, gpu, stream, q, k, v, log_decay, _scale(scale, q), lengths,
          s_init, s_final, o, ws)
    return o


def _scale(scale: Optional[float], q: torch.Tensor) -> float:
    return float(q.shape[-1]) ** -0.5 if scale is None else scale


def _linattn_floats(q, k, v, H: int, backward: int) -> int:
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [batch, L, heads, dim]")
    return lib().ss_linattn_workspace(q.shape[0], q.shape[1], H, q.shape[2], k.shape[2], v.shape[2], q.shape[3],
                                      v.shape[3], _CODES.get(q.dtype, -1), backward)


def linattn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, do: torch.Tensor, *,
                scale: Optional[float] = None, lengths: Optional[torch.Tensor] = None,
                s_init: Optional[torch.Tensor] = None, ds_final: Optional[torch.Tensor] = None,
                dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                dv: Optional[torch.Tensor] = None, ds_init: Optional[torch.Tensor] = None,
                stream: Optional[int] = None) -> dict:
    """Gradients of sum(do * o) + sum(ds_final * s_final) of linattn_fwd through ss_linattn_bwd.
    Returns a dict with dq, dk, dv (shapes and dtype of q, k, v; the given tensors where they are
    passed) and, when ``s_init`` or ``ds_init`` is given, ds_init [batch, heads, K, V] float32."""
    gpu = _gpu(q)
    ws = _workspace(gpu, stream, _on(gpu, _linattn_floats, q, k, v, log_decay.shape[0], 1))
    dq = torch.empty(q.shape, dtype=q.dtype, device=gpu) if dq is None else dq
    dk = torch.empty(k.shape, dtype=k.dtype, device=gpu) if dk is None else dk
    dv = torch.empty(v.shape, dtype=v.dtype, device=gpu) if dv is None else dv
    if ds_init is None and s_init is not None:
        ds_init = torch.empty(s_init.shape, dtype=torch.float32, device=gpu)
    _call((_lib or lib()).ss_linattn_bwd, gpu, stream, q, k, v, log_decay, _scale(scale, q), lengths,
          s_init, do, ds_final, dq, dk, dv, ds_init, ws)
    return dict(dq=dq, dk=dk, dv=dv, ds_init=ds_init)


def linattn_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, s: torch.Tensor, *,
                 scale: Optional[float] = None, s_out: Optional[torch.Tensor] = None,
                 o: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                 stream: Optional[int] = None) -> torch.Tensor:
    """One token through ss_linattn_step: q [batch, heads_q, K], k [batch, heads_k, K], v [batch, heads_v, V];
    the state s [batch, heads, K, V] float32 is updated in place, or written to ``s_out``.  Returns o
    [batch, heads, V] (the dtype of q unless out_dtype/o say so)."""
    gpu = _gpu(q)
    if o is None:
        o = torch.empty(q.shape[0], log_decay.shape[0], v.shape[-1], dtype=out_dtype or q.dtype, device=gpu)
    _call((_lib or lib()).ss_linattn_step, gpu, stream, q, k, v, log_decay, _scale(scale, q), s,
          s if s_out is None else s_out, o)
    return o


def rope_inv_freq(n: int, base: float = 10000.0, *, scaling: Optional[str] = None, factor: float = 1.0,
                  trained: int = 8192, beta_fast: float = 32.0, beta_slow: float = 1.0,
                  device=None) -> tuple:
    """(inv_freq [n] float32, amp) of ``rope`` for n pairs: inv_freq[i] = base ** (-i / n), computed in 64
    bits.  ``scaling`` stretches contexts of ``trained`` positions by ``factor``:
    None: as it is; "linear": every frequency divided by factor; "base": the base raised so that the
    slowest pair is slowed by factor and the fastest keeps its speed; "parts": pairs that turn more than
    beta_fast times over the trained context are kept, those that turn less than beta_slow times are
    divided by factor, a linear ramp over the pair index in between, and amp = 1 + 0.1 ln factor."""
    if n < 0 or base <= 1 or factor < 1:
        raise ValueError("n >= 0, base > 1 and factor >= 1 are required")
    i = torch.arange(n, dtype=torch.float64)
    amp = 1.0
    if scaling == "base" and n > 1:
        base = base * factor ** (n / (n - 1))
    freq = base ** (-i / max(n, 1))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        # the (fractional) index of the pair that turns `turns` times over the trained context
        at = lambda turns: n * math.log(trained / (2 * math.pi * turns)) / math.log(base)
        low, high = max(math.floor(at(beta_fast)), 0), min(math.ceil(at(beta_slow)), max(n - 1, 0))
        kept = 1.0 - ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        freq = freq / factor * (1 - kept) + freq * kept
        amp = 1.0 + 0.1 * math.log(factor)
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    return freq.float().to(device) if device is not None else freq.float(), amp


def rope(x: torch.Tensor, inv_freq: torch.Tensor, *, x2: Optional[torch.Tensor] = None,
         pos: Optional[torch.Tensor] = None, pos0: int = 0, amp: float = 1.0, interleaved: bool = False,
         inverse: bool = False, out: Optional[torch.Tensor] = None, out2: Optional[torch.Tensor] = None,
         stream: Optional[int] = None):
    """Rotary positions through ss_rope: x [batch, L, heads, dim] and optionally x2 [batch, L, heads2, dim]
    in one launch.  ``pos`` [batch, L] int32, or positions pos0, pos0 + 1, ...; ``inv_freq`` [n] float32
    rotates the first 2 n features, as pairs (i, i + n) or, ``interleaved``, (2 i, 2 i + 1), and ``amp``
    scales them.  ``inverse`` rotates back: the backward of the same call.  ``out=x`` (``out2=x2``) works
    in place.  Returns out, or (out, out2) when x2 is given."""
    gpu = _gpu(x)
    out = torch.empty(x.shape, dtype=x.dtype, device=gpu) if out is None else out
    if x2 is not None and out2 is None:
        out2 = torch.empty(x2.shape, dtype=x2.dtype, device=gpu)
    flags = (SS_ROPE_INTERLEAVED if interleaved else 0) | (SS_ROPE_INVERSE if inverse else 0)
    _call((_lib or lib()).ss_rope, gpu, stream, x, x2, pos, pos0, inv_freq, amp, flags, out, out2)
    return out if x2 is None else (out, out2)


def addnorm_fwd(x: torch.Tensor, weight: torch.Tensor, *, residual: Optional[torch.Tensor] = None,
                alpha: float = 1.0, eps: float = 1e-5, sum: Optional[torch.Tensor] = None,
                sum_dtype: Optional[torch.dtype] = None, y: Optional[torch.Tensor] = None,
                out_dtype: Optional[torch.dtype] = None, stream: Optional[int] = None) -> tuple:
    """The norm before a block through ss_addnorm_fwd: returns (y, sum), sum = residual + alpha x in the
    residual's dtype (``sum_dtype`` or x's without a residual) and y = sum / rms(sum) * weight in x's
    dtype (unless out_dtype/y say so).  x, residual: [batch, L, channels]; weight [channels] float32.
    ``sum=residual`` updates the residual stream in place."""
    gpu = _gpu(x)
    if sum is None:
        dt = residual.dtype if residual is not None else (sum_dtype or x.dtype)
        sum = torch.empty(x.shape, dtype=dt, device=gpu)
    if y is None:
        y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=gpu)
    _call((_lib or lib()).ss_addnorm_fwd, gpu, stream, x, residual, weight, alpha, eps, sum, y)
    return y, sum


def _norm_floats(x: torch.Tensor, groups: int) -> int:
    if x.dim() != 3:
        raise ValueError("norm tensors must be [batch, L, channels]")
    return lib().ss_norm_workspace(x.shape[0], x.shape[1], x.shape[2], groups)


def addnorm_bwd(dy: torch.Tensor, sum: torch.Tensor, weight: torch.Tensor, *, dsum: Optional[torch.Tensor] = None,
                alpha: float = 1.0, eps: float = 1e-5, dresidual: Optional[torch.Tensor] = None,
                dx: Optional[torch.Tensor] = None, x_dtype: Optional[torch.dtype] = None,
                dweight: Optional[torch.Tensor] = None, stream: Optional[int] = None) -> dict:
    """Gradients of addnorm_fwd through ss_addnorm_bwd, from its ``sum``; ``dsum`` is the gradient that
    reaches the sum by its later uses.  Returns a dict: dresidual (sum's dtype), dx = alpha dresidual
    (``x_dtype``, else dy's), dweight (float32)."""
    gpu = _gpu(dy)
    dresidual = torch.empty(sum.shape, dtype=sum.dtype, device=gpu) if dresidual is None else dresidual
    dx = torch.empty(sum.shape, dtype=x_dtype or dy.dtype, device=gpu) if dx is None else dx
    dweight = torch.empty(weight.shape, dtype=torch.float32, device=gpu) if dweight is None else dweight
    ws = _workspace(gpu, stream, _on(gpu, _norm_floats, sum, 1))
    _call((_lib or lib()).ss_addnorm_bwd, gpu, stream, dy, dsum, sum, weight, alpha, eps, dresidual, dx, dweight, ws)
    return dict(dresidual=dresidual, dx=dx, dweight=dweight)


def gatenorm_fwd(x: torch.Tensor, weight: torch.Tensor, *, z: Optional[torch.Tensor] = None, groups: int = 1,
                 gate_first: bool = False, eps: float = 1e-5, y: Optional[torch.Tensor] = None,
                 out_dtype: Optional[torch.dtype] = None, stream: Optional[int] = None) -> torch.Tensor:
    """The norm after a block's inner product, with its gate, through ss_gatenorm_fwd: x, z [batch, L,
    channels] (a transposed view of the scan's [batch, channels, L] output is taken as it is), weight
    [channels] float32, the norm over each of ``groups`` equal groups of channels; norm(x) weight silu(z),
    or norm(x silu(z)) weight with ``gate_first``.  Returns y, [batch, L, channels] contiguous unless y is
    given (x's dtype unless out_dtype/y say so)."""
    gpu = _gpu(x)
    y = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=gpu) if y is None else y
    _call((_lib or lib()).ss_gatenorm_fwd, gpu, stream, x, z, weight, groups, eps,
          SS_NORM_GATE_FIRST if gate_first else 0, y)
    return y


def gatenorm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor, *, z: Optional[torch.Tensor] = None,
                 groups: int = 1, gate_first: bool = False, eps: float = 1e-5, dx: Optional[torch.Tensor] = None,
                 dz: Optional[torch.Tensor] = None, dweight: Optional[torch.Tensor] = None,
                 stream: Optional[int] = None) -> dict:
    """Gradients of gatenorm_fwd through ss_gatenorm_bwd.  Returns a dict: dx and dz (the dtype and, unless
    they are given, the layout of x and z; dz None without z), dweight (float32)."""
    gpu = _gpu(dy)
    dx = torch.empty_like(x) if dx is None else dx
    dz = torch.empty_like(z) if dz is None and z is not None else dz
    dweight = torch.empty(weight.shape, dtype=torch.float32, device=gpu) if dweight is None else dweight
    ws = _workspace(gpu, stream, _on(gpu, _norm_floats, x, groups))
    _call((_lib or lib()).ss_gatenorm_bwd, gpu, stream, dy, x, z, weight, groups, eps,
          SS_NORM_GATE_FIRST if gate_first else 0, dx, dz, dweight, ws)
    return dict(dx=dx, dz=dz, dweight=dweight)
