"""ctypes binding of libssm.so (include/ssm.h): argument marshalling only.

Every step of the computation runs in the CUDA kernels behind the C ABI.  There is no
fallback: if the library is missing or was built for another architecture the calls
raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libssm.so")

SSM_F32, SSM_BF16 = 0, 1
SSM_OK, SSM_ERR_INVALID_ARG, SSM_ERR_UNSUPPORTED, SSM_ERR_ALIGNMENT, SSM_ERR_CUDA, SSM_ERR_SCRATCH = range(6)

_DTYPE_CODE = {torch.float32: SSM_F32, torch.bfloat16: SSM_BF16}

_lib = None
_lock = threading.Lock()


class SsmError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("%s (status %d)" % (msg, status))
        self.status = status


def load_library(path: str | None = None):
    """Load libssm.so once (raises if it is absent: build it with
    ``python -m selective_state_space_45_b200.build``)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libssm.so not found at %s; build it first "
                               "(python -m selective_state_space_45_b200.build)" % p)
        lib = ctypes.CDLL(p)
        vp, i = ctypes.c_void_p, ctypes.c_int
        lib.ssm_selective_scan_fwd.restype = i
        lib.ssm_selective_scan_fwd.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp,
                                               i, i, i, i, i, i, vp]
        lib.ssm_selective_scan_fwd_ex.restype = i
        lib.ssm_selective_scan_fwd_ex.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, vp, i,
                                                  i, i, i, i, i, i, vp]
        lib.ssm_selective_scan_fwd_noalloc.restype = i
        lib.ssm_selective_scan_fwd_noalloc.argtypes = list(lib.ssm_selective_scan_fwd.argtypes)
        lib.ssm_state_step.restype = i
        lib.ssm_state_step.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, vp]
        lib.ssm_causal_conv1d_fwd.restype = i
        lib.ssm_causal_conv1d_fwd.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
        lib.ssm_causal_conv1d_step.restype = i
        lib.ssm_causal_conv1d_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.ssm_ssd_fwd.restype = i
        lib.ssm_ssd_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, vp]
        lib.ssm_state_step_multi.restype = i
        lib.ssm_state_step_multi.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, vp]
        lib.ssm_selective_scan_bwd.restype = i
        lib.ssm_selective_scan_bwd.argtypes = [vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, vp,
                                               vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                               i, i, i, i, i, i, vp]
        fl, sz = ctypes.c_float, ctypes.c_size_t
        lib.ssm_delta_rule_fwd.restype = i
        lib.ssm_delta_rule_fwd.argtypes = [vp] * 8 + [fl] + [i] * 8 + [vp, sz, vp]
        lib.ssm_delta_rule_step.restype = i
        lib.ssm_delta_rule_step.argtypes = [vp] * 7 + [fl] + [i] * 8 + [vp]
        lib.ssm_delta_rule_bwd.restype = i
        lib.ssm_delta_rule_bwd.argtypes = [vp] * 14 + [fl] + [i] * 8 + [vp, sz, vp]
        lib.ssm_layer_norm_fwd.restype = i
        lib.ssm_layer_norm_fwd.argtypes = [vp] * 6 + [fl] + [i] * 4 + [vp]
        lib.ssm_layer_norm_bwd.restype = i
        lib.ssm_layer_norm_bwd.argtypes = [vp] * 8 + [i] * 4 + [vp, sz, vp]
        for name, n in (("ssm_delta_rule_fwd", 8), ("ssm_delta_rule_bwd", 8), ("ssm_layer_norm_bwd", 2)):
            getattr(lib, name + "_workspace").restype = sz
            getattr(lib, name + "_workspace").argtypes = [i] * n
        lib.ssm_status_string.restype = ctypes.c_char_p
        lib.ssm_status_string.argtypes = [i]
        lib.ssm_version.restype = i
        lib.ssm_version.argtypes = []
        lib.ssm_device_timeouts.restype = ctypes.c_uint
        lib.ssm_device_timeouts.argtypes = []
        lib.ssm_scan_force_segments.restype = i
        lib.ssm_scan_force_segments.argtypes = [i]
        lib.ssm_sfu_probe.restype = i
        lib.ssm_sfu_probe.argtypes = [vp, i, i, vp]
        _lib = lib
        return lib


def ssm_status_string(status: int) -> str:
    return load_library().ssm_status_string(int(status)).decode()


def ssm_version() -> int:
    return int(load_library().ssm_version())


def ssm_device_timeouts() -> int:
    """How many bounded waits inside the library's kernels gave up on this device (0 in
    normal operation; see include/ssm.h).  Synchronises with the device."""
    return int(load_library().ssm_device_timeouts())


def ssm_sfu_probe(out, blocks, iters, stream=None):
    """Diagnostic SFU throughput probe (see include/ssm.h): ``blocks`` CTAs of 256 threads,
    8 ex2 chains of ``iters`` steps per thread; ``out`` is a CUDA fp32 tensor of at least
    blocks * 256 elements.  Asynchronous on ``stream``."""
    if out.dtype.itemsize != 4 or out.numel() < int(blocks) * 256:
        raise ValueError("out must hold blocks * 256 fp32 values")
    _check(load_library().ssm_sfu_probe(_ptr(out), int(blocks), int(iters), _stream(stream, out)))


def ssm_scan_force_segments(segments: int) -> int:
    """Testing and tuning: force the time-segment count of the following scans (0 restores
    the automatic plan).  Returns the previous setting (see include/ssm.h)."""
    prev = int(load_library().ssm_scan_force_segments(int(segments)))
    if prev < 0:
        raise ValueError("segments must be >= 0")
    return prev


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors passed to libssm must be contiguous")
    return t.data_ptr()


def _stream(stream, *tensors):
    if stream is None:
        dev = next((t.device for t in tensors if isinstance(t, torch.Tensor) and t.is_cuda), None)
        if dev is None:
            return None
        return torch.cuda.current_stream(dev).cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _fits(what, *sizes):
    """Raise ValueError for a size that the library's int does not hold: ctypes would cut it down
    to 32 bits without a word."""
    if max(sizes) >= 2 ** 31:
        raise ValueError("%s: at most 2^31 - 1, got %d" % (what, max(sizes)))


def _current(stream, like):
    """The context that makes ``stream`` (of torch, or a handle) current on ``like``'s device.  A
    call that is given a stream runs whole in it: torch's allocator hands a block out again to
    the stream that it was taken on, so outputs and scratch have to be of the stream whose
    kernels write them."""
    if not like.is_cuda:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        # (an external stream of handle 0 would be some stream of torch's pool)
        stream = (torch.cuda.ExternalStream(raw, device=like.device) if raw else torch.cuda.default_stream(like.device))
    if stream.device != like.device:
        raise ValueError("a stream of %s for tensors on %s" % (stream.device, like.device))
    return torch.cuda.stream(stream)


def _check(status):
    if status != SSM_OK:
        raise SsmError(status, ssm_status_string(status))


def ssm_selective_scan_fwd(x, delta, delta_bias, delta_softplus, A, B, C, D, z, y, final_state,
                           stream=None):
    """Selective scan forward (see include/ssm.h).  Tensors are CUDA tensors in the
    layouts of the header: x, delta, z, y [batch, dim, L]; B, C [batch, L, N]; A [dim, N];
    D, delta_bias [dim]; final_state [batch, dim, N].  Writes y and final_state in place."""
    batch, dim, L = x.shape
    N = A.shape[1]
    _fits("sizes", batch, dim, L)
    _check(load_library().ssm_selective_scan_fwd(
        _ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(A), _ptr(B),
        _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(final_state), batch, dim, L, N,
        _DTYPE_CODE[x.dtype], _DTYPE_CODE[y.dtype], _stream(stream, x, y)))


def ssm_selective_scan_fwd_ex(x, delta, delta_bias, delta_softplus, A, B, C, D, z, y, final_state,
                              initial_state=None, zoh_exact=False, stream=None):
    """``ssm_selective_scan_fwd`` with a start state and the exact zero-order-hold gain
    (see include/ssm.h); initial_state is [batch, dim, N] fp32 or None."""
    batch, dim, L = x.shape
    N = A.shape[1]
    _fits("sizes", batch, dim, L)
    _check(load_library().ssm_selective_scan_fwd_ex(
        _ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(A), _ptr(B),
        _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(final_state), _ptr(initial_state),
        int(bool(zoh_exact)), batch, dim, L, N, _DTYPE_CODE[x.dtype], _DTYPE_CODE[y.dtype],
        _stream(stream, x, y)))


def ssm_selective_scan_fwd_noalloc(x, delta, delta_bias, delta_softplus, A, B, C, D, z, y,
                                   final_state, stream=None):
    """Allocation-free variant of ``ssm_selective_scan_fwd`` (see include/ssm.h): same
    arguments and results; long sequences use a fixed device array for their scratch."""
    batch, dim, L = x.shape
    N = A.shape[1]
    _fits("sizes", batch, dim, L)
    _check(load_library().ssm_selective_scan_fwd_noalloc(
        _ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(A), _ptr(B),
        _ptr(C), _ptr(D), _ptr(z), _ptr(y), _ptr(final_state), batch, dim, L, N,
        _DTYPE_CODE[x.dtype], _DTYPE_CODE[y.dtype], _stream(stream, x, y)))


def ssm_state_step(state, x, delta, A, B, C, D, z, y, stream=None):
    """One decode step (see include/ssm.h): state [batch, dim, N] fp32 updated in place;
    x, delta, z, y [batch, dim]; B, C [batch, N]."""
    batch, dim, N = state.shape
    _fits("sizes", batch, dim, N)
    _check(load_library().ssm_state_step(
        _ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y),
        batch, dim, N, _DTYPE_CODE[x.dtype], _DTYPE_CODE[y.dtype], _stream(stream, state, y)))


def ssm_ssd_fwd(x, a, B, C, y, initial_state=None, final_state=None, stream=None):
    """Mamba-2 SSD by chunks (see include/ssm.h): x, y [batch, L, heads, P]; a [batch, L,
    heads] fp32; B, C [batch, L, heads, N] bf16; states [batch, heads, P, N] fp32."""
    batch, L, heads, P = x.shape
    N = B.shape[-1]
    _fits("sizes", batch, L, heads, P)
    _check(load_library().ssm_ssd_fwd(
        _ptr(x), _ptr(a), _ptr(B), _ptr(C), _ptr(y), _ptr(initial_state), _ptr(final_state),
        batch, L, heads, P, N, _DTYPE_CODE[x.dtype], _DTYPE_CODE[y.dtype], _stream(stream, x, y)))


def ssd(x, a, B, C, initial_state=None, out_dtype=None, return_final_state=True, stream=None):
    """Allocate y (and the final state) with torch and run ``ssm_ssd_fwd``."""
    if stream is not None:
        with _current(stream, x):
            return ssd(x, a, B, C, initial_state, out_dtype, return_final_state)
    batch, L, heads, P = x.shape
    y = torch.empty(x.shape, device=x.device, dtype=out_dtype or torch.float32)
    fs = (torch.empty((batch, heads, P, B.shape[-1]), device=x.device, dtype=torch.float32)
          if return_final_state else None)
    ssm_ssd_fwd(x, a, B, C, y, initial_state, fs, stream)
    return (y, fs) if return_final_state else y


def ssm_state_step_multi(state, x, delta, A, B, C, D, z, y, stream=None):
    """Several decode tokens on the carried state (see include/ssm.h): state [batch, dim, N]
    fp32 updated in place; x, delta, z, y [ntok, batch, dim]; B, C [ntok, batch, N]."""
    batch, dim, N = state.shape
    ntok = x.shape[0]
    _fits("sizes", batch, dim, N, ntok)
    _check(load_library().ssm_state_step_multi(
        _ptr(state), _ptr(x), _ptr(delta), _ptr(A), _ptr(B), _ptr(C), _ptr(D), _ptr(z), _ptr(y),
        ntok, batch, dim, N, _DTYPE_CODE[x.dtype], _DTYPE_CODE[y.dtype], _stream(stream, state, y)))


def ssm_selective_scan_bwd(x, delta, delta_bias, delta_softplus, A, B, C, D, z, initial_state,
                           dy, dfinal_state, dx, ddelta, dA, dB, dC, dD, dz, ddelta_bias,
                           dinitial_state, stream=None):
    """Backward of the scan (see include/ssm.h).  Gradient tensors share dy's dtype
    (dx, ddelta, dz, dB, dC); dA, dD, ddelta_bias, dinitial_state are fp32.  Optional
    arguments are None.  Writes the gradients in place."""
    batch, dim, L = x.shape
    N = A.shape[1]
    _fits("sizes", batch, dim, L)
    _check(load_library().ssm_selective_scan_bwd(
        _ptr(x), _ptr(delta), _ptr(delta_bias), int(bool(delta_softplus)), _ptr(A), _ptr(B),
        _ptr(C), _ptr(D), _ptr(z), _ptr(initial_state), _ptr(dy), _ptr(dfinal_state),
        _ptr(dx), _ptr(ddelta), _ptr(dA), _ptr(dB), _ptr(dC), _ptr(dD), _ptr(dz),
        _ptr(ddelta_bias), _ptr(dinitial_state), batch, dim, L, N,
        _DTYPE_CODE[x.dtype], _DTYPE_CODE[dy.dtype], _stream(stream, x, dy)))


def selective_scan_bwd(dy, x, delta, A, B, C, D=None, z=None, delta_bias=None,
                       delta_softplus=False, initial_state=None, dfinal_state=None, stream=None):
    """Allocate the gradients with torch (dy's dtype for the tensor gradients) and run the
    backward; returns a dict dx, ddelta, dz, dA, dB, dC, dD, ddelta_bias, dinitial_state
    (None where the input was absent)."""
    if stream is not None:
        with _current(stream, x):
            return selective_scan_bwd(dy, x, delta, A, B, C, D, z, delta_bias, delta_softplus, initial_state, dfinal_state)
    batch, dim, L = x.shape
    N = A.shape[1]
    dev, gd, f32 = x.device, dy.dtype, torch.float32
    g = dict(dx=torch.empty((batch, dim, L), device=dev, dtype=gd),
             ddelta=torch.empty((batch, dim, L), device=dev, dtype=gd),
             dz=None if z is None else torch.empty((batch, dim, L), device=dev, dtype=gd),
             dA=torch.empty((dim, N), device=dev, dtype=f32),
             dB=torch.empty((batch, L, N), device=dev, dtype=gd),
             dC=torch.empty((batch, L, N), device=dev, dtype=gd),
             dD=None if D is None else torch.empty(dim, device=dev, dtype=f32),
             ddelta_bias=None if delta_bias is None else torch.empty(dim, device=dev, dtype=f32),
             dinitial_state=None if initial_state is None else
             torch.empty((batch, dim, N), device=dev, dtype=f32))
    ssm_selective_scan_bwd(x, delta, delta_bias, delta_softplus, A, B, C, D, z, initial_state,
                           dy, dfinal_state, g["dx"], g["ddelta"], g["dA"], g["dB"], g["dC"],
                           g["dD"], g["dz"], g["ddelta_bias"], g["dinitial_state"], stream)
    return g


def ssm_causal_conv1d_fwd(x, weight, bias, initial_window, u, final_window, silu=True,
                          stream=None):
    """Causal depthwise convolution + bias + SiLU (see include/ssm.h): x, u [batch, dim, L];
    weight [dim, width] fp32; bias [dim] fp32 or None; initial_window / final_window
    [batch, dim, width-1] fp32 or None.  Writes u (and final_window) in place."""
    batch, dim, L = x.shape
    width = weight.shape[1]
    _fits("sizes", batch, dim, L)
    _check(load_library().ssm_causal_conv1d_fwd(
        _ptr(x), _ptr(weight), _ptr(bias), _ptr(initial_window), _ptr(u), _ptr(final_window),
        batch, dim, L, width, int(bool(silu)), _DTYPE_CODE[x.dtype], _DTYPE_CODE[u.dtype],
        _stream(stream, x, u)))


def ssm_causal_conv1d_step(window, x, weight, bias, u, silu=True, stream=None):
    """One decode token of the convolution (see include/ssm.h): window [batch, dim, width-1]
    fp32 updated in place (may be None for width 1); x, u [batch, dim]."""
    batch, dim = x.shape
    width = weight.shape[1]
    _fits("sizes", batch, dim)
    _check(load_library().ssm_causal_conv1d_step(
        _ptr(window), _ptr(x), _ptr(weight), _ptr(bias), _ptr(u), batch, dim, width,
        int(bool(silu)), _DTYPE_CODE[x.dtype], _DTYPE_CODE[u.dtype], _stream(stream, x, u)))


def causal_conv1d(x, weight, bias=None, initial_window=None, silu=True, out_dtype=None,
                  return_final_window=False, stream=None):
    """Allocate u (and the final window) with torch and run the convolution."""
    if stream is not None:
        with _current(stream, x):
            return causal_conv1d(x, weight, bias, initial_window, silu, out_dtype, return_final_window)
    batch, dim, L = x.shape
    u = torch.empty((batch, dim, L), device=x.device, dtype=out_dtype or x.dtype)
    fw = (torch.empty((batch, dim, weight.shape[1] - 1), device=x.device, dtype=torch.float32)
          if return_final_window else None)
    ssm_causal_conv1d_fwd(x, weight, bias, initial_window, u, fw, silu, stream)
    return (u, fw) if return_final_window else u


def selective_scan(x, delta, A, B, C, D=None, z=None, delta_bias=None, delta_softplus=False,
                   out_dtype=None, return_final_state=True, initial_state=None, zoh_exact=False,
                   stream=None):
    """Allocate y (and the final state) with torch and run the scan."""
    if stream is not None:
        with _current(stream, x):
            return selective_scan(x, delta, A, B, C, D, z, delta_bias, delta_softplus, out_dtype, return_final_state,
                                  initial_state, zoh_exact)
    batch, dim, L = x.shape
    y = torch.empty((batch, dim, L), device=x.device, dtype=out_dtype or x.dtype)
    fs = (torch.empty((batch, dim, A.shape[1]), device=x.device, dtype=torch.float32)
          if return_final_state else None)
    ssm_selective_scan_fwd_ex(x, delta, delta_bias, delta_softplus, A, B, C, D, z, y, fs,
                              initial_state, zoh_exact, stream)
    return (y, fs) if return_final_state else y


def _require(shapes):
    """Raise ValueError unless every (name, tensor or None, shape, dtype) is given as asked and
    contiguous: the kernels read what the sizes say, so nothing else must reach them.  All
    tensors have to be on one CUDA device."""
    device = None
    for name, t, shape, dtype in shapes:
        if t is None:
            continue
        if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
            raise ValueError("%s must be a contiguous %s tensor of shape %s, got %s of shape %s and strides %s" % (
                name, dtype, tuple(shape), t.dtype, tuple(t.shape), t.stride()))
        if device is None:
            device = t.device
            if device.type != "cuda":
                raise ValueError("libssm needs CUDA tensors, got %s" % device)
        elif t.device != device:
            raise ValueError("%s is on %s, other tensors on %s" % (name, t.device, device))


def _rows(x, dim):
    """Rows of ``dim`` values."""
    rows = x.numel() // dim if dim else 0
    if rows >= 2 ** 31:
        _fits("rows", rows)
    return rows


def _dtype_code(name, t):
    code = _DTYPE_CODE.get(t.dtype)
    if code is None:
        raise ValueError("%s must be fp32 or bf16, got %s" % (name, t.dtype))
    return code


def _at(t):
    return None if t is None else t.data_ptr()


def _call_on(like, stream, name, *args, workspace=None):
    """Run a library call with ``like``'s device current (its kernels and scratch live there).  Scratch
    comes from torch's allocator, on the stream that the call runs on."""
    if stream is not None:
        with _current(stream, like):
            return _call_on(like, None, name, *args, workspace=workspace)
    index = like.device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _call_on(like, None, name, *args, workspace=workspace)
    lib = _lib or load_library()
    if workspace is not None:
        nbytes = getattr(lib, name + "_workspace")(*workspace)
        ws = like.new_empty(nbytes, dtype=torch.uint8)
        args += (ws.data_ptr() if nbytes else None, nbytes)
    _check(getattr(lib, name)(*args, torch._C._cuda_getCurrentRawStream(index)))


def _delta_dims(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must have four dimensions")


def _delta_shapes(lead, q, k, v, a, beta):
    _delta_dims(q, k, v)
    (H, P), (K, N) = v.shape[2:], q.shape[2:]
    return H, K, P, N, [("q", q, (*lead, K, N), v.dtype), ("k", k, (*lead, K, N), v.dtype),
                        ("v", v, (*lead, H, P), v.dtype), ("a", a, (*lead, H), torch.float32),
                        ("beta", beta, (*lead, H), torch.float32)]


def ssm_delta_rule_fwd(q, k, v, a, beta, y, initial_state=None, final_state=None, scale=1.0, stream=None):
    """Gated delta rule over whole sequences (see include/ssm.h): q, k [batch, L, qk_heads, N];
    v, y [batch, L, heads, P]; a, beta [batch, L, heads] fp32; states [batch, heads, P, N] fp32.
    Writes y and final_state in place."""
    lead = v.shape[:2]
    H, K, P, N, shapes = _delta_shapes(lead, q, k, v, a, beta)
    st = (lead[0], H, P, N)
    _require(shapes + [("y", y, v.shape, y.dtype), ("initial_state", initial_state, st, torch.float32),
                             ("final_state", final_state, st, torch.float32)])
    sizes = (lead[0], lead[1], H, K, P, N, _dtype_code("v", v), _dtype_code("y", y))
    _call_on(v, stream, "ssm_delta_rule_fwd", _at(q), _at(k), _at(v), _at(a), _at(beta), _at(y),
             _at(initial_state), _at(final_state), float(scale), *sizes, workspace=sizes)


def delta_rule(q, k, v, a, beta, initial_state=None, scale=1.0, out_dtype=None, return_final_state=True,
               stream=None):
    """Allocate y (and the final state) with torch and run ``ssm_delta_rule_fwd``."""
    if stream is not None:
        with _current(stream, v):
            return delta_rule(q, k, v, a, beta, initial_state, scale, out_dtype, return_final_state)
    _delta_dims(q, k, v)
    y = torch.empty_like(v, dtype=out_dtype)
    fs = a.new_empty((v.shape[0], v.shape[2], v.shape[3], k.shape[-1])) if return_final_state else None
    ssm_delta_rule_fwd(q, k, v, a, beta, y, initial_state, fs, scale, stream)
    return (y, fs) if return_final_state else y


def ssm_delta_rule_step(state, q, k, v, a, beta, y, scale=1.0, stream=None):
    """Decode tokens of the gated delta rule (see include/ssm.h): state [batch, heads, P, N]
    fp32 updated in place; q, k [ntok, batch, qk_heads, N]; v, y [ntok, batch, heads, P]; a,
    beta [ntok, batch, heads] fp32."""
    lead = v.shape[:2]
    H, K, P, N, shapes = _delta_shapes(lead, q, k, v, a, beta)
    _require(shapes + [("y", y, v.shape, y.dtype), ("state", state, (lead[1], H, P, N), torch.float32)])
    _call_on(v, stream, "ssm_delta_rule_step", _at(state), _at(q), _at(k), _at(v), _at(a), _at(beta),
             _at(y), float(scale), lead[0], lead[1], H, K, P, N, _dtype_code("v", v), _dtype_code("y", y))


def delta_rule_step(state, q, k, v, a, beta, scale=1.0, out_dtype=None, stream=None):
    """Allocate y with torch and run ``ssm_delta_rule_step``."""
    if stream is not None:
        with _current(stream, v):
            return delta_rule_step(state, q, k, v, a, beta, scale, out_dtype)
    y = torch.empty_like(v, dtype=out_dtype)
    ssm_delta_rule_step(state, q, k, v, a, beta, y, scale, stream)
    return y


def ssm_delta_rule_bwd(q, k, v, a, beta, initial_state, dy, dfinal_state, dq, dk, dv, da, dbeta,
                       dinitial_state=None, scale=1.0, stream=None):
    """Backward of the gated delta rule (see include/ssm.h).  dq, dk, dv share dy's dtype; da,
    dbeta, dinitial_state are fp32.  Writes the gradients in place."""
    lead = v.shape[:2]
    H, K, P, N, shapes = _delta_shapes(lead, q, k, v, a, beta)
    st, f32 = (lead[0], H, P, N), torch.float32
    _require(shapes + [
        ("initial_state", initial_state, st, f32), ("dy", dy, v.shape, dy.dtype),
        ("dfinal_state", dfinal_state, st, f32), ("dq", dq, q.shape, dy.dtype), ("dk", dk, k.shape, dy.dtype),
        ("dv", dv, v.shape, dy.dtype), ("da", da, a.shape, f32), ("dbeta", dbeta, beta.shape, f32),
        ("dinitial_state", dinitial_state, st, f32)])
    sizes = (lead[0], lead[1], H, K, P, N, _dtype_code("v", v), _dtype_code("dy", dy))
    _call_on(v, stream, "ssm_delta_rule_bwd", _at(q), _at(k), _at(v), _at(a), _at(beta),
             _at(initial_state), _at(dy), _at(dfinal_state), _at(dq), _at(dk), _at(dv), _at(da), _at(dbeta),
             _at(dinitial_state), float(scale), *sizes, workspace=sizes)


def delta_rule_bwd(dy, q, k, v, a, beta, initial_state=None, dfinal_state=None, scale=1.0, stream=None):
    """Allocate the gradients with torch and run ``ssm_delta_rule_bwd``; returns a dict dq, dk,
    dv (dy's dtype), da, dbeta, dinitial_state (fp32; None without an initial_state)."""
    if stream is not None:
        with _current(stream, v):
            return delta_rule_bwd(dy, q, k, v, a, beta, initial_state, dfinal_state, scale)
    g = dict(dq=torch.empty_like(q, dtype=dy.dtype), dk=torch.empty_like(k, dtype=dy.dtype),
             dv=torch.empty_like(v, dtype=dy.dtype), da=torch.empty_like(a), dbeta=torch.empty_like(beta),
             dinitial_state=None if initial_state is None else torch.empty_like(initial_state))
    ssm_delta_rule_bwd(q, k, v, a, beta, initial_state, dy, dfinal_state, g["dq"], g["dk"], g["dv"], g["da"],
                       g["dbeta"], g["dinitial_state"], scale, stream)
    return g


def ssm_layer_norm_fwd(x, weight, bias, y, mean=None, rstd=None, eps=1e-5, stream=None):
    """Layer norm over the last dimension (see include/ssm.h): x, y [..., dim]; weight, bias
    [dim] fp32 or None; mean, rstd fp32, one value per row, or None.  Writes in place."""
    shape, f32 = x.shape, torch.float32
    dim = shape[-1]
    _require((("x", x, shape, x.dtype), ("weight", weight, shape[-1:], f32), ("bias", bias, shape[-1:], f32),
                    ("y", y, shape, y.dtype), ("mean", mean, shape[:-1], f32), ("rstd", rstd, shape[:-1], f32)))
    _layer_norm_fwd(x, weight, bias, y, mean, rstd, eps, dim, stream)


def _layer_norm_fwd(x, weight, bias, y, mean, rstd, eps, dim, stream):
    _call_on(x, stream, "ssm_layer_norm_fwd", _at(x), _at(weight), _at(bias), _at(y), _at(mean),
             _at(rstd), float(eps), _rows(x, dim), dim, _dtype_code("x", x), _dtype_code("y", y))


def layer_norm(x, weight=None, bias=None, eps=1e-5, out_dtype=None, return_stats=False, stream=None):
    """Allocate y (and mean, rstd) with torch and run the layer norm; returns y, or (y, mean,
    rstd) for the backward."""
    if stream is not None:
        with _current(stream, x):
            return layer_norm(x, weight, bias, eps, out_dtype, return_stats)
    shape = x.shape
    mean, rstd = None, None
    y = torch.empty_like(x, dtype=out_dtype)
    if return_stats:
        mean = x.new_empty(shape[:-1], dtype=torch.float32)
        rstd = torch.empty_like(mean)
    _require((("x", x, shape, x.dtype), ("weight", weight, shape[-1:], torch.float32),
                    ("bias", bias, shape[-1:], torch.float32)))
    _layer_norm_fwd(x, weight, bias, y, mean, rstd, eps, shape[-1], stream)
    return (y, mean, rstd) if return_stats else y


def ssm_layer_norm_bwd(dy, x, weight, mean, rstd, dx, dweight=None, dbias=None, stream=None):
    """Backward of the layer norm (see include/ssm.h): dx in dy's dtype; dweight, dbias [dim]
    fp32 or None.  Writes the gradients in place."""
    dim, f32 = x.shape[-1], torch.float32
    _require([("dy", dy, x.shape, dy.dtype), ("x", x, x.shape, x.dtype), ("weight", weight, (dim,), f32),
                    ("mean", mean, x.shape[:-1], f32), ("rstd", rstd, x.shape[:-1], f32),
                    ("dx", dx, x.shape, dy.dtype), ("dweight", dweight, (dim,), f32), ("dbias", dbias, (dim,), f32)])
    rows = _rows(x, dim)
    _call_on(x, stream, "ssm_layer_norm_bwd", _at(dy), _at(x), _at(weight), _at(mean), _at(rstd),
             _at(dx), _at(dweight), _at(dbias), rows, dim, _dtype_code("x", x), _dtype_code("dy", dy),
             workspace=(rows, dim))


def layer_norm_bwd(dy, x, weight, mean, rstd, stream=None):
    """Allocate the gradients with torch and run ``ssm_layer_norm_bwd``; returns a dict dx
    (dy's dtype), dweight, dbias (fp32)."""
    if stream is not None:
        with _current(stream, x):
            return layer_norm_bwd(dy, x, weight, mean, rstd)
    dw = x.new_empty(x.shape[-1:], dtype=torch.float32)
    g = dict(dx=torch.empty_like(dy), dweight=dw, dbias=torch.empty_like(dw))
    ssm_layer_norm_bwd(dy, x, weight, mean, rstd, g["dx"], g["dweight"], g["dbias"], stream)
    return g
