"""Binding of the selective state space block's entry points: the short causal
convolution, the selective scan and gradient clipping (include/falcon.h).

Argument marshalling only, as in the package's other functions: the names are
the C names, the work is in the CUDA kernels, a nonzero return code raises
``FalconError``.  Activations may be views with any row strides as long as
consecutive channels are adjacent; parameters and states are dense.

A call runs on the current stream, or on ``stream``: the caller then orders the inputs
before it and the use of its results after it, as with any work on another stream.
"""
from __future__ import annotations

import array
import ctypes
import functools

import torch

FALCON_ACT_IDENTITY = 0
FALCON_ACT_SILU = 1
_ACT = {"identity": FALCON_ACT_IDENTITY, "silu": FALCON_ACT_SILU}
_DTYPE = {torch.bfloat16: 0, torch.float32: 1}

EXPORTS = (
    "falcon_short_conv_fwd", "falcon_short_conv_bwd_workspace_bytes", "falcon_short_conv_bwd",
    "falcon_short_conv_step", "falcon_selective_scan_fwd",
    "falcon_selective_scan_bwd_workspace_bytes", "falcon_selective_scan_bwd",
    "falcon_selective_scan_step", "falcon_clip_workspace_bytes", "falcon_clip_grad_norm",
)

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
_f32, _sz = ctypes.c_float, ctypes.c_size_t


class falcon_strides(ctypes.Structure):
    _fields_ = [("batch", _i64), ("head", _i64), ("time", _i64)]


class falcon_conv_shape(ctypes.Structure):
    _fields_ = [("B", _i64), ("H", _i64), ("T", _i64), ("m", _i32), ("width", _i32),
                ("dtype", _i32), ("activation", _i32)]


class falcon_scan_shape(ctypes.Structure):
    _fields_ = [("B", _i64), ("T", _i64), ("D", _i32), ("G", _i32), ("N", _i32),
                ("dtype", _i32), ("softplus", _i32)]


class falcon_grad(ctypes.Structure):
    _fields_ = [("grad", _vp), ("out", _vp), ("count", _i64), ("dtype", _i32)]


def declare(lib):
    """Sets the argument types of this module's entry points."""
    conv, scan = ctypes.POINTER(falcon_conv_shape), ctypes.POINTER(falcon_scan_shape)
    st, grads = ctypes.POINTER(falcon_strides), ctypes.POINTER(falcon_grad)
    sig = {
        "falcon_short_conv_fwd": [conv, _vp, st, _vp, _vp, _vp, _vp, _vp, st, _vp, _vp],
        "falcon_short_conv_bwd_workspace_bytes": [conv],
        "falcon_short_conv_bwd": [conv, _vp, st, _vp, _vp, _vp, _vp, _vp, st, _vp, _vp, st,
                                  _vp, _vp, _vp, _vp, _sz, _vp],
        "falcon_short_conv_step": [_i64, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i64,
                                   _vp, _vp, _vp, _vp],
        "falcon_selective_scan_fwd": [scan, _vp, st, _vp, st, _vp, _vp, st, _vp, st, _vp, _vp,
                                      st, _vp, _vp, _vp, _vp, st, _vp, _vp],
        "falcon_selective_scan_bwd_workspace_bytes": [scan],
        "falcon_selective_scan_bwd": [scan, _vp, st, _vp, st, _vp, _vp, st, _vp, st, _vp, _vp,
                                      st, _vp, _vp, _vp, _vp, st, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _sz, _vp],
        "falcon_selective_scan_step": [_i64, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _i64,
                                       _vp, _vp, st, _vp, st, _vp, _vp, _i64, _vp, _vp, _i64,
                                       _vp, _vp, _vp, _vp],
        "falcon_clip_workspace_bytes": [grads, _i64],
        "falcon_clip_grad_norm": [grads, _i64, _f32, _f32, _vp, _vp, _sz, _vp],
    }
    for name in EXPORTS:
        fn = getattr(lib, name)
        fn.argtypes = sig[name]
        fn.restype = _sz if name.endswith("_bytes") else ctypes.c_int


_lib = None


def _library():
    global _lib
    if _lib is None:
        from . import load_library
        _lib = load_library()
    return _lib


def _check(rc, what):
    if rc != 0:
        from . import FalconError
        raise FalconError(rc, what)


def _at(t):
    return None if t is None else t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream
_device_now = torch._C._cuda_getDevice


def refuse_other_device(t, name):
    """A launch goes to the current device, whatever its pointers belong to."""
    if t.get_device() != _device_now():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{_device_now()}")


def elsewhere(stream, fn, *args):
    """fn(*args) on a stream that need not be the current one.  Its new tensors come from
    that stream's memory: what the current stream's pool hands out may be in use by work
    still queued there, which nothing orders before this call.  The tensors that it
    returns are marked as used by the current stream as well, so that they may be dropped
    there as soon as what reads them is queued."""
    here = torch.cuda.current_stream(stream.device)
    if here.cuda_stream == stream.cuda_stream and stream.device.index == _device_now():
        return fn(*args)
    given = set()
    for a in args:
        given.update(map(id, a.values() if isinstance(a, dict) else (a,)))
    with torch.cuda.stream(stream):
        out = fn(*args)
    new = (out,) if isinstance(out, torch.Tensor) else \
        out.values() if isinstance(out, dict) else out
    for t in new:
        if t is not None and id(t) not in given:
            t.record_stream(here)
    return out


# Descriptions by their values: the structures of a shape met before are not built
# again.
@functools.lru_cache(maxsize=4096)
def _strides(batch, head, time):
    return ctypes.byref(falcon_strides(batch, head, time))


@functools.lru_cache(maxsize=1024)
def _conv_shape(*fields):
    return ctypes.byref(falcon_conv_shape(*fields))


@functools.lru_cache(maxsize=1024)
def _scan_shape(*fields):
    return ctypes.byref(falcon_scan_shape(*fields))


def _refuse(t, name, dtype, shape, device, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, x or u on {device}")
    raise ValueError(f"{name} must {what}")


# The checks run for every tensor of every call, small calls among them: what passes
# costs four attributes, and what fails is asked again for the words of the error.

def _rows(t, name, dtype, shape, device):
    """A tensor of this type, shape and GPU whose last dimension is adjacent."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.device == device and
                (t.stride(-1) == 1 or t.shape[-1] <= 1)):
            return t
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, device, "have adjacent channels")


def _dense(t, name, dtype, shape, device):
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.shape == shape and t.device == device and
                t.is_contiguous()):
            return t
    except AttributeError:
        pass
    _refuse(t, name, dtype, shape, device, "be contiguous")


def _dtype(t, name):
    """The dtype of a call's first tensor, whose GPU the others are held to."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _DTYPE:
        raise TypeError(f"{name} must be bfloat16 or float32")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    refuse_other_device(t, name)
    return t.dtype


_new = torch.empty


def _empty(shape, dtype, device):
    return _new(shape, dtype=dtype, device=device)


def _like(t):
    """A new dense tensor of t's shape, type and device."""
    return torch.empty_like(t) if t.is_contiguous() else _empty(t.shape, t.dtype, t.device)


def _workspace(need, workspace, device):
    if workspace is None:
        return (_empty(need, torch.uint8, device), need) if need else (None, 0)
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _conv_rows(t):
    """Strides of [B,T,m] or [B,H,T,m]."""
    s = t.stride()
    return _strides(s[0], 0, s[1]) if len(s) == 3 else _strides(s[0], s[1], s[2])


def _conv_setup(x, weight, bias, state, lengths, activation):
    dt = _dtype(x, "x")
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B,T,m] or [B,H,T,m]")
    if activation not in _ACT:
        raise ValueError(f"activation must be one of {sorted(_ACT)}")
    dev = x.device
    shape = x.shape
    _rows(x, "x", dt, shape, dev)
    B, T, m = shape[0], shape[-2], shape[-1]
    H = 1 if len(shape) == 3 else shape[1]
    C = H * m
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [channels, width]")
    W = weight.shape[1]
    _dense(weight, "weight", torch.float32, (C, W), dev)
    if bias is not None:
        _dense(bias, "bias", torch.float32, (C,), dev)
    if state is not None:
        _dense(state, "state", dt, (B, W - 1, C), dev)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (B,), dev)
    return _conv_shape(B, H, T, m, W, _DTYPE[dt], _ACT[activation]), dt, dev, B, C, W


def falcon_short_conv_fwd(x, weight, bias=None, state=None, lengths=None, activation="silu",
                          y=None, state_out=None, stream=None):
    """Depthwise causal convolution over time.  x [B,T,m], or [B,H,T,m] with
    H*m channels (bf16 or fp32, any row strides); weight [channels, width] fp32,
    width 2, 3 or 4; bias [channels] fp32; state [B, width-1, channels] in x's
    dtype (the inputs before token 0); lengths [B] int32; activation "silu" or
    "identity".  Returns (y, state_out): y of x's shape, dense unless passed in,
    and the last width-1 inputs of every row."""
    if stream is not None:
        return elsewhere(stream, falcon_short_conv_fwd, x, weight, bias, state, lengths,
                          activation, y, state_out)
    lib = _lib or _library()
    shape, dt, dev, B, C, W = _conv_setup(x, weight, bias, state, lengths, activation)
    y = _like(x) if y is None else _rows(y, "y", dt, x.shape, dev)
    state_out = _empty((B, W - 1, C), dt, dev) if state_out is None else \
        _dense(state_out, "state_out", dt, (B, W - 1, C), dev)
    rc = lib.falcon_short_conv_fwd(shape, x.data_ptr(), _conv_rows(x), weight.data_ptr(), _at(bias),
                                   _at(state), _at(lengths), y.data_ptr(), _conv_rows(y),
                                   state_out.data_ptr(), _raw_stream(dev.index))
    _check(rc, "falcon_short_conv_fwd")
    return y, state_out


def falcon_short_conv_bwd(x, weight, dy, bias=None, state=None, lengths=None, dstate_out=None,
                          activation="silu", grads=None, workspace=None, stream=None):
    """Gradients of <dy, y> + <dstate_out, state_out> of falcon_short_conv_fwd.
    Returns a dict with dx (dense, x's shape), dweight, dbias (fp32) and dstate;
    ``grads`` may pass preallocated outputs."""
    if stream is not None:
        return elsewhere(stream, falcon_short_conv_bwd, x, weight, dy, bias, state, lengths,
                          dstate_out, activation, grads, workspace)
    lib = _lib or _library()
    shape, dt, dev, B, C, W = _conv_setup(x, weight, bias, state, lengths, activation)
    _rows(dy, "dy", dt, x.shape, dev)
    _dense(dstate_out, "dstate_out", dt, (B, W - 1, C), dev)
    g = {} if grads is None else grads
    if "dx" not in g:
        g["dx"] = _like(x)
    if "dweight" not in g:
        g["dweight"] = _like(weight)
    if "dbias" not in g:
        g["dbias"] = _empty((C,), torch.float32, dev)
    if "dstate" not in g:
        g["dstate"] = _empty((B, W - 1, C), dt, dev)
    if grads is not None:
        _rows(g["dx"], "dx", dt, x.shape, dev)
        _dense(g["dweight"], "dweight", torch.float32, (C, W), dev)
        _dense(g["dbias"], "dbias", torch.float32, (C,), dev)
        _dense(g["dstate"], "dstate", dt, (B, W - 1, C), dev)
    workspace, have = _workspace(int(lib.falcon_short_conv_bwd_workspace_bytes(shape)),
                                 workspace, dev)
    rc = lib.falcon_short_conv_bwd(
        shape, x.data_ptr(), _conv_rows(x), weight.data_ptr(), _at(bias), _at(state),
        _at(lengths), dy.data_ptr(),
        _conv_rows(dy), _at(dstate_out), _at(g["dx"]), _conv_rows(g["dx"]), _at(g["dweight"]),
        _at(g["dbias"]), _at(g["dstate"]), _at(workspace), have, _raw_stream(dev.index))
    _check(rc, "falcon_short_conv_bwd")
    return g


def falcon_short_conv_step(x, weight, state, bias=None, slots=None, fresh=None,
                           activation="silu", y=None, stream=None):
    """One token of N sequences: x [N,channels]; state [pool, width-1, channels]
    (x's dtype) is updated in place; slots [N] int32 names each row's state (row i
    uses state i when absent), fresh [N] uint8 marks sequences that start here.
    Returns y [N,channels]."""
    if stream is not None:
        return elsewhere(stream, falcon_short_conv_step, x, weight, state, bias, slots, fresh,
                          activation, y)
    lib = _lib or _library()
    dt = _dtype(x, "x")
    if x.dim() != 2 or not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("x must be [N, channels] and weight [channels, width]")
    if activation not in _ACT:
        raise ValueError(f"activation must be one of {sorted(_ACT)}")
    N, C = x.shape
    W = weight.shape[1]
    dev = x.device
    _rows(x, "x", dt, x.shape, dev)
    _dense(weight, "weight", torch.float32, (C, W), dev)
    _dense(bias, "bias", torch.float32, (C,), dev)
    pool = _pool(state, "state", slots, N)
    _dense(state, "state", dt, (pool, W - 1, C), dev)
    _dense(slots, "slots", torch.int32, (N,), dev)
    _dense(fresh, "fresh", torch.uint8, (N,), dev)
    y = _like(x) if y is None else _dense(y, "y", dt, (N, C), dev)
    rc = lib.falcon_short_conv_step(N, C, W, _DTYPE[dt], _ACT[activation], x.data_ptr(),
                                    x.stride(0), weight.data_ptr(), _at(bias), _at(state), pool,
                                    _at(slots), _at(fresh), y.data_ptr(), _raw_stream(dev.index))
    _check(rc, "falcon_short_conv_step")
    return y


def _pool(state, name, slots, N):
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError(f"{name} must be a pool of states, [pool, ., .]")
    if slots is None and state.shape[0] != N:
        raise ValueError(f"{name} must hold one state a row where no slots are given")
    return state.shape[0]


def _time_rows(t):
    s = t.stride()
    return _strides(s[0], 0, s[1])


def _group_rows(t):
    s = t.stride()
    return _strides(s[0], s[2], s[1])


def _scan_setup(u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, softplus):
    dt = _dtype(u, "u")
    if u.dim() != 3:
        raise ValueError("u must be [B,T,D]")
    B, T, C = u.shape
    if not isinstance(A, torch.Tensor) or A.dim() != 2:
        raise ValueError("A must be [D, N]")
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
        raise ValueError("Bm and Cm must be [B,T,G,N]")
    N, G = A.shape[1], Bm.shape[2]
    dev, row, bc, f32 = u.device, (B, T, C), (B, T, G, N), torch.float32
    _rows(u, "u", dt, row, dev)
    _rows(delta, "delta", dt, row, dev)
    _rows(Bm, "Bm", dt, bc, dev)
    _rows(Cm, "Cm", dt, bc, dev)
    if z is not None:
        _rows(z, "z", dt, row, dev)
    _dense(A, "A", f32, (C, N), dev)
    _dense(D, "D", f32, (C,), dev)
    _dense(delta_bias, "delta_bias", f32, (C,), dev)
    if h0 is not None:
        _dense(h0, "h0", f32, (B, C, N), dev)
    if lengths is not None:
        _dense(lengths, "lengths", torch.int32, (B,), dev)
    return _scan_shape(B, T, C, G, N, _DTYPE[dt], 1 if softplus else 0), dt, dev, (B, C, N)


def falcon_selective_scan_fwd(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None, h0=None,
                              lengths=None, softplus=True, y=None, h_out=None, stream=None):
    """Selective scan h_t = exp(s_t A) h_{t-1} + s_t u_t Bm_t, y_t = (<Cm_t, h_t> +
    D u_t) silu(z_t), s_t = softplus(delta_t + delta_bias).  u, delta, z [B,T,D]
    and Bm, Cm [B,T,G,N] (bf16 or fp32, any row strides); A [D,N], D, delta_bias
    [D] and h0 [B,D,N] fp32; lengths [B] int32.  Returns (y, h_T)."""
    if stream is not None:
        return elsewhere(stream, falcon_selective_scan_fwd, u, delta, A, Bm, Cm, D, z, delta_bias,
                          h0, lengths, softplus, y, h_out)
    lib = _lib or _library()
    shape, dt, dev, hs = _scan_setup(u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, softplus)
    y = _like(delta) if y is None else _rows(y, "y", dt, u.shape, dev)
    h_out = _empty(hs, torch.float32, dev) if h_out is None else \
        _dense(h_out, "h_out", torch.float32, hs, dev)
    rc = lib.falcon_selective_scan_fwd(
        shape, u.data_ptr(), _time_rows(u), delta.data_ptr(), _time_rows(delta), A.data_ptr(),
        Bm.data_ptr(),
        _group_rows(Bm), Cm.data_ptr(), _group_rows(Cm), _at(D), _at(z),
        None if z is None else _time_rows(z), _at(delta_bias), _at(h0), _at(lengths), y.data_ptr(),
        _time_rows(y), h_out.data_ptr(), _raw_stream(dev.index))
    _check(rc, "falcon_selective_scan_fwd")
    return y, h_out


def falcon_selective_scan_bwd(u, delta, A, Bm, Cm, dy, D=None, z=None, delta_bias=None, h0=None,
                              lengths=None, dh_T=None, softplus=True, grads=None,
                              workspace=None, stream=None):
    """Gradients of <dy, y> + <dh_T, h_T> of falcon_selective_scan_fwd.  Returns a
    dict with du, ddelta, dz, dB, dC (u's dtype, dense) and dA, dD, ddelta_bias,
    dh0 (fp32); dz, dD and ddelta_bias are None where z, D or delta_bias is.
    ``grads`` may pass preallocated outputs."""
    if stream is not None:
        return elsewhere(stream, falcon_selective_scan_bwd, u, delta, A, Bm, Cm, dy, D, z,
                          delta_bias, h0, lengths, dh_T, softplus, grads, workspace)
    lib = _lib or _library()
    shape, dt, dev, hs = _scan_setup(u, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths, softplus)
    _rows(dy, "dy", dt, u.shape, dev)
    _dense(dh_T, "dh_T", torch.float32, hs, dev)
    # each gradient is shaped and typed as its input
    like = {"du": delta, "ddelta": delta, "dA": A, "dB": Bm, "dC": Bm, "dD": D, "dz": z,
            "ddelta_bias": delta_bias}
    g = {} if grads is None else grads
    for name, t in like.items():
        if t is None:
            g[name] = None
        elif name in g:
            _dense(g[name], name, t.dtype, t.shape, dev)
        else:
            g[name] = _like(t)
    if "dh0" in g:
        _dense(g["dh0"], "dh0", torch.float32, hs, dev)
    else:
        g["dh0"] = _empty(hs, torch.float32, dev)
    workspace, have = _workspace(int(lib.falcon_selective_scan_bwd_workspace_bytes(shape)),
                                 workspace, dev)
    rc = lib.falcon_selective_scan_bwd(
        shape, u.data_ptr(), _time_rows(u), delta.data_ptr(), _time_rows(delta), A.data_ptr(),
        Bm.data_ptr(),
        _group_rows(Bm), Cm.data_ptr(), _group_rows(Cm), _at(D), _at(z),
        None if z is None else _time_rows(z), _at(delta_bias), _at(h0), _at(lengths), dy.data_ptr(),
        _time_rows(dy), _at(dh_T), _at(g["du"]), _at(g["ddelta"]), _at(g["dA"]), _at(g["dB"]),
        _at(g["dC"]), _at(g["dD"]), _at(g["dz"]), _at(g["ddelta_bias"]), _at(g["dh0"]),
        _at(workspace), have, _raw_stream(dev.index))
    _check(rc, "falcon_selective_scan_bwd")
    return g


def falcon_selective_scan_step(u, delta, A, Bm, Cm, h, D=None, z=None, delta_bias=None,
                               slots=None, fresh=None, softplus=True, y=None, stream=None):
    """One token of N sequences: u, delta, z [N,D], Bm, Cm [N,G,S]; h [pool,D,S]
    fp32 is updated in place; slots and fresh as in falcon_short_conv_step.
    Returns y [N,D]."""
    if stream is not None:
        return elsewhere(stream, falcon_selective_scan_step, u, delta, A, Bm, Cm, h, D, z,
                          delta_bias, slots, fresh, softplus, y)
    lib = _lib or _library()
    dt = _dtype(u, "u")
    if u.dim() != 2 or not isinstance(A, torch.Tensor) or A.dim() != 2 or \
            not isinstance(Bm, torch.Tensor) or Bm.dim() != 3:
        raise ValueError("u must be [N,D], A [D,S] and Bm, Cm [N,G,S]")
    N, C = u.shape
    S, G = A.shape[1], Bm.shape[1]
    dev, row, bc, f32 = u.device, (N, C), (N, G, S), torch.float32
    _rows(u, "u", dt, row, dev)
    _rows(delta, "delta", dt, row, dev)
    _rows(Bm, "Bm", dt, bc, dev)
    _rows(Cm, "Cm", dt, bc, dev)
    if z is not None:
        _rows(z, "z", dt, row, dev)
    _dense(A, "A", f32, (C, S), dev)
    _dense(D, "D", f32, (C,), dev)
    _dense(delta_bias, "delta_bias", f32, (C,), dev)
    pool = _pool(h, "h", slots, N)
    _dense(h, "h", f32, (pool, C, S), dev)
    _dense(slots, "slots", torch.int32, (N,), dev)
    _dense(fresh, "fresh", torch.uint8, (N,), dev)
    y = _like(delta) if y is None else _dense(y, "y", dt, row, dev)
    b, c = Bm.stride(), Cm.stride()
    rc = lib.falcon_selective_scan_step(
        N, C, G, S, _DTYPE[dt], 1 if softplus else 0, u.data_ptr(), u.stride(0), delta.data_ptr(),
        delta.stride(0), A.data_ptr(), Bm.data_ptr(), _strides(b[0], b[1], 0), Cm.data_ptr(),
        _strides(c[0], c[1], 0), _at(D), _at(z), 0 if z is None else z.stride(0),
        _at(delta_bias), h.data_ptr(), pool, _at(slots), _at(fresh), y.data_ptr(),
        _raw_stream(dev.index))
    _check(rc, "falcon_selective_scan_step")
    return y


def falcon_clip_grad_norm(grads, max_norm, out=None, eps=1e-6, norm=None, workspace=None,
                          stream=None):
    """Scales a list of dense gradients (bf16 or fp32, mixed, any shapes) by
    min(1, max_norm / (n + eps)), n their global 2-norm: in place, or into the
    tensors of ``out`` (same sizes and dtypes).  Returns n, a 0-d fp32 tensor on
    the gradients' device; the host does not wait for it."""
    if stream is not None:
        return elsewhere(stream, falcon_clip_grad_norm, grads, max_norm, out, eps, norm, workspace)
    lib = _lib or _library()
    grads = list(grads)
    if not grads:
        raise ValueError("grads must hold at least one tensor")
    into = grads if out is None else list(out)
    if len(into) != len(grads):
        raise ValueError("out must hold one tensor a gradient")
    T = torch.Tensor
    counts = list(map(T.numel, grads))  # refuses what is no tensor
    kinds = [t.dtype for t in grads]
    if not _DTYPE.keys() >= set(kinds):
        raise TypeError("gradients must be bfloat16 or float32")
    index = grads[0].get_device()
    both = grads if into is grads else grads + into
    if index < 0 or list(map(T.get_device, both)).count(index) != len(both):
        raise ValueError("gradients and outputs must be CUDA tensors of one device")
    refuse_other_device(grads[0], "gradients")
    if not all(map(T.is_contiguous, both)):
        raise ValueError("gradients and outputs must be contiguous")
    at = array.array("q", map(T.data_ptr, grads))
    if into is grads:
        to = at
    else:
        if [t.dtype for t in into] != kinds:
            raise TypeError("outputs must have their gradients' dtypes")
        if list(map(T.numel, into)) != counts:
            raise ValueError("outputs must have their gradients' sizes")
        to = array.array("q", map(T.data_ptr, into))
    # the rows of falcon_grad: four 64-bit words each
    table = array.array("q", bytes(32 * len(grads)))
    table[0::4], table[1::4], table[2::4] = at, to, array.array("q", counts)
    table[3::4] = array.array("q", map(_DTYPE.__getitem__, kinds))
    rows = ctypes.cast(table.buffer_info()[0], ctypes.POINTER(falcon_grad))
    dev = grads[0].device
    if norm is None:
        norm = _empty((), torch.float32, dev)
    elif not isinstance(norm, torch.Tensor) or norm.dtype != torch.float32:
        raise TypeError("norm must be a float32 torch.Tensor")
    elif norm.numel() != 1 or norm.device != dev:
        raise ValueError(f"norm must be one element on {dev}")
    workspace, have = _workspace(int(lib.falcon_clip_workspace_bytes(rows, len(grads))),
                                 workspace, dev)
    rc = lib.falcon_clip_grad_norm(rows, len(grads), float(max_norm), float(eps), norm.data_ptr(),
                                   _at(workspace), have, _raw_stream(dev.index))
    _check(rc, "falcon_clip_grad_norm")
    return norm
