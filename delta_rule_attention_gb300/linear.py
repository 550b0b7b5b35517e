"""Binding of the linear attention block's entry points: attention with a fixed decay for
each head, and the norms around a block with its gate, scale and residual
(include/falcon.h).

Argument marshalling only, as in ``block.py``: the names are the C names, the work is in
the CUDA kernels, a nonzero return code raises ``FalconError``.  Activations may be views
with any strides as long as consecutive channels are adjacent; parameters and states are
dense.  A call runs on the current stream, or on ``stream``, as there.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import block
from .block import _DTYPE, _at, _check, _dense, _dtype, _rows, _strides, elsewhere

FALCON_ACT_SIGMOID = 2
_GATE = {**block._ACT, "sigmoid": FALCON_ACT_SIGMOID}

EXPORTS = (
    "falcon_decay_attn_workspace_bytes", "falcon_decay_attn_fwd",
    "falcon_decay_attn_bwd_workspace_bytes", "falcon_decay_attn_bwd", "falcon_decay_attn_step",
    "falcon_gated_norm_fwd", "falcon_gated_norm_bwd_workspace_bytes", "falcon_gated_norm_bwd",
)

_i64, _i32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
_f32, _sz = ctypes.c_float, ctypes.c_size_t


class falcon_decay_shape(ctypes.Structure):
    _fields_ = [("B", _i64), ("H", _i64), ("T", _i64), ("m", _i32), ("dv", _i32),
                ("dtype", _i32), ("scale", _f32)]


class falcon_norm_shape(ctypes.Structure):
    _fields_ = [("B", _i64), ("H", _i64), ("T", _i64), ("m", _i32), ("dtype", _i32),
                ("gate", _i32), ("eps", _f32)]


def declare(lib):
    """Sets the argument types of this module's entry points."""
    decay, norm = ctypes.POINTER(falcon_decay_shape), ctypes.POINTER(falcon_norm_shape)
    st = ctypes.POINTER(block.falcon_strides)
    act = [_vp, st]
    sig = {
        "falcon_decay_attn_workspace_bytes": [decay],
        "falcon_decay_attn_fwd": [decay, *act * 3, _vp, _vp, _vp, *act, _vp, _vp, _sz, _vp],
        "falcon_decay_attn_bwd_workspace_bytes": [decay],
        "falcon_decay_attn_bwd": [decay, *act * 3, _vp, _vp, _vp, *act, _vp, *act * 3, _vp, _vp,
                                  _sz, _vp],
        "falcon_decay_attn_step": [decay, *act * 3, _vp, _vp, _i64, _vp, _vp, _vp, _vp],
        "falcon_gated_norm_fwd": [norm, *act, _vp, *act, _vp, *act, _vp, _vp, *act * 2, _vp],
        "falcon_gated_norm_bwd_workspace_bytes": [norm],
        "falcon_gated_norm_bwd": [norm, *act, _vp, *act, _vp, *act, _vp, _vp, *act * 5, _vp, _vp,
                                  _vp, _vp, _sz, _vp],
    }
    for name in EXPORTS:
        fn = getattr(lib, name)
        fn.argtypes = sig[name]
        fn.restype = _sz if name.endswith("_bytes") else ctypes.c_int


@functools.lru_cache(maxsize=1024)
def _decay_shape(*fields):
    return ctypes.byref(falcon_decay_shape(*fields))


@functools.lru_cache(maxsize=1024)
def _norm_shape(*fields):
    return ctypes.byref(falcon_norm_shape(*fields))


# Workspace sizes by shape: the same shape is asked once.
@functools.lru_cache(maxsize=1024)
def _need(name, kind, *fields):
    return int(getattr(block._lib or block._library(), name)(kind(*fields)))


def _heads(t):
    """Strides of [B,H,T,m]."""
    s = t.stride()
    return _strides(s[0], s[1], s[2])


def _default_scale(m):
    return max(m, 1) ** -0.5  # keys of no channel are the library's to refuse


def _decay_setup(q, k, v, log_decay, S0, lengths, scale):
    dt = _dtype(q, "q")
    if q.dim() != 4 or not isinstance(v, torch.Tensor) or v.dim() != 4:
        raise ValueError("q and k must be [B,H,T,m] and v [B,H,T,dv]")
    B, H, T, m = q.shape
    dv, dev = v.shape[3], q.device
    _rows(q, "q", dt, q.shape, dev)
    _rows(k, "k", dt, q.shape, dev)
    _rows(v, "v", dt, (B, H, T, dv), dev)
    _dense(log_decay, "log_decay", torch.float32, (H,), dev)
    if log_decay is None:
        raise TypeError("log_decay must be a torch.Tensor")
    _dense(S0, "S0", torch.float32, (B, H, m, dv), dev)
    _dense(lengths, "lengths", torch.int32, (B,), dev)
    scale = _default_scale(m) if scale is None else float(scale)
    return (B, H, T, m, dv, _DTYPE[dt], scale), dt, dev


def falcon_decay_attn_fwd(q, k, v, log_decay, S0=None, lengths=None, scale=None, o=None,
                          S_out=None, workspace=None, stream=None):
    """S_t = gamma S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t with gamma =
    exp(log_decay) for each head.  q, k [B,H,T,m], v [B,H,T,dv] (bf16 or fp32, any
    strides, m and dv up to 128); log_decay [H] fp32, at most 0; S0 [B,H,m,dv] fp32;
    lengths [B] int32; scale m ** -0.5 where it is not given.  Returns (o, S_T): o
    [B,H,T,dv], dense unless passed in, and the state after every row's last token."""
    if stream is not None:
        return elsewhere(stream, falcon_decay_attn_fwd, q, k, v, log_decay, S0, lengths, scale,
                         o, S_out, workspace)
    lib = block._lib or block._library()
    fields, dt, dev = _decay_setup(q, k, v, log_decay, S0, lengths, scale)
    B, H, T, m, dv = fields[:5]
    o = block._empty((B, H, T, dv), dt, dev) if o is None else _rows(o, "o", dt, v.shape, dev)
    S_out = block._empty((B, H, m, dv), torch.float32, dev) if S_out is None else \
        _dense(S_out, "S_out", torch.float32, (B, H, m, dv), dev)
    workspace, have = block._workspace(_need("falcon_decay_attn_workspace_bytes", _decay_shape,
                                             *fields), workspace, dev)
    rc = lib.falcon_decay_attn_fwd(
        _decay_shape(*fields), q.data_ptr(), _heads(q), k.data_ptr(), _heads(k), v.data_ptr(),
        _heads(v), log_decay.data_ptr(), _at(S0), _at(lengths), o.data_ptr(), _heads(o),
        S_out.data_ptr(), _at(workspace), have, block._raw_stream(dev.index))
    _check(rc, "falcon_decay_attn_fwd")
    return o, S_out


def falcon_decay_attn_bwd(q, k, v, log_decay, dO, S0=None, lengths=None, dS_T=None, scale=None,
                          grads=None, workspace=None, stream=None):
    """Gradients of <dO, o> + <dS_T, S_T> of falcon_decay_attn_fwd.  Returns a dict with
    dq, dk, dv (dense, of q's, k's and v's shapes and type) and dS0 (fp32); ``grads`` may
    pass preallocated outputs."""
    if stream is not None:
        return elsewhere(stream, falcon_decay_attn_bwd, q, k, v, log_decay, dO, S0, lengths,
                         dS_T, scale, grads, workspace)
    lib = block._lib or block._library()
    fields, dt, dev = _decay_setup(q, k, v, log_decay, S0, lengths, scale)
    B, H, T, m, dv = fields[:5]
    st = (B, H, m, dv)
    _rows(dO, "dO", dt, v.shape, dev)
    _dense(dS_T, "dS_T", torch.float32, st, dev)
    g = {} if grads is None else grads
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        if name in g:
            _rows(g[name], name, dt, t.shape, dev)
        else:
            g[name] = block._empty(t.shape, dt, dev)
    if "dS0" in g:
        _dense(g["dS0"], "dS0", torch.float32, st, dev)
    else:
        g["dS0"] = block._empty(st, torch.float32, dev)
    workspace, have = block._workspace(_need("falcon_decay_attn_bwd_workspace_bytes",
                                             _decay_shape, *fields), workspace, dev)
    rc = lib.falcon_decay_attn_bwd(
        _decay_shape(*fields), q.data_ptr(), _heads(q), k.data_ptr(), _heads(k), v.data_ptr(),
        _heads(v), log_decay.data_ptr(), _at(S0), _at(lengths), dO.data_ptr(), _heads(dO),
        _at(dS_T), g["dq"].data_ptr(), _heads(g["dq"]), g["dk"].data_ptr(), _heads(g["dk"]),
        g["dv"].data_ptr(), _heads(g["dv"]), _at(g["dS0"]), _at(workspace), have,
        block._raw_stream(dev.index))
    _check(rc, "falcon_decay_attn_bwd")
    return g


def falcon_decay_attn_step(q, k, v, log_decay, S, slots=None, fresh=None, scale=None, o=None,
                           stream=None):
    """One token of N sequences: q, k [N,H,m], v [N,H,dv]; S [pool,H,m,dv] fp32 is updated
    in place; slots [N] int32 names each row's state (row i uses state i when absent),
    fresh [N] uint8 marks sequences that start here.  Returns o [N,H,dv]."""
    if stream is not None:
        return elsewhere(stream, falcon_decay_attn_step, q, k, v, log_decay, S, slots, fresh,
                         scale, o)
    lib = block._lib or block._library()
    dt = _dtype(q, "q")
    if q.dim() != 3 or not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError("q and k must be [N,H,m] and v [N,H,dv]")
    N, H, m = q.shape
    dv, dev = v.shape[2], q.device
    _rows(q, "q", dt, q.shape, dev)
    _rows(k, "k", dt, q.shape, dev)
    _rows(v, "v", dt, (N, H, dv), dev)
    _dense(log_decay, "log_decay", torch.float32, (H,), dev)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be a pool of states, [pool,H,m,dv]")
    pool = S.shape[0]
    if slots is None and pool != N:
        raise ValueError("S must hold one state a row where no slots are given")
    _dense(S, "S", torch.float32, (pool, H, m, dv), dev)
    _dense(slots, "slots", torch.int32, (N,), dev)
    _dense(fresh, "fresh", torch.uint8, (N,), dev)
    o = block._empty((N, H, dv), dt, dev) if o is None else _dense(o, "o", dt, (N, H, dv), dev)
    s, t, u = q.stride(), k.stride(), v.stride()
    rc = lib.falcon_decay_attn_step(
        _decay_shape(N, H, 1, m, dv, _DTYPE[dt],
                     _default_scale(m) if scale is None else float(scale)),
        q.data_ptr(), _strides(s[0], s[1], 0), k.data_ptr(), _strides(t[0], t[1], 0),
        v.data_ptr(), _strides(u[0], u[1], 0), log_decay.data_ptr(), S.data_ptr(), pool,
        _at(slots), _at(fresh), o.data_ptr(), block._raw_stream(dev.index))
    _check(rc, "falcon_decay_attn_step")
    return o


def _lines(t):
    """Strides of [B,T,D]."""
    if t is None:
        return None
    s = t.stride()
    return _strides(s[0], 0, s[1])


def _blocks(t):
    """Strides of [B,T,m] or [B,H,T,m]."""
    return None if t is None else _heads(t) if t.dim() == 4 else _lines(t)


def _norm_setup(h, first, name, gate, eps):
    """(shape of the rows, B, H, T, m, dtype, device) by h, or by `first` where h is None."""
    dt = _dtype(first if h is None else h, name if h is None else "h")
    if gate not in _GATE:
        raise ValueError(f"gate must be one of {sorted(_GATE)}")
    t = first if h is None else h
    if t.dim() == 3:
        (B, T, m), H = t.shape, 1
    elif t.dim() == 4 and h is not None:
        B, H, T, m = t.shape
    else:
        raise ValueError(f"{'h' if h is not None else name} must be [B,T,m]"
                         + (" or [B,H,T,m]" if h is not None else ""))
    if h is not None:
        _rows(h, "h", dt, h.shape, h.device)
    return (B, H, T, m, _DTYPE[dt], _GATE[gate], float(eps)), (B, T, H * m), dt, t.device


def _norm_params(D, dev, **params):
    for name, p in params.items():
        if p is not None:
            _dense(p, name, torch.float32, (D,), dev)


def falcon_gated_norm_fwd(h, weight=None, z=None, gate="silu", scale=None, x=None,
                          next_weight=None, lengths=None, eps=1e-6, out=None, next_out=None,
                          stream=None):
    """The norm behind a block with its gate, scale and residual, and the norm before the
    next block: out = x + scale act(z) norm(h) weight, next = norm(out) next_weight, norm
    over each head of h and over all channels of out.  h [B,T,m] or [B,H,T,m] (bf16 or
    fp32, any strides; H*m at most 8192); z, x [B,T,H*m]; weight, scale, next_weight
    [H*m] fp32; gate "silu", "sigmoid" or "identity".  Everything but h may be None; h
    may be where x and next_weight are given: next is then the norm before the first
    block, and out is x.  Returns (out, next), next None without next_weight; ``out`` may
    be x."""
    if stream is not None:
        return elsewhere(stream, falcon_gated_norm_fwd, h, weight, z, gate, scale, x,
                         next_weight, lengths, eps, out, next_out)
    lib = block._lib or block._library()
    if h is None and (x is None or next_weight is None or weight is not None or z is not None
                      or scale is not None or out is not None):
        raise ValueError("without h there are x and next_weight only")
    if next_out is not None and next_weight is None:
        raise ValueError("next_out needs next_weight")
    fields, row, dt, dev = _norm_setup(h, x, "x", gate, eps)
    for name, t in (("z", z), ("x", x)):
        if t is not None:
            _rows(t, name, dt, row, dev)
    _norm_params(row[2], dev, weight=weight, scale=scale, next_weight=next_weight)
    _dense(lengths, "lengths", torch.int32, row[:1], dev)
    if h is not None:
        out = block._empty(row, dt, dev) if out is None else _rows(out, "out", dt, row, dev)
    if next_weight is not None:
        next_out = block._empty(row, dt, dev) if next_out is None else \
            _rows(next_out, "next_out", dt, row, dev)
    rc = lib.falcon_gated_norm_fwd(
        _norm_shape(*fields), _at(h), _blocks(h), _at(weight), _at(z), _lines(z), _at(scale),
        _at(x), _lines(x), _at(next_weight), _at(lengths), _at(out), _lines(out), _at(next_out),
        _lines(next_out), block._raw_stream(dev.index))
    _check(rc, "falcon_gated_norm_fwd")
    return x if h is None else out, next_out


def falcon_gated_norm_bwd(h, dout, dnext=None, out=None, weight=None, z=None, gate="silu",
                          scale=None, residual=True, next_weight=None, lengths=None, eps=1e-6,
                          grads=None, workspace=None, stream=None):
    """Gradients of <dout, out> + <dnext, next> of falcon_gated_norm_fwd.  ``out`` is the
    stored output (x where h is None), needed with next_weight; dout may be None where
    dnext is given; ``residual`` says whether x was.  Returns a dict with dx, dh, dz
    (dense, h's type, dh of h's shape) and dweight, dscale, dnext_weight (fp32); those of
    what was not given are None.  ``grads`` may pass preallocated outputs of those that
    there are."""
    if stream is not None:
        return elsewhere(stream, falcon_gated_norm_bwd, h, dout, dnext, out, weight, z, gate,
                         scale, residual, next_weight, lengths, eps, grads, workspace)
    lib = block._lib or block._library()
    if h is None and (weight is not None or z is not None or scale is not None):
        raise ValueError("without h there are out, dout, dnext and next_weight only")
    if next_weight is None:
        if h is None or dnext is not None:
            raise ValueError("dnext, and a call without h, need next_weight")
        out = None
    elif out is None or dnext is None:
        raise ValueError("next_weight needs out and dnext")
    if dout is None and dnext is None:
        raise ValueError("one of dout and dnext is needed")
    fields, row, dt, dev = _norm_setup(h, out, "out", gate, eps)
    for name, t in (("z", z), ("out", out), ("dout", dout), ("dnext", dnext)):
        if t is not None:
            _rows(t, name, dt, row, dev)
    _norm_params(row[2], dev, weight=weight, scale=scale, next_weight=next_weight)
    _dense(lengths, "lengths", torch.int32, row[:1], dev)
    g = {} if grads is None else grads
    # each result with what it is the gradient of; `grads` may hold the None of an earlier call
    given = dict(dx=residual or h is None, dh=h is not None, dz=z is not None,
                 dweight=weight is not None, dscale=scale is not None,
                 dnext_weight=next_weight is not None)
    for name in g:
        if g[name] is not None and not given.get(name, True):
            raise ValueError(f"grads has {name}, whose argument was not given")
    for name, on in given.items():
        if not on:
            g[name] = None
        elif name in ("dx", "dh", "dz"):
            shape = h.shape if name == "dh" else row
            g[name] = block._empty(shape, dt, dev) if g.get(name) is None else \
                _rows(g[name], name, dt, shape, dev)
        else:
            g[name] = block._empty((row[2],), torch.float32, dev) if g.get(name) is None else \
                _dense(g[name], name, torch.float32, (row[2],), dev)
    workspace, have = block._workspace(_need("falcon_gated_norm_bwd_workspace_bytes",
                                             _norm_shape, *fields), workspace, dev)
    rc = lib.falcon_gated_norm_bwd(
        _norm_shape(*fields), _at(h), _blocks(h), _at(weight), _at(z), _lines(z), _at(scale),
        _at(out), _lines(out), _at(next_weight), _at(lengths), _at(dout), _lines(dout),
        _at(dnext), _lines(dnext), _at(g["dx"]), _lines(g["dx"]), _at(g["dh"]), _blocks(g["dh"]),
        _at(g["dz"]), _lines(g["dz"]), _at(g["dweight"]), _at(g["dscale"]),
        _at(g["dnext_weight"]), _at(workspace), have, block._raw_stream(dev.index))
    _check(rc, "falcon_gated_norm_bwd")
    return g
