"""Python front end of the sequence-mixer operators of libtitansmem: the short
causal convolution, the selective state-space scan and the group norm with an
activation (formulas: include/titansmem.h).

Token tensors are [B, H, T, d] (batch, head, token, channel) CUDA tensors,
float32 or bfloat16, with contiguous channels and any other strides: a
[B, T, H, d] tensor is passed as x.transpose(1, 2), a slice of a projection as
it is. Parameters, states and statistics are contiguous float32. Every function
runs on `stream` (default: the current stream of the tensors' device) and takes
its outputs and workspace from torch unless they are given. Gradients are calls
of their own (`*_backward`): outputs never require gradients, whatever the inputs do.

`lengths` ([B] int32 on the device) gives the tokens of each sequence of a
padded batch: rows behind them are not read, and are zero in outputs that are
made here (a given output keeps what it held there).
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _native as N

_F32, _BF16, _I32 = torch.float32, torch.bfloat16, torch.int32
_TYPES = {_F32: N.TM_F32, _BF16: N.TM_BF16}
_ACTS = {"silu": N.TM_ACT_SILU, "none": N.TM_ACT_NONE, None: N.TM_ACT_NONE}
_OVER = {"token": N.TM_NORM_TOKEN, "sequence": N.TM_NORM_SEQUENCE}


# A decode step is a few microseconds on the GPU, and its call should not take
# longer on the host: each entry point tests its tensors in one expression and
# only asks _check for the reason when that fails; tables of strides are packed
# bytes; workspace sizes are remembered by the problem's sizes.

def _dtype_code(name, t):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _named(table, name, value):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(map(str, table))}, got {value!r}")
    return table[value]


def _need(**tensors):
    """Raises for the first that is not a tensor."""
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor, got {type(t).__name__}")


def _check(device, **tensors):
    """name=(tensor or None, shape, dtype, strided): raises for the first that has
    another shape, type or device, or that is not contiguous (its channels, if
    `strided`)."""
    for name, (t, shape, dtype, strided) in tensors.items():
        if t is None:
            continue
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if t.device != device:
            raise ValueError(f"{name} must be on {device}, got {t.device}")
        if t.is_contiguous():
            continue
        if not strided:
            raise ValueError(f"{name} must be contiguous")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            raise ValueError(f"the channels of {name} must be contiguous")


def _par(t, shape, dev):
    """A float32 parameter or state as the library wants it (or absent)."""
    return t is None or (t.dtype is _F32 and t.get_device() == dev and t.shape == shape and t.is_contiguous())


def _len(t, B, dev):
    return t is None or (t.dtype is _I32 and t.get_device() == dev and t.shape == (B,) and t.is_contiguous())


def _tok(t, shape, kind, dev):
    """A token tensor (strides are looked at by _strides), or absent."""
    return t is None or (t.dtype is kind and t.get_device() == dev and t.shape == shape)


def _shape(name, t, n):
    shape = t.shape
    if len(shape) != n or 0 in shape:
        raise ValueError(f"{name} must be a non-empty tensor of {n} dimensions, got shape {tuple(shape)}")
    return shape


def _p(t):
    return None if t is None else t.data_ptr()


_PACK = {n: struct.Struct(f"{3 * n}q").pack for n in range(1, 10)}


def _strides(names, *tensors):
    """The library's table of (batch, head, token) strides; None when every tensor
    is contiguous. Tensors of single tokens have no token stride."""
    table, plain = [], True
    for i, t in enumerate(tensors):
        if t is None:
            table += (0, 0, 0)
            continue
        s = t.stride()
        if s[-1] != 1 and t.shape[-1] > 1:
            raise ValueError(f"the channels of {names.split()[i]} must be contiguous")
        if plain and not t.is_contiguous():
            plain = False
        table += s[:3] if len(s) == 4 else (s[0], s[1], 0)
    return None if plain else _PACK[len(tensors)](*table)


def _elsewhere(fn, stream, x, args, kwargs):
    """fn on another device than the current one, or on a given stream: with both
    made current, so that what fn allocates belongs to them, and the allocator
    told that the stream uses the caller's tensors."""
    _need(x=x)
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    with torch.cuda.device(x.device):
        if stream is None:
            return fn(x, *args, **kwargs)
        if stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, x on {x.device}")
        with torch.cuda.stream(stream):
            for t in (x, *args, *kwargs.values()):
                if isinstance(t, torch.Tensor) and t.is_cuda:
                    t.record_stream(stream)
            return fn(x, *args, **kwargs)


def _here(x, stream):
    """Whether x's device is the current one and the call goes to its current stream."""
    return stream is None and isinstance(x, _Tensor) and x.is_cuda and x.get_device() == _current_device()


_Tensor = torch.Tensor
# the current device and stream without the checks and the Stream object around them, where torch offers that
# (a CUDA tensor is there: CUDA is initialised)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


@functools.lru_cache(maxsize=4096)
def _workspace_size(fn, *sizes):
    n = ctypes.c_size_t()
    N.check(getattr(N.load(), fn)(*sizes, ctypes.byref(n)), fn)
    return n.value


def _like(x, dtype=None):
    """An output for x: in x's layout where that is dense, with contiguous channels
    always (x may repeat rows, or be overlapping windows of one signal)."""
    out = torch.empty_like(x) if dtype is None else torch.empty_like(x, dtype=dtype)
    if not x.is_contiguous() and out.stride(-1) != 1 and x.shape[-1] > 1:
        out = torch.empty_like(out, memory_format=torch.contiguous_format)
    return out


def _workspace(given, x, fn, *sizes):
    """(tensor or None, bytes)"""
    if given is None:
        n = _workspace_size(fn, *sizes)
        return (x.new_empty(n, dtype=torch.uint8) if n else None), n
    if given.dtype != torch.uint8 or not given.is_contiguous() or given.device != x.device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {x.device}")
    return given, given.numel()


def _conv_check(x, shape, filt, bias, hist, lengths, token2, tail):
    """Checks what the three convolution calls share; the width."""
    if filt is None:
        _need(filt=filt)
    w, dev, kind = filt.shape[-1], x.get_device(), x.dtype
    B, H, d = shape[0], shape[1], shape[-1]
    past = (B, H, w - 1, d)
    if not (_par(filt, (H, d, w), dev) and _par(bias, (H, d), dev) and _tok(token2, shape, kind, dev) and
            _tok(hist, past, kind, dev) and (hist is None or hist.is_contiguous()) and
            _tok(tail, past, kind, dev) and (tail is None or tail.is_contiguous()) and _len(lengths, B, dev)):
        _check(x.device, filt=(filt, (H, d, w), _F32, False), bias=(bias, (H, d), _F32, False),
               hist=(hist, past, kind, False), lengths=(lengths, (B,), _I32, False),
               **{"out or dy": (token2, shape, kind, True), "tail or its gradient": (tail, past, kind, False)})
    return w


def short_conv(x, filt, bias=None, *, hist=None, lengths=None, act="silu", out=None, tail=None, stream=None):
    """Depthwise causal convolution act(bias + sum_j filt[..., j] x[t - j]).

    x [B, H, T, d]; filt [H, d, width] (width <= 8) and bias [H, d] float32; hist
    [B, H, width-1, d], the tokens before the call. Returns (y, tail): tail, like
    hist, holds the last width-1 tokens, the history of the next call."""
    if not _here(x, stream):
        return _elsewhere(short_conv, stream, x, (filt, bias),
                          dict(hist=hist, lengths=lengths, act=act, out=out, tail=tail))
    shape = B, H, T, d = _shape("x", x, 4)
    code = _dtype_code("x", x)
    w = _conv_check(x, shape, filt, bias, hist, lengths, out, tail)
    fresh = out is None                                  # then rows behind the ends are written as zeros
    if fresh:
        out = _like(x)
    if tail is None:
        tail = x.new_empty((B, H, w - 1, d))
    N.check(N.load().tm_conv(B, H, T, d, w, code, _named(_ACTS, "act", act), fresh, x.data_ptr(), filt.data_ptr(), _p(bias),
                             _p(hist), _p(lengths), out.data_ptr(), tail.data_ptr(), _strides("x out", x, out),
                             _stream_of(x.get_device())), "tm_conv")
    return out, tail


def short_conv_backward(x, filt, dy, bias=None, *, hist=None, lengths=None, act="silu", dtail=None, workspace=None,
                        stream=None):
    """Gradients of sum <dy, y> + <dtail, tail> for short_conv of these inputs:
    a dict of dx, dfilt, dbias (with a bias) and dhist (with a history)."""
    if not _here(x, stream):
        return _elsewhere(short_conv_backward, stream, x, (filt, dy, bias),
                          dict(hist=hist, lengths=lengths, act=act, dtail=dtail, workspace=workspace))
    shape = B, H, T, d = _shape("x", x, 4)
    code = _dtype_code("x", x)
    if dy is None:
        _need(dy=dy)
    w = _conv_check(x, shape, filt, bias, hist, lengths, dy, dtail)
    ws, n = _workspace(workspace, x, "tm_conv_backward_workspace_size", B, H, T, d, w, code)
    out = {"dx": _like(x), "dfilt": torch.empty_like(filt)}
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    if hist is not None:
        out["dhist"] = torch.empty_like(hist)
    N.check(N.load().tm_conv_backward(
        B, H, T, d, w, code, _named(_ACTS, "act", act), _p(x), _p(filt), _p(bias), _p(hist), _p(lengths), _p(dy),
        _p(dtail), _p(out["dx"]), _p(out["dfilt"]), _p(out.get("dbias")), _p(out.get("dhist")),
        _strides("x dy dx", x, dy, out["dx"]), _p(ws), n, _stream_of(x.get_device())), "tm_conv_backward")
    return out


def short_conv_step(x, hist, filt, bias=None, *, act="silu", out=None, stream=None):
    """short_conv of one token per sequence, x [B, H, d]: returns y and moves
    hist [B, H, width-1, d] on in place."""
    if not _here(x, stream):
        return _elsewhere(short_conv_step, stream, x, (hist, filt, bias), dict(act=act, out=out))
    shape = B, H, d = _shape("x", x, 3)
    code = _dtype_code("x", x)
    if hist is None:
        _need(hist=hist)
    w = _conv_check(x, shape, filt, bias, hist, None, out, None)
    if out is None:
        out = x.new_empty(shape)
    N.check(N.load().tm_conv_step(B, H, d, w, code, _named(_ACTS, "act", act), x.data_ptr(), filt.data_ptr(), _p(bias),
                                  hist.data_ptr(), out.data_ptr(), _strides("x out", x, out), _stream_of(x.get_device())),
            "tm_conv_step")
    return out


def _scan_sizes(x, shape, dt, A, Bm, Cm, D, z, dt_bias, state, state2, token2, lengths):
    """Checks what the three scan calls share; (G, N)."""
    if dt is None or A is None or Bm is None or Cm is None:
        _need(dt=dt, A=A, Bm=Bm, Cm=Cm)
    kind, dev = x.dtype, x.get_device()
    B, H, d = shape[0], shape[1], shape[-1]
    if Bm.dim() != len(shape) or A.dim() != 3:
        raise ValueError(f"A must be [H, d, N] and Bm [B, G, {'T, ' if len(shape) == 4 else ''}N], got "
                         f"{tuple(A.shape)} and {tuple(Bm.shape)}")
    G, n = Bm.shape[1], A.shape[-1]
    if G == 0 or H % G:
        raise ValueError(f"the {G} groups of Bm must divide the {H} heads")
    group = (B, G, shape[2], n) if len(shape) == 4 else (B, G, n)
    par, held = (H, d), (B, H, d, n)
    if not (_tok(dt, shape, kind, dev) and _tok(z, shape, kind, dev) and _tok(token2, shape, kind, dev) and
            _tok(Bm, group, kind, dev) and _tok(Cm, group, kind, dev) and _par(A, (H, d, n), dev) and
            _par(D, par, dev) and _par(dt_bias, par, dev) and _par(state, held, dev) and _par(state2, held, dev) and
            _len(lengths, B, dev)):
        _check(x.device, dt=(dt, shape, kind, True), A=(A, (H, d, n), _F32, False), Bm=(Bm, group, kind, True),
               Cm=(Cm, group, kind, True), D=(D, par, _F32, False), z=(z, shape, kind, True),
               dt_bias=(dt_bias, par, _F32, False), state=(state, held, _F32, False),
               lengths=(lengths, (B,), _I32, False), **{"out or dy": (token2, shape, kind, True),
                                                       "state_end or its gradient": (state2, held, _F32, False)})
    return G, n


def selective_scan(x, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, state=None, lengths=None, softplus=True,
                   out=None, state_end=None, workspace=None, stream=None):
    """Selective state-space scan: h = exp(e A) h + e x Bm, y = (Cm h + D x) silu(z),
    e = softplus(dt + dt_bias).

    x, dt, z [B, H, T, d]; Bm, Cm [B, G, T, N] (G divides H); A [H, d, N], D and
    dt_bias [H, d], state [B, H, d, N] float32. Returns (y, state_end); pass
    state_end=state to update in place."""
    if not _here(x, stream):
        return _elsewhere(selective_scan, stream, x, (dt, A, Bm, Cm),
                          dict(D=D, z=z, dt_bias=dt_bias, state=state, lengths=lengths, softplus=softplus, out=out,
                               state_end=state_end, workspace=workspace))
    shape = B, H, T, d = _shape("x", x, 4)
    code = _dtype_code("x", x)
    G, n = _scan_sizes(x, shape, dt, A, Bm, Cm, D, z, dt_bias, state, state_end, out, lengths)
    fresh = out is None
    if fresh:
        out = _like(x)
    if state_end is None:
        state_end = A.new_empty((B, H, d, n))
    ws, nb = _workspace(workspace, x, "tm_scan_workspace_size", B, H, G, T, d, n, code)
    N.check(N.load().tm_scan(B, H, G, T, d, n, code, bool(softplus), fresh, x.data_ptr(), dt.data_ptr(), A.data_ptr(),
                             Bm.data_ptr(), Cm.data_ptr(), _p(D), _p(z), _p(dt_bias), _p(state), _p(lengths),
                             out.data_ptr(), state_end.data_ptr(),
                             _strides("x dt Bm Cm z out", x, dt, Bm, Cm, z, out), _p(ws), nb,
                             _stream_of(x.get_device())), "tm_scan")
    return out, state_end


def selective_scan_backward(x, dt, A, Bm, Cm, dy, *, D=None, z=None, dt_bias=None, state=None, dstate_end=None,
                            lengths=None, softplus=True, workspace=None, stream=None):
    """Gradients of sum <dy, y> + <dstate_end, state_end> for selective_scan of
    these inputs: a dict of dx, ddt, dA, dB, dC and, where the input is given,
    dD, dz, ddt_bias and dstate."""
    if not _here(x, stream):
        return _elsewhere(selective_scan_backward, stream, x, (dt, A, Bm, Cm, dy),
                          dict(D=D, z=z, dt_bias=dt_bias, state=state, dstate_end=dstate_end, lengths=lengths,
                               softplus=softplus, workspace=workspace))
    shape = B, H, T, d = _shape("x", x, 4)
    code = _dtype_code("x", x)
    if dy is None:
        _need(dy=dy)
    G, n = _scan_sizes(x, shape, dt, A, Bm, Cm, D, z, dt_bias, state, dstate_end, dy, lengths)
    ws, nb = _workspace(workspace, x, "tm_scan_backward_workspace_size", B, H, G, T, d, n, code)
    out = {"dx": _like(x), "ddt": _like(dt), "dA": torch.empty_like(A),
           "dB": x.new_empty((B, G, T, n)), "dC": x.new_empty((B, G, T, n))}
    if z is not None:
        out["dz"] = _like(z)
    for name, t in (("dD", D), ("ddt_bias", dt_bias), ("dstate", state)):
        if t is not None:
            out[name] = torch.empty_like(t)
    N.check(N.load().tm_scan_backward(
        B, H, G, T, d, n, code, bool(softplus), _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(z), _p(dt_bias),
        _p(state), _p(lengths), _p(dy), _p(dstate_end), _p(out["dx"]), _p(out["ddt"]), _p(out["dA"]), _p(out["dB"]),
        _p(out["dC"]), _p(out.get("dD")), _p(out.get("dz")), _p(out.get("ddt_bias")), _p(out.get("dstate")),
        _strides("x dt Bm Cm z dy dx ddt dz", x, dt, Bm, Cm, z, dy, out["dx"], out["ddt"], out.get("dz")), _p(ws), nb,
        _stream_of(x.get_device())), "tm_scan_backward")
    return out


def selective_scan_step(x, dt, A, Bm, Cm, state, *, D=None, z=None, dt_bias=None, softplus=True, out=None,
                        stream=None):
    """selective_scan of one token per sequence, x, dt, z [B, H, d], Bm, Cm
    [B, G, N]: returns y and updates state [B, H, d, N] in place."""
    if not _here(x, stream):
        return _elsewhere(selective_scan_step, stream, x, (dt, A, Bm, Cm, state),
                          dict(D=D, z=z, dt_bias=dt_bias, softplus=softplus, out=out))
    shape = B, H, d = _shape("x", x, 3)
    code = _dtype_code("x", x)
    if state is None:
        _need(state=state)
    G, n = _scan_sizes(x, shape, dt, A, Bm, Cm, D, z, dt_bias, state, None, out, None)
    if out is None:
        out = x.new_empty(shape)
    N.check(N.load().tm_scan_step(B, H, G, d, n, code, bool(softplus), x.data_ptr(), dt.data_ptr(), A.data_ptr(),
                                  Bm.data_ptr(), Cm.data_ptr(), _p(D), _p(z), _p(dt_bias), state.data_ptr(),
                                  out.data_ptr(), _strides("x dt Bm Cm z out", x, dt, Bm, Cm, z, out),
                                  _stream_of(x.get_device())), "tm_scan_step")
    return out


def _norm_check(x, shape, weight, bias, lengths, stats, over, token2, kind):
    """Checks what the two norm calls share; the shape of stats."""
    B, H, T, d = shape
    dev, par = x.get_device(), (H, d)
    kept = (B, H, T, 2) if over == "token" else (B, H, 2)
    if not (_par(weight, par, dev) and _par(bias, par, dev) and _par(stats, kept, dev) and
            _tok(token2, shape, kind, dev) and _len(lengths, B, dev)):
        _check(x.device, weight=(weight, par, _F32, False), bias=(bias, par, _F32, False),
               lengths=(lengths, (B,), _I32, False), stats=(stats, kept, _F32, False),
               **{"out or dy": (token2, shape, kind, True)})
    return kept


def group_norm(x, weight=None, bias=None, *, over="token", act=None, eps=1e-5, lengths=None, dtype=None, out=None,
               stats=None, workspace=None, stream=None):
    """act(weight (x - mean) / sqrt(var + eps) + bias), the statistics of each
    head over the channels of one token (over="token") or of the whole sequence
    (over="sequence": group norm of a channels-last [B, T, H * d] tensor, passed as
    x.view(B, T, H, d).transpose(1, 2)). weight, bias [H, d] float32; `dtype`: the
    output's type (default: x's). Returns (y, stats) with stats = (mean, 1 /
    sqrt(var + eps)) [B, H, T, 2] or [B, H, 2] for group_norm_backward."""
    if not _here(x, stream):
        return _elsewhere(group_norm, stream, x, (weight, bias),
                          dict(over=over, act=act, eps=eps, lengths=lengths, dtype=dtype, out=out, stats=stats,
                               workspace=workspace))
    shape = B, H, T, d = _shape("x", x, 4)
    kind = out.dtype if out is not None else dtype or x.dtype
    if dtype is not None and kind != dtype:
        raise TypeError(f"out must be {dtype}, got {kind}")
    if kind not in _TYPES:
        raise TypeError(f"the output must be float32 or bfloat16, got {kind}")
    code, where = _dtype_code("x", x), _named(_OVER, "over", over)
    kept = _norm_check(x, shape, weight, bias, lengths, stats, over, out, kind)
    fresh = out is None
    if fresh:
        out = _like(x, kind)
    if stats is None:
        # rows behind the ends: written with those of y, so zeroed here when those of a given y are left alone
        stats = (x.new_empty if lengths is None or fresh else x.new_zeros)(kept, dtype=_F32)
    ws, n = _workspace(workspace, x, "tm_group_norm_workspace_size", B, H, T, d, where, 0)
    N.check(N.load().tm_group_norm(B, H, T, d, where, code, _TYPES[kind], _named(_ACTS, "act", act), fresh, float(eps),
                                   x.data_ptr(), _p(weight), _p(bias), _p(lengths), out.data_ptr(), stats.data_ptr(),
                                   _strides("x out", x, out), _p(ws), n, _stream_of(x.get_device())), "tm_group_norm")
    return out, stats


def group_norm_backward(x, dy, stats, weight=None, bias=None, *, over="token", act=None, lengths=None, workspace=None,
                        stream=None):
    """Gradients of sum <dy, y> for group_norm of these inputs and the stats it
    returned: a dict of dx and, where the parameter is given, dweight and dbias."""
    if not _here(x, stream):
        return _elsewhere(group_norm_backward, stream, x, (dy, stats, weight, bias),
                          dict(over=over, act=act, lengths=lengths, workspace=workspace))
    shape = B, H, T, d = _shape("x", x, 4)
    if dy is None or stats is None:
        _need(dy=dy, stats=stats)
    code, where, out_code = _dtype_code("x", x), _named(_OVER, "over", over), _dtype_code("dy", dy)
    _norm_check(x, shape, weight, bias, lengths, stats, over, dy, dy.dtype)
    ws, n = _workspace(workspace, x, "tm_group_norm_workspace_size", B, H, T, d, where, 1)
    out = {"dx": _like(x)}
    if weight is not None:
        out["dweight"] = torch.empty_like(weight)
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    N.check(N.load().tm_group_norm_backward(
        B, H, T, d, where, code, out_code, _named(_ACTS, "act", act), _p(x), _p(dy), _p(stats), _p(weight), _p(bias),
        _p(lengths), _p(out["dx"]), _p(out.get("dweight")), _p(out.get("dbias")), _strides("x dy dx", x, dy, out["dx"]),
        _p(ws), n, _stream_of(x.get_device())), "tm_group_norm_backward")
    return out
