"""Python front end of the sequence-mixer operators of libtitansmem: the short
causal convolution, the selective state-space scan and the group norm with an
activation (formulas: include/titansmem.h).

Token tensors are [B, H, T, d] (batch, head, token, channel) CUDA tensors,
float32 or bfloat16, with contiguous channels and any other strides: a
[B, T, H, d] tensor is passed as x.transpose(1, 2), a slice of a projection as
it is. Parameters, states and statistics are contiguous float32. Every function
runs on `stream` (default: the current stream of the tensors' device) and takes
its outputs and workspace from torch unless they are given.

`lengths` ([B] int32 on the device) gives the tokens of each sequence of a
padded batch: rows behind them are not read, and are zero in outputs that are
made here (a given output keeps what it held there).
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _native as N

_TYPES = {torch.float32: N.TM_F32, torch.bfloat16: N.TM_BF16}
_ACTS = {"silu": N.TM_ACT_SILU, "none": N.TM_ACT_NONE, None: N.TM_ACT_NONE}
_OVER = {"token": N.TM_NORM_TOKEN, "sequence": N.TM_NORM_SEQUENCE}


def _dtype_code(name, t):
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    return code


def _named(table, name, value):
    if value not in table:
        raise ValueError(f"{name} must be one of {sorted(map(str, table))}, got {value!r}")
    return table[value]


def _check(device, **tensors):
    """name=(tensor or None, shape, dtype): the right shape, type and device,
    contiguous in the last dimension (token tensors) or altogether."""
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


def _rank(name, t, n):
    if t.dim() != n or t.numel() == 0:
        raise ValueError(f"{name} must be a non-empty tensor of {n} dimensions, got shape {tuple(t.shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")


def _p(t):
    return None if t is None else t.data_ptr()


def _strides(*tensors):
    """The library's table of (batch, head, token) strides; None when every
    tensor is contiguous. Tensors of single tokens have no token stride."""
    if all(t is None or t.is_contiguous() for t in tensors):
        return None
    table = []
    for t in tensors:
        if t is None:
            table += (0, 0, 0)
        else:
            s = t.stride()
            table += (s[0], s[1], s[2] if len(s) == 4 else 0)
    return (ctypes.c_longlong * len(table))(*table)


@contextlib.contextmanager
def _on_stream(device, stream, used):
    """Makes `stream` current, so that what is allocated belongs to it, and tells
    the allocator that it uses the caller's tensors."""
    with torch.cuda.device(device), torch.cuda.stream(stream):
        for t in used:
            if t is not None:
                t.record_stream(stream)
        yield


def _placed(fn):
    """Runs fn on its tensors' device and on the given stream."""
    def call(x, *args, stream=None, **kwargs):
        if not isinstance(x, torch.Tensor) or not x.is_cuda:
            raise ValueError("x must be a CUDA tensor")
        index = x.device.index
        if stream is None:
            if index == torch.cuda.current_device():
                return fn(x, *args, _stream=torch.cuda.current_stream(index).cuda_stream, **kwargs)
            with torch.cuda.device(index):
                return fn(x, *args, _stream=torch.cuda.current_stream(index).cuda_stream, **kwargs)
        if stream.device.index != index:
            raise ValueError(f"stream is on {stream.device}, x on {x.device}")
        used = [t for t in (x, *args, *kwargs.values()) if isinstance(t, torch.Tensor)]
        with _on_stream(x.device, stream, used):
            return fn(x, *args, _stream=stream.cuda_stream, **kwargs)
    call.__name__, call.__doc__, call.__wrapped__ = fn.__name__, fn.__doc__, fn
    return call


def _fresh(like, lengths, dtype=None):
    """An output: zeros where rows behind a sequence's end are not written."""
    return torch.empty_like(like, dtype=dtype) if lengths is None else torch.zeros_like(like, dtype=dtype)


def _workspace(given, size_fn, *args, device):
    n = ctypes.c_size_t()
    N.check(getattr(N.load(), size_fn)(*args, ctypes.byref(n)), size_fn)
    if given is None:
        return (None, 0) if n.value == 0 else _pair(torch.empty(n.value, dtype=torch.uint8, device=device))
    if given.dtype != torch.uint8 or not given.is_contiguous() or given.device != device:
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    return _pair(given)


def _pair(ws):
    return ws, ws.numel()


@_placed
def short_conv(x, filt, bias=None, *, hist=None, lengths=None, act="silu", out=None, tail=None, _stream=None):
    """Depthwise causal convolution act(bias + sum_j filt[..., j] x[t - j]).

    x [B, H, T, d]; filt [H, d, width] (width <= 8) and bias [H, d] float32; hist
    [B, H, width-1, d], the tokens before the call. Returns (y, tail): tail, like
    hist, holds the last width-1 tokens, the history of the next call."""
    _rank("x", x, 4)
    B, H, T, d = x.shape
    w, dev, dt = filt.shape[-1], x.device, x.dtype
    code = _dtype_code("x", x)
    _check(dev, x=(x, (B, H, T, d), dt, True), filt=(filt, (H, d, w), torch.float32, False),
           bias=(bias, (H, d), torch.float32, False), hist=(hist, (B, H, w - 1, d), dt, False),
           lengths=(lengths, (B,), torch.int32, False), out=(out, (B, H, T, d), dt, True),
           tail=(tail, (B, H, w - 1, d), dt, False))
    if out is None:
        out = _fresh(x, lengths)
    if tail is None:
        tail = torch.empty((B, H, w - 1, d), dtype=dt, device=dev)
    N.check(N.load().tm_conv(B, H, T, d, w, code, _named(_ACTS, "act", act), _p(x), _p(filt), _p(bias), _p(hist),
                             _p(lengths), _p(out), _p(tail), _strides(x, out), _stream), "tm_conv")
    return out, tail


@_placed
def short_conv_backward(x, filt, dy, bias=None, *, hist=None, lengths=None, act="silu", dtail=None, workspace=None,
                        _stream=None):
    """Gradients of sum <dy, y> + <dtail, tail> for short_conv of these inputs:
    a dict of dx, dfilt, dbias (with a bias) and dhist (with a history)."""
    _rank("x", x, 4)
    B, H, T, d = x.shape
    w, dev, dt = filt.shape[-1], x.device, x.dtype
    code = _dtype_code("x", x)
    _check(dev, x=(x, (B, H, T, d), dt, True), filt=(filt, (H, d, w), torch.float32, False),
           dy=(dy, (B, H, T, d), dt, True), bias=(bias, (H, d), torch.float32, False),
           hist=(hist, (B, H, w - 1, d), dt, False), lengths=(lengths, (B,), torch.int32, False),
           dtail=(dtail, (B, H, w - 1, d), dt, False))
    ws, n = _workspace(workspace, "tm_conv_backward_workspace_size", B, H, T, d, w, code, device=dev)
    out = {"dx": torch.empty_like(x), "dfilt": torch.empty_like(filt)}
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    if hist is not None:
        out["dhist"] = torch.empty_like(hist)
    N.check(N.load().tm_conv_backward(
        B, H, T, d, w, code, _named(_ACTS, "act", act), _p(x), _p(filt), _p(bias), _p(hist), _p(lengths), _p(dy),
        _p(dtail), _p(out["dx"]), _p(out["dfilt"]), _p(out.get("dbias")), _p(out.get("dhist")),
        _strides(x, dy, out["dx"]), _p(ws), n, _stream), "tm_conv_backward")
    return out


@_placed
def short_conv_step(x, hist, filt, bias=None, *, act="silu", out=None, _stream=None):
    """short_conv of one token per sequence, x [B, H, d]: returns y and moves
    hist [B, H, width-1, d] on in place."""
    _rank("x", x, 3)
    B, H, d = x.shape
    w, dev, dt = filt.shape[-1], x.device, x.dtype
    code = _dtype_code("x", x)
    _check(dev, x=(x, (B, H, d), dt, True), hist=(hist, (B, H, w - 1, d), dt, False),
           filt=(filt, (H, d, w), torch.float32, False), bias=(bias, (H, d), torch.float32, False),
           out=(out, (B, H, d), dt, True))
    if out is None:
        out = torch.empty((B, H, d), dtype=dt, device=dev)
    N.check(N.load().tm_conv_step(B, H, d, w, code, _named(_ACTS, "act", act), _p(x), _p(filt), _p(bias), _p(hist),
                                  _p(out), _strides(x, out), _stream), "tm_conv_step")
    return out


def _scan_check(x, dt, A, Bm, Cm, D, z, dt_bias, state, more):
    shape, dev, kind, f32 = x.shape, x.device, x.dtype, torch.float32
    B, H, d = shape[0], shape[1], shape[-1]
    if Bm.dim() != len(shape) or A.dim() != 3:
        raise ValueError(f"A must be [H, d, N] and Bm [B, G, {'T, ' if len(shape) == 4 else ''}N], got "
                         f"{tuple(A.shape)} and {tuple(Bm.shape)}")
    G, n = Bm.shape[1], A.shape[-1]
    if G == 0 or H % G:
        raise ValueError(f"the {G} groups of Bm must divide the {H} heads")
    group = (B, G, *shape[2:-1], n)
    _check(dev, x=(x, shape, kind, True), dt=(dt, shape, kind, True), A=(A, (H, d, n), f32, False),
           Bm=(Bm, group, kind, True), Cm=(Cm, group, kind, True), D=(D, (H, d), f32, False),
           z=(z, shape, kind, True), dt_bias=(dt_bias, (H, d), f32, False), state=(state, (B, H, d, n), f32, False),
           **more)
    return G, n


@_placed
def selective_scan(x, dt, A, Bm, Cm, *, D=None, z=None, dt_bias=None, state=None, lengths=None, softplus=True,
                   out=None, state_end=None, workspace=None, _stream=None):
    """Selective state-space scan: h = exp(e A) h + e x Bm, y = (Cm h + D x) silu(z),
    e = softplus(dt + dt_bias).

    x, dt, z [B, H, T, d]; Bm, Cm [B, G, T, N] (G divides H); A [H, d, N], D and
    dt_bias [H, d], state [B, H, d, N] float32. Returns (y, state_end); pass
    state_end=state to update in place."""
    _rank("x", x, 4)
    B, H, T, d = x.shape
    code = _dtype_code("x", x)
    G, n = _scan_check(x, dt, A, Bm, Cm, D, z, dt_bias, state, {"lengths": (lengths, (B,), torch.int32, False),
                                                               "out": (out, x.shape, x.dtype, True)})
    _check(x.device, state_end=(state_end, (B, H, d, n), torch.float32, False))
    if out is None:
        out = _fresh(x, lengths)
    if state_end is None:
        state_end = torch.empty((B, H, d, n), dtype=torch.float32, device=x.device)
    ws, nb = _workspace(workspace, "tm_scan_workspace_size", B, H, G, T, d, n, code, device=x.device)
    N.check(N.load().tm_scan(B, H, G, T, d, n, code, int(softplus), _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(z),
                             _p(dt_bias), _p(state), _p(lengths), _p(out), _p(state_end),
                             _strides(x, dt, Bm, Cm, z, out), _p(ws), nb, _stream), "tm_scan")
    return out, state_end


@_placed
def selective_scan_backward(x, dt, A, Bm, Cm, dy, *, D=None, z=None, dt_bias=None, state=None, dstate_end=None,
                            lengths=None, softplus=True, workspace=None, _stream=None):
    """Gradients of sum <dy, y> + <dstate_end, state_end> for selective_scan of
    these inputs: a dict of dx, ddt, dA, dB, dC and, where the input is given,
    dD, dz, ddt_bias and dstate."""
    _rank("x", x, 4)
    B, H, T, d = x.shape
    code = _dtype_code("x", x)
    G, n = _scan_check(x, dt, A, Bm, Cm, D, z, dt_bias, state, {"lengths": (lengths, (B,), torch.int32, False),
                                                               "dy": (dy, x.shape, x.dtype, True)})
    _check(x.device, dstate_end=(dstate_end, (B, H, d, n), torch.float32, False))
    ws, nb = _workspace(workspace, "tm_scan_backward_workspace_size", B, H, G, T, d, n, code, device=x.device)
    group = dict(dtype=x.dtype, device=x.device)
    out = {"dx": torch.empty_like(x), "ddt": torch.empty_like(dt), "dA": torch.empty_like(A),
           "dB": torch.empty((B, G, T, n), **group), "dC": torch.empty((B, G, T, n), **group)}
    for name, t in (("dD", D), ("dz", z), ("ddt_bias", dt_bias), ("dstate", state)):
        if t is not None:
            out[name] = torch.empty_like(t)
    N.check(N.load().tm_scan_backward(
        B, H, G, T, d, n, code, int(softplus), _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D), _p(z), _p(dt_bias),
        _p(state), _p(lengths), _p(dy), _p(dstate_end), _p(out["dx"]), _p(out["ddt"]), _p(out["dA"]), _p(out["dB"]),
        _p(out["dC"]), _p(out.get("dD")), _p(out.get("dz")), _p(out.get("ddt_bias")), _p(out.get("dstate")),
        _strides(x, dt, Bm, Cm, z, dy, out["dx"], out["ddt"], out.get("dz")), _p(ws), nb, _stream), "tm_scan_backward")
    return out


@_placed
def selective_scan_step(x, dt, A, Bm, Cm, state, *, D=None, z=None, dt_bias=None, softplus=True, out=None,
                        _stream=None):
    """selective_scan of one token per sequence, x, dt, z [B, H, d], Bm, Cm
    [B, G, N]: returns y and updates state [B, H, d, N] in place."""
    _rank("x", x, 3)
    B, H, d = x.shape
    code = _dtype_code("x", x)
    G, n = _scan_check(x, dt, A, Bm, Cm, D, z, dt_bias, state, {"out": (out, x.shape, x.dtype, True)})
    if out is None:
        out = torch.empty((B, H, d), dtype=x.dtype, device=x.device)
    N.check(N.load().tm_scan_step(B, H, G, d, n, code, int(softplus), _p(x), _p(dt), _p(A), _p(Bm), _p(Cm), _p(D),
                                  _p(z), _p(dt_bias), _p(state), _p(out), _strides(x, dt, Bm, Cm, z, out), _stream),
            "tm_scan_step")
    return out


def _norm_shapes(x, over):
    B, H, T, d = x.shape
    return (B, H, T, 2) if over == "token" else (B, H, 2)


@_placed
def group_norm(x, weight=None, bias=None, *, over="token", act=None, eps=1e-5, lengths=None, dtype=None, out=None,
               stats=None, workspace=None, _stream=None):
    """act(weight (x - mean) / sqrt(var + eps) + bias), the statistics of each
    head over the channels of one token (over="token") or of the whole sequence
    (over="sequence": group norm of a channels-last [B, T, H * d] tensor, passed as
    x.view(B, T, H, d).transpose(1, 2)). weight, bias [H, d] float32; `dtype`: the
    output's type (default: x's). Returns (y, stats) with stats = (mean, 1 /
    sqrt(var + eps)) [B, H, T, 2] or [B, H, 2] for group_norm_backward."""
    _rank("x", x, 4)
    B, H, T, d = x.shape
    dev = x.device
    kind = out.dtype if out is not None else dtype or x.dtype
    if dtype is not None and kind != dtype:
        raise TypeError(f"out must be {dtype}, got {kind}")
    code, where = _dtype_code("x", x), _named(_OVER, "over", over)
    if kind not in _TYPES:
        raise TypeError(f"the output must be float32 or bfloat16, got {kind}")
    _check(dev, x=(x, (B, H, T, d), x.dtype, True), weight=(weight, (H, d), torch.float32, False),
           bias=(bias, (H, d), torch.float32, False), lengths=(lengths, (B,), torch.int32, False),
           out=(out, (B, H, T, d), kind, True), stats=(stats, _norm_shapes(x, over), torch.float32, False))
    if out is None:
        out = _fresh(x, lengths, kind)
    if stats is None:
        make = torch.empty if lengths is None else torch.zeros
        stats = make(_norm_shapes(x, over), dtype=torch.float32, device=dev)
    ws, n = _workspace(workspace, "tm_group_norm_workspace_size", B, H, T, d, where, 0, device=dev)
    N.check(N.load().tm_group_norm(B, H, T, d, where, code, _TYPES[kind], _named(_ACTS, "act", act), float(eps), _p(x),
                                   _p(weight), _p(bias), _p(lengths), _p(out), _p(stats), _strides(x, out), _p(ws), n,
                                   _stream), "tm_group_norm")
    return out, stats


@_placed
def group_norm_backward(x, dy, stats, weight=None, bias=None, *, over="token", act=None, lengths=None, workspace=None,
                        _stream=None):
    """Gradients of sum <dy, y> for group_norm of these inputs and the stats it
    returned: a dict of dx and, where the parameter is given, dweight and dbias."""
    _rank("x", x, 4)
    B, H, T, d = x.shape
    dev = x.device
    code, where = _dtype_code("x", x), _named(_OVER, "over", over)
    _check(dev, x=(x, (B, H, T, d), x.dtype, True), dy=(dy, (B, H, T, d), dy.dtype, True),
           weight=(weight, (H, d), torch.float32, False), bias=(bias, (H, d), torch.float32, False),
           lengths=(lengths, (B,), torch.int32, False), stats=(stats, _norm_shapes(x, over), torch.float32, False))
    ws, n = _workspace(workspace, "tm_group_norm_workspace_size", B, H, T, d, where, 1, device=dev)
    out = {"dx": torch.empty_like(x)}
    if weight is not None:
        out["dweight"] = torch.empty_like(weight)
    if bias is not None:
        out["dbias"] = torch.empty_like(bias)
    N.check(N.load().tm_group_norm_backward(
        B, H, T, d, where, code, _dtype_code("dy", dy), _named(_ACTS, "act", act), _p(x), _p(dy), _p(stats), _p(weight),
        _p(bias), _p(lengths), _p(out["dx"]), _p(out.get("dweight")), _p(out.get("dbias")), _strides(x, dy, out["dx"]),
        _p(ws), n, _stream), "tm_group_norm_backward")
    return out
