"""Refusals of the sequence-mixer operators: every call here returns before its
first CUDA call, so no GPU is needed."""
import ctypes

import pytest
import torch

import test_trained_neural_b200 as tm
from test_trained_neural_b200 import _native as N

BAD, UNSUPPORTED, OOM = N.TM_ERR_INVALID_ARG, N.TM_ERR_UNSUPPORTED, N.TM_ERR_OOM


def addresses(n):
    """Distinct addresses far apart, never dereferenced."""
    return [0x10_0000_0000_00 + i * 0x1_0000_0000_00 for i in range(n)]


def table(*rows):
    flat = [v for r in rows for v in r]
    return (ctypes.c_longlong * len(flat))(*flat)


CONV = ["x", "filt", "bias", "hist", "lengths", "y", "tail"]
CONV_B = ["x", "filt", "bias", "hist", "lengths", "dy", "dtail", "dx", "dfilt", "dbias", "dhist"]
SCAN = ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state0", "lengths", "y", "state_end"]
SCAN_B = SCAN[:10] + ["dy", "dstate_end", "dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate0"]
STEP = ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state", "y"]
NORM = ["x", "weight", "bias", "lengths", "y", "stats"]
NORM_B = ["x", "dy", "stats", "weight", "bias", "lengths", "dx", "dweight", "dbias"]


def call(fn, names, sizes, ws=1 << 40, strides=None, eps=None, **change):
    """Status of the entry point with distinct pointers, but for the changed ones
    (another tensor's name + an offset, or a number)."""
    ptr = dict(zip(names + ["workspace"], addresses(len(names) + 1)))
    for k, v in change.items():
        if isinstance(v, tuple):
            v = ptr[v[0]] + v[1]
        ptr[k] = v
    args = list(sizes) + ([eps] if eps is not None else []) + [ptr[k] for k in names]
    args += [strides]
    if fn not in ("tm_conv", "tm_conv_step", "tm_scan_step"):
        args += [ptr["workspace"], ws]
    return getattr(N.load(), fn)(*args, None)


def conv(B=2, H=2, T=64, d=8, w=4, kind=N.TM_F32, act=0, **k):
    return call("tm_conv", CONV, (B, H, T, d, w, kind, act, 0), **k)


def conv_b(B=2, H=2, T=64, d=8, w=4, kind=N.TM_F32, act=0, **k):
    return call("tm_conv_backward", CONV_B, (B, H, T, d, w, kind, act), **k)


def conv_s(B=2, H=2, d=8, w=4, kind=N.TM_F32, act=0, **k):
    return call("tm_conv_step", ["x", "filt", "bias", "hist", "y"], (B, H, d, w, kind, act), **k)


def scan(B=2, H=2, G=1, T=64, d=8, n=16, kind=N.TM_F32, sp=1, **k):
    return call("tm_scan", SCAN, (B, H, G, T, d, n, kind, sp, 0), **k)


def scan_b(B=2, H=2, G=1, T=64, d=8, n=16, kind=N.TM_F32, sp=1, **k):
    return call("tm_scan_backward", SCAN_B, (B, H, G, T, d, n, kind, sp), **k)


def scan_s(B=2, H=2, G=1, d=8, n=16, kind=N.TM_F32, sp=1, **k):
    return call("tm_scan_step", STEP, (B, H, G, d, n, kind, sp), **k)


def norm(B=2, H=2, T=64, d=8, over=1, a=N.TM_F32, b=N.TM_F32, act=0, eps=1e-5, **k):
    return call("tm_group_norm", NORM, (B, H, T, d, over, a, b, act, 0), eps=eps, **k)


def norm_b(B=2, H=2, T=64, d=8, over=1, a=N.TM_F32, b=N.TM_F32, act=0, **k):
    return call("tm_group_norm_backward", NORM_B, (B, H, T, d, over, a, b, act), **k)


@pytest.mark.parametrize("fn", [conv, conv_b, conv_s, scan, scan_b, scan_s, norm, norm_b])
def test_sizes(fn):
    for bad in (dict(B=0), dict(H=0), dict(d=0), dict(d=1 << 21), dict(B=1 << 20, H=1 << 10), dict(H=-1)):
        assert fn(**bad) == BAD, bad
    if fn not in (conv_s, scan_s):
        for t in (0, -5, 1 << 30):
            assert fn(T=t) == BAD
    if fn not in (norm, norm_b):
        assert fn(kind=2) == BAD


@pytest.mark.parametrize("fn", [conv, conv_b, conv_s])
def test_conv_width_and_activation(fn):
    for bad in (dict(w=0), dict(w=9), dict(act=2), dict(act=-1)):
        assert fn(**bad) == BAD


@pytest.mark.parametrize("fn", [scan, scan_b, scan_s])
def test_scan_states_and_groups(fn):
    for bad in (dict(n=0), dict(n=129), dict(G=0), dict(H=3, G=2), dict(H=2, G=4)):
        assert fn(**bad) == BAD


@pytest.mark.parametrize("fn", [norm, norm_b])
def test_norm_choices(fn):
    for bad in (dict(over=2), dict(over=-1), dict(a=3), dict(b=3), dict(act=5)):
        assert fn(**bad) == BAD
    if fn is norm:
        assert fn(eps=-1.0) == BAD and fn(eps=float("nan")) == BAD


@pytest.mark.parametrize("fn,needed", [
    (conv, ["x", "filt", "y"]), (conv_b, ["x", "filt", "dy", "dx", "dfilt", "workspace"]),
    (conv_s, ["x", "filt", "hist", "y"]), (scan, ["x", "dt", "A", "Bm", "Cm", "y"]),
    (scan_b, ["x", "dt", "A", "Bm", "Cm", "dy", "dx", "ddt", "dA", "dB", "dC", "workspace"]),
    (scan_s, ["x", "dt", "A", "Bm", "Cm", "state", "y"]), (norm, ["x", "y", "workspace"]),
    (norm_b, ["x", "dy", "stats", "dx", "workspace"])])
def test_missing_and_misaligned_pointers(fn, needed):
    for name in needed:
        assert fn(**{name: None}) == BAD, name
        assert fn(**{name: (name, 1)}) == BAD, name
    if "workspace" in needed:
        assert fn(workspace=("workspace", 128)) == BAD


def test_gradients_of_what_is_not_there():
    assert scan_b(D=None) == BAD                     # dD without D
    assert scan_b(z=None) == BAD                     # dz without z
    assert scan_b(dz=None) == BAD                    # z without dz


@pytest.mark.parametrize("fn,outs,ins", [
    (conv, ["y", "tail"], ["x", "filt", "bias", "hist", "lengths"]),
    (conv_b, ["dx", "dfilt", "dbias", "dhist"], ["x", "filt", "bias", "hist", "lengths", "dy", "dtail"]),
    (conv_s, ["y", "hist"], ["x", "filt", "bias"]),
    (scan, ["y", "state_end"], ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "lengths"]),
    (scan_b, ["dx", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dstate0"],
     ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state0", "lengths", "dy", "dstate_end"]),
    (scan_s, ["y", "state"], ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias"]),
    (norm, ["y", "stats"], ["x", "weight", "bias", "lengths"]),
    (norm_b, ["dx", "dweight", "dbias"], ["x", "dy", "stats", "weight", "bias", "lengths"])])
def test_overlapping_buffers(fn, outs, ins):
    for o in outs:
        for i in ins:
            assert fn(**{o: (i, 0)}) == BAD, (o, i)
        for q in outs:
            if q != o:
                assert fn(**{o: (q, 0)}) == BAD, (o, q)
        if fn not in (conv, conv_s, scan_s):
            assert fn(**{o: ("workspace", 0)}) == BAD, o
    # the state may be updated in place, but not half of it
    if fn is scan:
        assert fn(state_end=("state0", 256)) == BAD


def test_strides():
    whole, rows = (8 * 64 * 2, 8 * 64, 8), (0, 0, 8)
    assert conv(strides=table((-1, 512, 8), whole)) == BAD
    assert conv(strides=table((1 << 50, 512, 8), whole)) == BAD
    assert conv(strides=table(whole, rows)) == BAD               # an output that overlaps itself
    assert conv(strides=table(whole, (1024, 512, 7))) == BAD
    assert conv(strides=table(whole, (1024, 4, 8))) == BAD
    assert conv_b(strides=table(whole, whole, rows)) == BAD
    assert scan(strides=table(*[whole] * 2, *[(1024, 0, 16)] * 2, whole, rows)) == BAD
    assert norm(strides=table(whole, rows)) == BAD


@pytest.mark.parametrize("fn", [conv_b, scan_b, norm, norm_b])
def test_small_workspace(fn):
    assert fn(ws=64) == OOM


def test_scan_workspace_only_when_it_splits():
    n = ctypes.c_size_t()
    lib = N.load()
    assert lib.tm_scan_workspace_size(1, 1, 1, 8192, 512, 16, N.TM_BF16, ctypes.byref(n)) == N.TM_OK and n.value > 0
    assert scan(B=1, H=1, T=8192, d=512, ws=64) == OOM
    assert scan(B=1, H=1, T=8192, d=512, workspace=None) == BAD
    assert lib.tm_scan_workspace_size(64, 8, 8, 16, 512, 16, N.TM_BF16, ctypes.byref(n)) == N.TM_OK and n.value == 0


def test_workspace_queries_refuse():
    lib, n = N.load(), ctypes.c_size_t()
    assert lib.tm_conv_backward_workspace_size(1, 1, 8, 8, 9, 0, ctypes.byref(n)) == BAD
    assert lib.tm_conv_backward_workspace_size(1, 1, 8, 8, 4, 0, None) == BAD
    assert lib.tm_scan_workspace_size(1, 3, 2, 8, 8, 16, 0, ctypes.byref(n)) == BAD
    assert lib.tm_scan_backward_workspace_size(1, 2, 2, 8, 8, 200, 0, ctypes.byref(n)) == BAD
    assert lib.tm_group_norm_workspace_size(1, 2, 8, 8, 7, 0, ctypes.byref(n)) == BAD


def test_memory_contexts_take_silu_only():
    h = ctypes.c_void_p()
    assert N.load().tm_create(2, 64, 4, N.TM_ACT_NONE, ctypes.byref(h)) == BAD


def test_python_takes_cuda_tensors_only():
    x, f = torch.zeros(1, 1, 4, 8), torch.zeros(1, 8, 4)
    with pytest.raises(ValueError):
        tm.short_conv(x, f)
    with pytest.raises(ValueError):
        tm.short_conv_step(x[:, :, 0], torch.zeros(1, 1, 3, 8), f)
    with pytest.raises(ValueError):
        tm.selective_scan(x, x, torch.zeros(1, 8, 4), torch.zeros(1, 1, 4, 4), torch.zeros(1, 1, 4, 4))
    with pytest.raises(ValueError):
        tm.group_norm(x)
