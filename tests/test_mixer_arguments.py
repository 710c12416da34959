"""Missing tensors are refused by name. The checks come before the library is called; CPU tensors stand in for CUDA
ones, past the test of the device."""
import pytest
import torch

from test_trained_neural_b200 import mixer

B, H, T, d, n, w = 2, 2, 6, 8, 4, 3


def zeros(*shape):
    return torch.zeros(*shape)


def conv():
    return dict(x=zeros(B, H, T, d), filt=zeros(H, d, w))


def conv_backward():
    return dict(conv(), dy=zeros(B, H, T, d))


def conv_step():
    return dict(x=zeros(B, H, d), hist=zeros(B, H, w - 1, d), filt=zeros(H, d, w))


def scan():
    return dict(x=zeros(B, H, T, d), dt=zeros(B, H, T, d), A=zeros(H, d, n), Bm=zeros(B, 1, T, n), Cm=zeros(B, 1, T, n))


def scan_backward():
    return dict(scan(), dy=zeros(B, H, T, d))


def scan_step():
    return dict(x=zeros(B, H, d), dt=zeros(B, H, d), A=zeros(H, d, n), Bm=zeros(B, 1, n), Cm=zeros(B, 1, n),
                state=zeros(B, H, d, n))


def norm():
    return dict(x=zeros(B, H, T, d))


def norm_backward():
    return dict(x=zeros(B, H, T, d), dy=zeros(B, H, T, d), stats=zeros(B, H, T, 2))


CALLS = [(mixer.short_conv, conv), (mixer.short_conv_backward, conv_backward), (mixer.short_conv_step, conv_step),
         (mixer.selective_scan, scan), (mixer.selective_scan_backward, scan_backward),
         (mixer.selective_scan_step, scan_step), (mixer.group_norm, norm), (mixer.group_norm_backward, norm_backward)]


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def on_cpu(monkeypatch):
    """The device test passes, and a call that gets as far as the library is told so instead of making it."""
    def load():
        raise Reached
    monkeypatch.setattr(mixer, "_here", lambda x, stream: isinstance(x, torch.Tensor))
    monkeypatch.setattr(mixer.N, "load", load)
    monkeypatch.setattr(mixer, "_workspace", lambda *a: (None, 0))


@pytest.mark.parametrize("call,inputs", CALLS, ids=[c.__name__ for c, _ in CALLS])
def test_missing_tensors_are_named(call, inputs):
    with pytest.raises(Reached):
        call(**inputs())
    for name in inputs():
        with pytest.raises(TypeError, match=rf"\b{name} must be a tensor"):
            call(**{**inputs(), name: None})
    with pytest.raises(TypeError, match=r"\bx must be a tensor"):
        call(**{**inputs(), "x": 3.0})
