"""Inputs whose token rows overlap (windows of one signal) and what the outputs that the calls make for them look
like: whole tensors with contiguous channels. The CPU tests hand CPU tensors to a stand-in for the library."""
import pytest
import torch

import test_trained_neural_b200 as tm
from test_trained_neural_b200 import mixer

BF, F = torch.bfloat16, torch.float32


def windows(g, B, H, T, d, kind=F, hop=1, device="cpu"):
    """[B, H, T, d] whose row t is signal[hop t : hop t + d]."""
    s = torch.randn(B, H, hop * (T - 1) + d, generator=g).to(device=device, dtype=kind)
    return s.unfold(2, d, hop)


def calls(g, B, H, T, d, N, kind, hop, device="cpu"):
    """name -> (function, its tensors, keywords): x, dt, z and dy are windows."""
    def win():
        return windows(g, B, H, T, d, kind, hop, device)

    def normal(*shape, kind=F):
        return torch.randn(*shape, generator=g).to(device=device, dtype=kind)

    x, dy = win(), win()
    filt, w = normal(H, d, 4), normal(H, d)
    c = dict(x=x, dt=win(), A=-normal(H, d, N).abs(), Bm=normal(B, 1, T, N, kind=kind), Cm=normal(B, 1, T, N, kind=kind),
             z=win())
    st = torch.stack([x.float().mean(-1), torch.rsqrt(x.float().var(-1, unbiased=False) + 1e-5)], -1)
    return {"conv": (tm.short_conv, dict(x=x, filt=filt), {}),
            "conv_backward": (tm.short_conv_backward, dict(x=x, filt=filt, dy=dy), {}),
            "scan": (tm.selective_scan, c, {}),
            "scan_backward": (tm.selective_scan_backward, dict(c, dy=dy), {}),
            "norm": (tm.group_norm, dict(x=x, weight=w), {}),
            "norm_sequence": (tm.group_norm, dict(x=x, weight=w), dict(over="sequence", dtype=F)),
            "norm_backward": (tm.group_norm_backward, dict(x=x, dy=dy, stats=st.contiguous(), weight=w), {})}


def outputs(r):
    return list(r.values()) if isinstance(r, dict) else list(r)


class Library:
    """Every entry point succeeds and does nothing."""
    def __getattr__(self, name):
        return lambda *args: mixer.N.TM_OK


@pytest.fixture
def stand_in(monkeypatch):
    monkeypatch.setattr(mixer, "_here", lambda x, stream: True)
    monkeypatch.setattr(mixer, "_stream_of", lambda dev: 0)
    monkeypatch.setattr(mixer, "_workspace", lambda *a: (None, 0))
    monkeypatch.setattr(mixer.N, "load", Library)


@pytest.mark.parametrize("B,H,T,d,hop", [(1, 1, 4, 16, 1), (2, 3, 5, 5, 1), (2, 1, 3, 12, 1), (1, 2, 16, 4, 1), (2, 2, 7, 8, 3),
                                         (1, 2, 6, 1, 1)])
def test_outputs_for_windows_have_contiguous_channels(stand_in, B, H, T, d, hop):
    for name, (fn, tensors, more) in calls(torch.Generator().manual_seed(1), B, H, T, d, 4, F, hop).items():
        for t in outputs(fn(**tensors, **more)):
            assert t.shape[-1] == 1 or t.stride(-1) == 1, name
            # one element an address
            reach = 1 + sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
            assert reach == t.numel(), name


@pytest.mark.parametrize("layout", ["bhtd", "bthd", "tbhd"])
def test_outputs_keep_a_dense_layout(stand_in, layout):
    order = [layout.index(v) for v in "bhtd"]
    x = torch.zeros([dict(b=2, h=3, t=5, d=8)[v] for v in layout]).permute(order)
    y, _ = tm.short_conv(x, torch.zeros(3, 8, 4))
    assert y.shape == x.shape and y.stride() == x.stride()


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,T,d,N,kind,hop", [(1, 1, 40, 64, 16, F, 1), (2, 2, 30, 48, 16, BF, 1), (1, 2, 9, 16, 4, F, 3),
                                                (2, 1, 70, 24, 16, BF, 8)])
def test_windows_equal_their_copies(B, H, T, d, N, kind, hop):
    """The copies may be read in wider pieces, so sums over up to 140 rows or 64 channels may run in another order: n
    roundings of a sum of n terms of random sign and size m come to about n u m, its value to sqrt(n) m, so 2 sqrt(n) u
    = 24 u of the largest entry for both sides together, and ten times that for the chain behind it. An output in bf16
    may be rounded the other way then: one step, 2^-7."""
    g = torch.Generator().manual_seed(7)
    for name, (fn, tensors, more) in calls(g, B, H, T, d, N, kind, hop, "cuda").items():
        got = outputs(fn(**tensors, **more))
        want = outputs(fn(**{k: v.contiguous() for k, v in tensors.items()}, **more))
        for p, q in zip(got, want):
            assert torch.isfinite(p).all() and p.shape == q.shape, name
            kinds = (p.dtype, q.dtype)
            assert kinds[0] == kinds[1], name
            p, q = p.float(), q.float()
            bound = 256 * 2.0 ** -24 * q.abs().max() + (2.0 ** -7 * q.abs() if kinds[0] == BF else 0)
            assert ((p - q).abs() <= bound).all(), name
