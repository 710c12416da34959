"""The sequence-mixer operators on the GPU against the float64 oracle.

Tolerances. u = 2^-24 is half a step of fp32, `half` half a step of the output's
type (bf16: 2^-8). The special-function unit's exp and reciprocal are within
2^-22, so an activation and its gradient are within 16 u. An output is compared
by norm, ||got - ref|| <= tol ||ref||, and entry by entry within 8 tol of the
larger of the entry and the root mean square (cancellation may leave an entry
that is small beside its terms). `tol` is half + the fp32 part:
  convolution    w products and sums, activation                  (2 w + 16) u
  scan           each step of the recurrence multiplies by exp(e A) known to
                 2^-22 + |e A| u and rounds twice: below 8 u a token for the |e A|
                 here, at most linear in the tokens that a state remembers,
                 bounded by T; softplus 8 u, N products      (8 T + 2 N + 32) u
  its gradients  the same in both directions                (24 T + 2 N + 64) u
  sums over n rows (parameters): a tree or chunks of at most 128 rows, terms
                 of random sign                              + 128 u
  group norm     mean and variance over the group in trees, two passes; rsqrt
                 and the activation                                     64 u
"""
import zlib

import numpy as np
import pytest
import torch

import test_trained_neural_b200 as tm
from oracle import mixer as M

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


def half(kind):
    return torch.finfo(kind).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, tol, what=""):
    got, ref = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(ref, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), what
    if not ref.size:
        return
    d, rms = np.abs(got - ref), np.sqrt((ref ** 2).mean())
    assert np.linalg.norm(d) <= tol * np.linalg.norm(ref) + 1e-30, (what, np.linalg.norm(d) / np.linalg.norm(ref), tol)
    assert (d <= 8 * tol * np.maximum(np.abs(ref), rms) + 1e-30).all(), (what, (d / np.maximum(np.abs(ref), rms)).max())


class Draw:
    def __init__(self, *key):
        self.g = torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))

    def normal(self, *shape, kind=F):
        return torch.randn(*shape, generator=self.g, device="cuda").to(kind)

    def uniform(self, lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=self.g, device="cuda")

    def tokens(self, B, H, T, d, kind, layout="bhtd"):
        """[B, H, T, d]: contiguous; [B, T, H, d] underneath; a slice of a wider projection; or with a
        base and strides that are odd."""
        if layout == "bthd":
            return self.normal(B, T, H, d, kind=kind).transpose(1, 2)
        if layout == "proj":
            return self.normal(B, T, 3, H, d, kind=kind)[:, :, 1].transpose(1, 2)
        if layout == "odd":
            return self.normal(B, H, T, d + 3, kind=kind)[..., 1:d + 1]
        return self.normal(B, H, T, d, kind=kind)


def each(B, H, lengths, T):
    n = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths]
    return [(b, h, n[b]) for b in range(B) for h in range(H)]


def lens(lengths):
    return None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")


def poison(t, lengths):
    """Rows behind each sequence's end hold NaN: nothing may read them."""
    if lengths is not None:
        for b, n in enumerate(lengths):
            t[b, :, max(0, n):] = float("nan")
    return t


# ------------------------------------------------------------- convolution

CONV = [  # B, H, T, d, w, kind, layout, act, bias, hist, lengths
    (2, 2, 40, 64, 4, BF, "bhtd", "silu", True, True, None),
    (1, 1, 1, 8, 4, BF, "bhtd", "silu", True, False, None),          # one token, shorter than the filter
    (2, 3, 2, 24, 4, F, "bthd", "none", True, True, None),
    (3, 2, 33, 50, 3, F, "proj", "silu", True, True, [33, 0, 7]),
    (2, 1, 100, 5, 4, BF, "odd", "silu", False, True, [1, 100]),
    (2, 4, 70, 16, 1, BF, "bthd", "silu", True, False, [70, 3]),     # width 1: no history
    (1, 2, 64, 12, 8, F, "odd", "none", True, True, None),
    (2, 2, 37, 40, 7, BF, "proj", "silu", True, True, [2, 37]),
    (1, 3, 300, 136, 4, BF, "bthd", "silu", True, True, None),
    (1, 1, 17, 2100, 2, F, "bhtd", "silu", False, False, None),      # channels beyond one block
    (2, 16, 130, 128, 4, BF, "proj", "silu", True, False, None),
    (1, 1, 2049, 6, 5, F, "bhtd", "silu", True, True, [2048]),
]


@pytest.mark.parametrize("B,H,T,d,w,kind,layout,act,bias,hist,lengths", CONV)
def test_conv(B, H, T, d, w, kind, layout, act, bias, hist, lengths):
    r = Draw("conv", B, H, T, d, w)
    x = poison(r.tokens(B, H, T, d, kind, layout), lengths)
    f, b = r.normal(H, d, w) / w ** 0.5, r.normal(H, d) if bias else None
    h = r.normal(B, H, w - 1, d, kind=kind) if hist else None
    y, tail = tm.short_conv(x, f, b, hist=h, lengths=lens(lengths), act=act)
    dy, dtail = poison(r.tokens(B, H, T, d, kind, layout), lengths), r.normal(B, H, w - 1, d, kind=kind)
    g = tm.short_conv_backward(x, f, dy, b, hist=h, lengths=lens(lengths), act=act, dtail=dtail)
    assert set(g) == {"dx", "dfilt"} | ({"dbias"} if bias else set()) | ({"dhist"} if hist else set())
    tol = (2 * w + 16) * U
    df, db = np.zeros((H, d, w)), np.zeros((H, d))
    for i, j, n in each(B, H, lengths, T):
        a = (f64(x[i, j, :n]), f64(f[j]))
        more = dict(bias=None if b is None else f64(b[j]), hist=None if h is None else f64(h[i, j]), silu=act == "silu")
        ry, rt, _, _ = M.conv(*a, **more)
        close(y[i, j, :n], ry, half(kind) + tol, "y")
        assert not f64(y[i, j, n:]).any()
        np.testing.assert_array_equal(f64(tail[i, j]), rt)
        dx, dfi, dbi, dh = M.conv_backward(*a, f64(dy[i, j, :n]), dtail=f64(dtail[i, j]), **more)
        close(g["dx"][i, j, :n], dx, half(kind) + 2 * tol, "dx")
        assert not f64(g["dx"][i, j, n:]).any()
        if hist and w > 1:
            close(g["dhist"][i, j], dh, half(kind) + 2 * tol, "dhist")
        df[j] += dfi
        db[j] += dbi
    close(g["dfilt"], df, 2 * tol + 128 * U, "dfilt")
    if bias:
        close(g["dbias"], db, 2 * tol + 128 * U, "dbias")


@pytest.mark.parametrize("B,H,d,w,kind", [(3, 2, 64, 4, BF), (1, 1, 5, 4, F), (2, 3, 6, 8, BF), (5, 1, 48, 1, F),
                                          (200, 4, 96, 4, BF), (2, 2, 20, 3, F)])
@pytest.mark.parametrize("sliced", [False, True])
def test_conv_steps_continue_a_prompt(B, H, d, w, kind, sliced):
    """A prompt and then tokens one by one give what one longer call gives, bit for bit in the history."""
    r = Draw("step", B, H, d, w)
    T, more = 6, 5
    x = r.tokens(B, H, T + more, d, kind, "proj" if sliced else "bhtd")
    f, b = r.normal(H, d, w) / w ** 0.5, r.normal(H, d)
    want, last = tm.short_conv(x, f, b)
    _, hist = tm.short_conv(x[:, :, :T].contiguous(), f, b)
    for t in range(T, T + more):
        y = tm.short_conv_step(x[:, :, t], hist, f, b)
        close(y, f64(want[:, :, t]), 2 * (half(kind) + (2 * w + 16) * U))
    np.testing.assert_array_equal(f64(hist), f64(last))


def test_conv_taps_beyond_the_filter_do_not_touch_infinities():
    for w in (1, 2, 3, 5):
        x = torch.zeros(1, 1, 32, 8, device="cuda", dtype=BF)
        x[0, 0, 9] = float("inf")
        f = torch.ones(1, 8, w, device="cuda")
        y, _ = tm.short_conv(x, f, act="none")
        bad = ~torch.isfinite(y[0, 0, :, 0])
        assert bad.nonzero().flatten().tolist() == list(range(9, 9 + w))


# -------------------------------------------------------------------- scan

def scan_case(B, H, G, T, d, N, kind, layout="bhtd", D=True, z=True, bias=True, state=True, lengths=None, strong=1.0):
    r = Draw("scan", B, H, G, T, d, N, layout)
    c = dict(x=poison(r.tokens(B, H, T, d, kind, layout), lengths),
             dt=poison(r.tokens(B, H, T, d, kind, "bthd" if layout == "proj" else layout), lengths),
             A=-r.uniform(0.2, 4.0, H, d, N) * strong,
             Bm=poison(r.tokens(B, G, T, N, kind, layout), lengths), Cm=poison(r.tokens(B, G, T, N, kind, layout), lengths))
    o = dict(D=r.normal(H, d) if D else None, z=poison(r.tokens(B, H, T, d, kind, layout), lengths) if z else None,
             dt_bias=r.uniform(-5, -2, H, d) if bias else None, state=r.normal(B, H, d, N) if state else None)
    return r, c, o


def scan_ref(c, o, b, h, n, G, H):
    g = h // (H // G)
    a = dict(x=f64(c["x"][b, h, :n]), dt=f64(c["dt"][b, h, :n]), A=f64(c["A"][h]), Bm=f64(c["Bm"][b, g, :n]),
             Cm=f64(c["Cm"][b, g, :n]))
    a["D"] = None if o["D"] is None else f64(o["D"][h])
    a["z"] = None if o["z"] is None else f64(o["z"][b, h, :n])
    a["dt_bias"] = None if o["dt_bias"] is None else f64(o["dt_bias"][h])
    a["state"] = None if o["state"] is None else f64(o["state"][b, h])
    return a


SCAN = [  # B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths
    (2, 2, 1, 40, 32, 16, BF, "bhtd", True, True, True, True, None),
    (1, 1, 1, 1, 8, 16, F, "bhtd", True, True, True, False, None),            # one token
    (2, 3, 3, 17, 5, 3, F, "odd", True, False, True, True, None),
    (3, 4, 2, 50, 24, 12, BF, "proj", True, True, True, True, [50, 0, 13]),
    (2, 2, 1, 70, 20, 8, F, "bthd", False, True, False, False, [1, 70]),
    (1, 4, 4, 33, 64, 32, BF, "bthd", True, True, True, True, None),
    (2, 1, 1, 30, 6, 64, F, "bhtd", True, True, True, True, [29, 30]),
    (1, 2, 1, 20, 3, 128, BF, "proj", True, True, True, True, None),
    (1, 1, 1, 129, 300, 16, F, "bhtd", False, False, False, False, None),
    (2, 2, 2, 65, 9, 100, F, "odd", True, True, True, True, [0, 65]),
    (1, 2, 1, 1500, 16, 16, BF, "proj", True, True, True, True, None),        # the sequence is split
    (2, 1, 1, 1025, 7, 5, F, "odd", True, True, True, True, [1025, 300]),     # split, one ends in an early part
    (2, 2, 2, 700, 40, 40, F, "bthd", True, True, True, True, [0, 511]),
    (1, 1, 1, 640, 33, 128, BF, "bhtd", True, False, True, True, None),
    (1, 8, 8, 321, 4, 16, F, "bhtd", True, True, True, False, None),
]
LENGTHY = [c for c in SCAN if c[3] >= 300]


def scan_tol(T, N):
    return (8 * T + 2 * N + 32) * U


@pytest.mark.parametrize("B,H,G,T,d,N,kind,layout,D,z,bias,state,lengths", SCAN)
def test_scan(B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths):
    r, c, o = scan_case(B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths)
    y, end = tm.selective_scan(**c, **o, lengths=lens(lengths))
    for b, h, n in each(B, H, lengths, T):
        ry, rh, _ = M.scan(**scan_ref(c, o, b, h, n, G, H))
        close(y[b, h, :n], ry, half(kind) + scan_tol(n, N), "y")
        assert not f64(y[b, h, n:]).any()
        close(end[b, h], rh, scan_tol(n, N), "state")


@pytest.mark.parametrize("B,H,G,T,d,N,kind,layout,D,z,bias,state,lengths", SCAN)
def test_scan_backward(B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths):
    r, c, o = scan_case(B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths)
    dy, ds = poison(r.tokens(B, H, T, d, kind, layout), lengths), r.normal(B, H, d, N) if state else None
    g = tm.selective_scan_backward(**c, dy=dy, **o, dstate_end=ds, lengths=lens(lengths))
    assert set(g) == {"dx", "ddt", "dA", "dB", "dC"} | {k for k, v in (("dD", D), ("dz", z), ("ddt_bias", bias),
                                                                      ("dstate", state)) if v}
    tol = (24 * T + 2 * N + 64) * U
    total = {k: np.zeros(g[k].shape) for k in ("dA", "dB", "dC", "dD", "ddt_bias") if k in g}
    for b, h, n in each(B, H, lengths, T):
        ref = M.scan_backward(dy=f64(dy[b, h, :n]), dstate_end=None if ds is None else f64(ds[b, h]),
                              **scan_ref(c, o, b, h, n, G, H))
        for k in ("dx", "ddt", "dz"):
            if k in g:
                close(g[k][b, h, :n], ref[k], half(kind) + tol, k)
                assert not f64(g[k][b, h, n:]).any(), k
        if state:
            close(g["dstate"][b, h], ref["dstate"], tol, "dstate")
        for k in total:
            if k in ("dB", "dC"):
                total[k][b, h // (H // G), :n] += ref[k]
            else:
                total[k][h] += ref[k]
    for k in total:
        close(g[k], total[k], (half(kind) if k in ("dB", "dC") else 128 * U) + tol, k)


def test_scan_without_softplus_and_with_growth():
    """e = dt + dt_bias as it is, negative too: the decay may grow the state."""
    r, c, o = scan_case(2, 2, 1, 37, 16, 16, F)
    c["dt"] = r.uniform(-0.1, 0.2, 2, 2, 37, 16)
    o["dt_bias"] = r.uniform(-0.05, 0.05, 2, 16)
    y, end = tm.selective_scan(**c, **o, softplus=False)
    dy, ds = r.normal(2, 2, 37, 16), r.normal(2, 2, 16, 16)
    g = tm.selective_scan_backward(**c, dy=dy, **o, dstate_end=ds, softplus=False)
    for b, h, n in each(2, 2, None, 37):
        a = scan_ref(c, o, b, h, n, 1, 2)
        ry, rh, _ = M.scan(softplus=False, **a)
        close(y[b, h], ry, scan_tol(n, 16))
        close(end[b, h], rh, scan_tol(n, 16))
        ref = M.scan_backward(dy=f64(dy[b, h]), dstate_end=f64(ds[b, h]), softplus=False, **a)
        for k in ("dx", "ddt", "dz", "dstate"):
            close(g[k][b, h], ref[k], (24 * n + 96) * U, k)


@pytest.mark.parametrize("v", [-200.0, -88.0, -30.0, -5.0, 0.0, 5.0, 30.0, 88.0, 1e4])
def test_softplus_over_its_range(v):
    """e x Bm Cm with A = 0 and one token is softplus(dt) itself: 16 u relative over the whole range; below
    -87 the special-function unit flushes denormal values."""
    one = torch.ones(1, 1, 1, 8, device="cuda")
    y, _ = tm.selective_scan(one, one * v, torch.zeros(1, 8, 4, device="cuda"), one[..., :4], one[..., :4])
    want = 4 * np.logaddexp(np.float64(np.float32(v)), 0.0)
    # exp(v) carries the rounding of v log2(e): |v| u
    assert abs(f64(y)[0, 0, 0, 0] - want) <= want * (32 + 2 * abs(v)) * U + 4 * 2.0 ** -126


def test_scan_decays_to_nothing_and_not_at_all():
    """exp(e A) of 0 (A = -1e30) and of 1 (A = 0), split and not, with their gradients finite and right."""
    for T in (24, 400):
        for a in (-1e30, 0.0):
            r, c, o = scan_case(1, 1, 1, T, 16, 16, F)
            c["A"].fill_(a)
            y, end = tm.selective_scan(**c, **o)
            ref = scan_ref(c, o, 0, 0, T, 1, 1)
            ry, rh, _ = M.scan(**ref)
            close(y[0, 0], ry, scan_tol(T, 16))
            close(end[0, 0], rh, scan_tol(T, 16))
            if a == 0.0:
                dy = r.normal(1, 1, T, 16)
                g = tm.selective_scan_backward(**c, dy=dy, **o)
                rg = M.scan_backward(dy=f64(dy[0, 0]), **ref)
                for k in ("dx", "ddt", "dz", "dstate"):
                    close(g[k][0, 0], rg[k], (24 * T + 96) * U, k)
                close(g["dA"][0], rg["dA"], (24 * T + 96) * U, "dA")


@pytest.mark.parametrize("B,H,G,d,N,kind,sliced", [(3, 2, 1, 32, 16, BF, True), (1, 1, 1, 5, 3, F, False),
                                                   (2, 4, 2, 24, 12, F, True), (2, 2, 2, 7, 64, BF, False),
                                                   (1, 3, 1, 4, 128, F, False), (150, 2, 1, 40, 16, BF, True)])
def test_scan_steps_continue_a_prompt(B, H, G, d, N, kind, sliced):
    T, more = 9, 4
    r, c, o = scan_case(B, H, G, T + more, d, N, kind, "proj" if sliced else "bhtd")
    want, last = tm.selective_scan(**c, **o)
    cut = {k: c[k][:, :, :T] for k in ("x", "dt", "Bm", "Cm")}
    _, state = tm.selective_scan(**cut, A=c["A"], **{**o, "z": o["z"][:, :, :T]})
    for t in range(T, T + more):
        y = tm.selective_scan_step(c["x"][:, :, t], c["dt"][:, :, t], c["A"], c["Bm"][:, :, t], c["Cm"][:, :, t], state,
                                   D=o["D"], z=o["z"][:, :, t], dt_bias=o["dt_bias"])
        close(y, f64(want[:, :, t]), 2 * (half(kind) + scan_tol(T + more, N)))
    close(state, f64(last), 2 * scan_tol(T + more, N))


@pytest.mark.parametrize("T", [20, 400])
def test_scan_decay_of_the_lowest_values(T):
    """A of -inf and of fp32's lowest value: every token alone where it writes, and the state left alone by rows
    behind the end and by tokens whose e is 0 (softplus(-200))."""
    r, c, o = scan_case(2, 1, 1, T, 16, 16, F, lengths=[T, 7])
    c["A"][:, :8] = float("-inf")
    c["A"][:, 8:] = torch.finfo(F).min
    c["dt"][0, :, 11:] = -200.0
    n = lens([T, 7])
    y, end = tm.selective_scan(**c, **o, lengths=n)
    assert torch.isfinite(end).all() and torch.isfinite(y[0]).all()
    # sequence 0: the state stays what token 10 wrote; sequence 1: what token 6 wrote
    for b, t in ((0, 10), (1, 6)):
        e = np.logaddexp(f64(c["dt"][b, 0, t]) + f64(o["dt_bias"][0]), 0.0)
        want = (e * f64(c["x"][b, 0, t]))[:, None] * f64(c["Bm"][b, 0, t])
        close(end[b, 0], want, 64 * U)
    dy = poison(r.tokens(2, 1, T, 16, F), [T, 7])
    g = tm.selective_scan_backward(**c, dy=dy, **o, lengths=n)
    for k in ("dx", "dB", "dC", "dz", "dstate"):
        assert torch.isfinite(g[k]).all(), k


@pytest.mark.parametrize("T", [1, 40, 3000])
def test_tokens_that_write_nothing_leave_the_state_bit_for_bit(T):
    """e = softplus(-200 ...) = 0: exp(e A) is 1 exactly, however often, in prompts, split prompts and steps."""
    r, c, o = scan_case(2, 2, 1, T, 16, 16, F)
    c["dt"].fill_(-200.0)
    _, end = tm.selective_scan(**c, **o)
    assert torch.equal(end, o["state"])
    state = o["state"].clone()
    tm.selective_scan_step(c["x"][:, :, 0], c["dt"][:, :, 0], c["A"], c["Bm"][:, :, 0], c["Cm"][:, :, 0], state,
                           dt_bias=o["dt_bias"])
    assert torch.equal(state, o["state"])
    ds = r.normal(2, 2, 16, 16)
    g = tm.selective_scan_backward(**c, dy=torch.zeros_like(c["x"]), **o, dstate_end=ds)
    assert torch.equal(g["dstate"], ds)


def test_expanded_inputs():
    """x itself repeated over the batch: outputs are whole tensors of their own."""
    r = Draw("expand")
    B, H, T, d, N = 3, 2, 40, 16, 16
    x = r.normal(1, H, T, d, kind=BF).expand(B, H, T, d)
    f, w = r.normal(H, d, 4), r.normal(H, d)
    _, c, o = scan_case(B, H, 1, T, d, N, BF)
    c["x"] = x
    whole = {**c, "x": x.contiguous()}
    dy = r.normal(B, H, T, d, kind=BF)
    st = tm.group_norm(x, w)[1]
    for got, want in ((tm.short_conv(x, f), tm.short_conv(x.contiguous(), f)),
                      (tm.short_conv_backward(x, f, dy), tm.short_conv_backward(x.contiguous(), f, dy)),
                      (tm.selective_scan(**c, **o), tm.selective_scan(**whole, **o)),
                      (tm.selective_scan_backward(**c, dy=dy, **o), tm.selective_scan_backward(**whole, dy=dy, **o)),
                      (tm.group_norm(x, w), tm.group_norm(x.contiguous(), w)),
                      (tm.group_norm_backward(x, dy, st, w), tm.group_norm_backward(x.contiguous(), dy, st, w))):
        for p, q in zip(flat(got), flat(want)):
            assert torch.equal(p, q)


def test_offsets_past_32_bits():
    """2^31 elements and more in one tensor: the last rows are those of a call on the end alone."""
    d, T = 2048, (1 << 20) + 77
    r = Draw("long")
    x = torch.empty(1, 1, T, d, device="cuda", dtype=BF)
    for i in range(0, T, 1 << 16):
        x[0, 0, i:i + (1 << 16)] = r.normal(min(1 << 16, T - i), d, kind=BF)
    f, w = r.normal(1, d, 4), r.normal(1, d)
    n = 300
    y, tail = tm.short_conv(x, f)
    end, tail_end = tm.short_conv(x[:, :, -n:], f, hist=x[:, :, -n - 3:-n].contiguous())
    assert torch.equal(y[:, :, -n:], end) and torch.equal(tail, tail_end)
    g = tm.short_conv_backward(x, f, y)["dx"]
    g_end = tm.short_conv_backward(x[:, :, -n:], f, y[:, :, -n:], hist=x[:, :, -n - 3:-n].contiguous())["dx"]
    assert torch.equal(g[:, :, -n:], g_end)
    del g, y
    y, st = tm.group_norm(x, w)
    assert torch.equal(y[:, :, -n:], tm.group_norm(x[:, :, -n:], w)[0])
    del y
    # the scan forgets within a few hundred tokens (e A below -0.3): its end does not know its beginning
    A = torch.full((1, d, 16), -4.0, device="cuda")
    bias = torch.full((1, d), -2.0, device="cuda")
    Bm = r.normal(1, 1, T, 16, kind=BF)
    y, state = tm.selective_scan(x, torch.zeros_like(x), A, Bm, Bm, dt_bias=bias)
    y_end, state_end = tm.selective_scan(x[:, :, -n:], torch.zeros_like(x[:, :, -n:]), A, Bm[:, :, -n:], Bm[:, :, -n:],
                                         dt_bias=bias)
    # e = softplus(-2) = 0.127: exp(-0.5 n / 2) of the difference is left after half of the rows
    close(state, f64(state_end), scan_tol(n, 16))
    close(y[:, :, -n // 2:], f64(y_end[:, :, -n // 2:]), 2 * half(BF))


def test_scan_state_in_place_and_broadcast_inputs():
    """state_end = state, a B and C shared by the batch (stride 0) and a z that repeats over heads."""
    B, H, T, d, N = 3, 2, 200, 16, 16
    r, c, o = scan_case(B, H, 1, T, d, N, F)
    c["Bm"], c["Cm"] = (c[k][:1].expand(B, 1, T, N) for k in ("Bm", "Cm"))
    o["z"] = o["z"][:, :1].expand(B, H, T, d)
    y, end = tm.selective_scan(**c, **o)
    full, _ = tm.selective_scan(**{k: v.contiguous() for k, v in c.items()},
                                **{k: v.contiguous() for k, v in o.items()})
    assert torch.equal(y, full)
    state = o.pop("state").clone()
    _, same = tm.selective_scan(**c, **o, state=state, state_end=state)
    assert same is state and torch.equal(state, end)
    dy = r.normal(B, H, T, d)
    g = tm.selective_scan_backward(**c, dy=dy, **o)
    w = tm.selective_scan_backward(**{k: v.contiguous() for k, v in c.items()}, dy=dy,
                                   **{k: v.contiguous() if v is not None else v for k, v in o.items()})
    for k in g:
        assert torch.equal(g[k], w[k]), k


# -------------------------------------------------------------- group norm

NORM = [  # B, H, T, d, kind, out, layout, over, act, affine, lengths
    (2, 2, 40, 64, BF, BF, "bthd", "token", "silu", True, None),
    (1, 1, 1, 1, F, F, "bhtd", "token", None, True, None),              # one channel: its own mean
    (2, 3, 17, 48, F, BF, "bhtd", "token", "silu", True, [17, 0]),
    (1, 2, 33, 7, BF, F, "odd", "token", None, False, None),
    (2, 1, 9, 200, F, F, "odd", "token", "silu", True, [9, 2]),
    (1, 2, 20, 128, BF, BF, "proj", "token", None, True, None),
    (2, 2, 11, 512, BF, BF, "bhtd", "token", "silu", True, None),
    (1, 1, 13, 1000, BF, F, "bhtd", "token", "silu", True, None),
    (1, 2, 5, 1024, F, F, "bthd", "token", "silu", True, None),
    (1, 1, 7, 3001, F, F, "bhtd", "token", "silu", True, [5]),          # a row beyond the registers
    (2, 1, 4, 1536, BF, BF, "odd", "token", None, True, None),
    (2, 1, 9, 2048, BF, BF, "bhtd", "token", "silu", True, [9, 4]),     # a row over a whole block
    (1, 1, 5, 4096, BF, F, "bthd", "token", "silu", True, None),
    (1, 1, 3, 8200, BF, BF, "bhtd", "token", None, True, None),
    (1, 2, 6, 4100, F, F, "bhtd", "token", "silu", True, None),
    (2, 4, 50, 8, BF, BF, "bthd", "sequence", "silu", True, None),
    (3, 2, 300, 24, F, F, "bhtd", "sequence", "silu", True, [300, 0, 1]),
    (2, 32, 130, 48, F, F, "bthd", "sequence", "silu", True, [130, 77]),
    (1, 3, 33, 5, BF, F, "odd", "sequence", None, False, None),
    (1, 1, 1, 16, F, F, "bhtd", "sequence", None, True, None),
    (2, 1, 1025, 520, BF, BF, "proj", "sequence", "silu", True, None),
    (1, 6, 700, 10, F, BF, "bthd", "sequence", "silu", True, [500]),
]


@pytest.mark.parametrize("B,H,T,d,kind,out,layout,over,act,affine,lengths", NORM)
def test_norm(B, H, T, d, kind, out, layout, over, act, affine, lengths):
    r = Draw("norm", B, H, T, d, layout)
    x = r.tokens(B, H, T, d, kind, layout)
    x += 3                                               # a mean beside the spread
    poison(x, lengths)
    w, b = (r.normal(H, d), r.normal(H, d)) if affine else (None, None)
    y, stats = tm.group_norm(x, w, b, over=over, act=act, lengths=lens(lengths), dtype=out)
    assert y.dtype == out
    dy = poison(r.tokens(B, H, T, d, out, layout), lengths)
    g = tm.group_norm_backward(x, dy, stats, w, b, over=over, act=act, lengths=lens(lengths))
    # the mean's rounding (u |mean|, here 4) is relative to the spread; one channel has no spread: the
    # value minus its mean is 0, and 1 / sqrt(eps) makes 300 of what rounding is left
    tol = 64 * U * 4
    dw, db = np.zeros((H, d)), np.zeros((H, d))
    for i, h, n in each(B, H, lengths, T):
        a = dict(weight=None if w is None else f64(w[h]), bias=None if b is None else f64(b[h]), over=over,
                 silu=act == "silu")
        ry, m, rs = M.norm(f64(x[i, h, :n]), **a)
        close(y[i, h, :n], ry, half(out) + tol, "y")
        assert not f64(y[i, h, n:]).any()
        if over == "token":
            assert not f64(stats[i, h, n:]).any()
        if n:
            got = stats[i, h, :n] if over == "token" else stats[i, h]
            close(got[..., 0], m, 64 * U, "mean")
            close(got[..., 1], rs, tol, "rstd")
        elif over == "sequence":
            assert not f64(stats[i, h]).any()
        dx, dwi, dbi = M.norm_backward(f64(x[i, h, :n]), f64(dy[i, h, :n]), **a)
        if d > 1:
            close(g["dx"][i, h, :n], dx, half(kind) + 2 * tol, "dx")
        assert not f64(g["dx"][i, h, n:]).any()
        dw[h] += dwi
        db[h] += dbi
    if affine:
        close(g["dbias"], db, 2 * tol + 128 * U, "dbias")
        if d > 1:
            close(g["dweight"], dw, 2 * tol + 128 * U, "dweight")


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_norm_beside_a_large_mean(over):
    """A mean of 1000 and a spread of 1: the variance does not cancel. x itself is rounded before the call; x - mean
    is exact to 1000 u."""
    r = Draw("mean", over)
    x = r.normal(2, 4, 200, 64) + 1000
    y, _ = tm.group_norm(x, over=over)
    for i, h, n in each(2, 4, None, 200):
        close(y[i, h], M.norm(f64(x[i, h]), over=over)[0], 64 * U + 4 * 1000 * U)


def test_norm_of_constant_rows_is_the_bias():
    x = torch.full((1, 2, 5, 64), 2.5, device="cuda", dtype=BF)
    b = torch.randn(2, 64, device="cuda")
    for over in ("token", "sequence"):
        y, _ = tm.group_norm(x, None, b, over=over, dtype=F)
        assert torch.equal(y, b[None, :, None].expand(1, 2, 5, 64))


# -------------------------------------------------- streams, graphs, buffers

def all_calls(r, kind=BF, lengths=None):
    """One call of every operator, as closures over their inputs."""
    B, H, T, d, N = 2, 2, 400, 64, 16
    _, c, o = scan_case(B, H, 1, T, d, N, kind)
    dy = r.tokens(B, H, T, d, kind)
    f, b, w = r.normal(H, d, 4), r.normal(H, d), r.normal(H, d)
    hist = r.normal(B, H, 3, d, kind=kind)
    st_t, st_s = (tm.group_norm(c["x"], w, b, over=v, act="silu")[1] for v in ("token", "sequence"))
    n = lens(lengths)

    def steps(**k):
        h, s = hist.clone(), o["state"].clone()
        y = tm.short_conv_step(c["x"][:, :, 0], h, f, b, **k)
        q = tm.selective_scan_step(y, c["dt"][:, :, 0], c["A"], c["Bm"][:, :, 0], c["Cm"][:, :, 0], s, **k)
        return y, q, h, s
    return {
        "conv": lambda **k: tm.short_conv(c["x"], f, b, hist=hist, lengths=n, **k),
        "conv_backward": lambda **k: tm.short_conv_backward(c["x"], f, dy, b, hist=hist, lengths=n, **k),
        "scan": lambda **k: tm.selective_scan(**c, **o, lengths=n, **k),
        "scan_backward": lambda **k: tm.selective_scan_backward(**c, dy=dy, **o, lengths=n, **k),
        "token": lambda **k: tm.group_norm(c["x"], w, b, act="silu", lengths=n, **k),
        "sequence": lambda **k: tm.group_norm(c["x"], w, b, over="sequence", act="silu", lengths=n, **k),
        "token_backward": lambda **k: tm.group_norm_backward(c["x"], dy, st_t, w, b, act="silu", lengths=n, **k),
        "sequence_backward": lambda **k: tm.group_norm_backward(c["x"], dy, st_s, w, b, over="sequence", act="silu",
                                                                lengths=n, **k),
        "steps": steps,
    }


def flat(v):
    return list(v.values()) if isinstance(v, dict) else list(v)


def test_same_inputs_same_bits():
    for name, call in all_calls(Draw("bits"), lengths=[400, 123]).items():
        one, two = flat(call()), flat(call())
        assert all(torch.equal(p, q) for p, q in zip(one, two)), name


def test_other_stream():
    calls = all_calls(Draw("stream"))
    want = {k: flat(v()) for k, v in calls.items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for name, call in calls.items():
        if name == "steps":
            continue
        got = flat(call(stream=side))
        # memory that the call freed on its side stream is not handed to this one before it is done
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        side.synchronize()
        del junk
        assert all(torch.equal(p, q) for p, q in zip(got, want[name])), name


def test_two_streams_at_once():
    """The same calls on two streams at the same time, each with its own buffers."""
    calls = all_calls(Draw("two"))
    want = {k: flat(v()) for k, v in calls.items()}
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[(k, flat(v(stream=s))) for k, v in calls.items() if k != "steps"] for _ in range(3) for s in (one, two)]
    torch.cuda.synchronize()
    for each_call in got:
        for k, out in each_call:
            assert all(torch.equal(p, q) for p, q in zip(out, want[k])), k


def test_captured_and_replayed():
    """Every call in one graph, replayed after its inputs changed."""
    calls = all_calls(Draw("graph"))
    first = {k: flat(v()) for k, v in calls.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = {k: flat(v()) for k, v in calls.items()}
    for v in out.values():
        for t in v:
            t.fill_(float("nan"))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for k in out:
            assert all(torch.equal(p, q) for p, q in zip(out[k], first[k])), k


def test_given_buffers_keep_the_rows_behind():
    B, H, T, d, N = 2, 2, 50, 32, 16
    n = [50, 20]
    r, c, o = scan_case(B, H, 1, T, d, N, F, lengths=n)
    f, w = r.normal(H, d, 4), r.normal(H, d)
    out = torch.full((B, H, T, d), 7.0, device="cuda")
    for call in (lambda: tm.short_conv(c["x"], f, lengths=lens(n), out=out),
                 lambda: tm.selective_scan(**c, **o, lengths=lens(n), out=out),
                 lambda: tm.group_norm(c["x"], w, lengths=lens(n), out=out),
                 lambda: tm.group_norm(c["x"], w, over="sequence", lengths=lens(n), out=out)):
        out.fill_(7.0)
        y = call()[0]
        assert y is out and torch.isfinite(out).all()
        assert (out[1, :, 20:] == 7).all() and (out[:, :, :20] != 7).any()


def test_lengths_outside_the_batch_are_held_to_it():
    B, H, T, d, N = 2, 1, 30, 16, 16
    r, c, o = scan_case(B, H, 1, T, d, N, F)
    y, end = tm.selective_scan(**c, **o, lengths=lens([100, -3]))
    full, last = tm.selective_scan(**c, **o)
    assert torch.equal(y[0], full[0]) and torch.equal(end[0], last[0])
    assert not y[1].any() and torch.equal(end[1], o["state"][1])


def test_python_refusals():
    B, H, T, d, N = 1, 2, 8, 16, 16
    r, c, o = scan_case(B, H, 1, T, d, N, BF)
    f = r.normal(H, d, 4)
    for bad in (lambda: tm.short_conv(c["x"].half(), f), lambda: tm.short_conv(c["x"], f.double()),
                lambda: tm.short_conv(c["x"], f, lengths=torch.zeros(B, dtype=torch.int64, device="cuda")),
                lambda: tm.selective_scan(**{**c, "dt": c["dt"].float()}, **o),
                lambda: tm.group_norm(c["x"], dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: tm.short_conv(c["x"], f[:1]), lambda: tm.short_conv(c["x"], f.cpu()),
                lambda: tm.short_conv(c["x"], f, act="relu"), lambda: tm.short_conv(c["x"][..., ::2], f[:, ::2]),
                lambda: tm.short_conv(c["x"][:, :, :0], f), lambda: tm.short_conv_step(c["x"], c["x"], f),
                lambda: tm.selective_scan(**{**c, "Bm": c["Bm"].expand(B, 3, T, N)}, **o),
                lambda: tm.selective_scan(**{**c, "A": c["A"].transpose(1, 2)}, **o),
                lambda: tm.group_norm(c["x"], over="batch"),
                lambda: tm.group_norm_backward(c["x"], c["x"], torch.zeros(B, H, 2, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    out = torch.empty(1, H, T, d, device="cuda", dtype=BF)
    with pytest.raises(tm.TitansMemError):
        tm.short_conv(c["x"], f, out=c["x"])                       # in place
    with pytest.raises(tm.TitansMemError):
        tm.short_conv(c["x"], f, out=out[:, :, :1].expand(B, H, T, d))
    with pytest.raises(tm.TitansMemError):
        tm.short_conv(c["x"], r.normal(H, d, 9))


# ------------------------------------------------------------- in a layer

def layer_weights(r, dim, H, d, N, w):
    s = dim ** -0.5
    return dict(inp=r.normal(dim, 2 * H * d) * s, filt=r.normal(H, d, w) * 0.5, cb=r.normal(H, d) * 0.1,
                par=r.normal(H * d, H * d + 2 * N) * (H * d) ** -0.5, A=-r.uniform(0.5, 4, H, d, N), D=r.normal(H, d),
                dtb=r.uniform(-5, -2, H, d), nw=r.normal(H, d), nb=r.normal(H, d), out=r.normal(H * d, dim) * s)


def layer(p, u, H, d, N, kind, hist=None, state=None, lengths=None):
    """One block as it is used: projection, convolution, scan gated by z, per-head norm, projection."""
    B, T, _ = u.shape
    xz = (u @ p["inp"].to(kind)).view(B, T, 2, H, d)
    x, z = xz[:, :, 0].transpose(1, 2), xz[:, :, 1].transpose(1, 2)
    x, tail = tm.short_conv(x, p["filt"], p["cb"], hist=hist, lengths=lengths)
    q = x.transpose(1, 2).reshape(B, T, H * d) @ p["par"].to(kind)
    dt = q[..., :H * d].view(B, T, H, d).transpose(1, 2)
    Bm, Cm = q[:, None, :, H * d:H * d + N], q[:, None, :, H * d + N:]
    y, state = tm.selective_scan(x, dt, p["A"], Bm, Cm, D=p["D"], z=z, dt_bias=p["dtb"], state=state, lengths=lengths)
    y, _ = tm.group_norm(y, p["nw"], p["nb"], over="token")
    return y.transpose(1, 2).reshape(B, T, H * d) @ p["out"].to(kind), tail, state


def layer_step(p, u, hist, state, H, d, N, kind):
    B = u.shape[0]
    xz = (u @ p["inp"].to(kind)).view(B, 2, H, d)
    x = tm.short_conv_step(xz[:, 0], hist, p["filt"], p["cb"])
    q = x.reshape(B, H * d) @ p["par"].to(kind)
    y = tm.selective_scan_step(x, q[:, :H * d].view(B, H, d), p["A"], q[:, None, H * d:H * d + N], q[:, None, H * d + N:],
                               state, D=p["D"], z=xz[:, 1], dt_bias=p["dtb"])
    y, _ = tm.group_norm(y[:, :, None], p["nw"], p["nb"], over="token")
    return y[:, :, 0].reshape(B, H * d) @ p["out"].to(kind)


@pytest.mark.parametrize("kind,tol", [(F, 2e-5), (BF, 6e-2)])
def test_prompt_then_tokens_equal_one_prompt(kind, tol):
    """A padded batch of prompts, then tokens one by one, against the whole sequences at once. fp32: the products of
    64 to 256 terms and a scan of 90 tokens, 1000 u. bf16: eight roundings to bf16 (2^-8 each) along the block."""
    r = Draw("layer")
    B, H, d, N, dim, T, more = 3, 4, 32, 16, 64, 80, 9
    p = layer_weights(r, dim, H, d, N, 4)
    n = [80, 33, 0]
    u = r.normal(B, T + more, dim, kind=kind)
    _, hist, state = layer(p, u[:, :T], H, d, N, kind, lengths=lens(n))
    whole = [layer(p, u[i:i + 1, :n[i] + more], H, d, N, kind)[0] for i in range(B)]
    for k in range(more):
        tok = torch.stack([u[i, n[i] + k] for i in range(B)])
        y = layer_step(p, tok, hist, state, H, d, N, kind)
        for i in range(B):
            close(y[i], f64(whole[i][0, n[i] + k]), tol)


def test_block_gradients_are_the_oracles():
    """Convolution, scan and norm chained, gradients from the loss back to x, in fp32 against the oracle's chain."""
    r = Draw("chain")
    B, H, T, d, N, w = 2, 2, 70, 24, 16, 4
    _, c, o = scan_case(B, H, 2, T, d, N, F, state=False)
    f, cb, nw, nb = r.normal(H, d, w) * 0.5, r.normal(H, d), r.normal(H, d), r.normal(H, d)
    dy = r.normal(B, H, T, d)
    x = c.pop("x")
    a, _ = tm.short_conv(x, f, cb)
    s, _ = tm.selective_scan(a, **c, **o)
    _, st = tm.group_norm(s, nw, nb, act="silu")
    g3 = tm.group_norm_backward(s, dy, st, nw, nb, act="silu")
    g2 = tm.selective_scan_backward(a, **c, dy=g3["dx"], **o)
    g1 = tm.short_conv_backward(x, f, g2["dx"], cb)
    df = np.zeros((H, d, w))
    for b in range(B):
        for h in range(H):
            ra = M.conv(f64(x[b, h]), f64(f[h]), f64(cb[h]))[0]
            k = scan_ref({**c, "x": a}, o, b, h, T, 2, H)
            k["x"] = ra
            rs, _, _ = M.scan(**k)
            r3, _, _ = M.norm_backward(rs, f64(dy[b, h]), f64(nw[h]), f64(nb[h]), "token", True)
            r2 = M.scan_backward(dy=r3, **k)
            r1, dfi, _, _ = M.conv_backward(f64(x[b, h]), f64(f[h]), r2["dx"], f64(cb[h]))
            # the three operators' own bounds, the norm's carrying the scan's rounding through 1 / spread
            close(g1["dx"][b, h], r1, 20 * (24 * T + 200) * U)
            df[h] += dfi
    close(g1["dfilt"], df, 20 * (24 * T + 200) * U)


def test_norm_of_the_memorys_reads():
    """The reads of a neural memory (fp32, [B, H, T, d]) normalised per head into bf16 for the next projection."""
    from gen import workloads as W
    from gpu_util import run_lib, to_dev
    w = W.make(2, 64, 4, 2, 4, 256, 64, index=955, theta_damping=0.03, alpha_damping=0.01)
    mem = tm.NeuralMemory(w.L, w.d, w.expansion)
    y, _, _ = run_lib(mem, to_dev(W.generate(w), w.B, w.H, w.dtype), w.C)
    r = Draw("reads")
    nw, nb = r.normal(4, 64), r.normal(4, 64)
    got, _ = tm.group_norm(y, nw, nb, over="token", act="silu", dtype=BF)
    for b, h, n in each(2, 4, None, 256):
        # reads may be far smaller than sqrt(eps); the norm's own bound holds all the same
        close(got[b, h], M.norm(f64(y[b, h]), f64(nw[h]), f64(nb[h]), "token", True)[0], half(BF) + 256 * U)
