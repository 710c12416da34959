"""The sequence-mixer kernels in their long runs: many (batch, head) units, so that every thread walks many batches of
rows, with copies in flight and sums carried from batch to batch; split and unsplit scans; calls captured into a
graph and replayed on other inputs. Against tests/mixer_bounds.py, whose values are pinned to the oracle here."""
import numpy as np
import pytest
import torch

import mixer_bounds as R
import test_trained_neural_b200 as tm
from oracle import mixer as M
from test_mixer import BF, F, LENGTHY, Draw, flat, lens, poison, scan_case

gpu = pytest.mark.gpu
U = R.U


# ------------------------------------------------- the definitions themselves

def host(seed, *shape, scale=1.0, shift=0.0):
    return torch.from_numpy(np.random.default_rng([seed, *shape]).standard_normal(shape) * scale + shift)


def same(check, want, what):
    """The batched definition's value is the oracle's (both float64), its bound a number."""
    want = torch.from_numpy(want)
    assert check.ref.shape == check.bound.shape == want.shape, what
    assert torch.allclose(check.ref, want, rtol=1e-11, atol=1e-12), what
    assert (check.bound >= 0).all() and torch.isfinite(check.bound).all(), what


@pytest.mark.parametrize("w,lengths,silu", [(4, None, True), (1, [5, 0], True), (3, [2, 7], False), (7, [7, 3], True)])
def test_conv_definition(w, lengths, silu):
    B, H, T, d = 2, 2, 7, 3
    x, dy, f, b = host(1, B, H, T, d), host(2, B, H, T, d), host(3, H, d, w), host(4, H, d)
    hist, dtail = host(5, B, H, w - 1, d), host(6, B, H, w - 1, d)
    got = R.conv(x, f, b, hist, dy, dtail, lengths, silu, 10)
    out = {k: np.zeros((B, H, T, d)) for k in ("y", "dx")}
    out.update(tail=np.zeros(hist.shape), dhist=np.zeros(hist.shape), dfilt=np.zeros(f.shape), dbias=np.zeros(b.shape))
    for i in range(B):
        for h in range(H):
            n = T if lengths is None else lengths[i]
            a = (x[i, h, :n].numpy(), f[h].numpy())
            more = dict(bias=b[h].numpy(), hist=hist[i, h].numpy(), silu=silu)
            out["y"][i, h, :n], out["tail"][i, h] = M.conv(*a, **more)[:2]
            dx, df, db, dh = M.conv_backward(*a, dy[i, h, :n].numpy(), dtail=dtail[i, h].numpy(), **more)
            out["dx"][i, h, :n], out["dhist"][i, h] = dx, dh
            out["dfilt"][h] += df
            out["dbias"][h] += db
    for k in out:
        same(got[k], out[k], k)


@pytest.mark.parametrize("over,lengths", [("token", None), ("token", [4, 0]), ("sequence", None), ("sequence", [6, 0])])
def test_norm_definition(over, lengths):
    B, H, T, d = 2, 2, 6, 5
    x, dy, w, b = host(1, B, H, T, d, shift=2), host(2, B, H, T, d), host(3, H, d), host(4, H, d)
    got = R.norm(x, w, b, dy, lengths, over, True, 1e-5, 10, 10)
    out = {k: np.zeros((B, H, T, d)) for k in ("y", "dx")}
    kept = (B, H, T) if over == "token" else (B, H)
    out.update(mean=np.zeros(kept), rstd=np.zeros(kept), dweight=np.zeros((H, d)), dbias=np.zeros((H, d)))
    for i in range(B):
        for h in range(H):
            n = T if lengths is None else lengths[i]
            a = dict(weight=w[h].numpy(), bias=b[h].numpy(), over=over, silu=True)
            y, m, r = M.norm(x[i, h, :n].numpy(), **a)
            dx, dw, db = M.norm_backward(x[i, h, :n].numpy(), dy[i, h, :n].numpy(), **a)
            out["y"][i, h, :n], out["dx"][i, h, :n] = y, dx
            out["dweight"][h] += dw
            out["dbias"][h] += db
            if n and over == "token":
                out["mean"][i, h, :n], out["rstd"][i, h, :n] = m, r
            elif n:
                out["mean"][i, h], out["rstd"][i, h] = m, r
    for k in out:
        same(got[k], out[k], k)


@pytest.mark.parametrize("z,lengths,G", [(True, None, 1), (True, [9, 0], 2), (False, [4, 9], 4)])
def test_scan_definition(z, lengths, G):
    B, H, T, d, N = 2, 4, 9, 3, 5
    c = dict(x=host(1, B, H, T, d), dt=host(2, B, H, T, d), A=-host(3, H, d, N).abs(), Bm=host(4, B, G, T, N),
             Cm=host(5, B, G, T, N), D=host(6, H, d), z=host(7, B, H, T, d) if z else None,
             dt_bias=host(8, H, d, shift=-2), state=host(9, B, H, d, N))
    dy, ds = host(10, B, H, T, d), host(11, B, H, d, N)
    got = R.scan(**c, dy=dy, dstate_end=ds, lengths=lengths, segment=16, sums=20)
    out = {k: np.zeros((B, H, T, d)) for k in ("y", "dx", "ddt") + (("dz",) if z else ())}
    out.update({k: np.zeros((B, H, d, N)) for k in ("state_end", "dstate")}, dA=np.zeros((H, d, N)),
               dB=np.zeros((B, G, T, N)), dC=np.zeros((B, G, T, N)), dD=np.zeros((H, d)), ddt_bias=np.zeros((H, d)))
    for i in range(B):
        for h in range(H):
            n, g = (T if lengths is None else lengths[i]), h // (H // G)
            a = dict(x=c["x"][i, h, :n], dt=c["dt"][i, h, :n], A=c["A"][h], Bm=c["Bm"][i, g, :n], Cm=c["Cm"][i, g, :n],
                     D=c["D"][h], z=c["z"][i, h, :n] if z else None, dt_bias=c["dt_bias"][h], state=c["state"][i, h])
            a = {k: None if v is None else v.numpy() for k, v in a.items()}
            out["y"][i, h, :n], out["state_end"][i, h], _ = M.scan(**a)
            ref = M.scan_backward(dy=dy[i, h, :n].numpy(), dstate_end=ds[i, h].numpy(), **a)
            for k in ("dx", "ddt") + (("dz",) if z else ()):
                out[k][i, h, :n] = ref[k]
            out["dstate"][i, h] = ref["dstate"]
            for k in ("dA", "dD", "ddt_bias"):
                out[k][h] += ref[k]
            for k in ("dB", "dC"):
                out[k][i, g, :n] += ref[k]
    for k in out:
        same(got[k], out[k], k)


# ------------------------------------------------------------------ the runs

CONV = [  # B, H, T, d, w, kind, layout, hist, ragged: 300 (batch, head) units, runs of 50 to 84 rows
    (75, 4, 200, 256, 4, BF, "bhtd", False, False),
    (75, 4, 200, 256, 4, F, "bhtd", True, True),
    (75, 4, 201, 130, 3, BF, "bthd", True, True),
    (75, 4, 199, 130, 3, F, "proj", True, False),
    (75, 4, 203, 128, 7, BF, "bhtd", True, True),
    (75, 4, 203, 64, 7, F, "bthd", True, False),
    (150, 2, 333, 65, 4, BF, "odd", True, True),
    (150, 2, 331, 65, 2, F, "bhtd", False, True),
    (300, 1, 230, 100, 1, BF, "bhtd", False, True),
    (150, 2, 222, 66, 8, F, "proj", True, True),
    (100, 3, 250, 68, 5, BF, "bthd", True, False),
    (75, 4, 200, 96, 4, BF, "bthd", False, True),             # heads walked as one row in the gradient
]


def ragged(B, T, on):
    """Whole, empty, shorter than a filter, and anything between."""
    return [[T, 0, 1, T - 1, T // 2, 2, 3 * T // 4, 33][i % 8] for i in range(B)] if on else None


@gpu
@pytest.mark.parametrize("B,H,T,d,w,kind,layout,hist,rag", CONV)
def test_conv_runs(B, H, T, d, w, kind, layout, hist, rag):
    r, n = Draw("conv run", B, H, T, d, w), ragged(B, T, rag)
    x, dy = (poison(r.tokens(B, H, T, d, kind, layout), n) for _ in range(2))
    f, b = r.normal(H, d, w) / w ** 0.5, r.normal(H, d)
    h, dtail = (r.normal(B, H, w - 1, d, kind=kind) if hist else None for _ in range(2))
    y, tail = tm.short_conv(x, f, b, hist=h, lengths=lens(n))
    g = tm.short_conv_backward(x, f, dy, b, hist=h, lengths=lens(n), dtail=dtail)
    # a run of T / 4 rows (or fewer), 4 groups and more of them, the parts of the batch entries 8 at a time
    want = R.conv(x, f, b, h, dy, dtail, n, True, depth=T // 4 + B // 8 + 48)
    for k, t in dict(g, y=y, tail=tail).items():
        want[k](t, k)


NORM = [  # B, H, T, d, kind, out, layout, ragged: 600 units, each CTA steps through all of its unit's rows
    (75, 8, 200, 64, BF, BF, "bhtd", True), (75, 8, 200, 128, BF, BF, "bthd", False), (150, 4, 300, 64, F, F, "bhtd", True),
    (75, 8, 203, 128, F, BF, "proj", True), (75, 8, 101, 256, BF, F, "bhtd", False), (300, 2, 90, 50, BF, BF, "bhtd", True),
    (300, 2, 90, 300, F, F, "bhtd", False), (600, 1, 24, 1536, BF, BF, "bhtd", True), (600, 1, 9, 4096, BF, BF, "bhtd", False),
    (600, 1, 11, 301, F, F, "odd", True), (300, 2, 130, 8, F, F, "bhtd", True),
]


@gpu
@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("B,H,T,d,kind,out,layout,rag", NORM)
def test_norm_runs(B, H, T, d, kind, out, layout, rag, over):
    r, n = Draw("norm run", B, H, T, d), ragged(B, T, rag)
    x = poison(r.tokens(B, H, T, d, kind, layout) + 0.5, n)
    dy = poison(r.tokens(B, H, T, d, out, layout), n)
    w, b = r.normal(H, d) + 1, r.normal(H, d)
    y, stats = tm.group_norm(x, w, b, over=over, act="silu", lengths=lens(n), dtype=out)
    g = tm.group_norm_backward(x, dy, stats, w, b, over=over, act="silu", lengths=lens(n))
    # a token's mean: up to 32 values a lane and 8 joins (301 channels at once a CTA: as many); a sequence's: a run of
    # 64 rows of 8 channels, two at a time, and the row groups
    depth = 48 if over == "token" else 64 * 4 + 64
    # the parameters' sums: the rows of a lane, the row groups, the parts; a sequence's d channels are added up too
    want = R.norm(x, w, b, dy, n, over, True, 1e-5, depth, sums=T + B // 8 + 64)
    for k, t in dict(g, y=y, mean=stats[..., 0], rstd=stats[..., 1]).items():
        want[k](t, k)


def check_scan(c, o, dy, ds, n, segment, sums):
    y, end = tm.selective_scan(**c, **o, lengths=lens(n))
    g = tm.selective_scan_backward(**c, dy=dy, **o, dstate_end=ds, lengths=lens(n))
    want = R.scan(**c, **o, dy=dy, dstate_end=ds, lengths=n, segment=segment, sums=sums)
    for k, t in dict(g, y=y, state_end=end).items():
        want[k](t, k)


@gpu
@pytest.mark.parametrize("strong", [1.0, 20.0])
@pytest.mark.parametrize("B,H,G,T,d,N,kind,layout,D,z,bias,state,lengths", LENGTHY)
def test_scan_split(B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths, strong):
    """Split scans within the bound of their own arithmetic: 20 times stronger decays remember some tens of tokens, so
    that a state, a kept state or a segment's join held in fewer bits would show. Segments of at most 48 tokens here."""
    r, c, o = scan_case(B, H, G, T, d, N, kind, layout, D, z, bias, state, lengths, strong)
    dy, ds = poison(r.tokens(B, H, T, d, kind, layout), lengths), r.normal(B, H, d, N) if state else None
    check_scan(c, o, dy, ds, lengths, segment=64, sums=128)


@gpu
@pytest.mark.parametrize("B,H,G,T,d,N,kind,layout,rag", [
    (60, 8, 8, 700, 64, 16, BF, "bhtd", False), (60, 8, 1, 500, 60, 16, F, "bthd", True), (40, 8, 2, 301, 132, 8, F, "bhtd", True),
    (75, 8, 8, 300, 34, 32, BF, "proj", True)])
def test_scan_unsplit(B, H, G, T, d, N, kind, layout, rag):
    """So many channels that nothing is split: a thread walks all T tokens and sums over them."""
    n = ragged(B, T, rag)
    r, c, o = scan_case(B, H, G, T, d, N, kind, layout, lengths=n)
    dy, ds = poison(r.tokens(B, H, T, d, kind, layout), n), r.normal(B, H, d, N)
    check_scan(c, o, dy, ds, n, segment=T, sums=T + B // 8 + 16)


# -------------------------------------------------------------------- graphs

@gpu
@pytest.mark.parametrize("kind", [BF, F])
def test_replayed_on_other_inputs(kind):
    """Every call captured once, the steps on a stream that forks off and joins; then every input, state, history and
    length changes in place, and a replay gives what eager calls give on the new values."""
    B, H, T, d, N = 3, 2, 400, 64, 16
    r, c, o = scan_case(B, H, 1, T, d, N, kind)
    dy, hist = r.tokens(B, H, T, d, kind), r.normal(B, H, 3, d, kind=kind)
    f, b, w = r.normal(H, d, 4), r.normal(H, d), r.normal(H, d)
    n = lens([400, 123, 0])
    step_hist, step_state = hist.clone(), o["state"].clone()
    changing = [t for t in (*c.values(), *o.values(), dy, hist, f, b, w)]

    def calls():
        out = flat(tm.short_conv(c["x"], f, b, hist=hist, lengths=n))
        out += flat(tm.short_conv_backward(c["x"], f, dy, b, hist=hist, lengths=n))
        out += flat(tm.selective_scan(**c, **o, lengths=n))
        out += flat(tm.selective_scan_backward(**c, dy=dy, **o, lengths=n))
        for over in ("token", "sequence"):
            y, st = tm.group_norm(c["x"], w, b, over=over, act="silu", lengths=n)
            out += [y, st] + flat(tm.group_norm_backward(c["x"], dy, st, w, b, over=over, act="silu", lengths=n))
        return out

    def steps():
        q = tm.short_conv_step(c["x"][:, :, 0], step_hist, f, b)
        y = tm.selective_scan_step(q, c["dt"][:, :, 0], c["A"], c["Bm"][:, :, 0], c["Cm"][:, :, 0], step_state, D=o["D"],
                                   z=o["z"][:, :, 0], dt_bias=o["dt_bias"])
        return [q, y, step_hist, step_state]

    calls(), steps()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            stepped = steps()
        out = calls()
        main.wait_stream(side)
    for k, more in enumerate(([77, 0, 400], [400, 400, 1])):
        for t in changing:
            t.copy_(t.float().flip(0) if t.dim() == 4 else t.float() * (0.5 + k))
        n.copy_(lens(more))
        held = [step_hist.normal_(generator=r.g).clone(), step_state.normal_(generator=r.g).clone()]
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out + stepped]
        step_hist.copy_(held[0])
        step_state.copy_(held[1])
        want = calls() + steps()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(got, want)):
            assert torch.equal(p, q), i


@gpu
def test_steps_on_a_given_stream():
    """`stream=`: the step waits for nothing but its stream, updates hist and state there, and its output belongs to it."""
    B, H, d, N = 64, 4, 96, 16
    r = Draw("step stream")
    x, dt, z = (r.normal(B, H, d, kind=BF) for _ in range(3))
    f, A = r.normal(H, d, 4), -r.uniform(0.5, 4, H, d, N)
    Bm, Cm = r.normal(B, 2, N, kind=BF), r.normal(B, 2, N, kind=BF)
    hist, state = r.normal(B, H, 3, d, kind=BF), r.normal(B, H, d, N)
    h, s = [[t.clone() for _ in range(2)] for t in (hist, state)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        q = tm.short_conv_step(x, h[0], f, stream=side)
        got += [q, tm.selective_scan_step(q, dt, A, Bm, Cm, s[0], z=z, stream=side)]
        junk = torch.full((B, H, d), float("nan"), device="cuda", dtype=BF)   # the current stream's memory, not the side's
        del junk
    side.synchronize()
    for i in range(20):
        q = tm.short_conv_step(x, h[1], f)
        y = tm.selective_scan_step(q, dt, A, Bm, Cm, s[1], z=z)
        assert torch.equal(q, got[2 * i]) and torch.equal(y, got[2 * i + 1])
    assert torch.equal(h[0], h[1]) and torch.equal(s[0], s[1])
