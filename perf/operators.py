"""Timed cases of the sequence-mixer operators that stand beside the neural memory: the short causal
convolution, the selective state-space scan and the group norm with an activation, each forward, backward and
(convolution and scan) for single tokens.

Every tensor of tokens is [B, H, T, d] (batch, head, token, channel) with the channels contiguous and the other
strides free. Formulas, per (batch, head), channel c, token t, state n:

  convolution   p_t[c] = bias[c] + sum_j filt[c, j] x_{t-j}[c],  y = p or p sigmoid(p)
  scan          e = softplus(dt + dt_bias),  h_t[c, n] = exp(e A[c, n]) h_{t-1}[c, n] + e x_t[c] Bm_t[n],
                y_t[c] = (sum_n Cm_t[n] h_t[c, n] + D[c] x_t[c]) * z_t[c] sigmoid(z_t[c])
  group norm    p = weight (x - mean) / sqrt(var + eps) + bias over the d channels of one token, or of all the
                tokens of a sequence;  y = p or p sigmoid(p)

`lengths` gives the tokens of each sequence of a padded batch; rows behind them are zero in the outputs.
"""
import math

import torch

own = False

F32, F64 = torch.float32, torch.float64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token for each of 64 requests, at the framework's 1536-wide hidden layer
        dict(name="conv step 64x1536", op="conv", way="step", B=64, H=1, T=1, d=1536, w=4, dtype="bf16"),
        # one long prompt over 16 heads of 128, read as [B, T, H d]
        dict(name="conv prompt 65536x2048", op="conv", way="forward", B=1, H=16, T=65536, d=128, w=4, dtype="bf16",
             layout="bthd"),
        # a padded batch of odd sizes in fp32, with the tokens before the call
        dict(name="conv ragged f32", op="conv", way="forward", B=5, H=3, T=1021, d=50, w=3, dtype="f32", hist=True,
             ragged=True),
        # training: the eight-head workload of the memory
        dict(name="conv gradient 4x8x8192x64", op="conv", way="backward", B=4, H=8, T=8192, d=64, w=4, dtype="bf16"),
        # one token for each of 64 requests
        dict(name="scan step 64x1536", op="scan", way="step", B=64, H=1, T=1, d=1536, N=16, G=1, dtype="bf16",
             layout="proj"),
        # one prompt on its own: few rows, a long axis; x and z are the halves of one projection
        dict(name="scan prompt 8192x2048", op="scan", way="forward", B=1, H=16, T=8192, d=128, N=16, G=1,
             dtype="bf16", layout="proj"),
        # a padded batch of odd sizes in fp32, carried on from a state
        dict(name="scan ragged f32", op="scan", way="forward", B=3, H=6, T=1021, d=52, N=12, G=3, dtype="f32",
             state=True, ragged=True),
        # training: the eight-head workload of the memory, B and C of each head its own
        dict(name="scan gradient 4x8x8192x64", op="scan", way="backward", B=4, H=8, T=8192, d=64, N=16, G=8,
             dtype="bf16"),
        # gradients of a short odd padded batch in fp32, through its initial state
        dict(name="scan gradient ragged f32", op="scan", way="backward", B=2, H=2, T=301, d=100, N=8, G=1,
             dtype="f32", state=True, ragged=True),
        # the reads of 8 heads, normalised token by token
        dict(name="norm token 4x8x8192x64", op="norm", way="forward", B=4, H=8, T=8192, d=64, dtype="bf16",
             over="token", layout="bthd"),
        # training: normalised token by token
        dict(name="norm gradient 8x8x8192x128", op="norm", way="backward", B=8, H=8, T=8192, d=128, dtype="bf16",
             over="token"),
        # 32 groups of the 1536 channels over a whole odd-sized sequence, channels last, fp32
        dict(name="norm sequence 2x4001x1536", op="norm", way="forward", B=2, H=32, T=4001, d=48, dtype="f32",
             over="sequence", layout="bthd"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op, way = rng.choice([("conv", "forward"), ("conv", "backward"), ("conv", "step"), ("scan", "forward"),
                          ("scan", "backward"), ("scan", "step"), ("norm", "forward"), ("norm", "backward")])
    c = dict(op=op, way=way, dtype=rng.choice(["bf16", "bf16", "f32"]))
    c["H"] = rng.choice([1, 2, 3, 4, 8, 16])
    c["d"] = rng.choice([spread(16, 2048 // c["H"]), 16 * spread(1, 128 // c["H"])])
    if way == "step":
        c["B"], c["T"] = spread(1, 256), 1
    else:
        most = 1 << (24 if op == "scan" else 26)         # elements of one tensor
        c["B"] = spread(1, 8)
        c["T"] = max(1, min(spread(1, 32768), most // (c["B"] * c["H"] * c["d"])))
    c["layout"] = rng.choice(["bhtd", "bthd", "proj"])
    if op == "conv":
        c["w"] = rng.choice([2, 3, 4, 4, 4, 7])
        c["hist"] = way == "step" or rng.random() < 0.5
    if op == "scan":
        c["N"] = rng.choice([4, 8, 16, 16, 12])
        c["G"] = rng.choice([g for g in (1, 2, 4, c["H"]) if c["H"] % g == 0])
        c["state"] = way == "step" or rng.random() < 0.5
    if op == "norm":
        c["over"] = rng.choice(["token", "token", "sequence"])
        c["act"] = rng.choice(["silu", "none"])
    c["ragged"] = way != "step" and rng.random() < 0.3
    return c


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    rows = c["B"] * c["H"] * c["T"]
    n = rows * c["d"]
    ch = c["H"] * c["d"]
    op, way = c["op"], c["way"]
    if op == "conv":
        w = c["w"]
        par = ch * (w + 1) * 4
        hist = c["B"] * ch * (w - 1) * e
        if way == "step":
            return {"bytes": 2 * n * e + 2 * hist + par, "flops": n * (2 * w + 6)}
        if way == "forward":
            return {"bytes": 2 * n * e + (2 if c.get("hist") else 1) * hist + par, "flops": n * (2 * w + 6)}
        return {"bytes": 3 * n * e + 2 * par + (2 * hist if c.get("hist") else 0), "flops": n * (6 * w + 12)}
    if op == "scan":
        N = c["N"]
        bc = 2 * c["B"] * c["G"] * c["T"] * N * e
        par = ch * (N + 2) * 4
        st = c["B"] * ch * N * 4
        if way in ("step", "forward"):
            return {"bytes": 4 * n * e + bc + par + st * (2 if way == "step" or c.get("state") else 1),
                    "flops": n * (7 * N + 16)}
        return {"bytes": 7 * n * e + 2 * bc + 2 * par + st * (3 if c.get("state") else 1), "flops": n * (25 * N + 40)}
    stat = (rows if c["over"] == "token" else c["B"] * c["H"]) * 8
    if way == "forward":
        return {"bytes": 2 * n * e + stat + 2 * ch * 4, "flops": n * 12}
    return {"bytes": 3 * n * e + stat + 4 * ch * 4, "flops": n * 22}


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    c = dict(case)
    B, H, T, d, dtype = c["B"], c["H"], c["T"], c["d"], TYPES[c["dtype"]]
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    layout = c.get("layout", "bhtd")

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=F32)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda", dtype=F32)

    def tokens(many=1):
        """`many` token tensors [B, H, T, d] in the case's layout; "proj": slices of one projection."""
        if layout == "proj":
            both = normal(B, T, max(2, many), H, d).to(dtype)
            return [both[:, :, i].transpose(1, 2) for i in range(many)]
        if layout == "bthd":
            return [normal(B, T, H, d).to(dtype).transpose(1, 2) for _ in range(many)]
        return [normal(B, H, T, d).to(dtype) for _ in range(many)]

    s = {"case": c, "lengths": None}
    if c.get("ragged"):
        # one full sequence, one empty where there are three, the rest anywhere
        n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        n[0] = T
        if B > 2:
            n[B - 1] = 0
        s["lengths"] = n
    back = c["way"] == "backward"
    if c["op"] == "conv":
        w = c["w"]
        s["x"] = tokens()[0]
        s["filt"] = normal(H, d, w) / math.sqrt(w)
        s["bias"] = 0.1 * normal(H, d)
        s["hist"] = normal(B, H, w - 1, d).to(dtype) if c["way"] == "step" or c.get("hist") else None
        if back:
            s["dy"] = tokens()[0]
    elif c["op"] == "scan":
        N, G = c["N"], c["G"]
        s["x"], s["z"] = tokens(2)
        s["dt"] = tokens()[0].mul_(0.5)
        # softplus(dt_bias) spread over [1e-3, 1e-1] in its logarithm; A near -(1 .. N)
        e = torch.exp(uniform(H, d) * math.log(100.0) + math.log(1e-3))
        s["dt_bias"] = e + torch.log(-torch.expm1(-e))
        s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=F32) * torch.exp(0.1 * normal(H, d, N))
        s["D"] = 1 + 0.1 * normal(H, d)
        s["Bm"] = normal(B, G, T, N).to(dtype)
        s["Cm"] = normal(B, G, T, N).to(dtype)
        s["state"] = normal(B, H, d, N) if c["way"] == "step" or c.get("state") else None
        if back:
            s["dy"] = tokens()[0]
            s["dstate_end"] = normal(B, H, d, N) if c.get("state") else None
    else:
        s["x"] = tokens()[0]
        s["weight"] = 1 + 0.1 * normal(H, d)
        s["bias"] = 0.1 * normal(H, d)
        s["act"] = c.get("act", "silu")
        if back:
            s["dy"] = tokens()[0]
            # what the forward call kept
            x, n = s["x"].double(), s["lengths"]
            n = torch.full((B,), T, device="cuda") if n is None else n.long()
            live = (torch.arange(T, device="cuda") < n[:, None])[:, None, :, None]
            x = torch.where(live, x, 0.0)
            if c["over"] == "token":
                m = x.mean(-1)
                r = torch.rsqrt((x - m[..., None]).square().mean(-1) + 1e-5) * live[..., 0]
            else:
                k = (n * d).clamp(min=1).view(B, 1)
                m = x.sum((2, 3)) / k
                v = (torch.where(live, x - m[..., None, None], 0.0)).square().sum((2, 3)) / k
                r = torch.rsqrt(v + 1e-5) * (n > 0).view(B, 1)
            s["stats"] = torch.stack([m, r], -1).float()
    return s


# ------------------------------------------------------------ plain forms

def _live(s):
    """[B, 1, T, 1]: whether a row is one of its sequence's tokens; None where all are."""
    if s["lengths"] is None:
        return None
    T = s["x"].shape[2]
    return (torch.arange(T, device="cuda", dtype=torch.int32) < s["lengths"][:, None])[:, None, :, None]


def _masked(x, live):
    x = x.to(F32)
    return x if live is None else torch.where(live, x, torch.zeros((), device=x.device))


def _taps(full, w, T):
    """full [B, H, w - 1 + T, d] -> [B, H, T, d, w], tap j the row j tokens back."""
    return full.unfold(2, w, 1).flip(-1)[:, :, :T]


def _conv_pre(s):
    live = _live(s)
    x = _masked(s["x"], live)
    B, H, T, d = x.shape
    w = s["filt"].shape[-1]
    old = s["hist"].to(F32) if s["hist"] is not None else x.new_zeros(B, H, w - 1, d)
    full = torch.cat([old, x], 2)
    taps = _taps(full, w, T)
    return live, full, taps, (taps * s["filt"][None, :, None]).sum(-1) + s["bias"][None, :, None]


def _conv_forward(s):
    live, full, _, p = _conv_pre(s)
    dtype = s["x"].dtype
    B, H, T, d = s["x"].shape
    w = s["filt"].shape[-1]
    y = _masked(p * torch.sigmoid(p), live).to(dtype)
    n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
    rows = (n[:, None] + torch.arange(w - 1, device="cuda"))[:, None, :, None].expand(B, H, w - 1, d)
    return y, torch.gather(full, 2, rows).to(dtype)


def _conv_step(s):
    x, hist = s["x"][:, :, 0], s["hist"]
    full = torch.cat([hist.to(F32), x[:, :, None].to(F32)], 2)
    p = (full.flip(2).transpose(2, 3) * s["filt"]).sum(-1) + s["bias"]
    hist.copy_(full[:, :, 1:])
    return (p * torch.sigmoid(p)).to(x.dtype), hist


def _conv_backward(s):
    live, full, taps, p = _conv_pre(s)
    dtype = s["x"].dtype
    B, H, T, d = s["x"].shape
    w = s["filt"].shape[-1]
    q = torch.sigmoid(p)
    g = _masked(_masked(s["dy"], live) * (q * (1 + p * (1 - q))), live)
    df = (g[..., None] * taps).sum((0, 2))
    db = g.sum((0, 2))
    # row t of the inputs feeds outputs t .. t + w - 1; rows before the call are the history's
    pad = g.new_zeros(B, H, w - 1, d)
    ahead = torch.cat([pad, g, pad], 2).unfold(2, w, 1)
    dfull = (ahead * s["filt"][None, :, None]).sum(-1)
    out = {"dx": _masked(dfull[:, :, w - 1:], live).to(dtype), "dfilt": df, "dbias": db}
    if s["hist"] is not None:
        out["dhist"] = dfull[:, :, :w - 1].to(dtype)
    return out


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 2, all tokens at once: spans of 1, 2, 4, ... tokens are joined, so
    the loop runs over the logarithm of the length."""
    a, b, k = a.clone(), b.clone(), 1
    while k < b.shape[2]:
        b[:, :, k:] = b[:, :, k:] + a[:, :, k:] * b[:, :, :-k]
        a[:, :, k:] = a[:, :, k:] * a[:, :, :-k]
        k *= 2
    return b


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _scan_parts(s):
    live = _live(s)
    x, z = _masked(s["x"], live), _masked(s["z"], live)
    v = _masked(s["dt"], live) + s["dt_bias"][None, :, None]
    e = _masked(_softplus(v), live)
    each = x.shape[1] // s["Bm"].shape[1]
    Bm = _masked(s["Bm"], live).repeat_interleave(each, 1)
    Cm = _masked(s["Cm"], live).repeat_interleave(each, 1)
    a = torch.exp(e[..., None] * s["A"][None, :, None])
    b = (e * x)[..., None] * Bm[:, :, :, None]
    if s["state"] is not None:
        b[:, :, 0] += a[:, :, 0] * s["state"]
    return live, x, z, v, e, Bm, Cm, a, _recurrence(a, b)


def _scan_forward(s):
    live, x, z, _, _, _, Cm, _, h = _scan_parts(s)
    y = (h * Cm[:, :, :, None]).sum(-1) + s["D"][None, :, None] * x
    y = y * (z * torch.sigmoid(z))
    return _masked(y, live).to(s["x"].dtype), h[:, :, -1].contiguous()


def _scan_step(s):
    x, z, dt = (s[k][:, :, 0].to(F32) for k in ("x", "z", "dt"))
    each = x.shape[1] // s["Bm"].shape[1]
    Bm, Cm = (s[k][:, :, 0].to(F32).repeat_interleave(each, 1) for k in ("Bm", "Cm"))
    e = _softplus(dt + s["dt_bias"])
    h = torch.exp(e[..., None] * s["A"]) * s["state"] + (e * x)[..., None] * Bm[:, :, None]
    s["state"].copy_(h)
    y = (h * Cm[:, :, None]).sum(-1) + s["D"] * x
    return (y * (z * torch.sigmoid(z))).to(s["x"].dtype), s["state"]


def _scan_backward(s):
    live, x, z, v, e, Bm, Cm, a, h = _scan_parts(s)
    dtype = s["x"].dtype
    B, H, T, d = x.shape
    G, N = s["Bm"].shape[1], s["Bm"].shape[3]
    D = s["D"][None, :, None]
    dy = _masked(s["dy"], live)
    q = torch.sigmoid(z)
    y = (h * Cm[:, :, :, None]).sum(-1) + D * x
    dz = dy * y * (q * (1 + z * (1 - q)))
    dy = dy * (z * q)
    # g_t = dL/dh_t = Cm_t dy_t + a_{t+1} g_{t+1}
    k = Cm[:, :, :, None] * dy[..., None]
    if s["dstate_end"] is not None:
        k[:, :, -1] += s["dstate_end"]
    later = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], 2)
    g = _recurrence(later.flip(2), k.flip(2)).flip(2)
    del later, k
    first = s["state"] if s["state"] is not None else torch.zeros_like(h[:, :, 0])
    before = torch.cat([first[:, :, None], h[:, :, :-1]], 2)
    ga = g * a * before                                # dL/d(e A)
    gB = (g * Bm[:, :, :, None]).sum(-1)               # dL/d(e x)
    de = gB * x + (ga * s["A"][None, :, None]).sum(-1)
    ddt = de * torch.sigmoid(v)
    out = {"dx": _masked(gB * e + D * dy, live).to(dtype), "ddt": _masked(ddt, live).to(dtype),
           "dA": (ga * e[..., None]).sum((0, 2)),
           "dB": (g * (e * x)[..., None]).sum(3).view(B, G, H // G, T, N).sum(2).to(dtype),
           "dC": (h * dy[..., None]).sum(3).view(B, G, H // G, T, N).sum(2).to(dtype),
           "dD": (dy * x).sum((0, 2)), "dz": dz.to(dtype), "ddt_bias": _masked(ddt, live).sum((0, 2))}
    if s["state"] is not None:
        out["dstate"] = a[:, :, 0] * g[:, :, 0]
    return out


def _norm_forward(s):
    live = _live(s)
    x = _masked(s["x"], live)
    B, H, T, d = x.shape
    if s["case"]["over"] == "token":
        m = x.mean(-1)
        r = torch.rsqrt((x - m[..., None]).square().mean(-1) + 1e-5)
        r = r if live is None else torch.where(live[..., 0], r, torch.zeros((), device="cuda"))
        mm, rr = m[..., None], r[..., None]
    else:
        n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
        k = (n * d).clamp(min=1).view(B, 1)
        m = (x.double().sum((2, 3)) / k).float()
        v = _masked(x - m[..., None, None], live).double().square().sum((2, 3)) / k
        r = (torch.rsqrt(v + 1e-5) * (n > 0).view(B, 1)).float()
        mm, rr = m[..., None, None], r[..., None, None]
    p = (x - mm) * rr * s["weight"][None, :, None] + s["bias"][None, :, None]
    y = p * torch.sigmoid(p) if s["act"] == "silu" else p
    return _masked(y, live).to(s["x"].dtype), torch.stack([m, r], -1)


def _norm_backward(s):
    live = _live(s)
    x = _masked(s["x"], live)
    dy = _masked(s["dy"], live)
    B, H, T, d = x.shape
    token = s["case"]["over"] == "token"
    m, r = s["stats"].unbind(-1)
    m, r = (m[..., None], r[..., None]) if token else (m[..., None, None], r[..., None, None])
    xh = (x - m) * r
    if s["act"] == "silu":
        p = xh * s["weight"][None, :, None] + s["bias"][None, :, None]
        q = torch.sigmoid(p)
        dy = dy * (q * (1 + p * (1 - q)))
    dy, xh = _masked(dy, live), _masked(xh, live)
    g = dy * s["weight"][None, :, None]
    if token:
        g1, g2 = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    else:
        n = torch.full((B,), T, device="cuda") if s["lengths"] is None else s["lengths"].long()
        k = (n * d).clamp(min=1).view(B, 1, 1, 1)
        g1, g2 = (t.sum((2, 3), keepdim=True) / k for t in (g, g * xh))
    return {"dx": _masked((g - g1 - xh * g2) * r, live).to(s["x"].dtype),
            "dweight": (dy * xh).sum((0, 2)), "dbias": dy.sum((0, 2))}


def _own(s):
    import test_trained_neural_b200 as tm
    c = s["case"]
    op, way = c["op"], c["way"]
    if op == "conv":
        if way == "step":
            return tm.short_conv_step(s["x"][:, :, 0], s["hist"], s["filt"], s["bias"]), s["hist"]
        if way == "forward":
            return tm.short_conv(s["x"], s["filt"], s["bias"], hist=s["hist"], lengths=s["lengths"])
        return tm.short_conv_backward(s["x"], s["filt"], s["dy"], s["bias"], hist=s["hist"], lengths=s["lengths"])
    if op == "scan":
        if way == "step":
            y = tm.selective_scan_step(s["x"][:, :, 0], s["dt"][:, :, 0], s["A"], s["Bm"][:, :, 0], s["Cm"][:, :, 0],
                                       s["state"], D=s["D"], z=s["z"][:, :, 0], dt_bias=s["dt_bias"])
            return y, s["state"]
        more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"], state=s["state"], lengths=s["lengths"])
        if way == "forward":
            return tm.selective_scan(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], **more)
        return tm.selective_scan_backward(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["dy"],
                                          dstate_end=s["dstate_end"], **more)
    more = dict(over=c["over"], act=s["act"], lengths=s["lengths"])
    if way == "forward":
        return tm.group_norm(s["x"], s["weight"], s["bias"], **more)
    return tm.group_norm_backward(s["x"], s["dy"], s["stats"], s["weight"], s["bias"], **more)


PLAIN = {("conv", "forward"): _conv_forward, ("conv", "backward"): _conv_backward, ("conv", "step"): _conv_step,
         ("scan", "forward"): _scan_forward, ("scan", "backward"): _scan_backward, ("scan", "step"): _scan_step,
         ("norm", "forward"): _norm_forward, ("norm", "backward"): _norm_backward}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"], state["case"]["way"]](state)


# ------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """run()'s outputs from the definitions in 64 bits, sequence by sequence and token by token; the gradients by
    differentiating that."""
    s = prepare(case, seed)
    c = s["case"]
    op, way = c["op"], c["way"]
    B, H, T, d = s["x"].shape
    lens = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    names = {"conv": ["x", "filt", "bias", "hist"], "scan": ["x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state"],
             "norm": ["x", "weight", "bias"]}[op]
    back = way == "backward"
    if back and op == "scan" and B * H * d * T * c["N"] * 8 > 12e9:
        return None
    v = {k: s[k].to(F64).requires_grad_(back) for k in names if s[k] is not None}
    zero = torch.zeros((), device="cuda", dtype=F64)

    def conv():
        w = c["w"]
        hist = v["hist"] if "hist" in v else torch.zeros(B, H, w - 1, d, device="cuda", dtype=F64)
        ys, tails = [], []
        for b in range(B):
            n = lens[b]
            rows = torch.cat([hist[b], v["x"][b, :, :n]], 1)
            y = v["bias"][:, None].expand(H, n, d)
            for j in range(w):
                y = y + v["filt"][:, None, :, j] * rows[:, w - 1 - j:w - 1 - j + n]
            y = y / (1 + torch.exp(-y))
            ys.append(torch.cat([y, zero.expand(H, T - n, d)], 1))
            tails.append(rows[:, n:])
        return torch.stack(ys), torch.stack(tails)

    def scan():
        e = torch.logaddexp(v["dt"] + v["dt_bias"][:, None], zero)
        each = H // c["G"]
        h = v["state"] if "state" in v else torch.zeros(B, H, d, c["N"], device="cuda", dtype=F64)
        n = torch.tensor(lens, device="cuda")
        on_all = (torch.arange(T, device="cuda")[:, None] < n)[:, :, None, None, None]
        ragged = min(lens) < T
        Bs, Cs = (v[k].repeat_interleave(each, 1)[:, :, :, None].unbind(2) for k in ("Bm", "Cm"))
        es, us = e[..., None].unbind(2), (e * v["x"])[..., None].unbind(2)
        ys = []
        for t in range(T):
            new = torch.exp(es[t] * v["A"]) * h + us[t] * Bs[t]
            h = torch.where(on_all[t], new, h) if ragged else new
            ys.append((h * Cs[t]).sum(-1))
        y = (torch.stack(ys, 2) + v["D"][:, None] * v["x"]) * v["z"] / (1 + torch.exp(-v["z"]))
        return torch.where(on_all[..., 0].permute(1, 2, 0, 3), y, zero), h

    def norm():
        ys, stats = [], []
        for b in range(B):
            n = lens[b]
            x = v["x"][b, :, :n]
            dims = -1 if c["over"] == "token" else (1, 2)
            if n:
                m = x.mean(dims, keepdim=True)
                r = ((x - m).square().mean(dims, keepdim=True) + 1e-5) ** -0.5
                p = (x - m) * r * v["weight"][:, None] + v["bias"][:, None]
                p = p / (1 + torch.exp(-p)) if s["act"] == "silu" else p
            else:
                p = x
                m = r = torch.zeros(H, 0 if c["over"] == "token" else 1, 1, device="cuda", dtype=F64)
            ys.append(torch.cat([p, zero.expand(H, T - n, d)], 1))
            st = torch.cat([m, r], -1)
            stats.append(torch.cat([st, zero.expand(H, T - n, 2)], 1) if c["over"] == "token" else st[:, 0])
        return torch.stack(ys), torch.stack(stats)

    y, more = {"conv": conv, "scan": scan, "norm": norm}[op]()
    if not back:
        return (y[:, :, 0], more) if way == "step" else (y, more)
    loss = (y * s["dy"].to(F64)).sum()
    if s.get("dstate_end") is not None:
        loss = loss + (more * s["dstate_end"].to(F64)).sum()
    grads = dict(zip(v, torch.autograd.grad(loss, list(v.values()))))
    said = {"Bm": "dB", "Cm": "dC"}
    return {said.get(k, "d" + k): t for k, t in grads.items()}
