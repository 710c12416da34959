"""Float64 oracle of the sequence-mixer operators (test infrastructure only):
plain loops over the definitions in include/titansmem.h, for one sequence of one
head at a time, and their gradients written out by hand.
"""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    x = np.asarray(x, dtype=np.float64)
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(p, silu):
    return p * sigmoid(p) if silu else p


def act_grad(p, silu):
    q = sigmoid(p)
    return q * (1 + p * (1 - q)) if silu else np.ones_like(p)


def conv(x, filt, bias=None, hist=None, silu=True):
    """x [T, d], filt [d, w], bias [d], hist [w-1, d] -> (y [T, d], tail [w-1, d], pre-activation, rows)."""
    T, d = x.shape
    w = filt.shape[1]
    rows = np.concatenate([np.zeros((w - 1, d)) if hist is None else hist, x])
    p = np.zeros((T, d)) + (0 if bias is None else bias)
    for t in range(T):
        for j in range(w):
            p[t] += filt[:, j] * rows[w - 1 + t - j]
    return act(p, silu), rows[T:], p, rows


def conv_backward(x, filt, dy, bias=None, hist=None, silu=True, dtail=None):
    """-> dx [T, d], dfilt [d, w], dbias [d], dhist [w-1, d]."""
    T, d = x.shape
    w = filt.shape[1]
    _, _, p, rows = conv(x, filt, bias, hist, silu)
    g = dy * act_grad(p, silu)
    drows = np.zeros_like(rows)
    dfilt = np.zeros((d, w))
    for t in range(T):
        for j in range(w):
            drows[w - 1 + t - j] += filt[:, j] * g[t]
            dfilt[:, j] += g[t] * rows[w - 1 + t - j]
    if dtail is not None and w > 1:
        drows[T:] += dtail
    return drows[w - 1:], dfilt, g.sum(0), drows[:w - 1]


def scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, state=None, softplus=True):
    """x, dt, z [T, d]; Bm, Cm [T, N]; A, state [d, N]; D, dt_bias [d] -> (y [T, d], state_end, kept values)."""
    T, d = x.shape
    v = dt + (0 if dt_bias is None else dt_bias)
    e = np.logaddexp(v, 0.0) if softplus else v
    h = np.zeros((d, A.shape[1])) if state is None else state.copy()
    hs, s = [h.copy()], np.zeros((T, d))
    for t in range(T):
        h = np.exp(e[t][:, None] * A) * h + (e[t] * x[t])[:, None] * Bm[t]
        hs.append(h.copy())
        s[t] = h @ Cm[t]
    s = s + (0 if D is None else D) * x
    y = s if z is None else s * act(z, True)
    return y, h, (v, e, hs, s)


def scan_backward(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, state=None, softplus=True, dstate_end=None):
    """-> dict of dx, ddt, dA, dB, dC, dD, dz, ddt_bias, dstate."""
    T, d = x.shape
    _, _, (v, e, hs, s) = scan(x, dt, A, Bm, Cm, D, z, dt_bias, state, softplus)
    k = dy if z is None else dy * act(z, True)
    out = {"dx": np.zeros((T, d)), "dA": np.zeros_like(A), "dB": np.zeros_like(Bm), "dC": np.zeros_like(Cm)}
    out["dz"] = None if z is None else dy * act_grad(z, True) * s
    out["dD"] = (k * x).sum(0)
    de = np.zeros((T, d))
    R = np.zeros_like(A) if dstate_end is None else dstate_end.copy()    # gradient of h_t from later tokens
    for t in range(T - 1, -1, -1):
        g = R + k[t][:, None] * Cm[t]
        a = np.exp(e[t][:, None] * A)
        du = g @ Bm[t]
        q = g * a * hs[t]
        out["dx"][t] = du * e[t] + (0 if D is None else D) * k[t]
        out["dB"][t] = (e[t] * x[t]) @ g
        out["dC"][t] = k[t] @ hs[t + 1]
        out["dA"] += e[t][:, None] * q
        de[t] = du * x[t] + (q * A).sum(1)
        R = g * a
    out["ddt"] = de * sigmoid(v) if softplus else de
    out["ddt_bias"] = out["ddt"].sum(0)
    out["dstate"] = R
    return out


def norm(x, weight=None, bias=None, over="token", silu=False, eps=1e-5):
    """x [T, d] -> (y [T, d], mean, 1 / sqrt(var + eps)): per token, or scalars; None for no tokens."""
    if x.shape[0] == 0:
        return x.copy(), None, None
    axes = 1 if over == "token" else (0, 1)
    m = x.mean(axis=axes, keepdims=True)
    r = 1 / np.sqrt(((x - m) ** 2).mean(axis=axes, keepdims=True) + eps)
    p = (x - m) * r * (1 if weight is None else weight) + (0 if bias is None else bias)
    return act(p, silu), m[:, 0] if over == "token" else m[0, 0], r[:, 0] if over == "token" else r[0, 0]


def norm_backward(x, dy, weight=None, bias=None, over="token", silu=False, eps=1e-5):
    """-> dx [T, d], dweight [d], dbias [d]."""
    if x.shape[0] == 0:
        return x.copy(), np.zeros(x.shape[1]), np.zeros(x.shape[1])
    axes = 1 if over == "token" else (0, 1)
    m = x.mean(axis=axes, keepdims=True)
    r = 1 / np.sqrt(((x - m) ** 2).mean(axis=axes, keepdims=True) + eps)
    xh = (x - m) * r
    w = 1 if weight is None else weight
    q = dy * act_grad(xh * w + (0 if bias is None else bias), silu)
    k = q * w
    dx = r * (k - k.mean(axis=axes, keepdims=True) - xh * (k * xh).mean(axis=axes, keepdims=True))
    return dx, (q * xh).sum(0), q.sum(0)
