"""The float64 oracle of the sequence-mixer operators, held to library routines,
closed forms and finite differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import mixer as M


def rng_of(*key):
    return np.random.default_rng(key)


def test_conv_is_numpy_convolve_and_carries_its_tail():
    r = rng_of(1)
    x, f, b = r.standard_normal((23, 3)), r.standard_normal((3, 4)), r.standard_normal(3)
    y, tail, _, _ = M.conv(x, f, b, silu=False)
    for c in range(3):
        np.testing.assert_allclose(y[:, c], np.convolve(x[:, c], f[c])[:23] + b[c], rtol=1e-13, atol=1e-13)
    np.testing.assert_array_equal(tail, x[-3:])
    y1, t1, _, _ = M.conv(x[:2], f, b)
    y2, t2, _, _ = M.conv(x[2:], f, b, hist=t1)
    np.testing.assert_allclose(np.concatenate([y1, y2]), M.conv(x, f, b)[0], rtol=1e-13, atol=1e-13)
    np.testing.assert_array_equal(t2, tail)


def test_silu_is_torchs():
    x = np.linspace(-40, 40, 101)
    np.testing.assert_allclose(M.act(x, True), torch.nn.functional.silu(torch.from_numpy(x)).numpy(), rtol=1e-13)
    t = torch.from_numpy(x).requires_grad_()
    torch.nn.functional.silu(t).sum().backward()
    np.testing.assert_allclose(M.act_grad(x, True), t.grad.numpy(), rtol=1e-12, atol=1e-15)


def test_scan_without_decay_is_a_running_sum():
    r = rng_of(2)
    T, d, N = 9, 3, 2
    x, Bm, Cm = r.standard_normal((T, d)), r.standard_normal((T, N)), r.standard_normal((T, N))
    dt = r.uniform(0.1, 1, (T, d))
    y, h, _ = M.scan(x, dt, np.zeros((d, N)), Bm, Cm, softplus=False)
    run = np.cumsum((dt * x)[:, :, None] * Bm[:, None], 0)
    np.testing.assert_allclose(y, (run * Cm[:, None]).sum(2), rtol=1e-12)
    np.testing.assert_allclose(h, run[-1], rtol=1e-12)


def test_scan_forgets_under_a_strong_decay_and_carries_its_state():
    r = rng_of(3)
    T, d, N = 8, 2, 3
    x, dt, z = (r.standard_normal((T, d)) for _ in range(3))
    A, Bm, Cm = -r.uniform(0.1, 2, (d, N)), r.standard_normal((T, N)), r.standard_normal((T, N))
    D, bias, h0 = r.standard_normal(d), r.standard_normal(d), r.standard_normal((d, N))
    y, h, _ = M.scan(x, dt, A, Bm, Cm, D, z, bias, h0)
    y1, h1, _ = M.scan(x[:5], dt[:5], A, Bm[:5], Cm[:5], D, z[:5], bias, h0)
    y2, h2, _ = M.scan(x[5:], dt[5:], A, Bm[5:], Cm[5:], D, z[5:], bias, h1)
    np.testing.assert_allclose(np.concatenate([y1, y2]), y, rtol=1e-12)
    np.testing.assert_allclose(h2, h, rtol=1e-12)
    # exp(e A) = 0: every token alone
    y, _, _ = M.scan(x, np.ones((T, d)), np.full((d, N), -1e9), Bm, Cm, softplus=False)
    np.testing.assert_allclose(y, x * (Bm * Cm).sum(1)[:, None], rtol=1e-12)


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_norm_is_torchs_group_norm(over):
    r = rng_of(4)
    B, H, T, d = 2, 3, 5, 4
    x, w, b = r.standard_normal((B, H, T, d)), r.standard_normal((H, d)), r.standard_normal((H, d))
    y = np.stack([[M.norm(x[i, h], w[h], b[h], over, silu=False)[0] for h in range(H)] for i in range(B)])
    t = torch.from_numpy(x).transpose(1, 2).reshape(B, T, H * d)          # channels last
    rows = t.reshape(B * T, H * d, 1) if over == "token" else t.transpose(1, 2)
    ref = torch.nn.functional.group_norm(rows, H, torch.from_numpy(w).reshape(-1), torch.from_numpy(b).reshape(-1))
    ref = ref.reshape(B, T, H * d) if over == "token" else ref.transpose(1, 2)
    ref = ref.reshape(B, T, H, d).transpose(1, 2).numpy()
    np.testing.assert_allclose(y, ref, rtol=1e-12, atol=1e-12)


def differences(f, args, grads, eps=1e-6):
    """Central differences of f(**args) against the claimed gradients, every entry."""
    for name, g in grads.items():
        x = args[name]
        for i in np.ndindex(x.shape):
            old = x[i]
            x[i] = old + eps
            up = f(**args)
            x[i] = old - eps
            down = f(**args)
            x[i] = old
            # truncation eps^2 f''' and rounding 1e-16 |f| / eps are both below 1e-8 at these sizes
            assert abs((up - down) / (2 * eps) - g[i]) < 1e-7 * max(1, abs(g[i])), (name, i)


@pytest.mark.parametrize("T", [1, 2, 6])
@pytest.mark.parametrize("silu", [False, True])
def test_conv_gradient_is_the_difference_quotient(T, silu):
    r = rng_of(5, T)
    a = dict(x=r.standard_normal((T, 2)), filt=r.standard_normal((2, 4)), bias=r.standard_normal(2),
             hist=r.standard_normal((3, 2)))
    dy, dt = r.standard_normal((T, 2)), r.standard_normal((3, 2))

    def loss(x, filt, bias, hist):
        y, tail, _, _ = M.conv(x, filt, bias, hist, silu)
        return (y * dy).sum() + (tail * dt).sum()
    dx, df, db, dh = M.conv_backward(a["x"], a["filt"], dy, a["bias"], a["hist"], silu, dt)
    differences(loss, a, dict(x=dx, filt=df, bias=db, hist=dh))


@pytest.mark.parametrize("T,softplus,gate", [(1, True, True), (5, True, True), (5, False, False)])
def test_scan_gradient_is_the_difference_quotient(T, softplus, gate):
    r = rng_of(6, T)
    d, N = 2, 3
    a = dict(x=r.standard_normal((T, d)), dt=r.standard_normal((T, d)), A=-r.uniform(0.2, 1.5, (d, N)),
             Bm=r.standard_normal((T, N)), Cm=r.standard_normal((T, N)), D=r.standard_normal(d),
             dt_bias=r.standard_normal(d), state=r.standard_normal((d, N)))
    if gate:
        a["z"] = r.standard_normal((T, d))
    dy, ds = r.standard_normal((T, d)), r.standard_normal((d, N))

    def loss(**k):
        y, h, _ = M.scan(softplus=softplus, **k)
        return (y * dy).sum() + (h * ds).sum()
    g = M.scan_backward(dy=dy, softplus=softplus, dstate_end=ds, **a)
    said = {"Bm": "dB", "Cm": "dC"}
    differences(loss, a, {k: g[said.get(k, "d" + k)] for k in a})


@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("silu", [False, True])
def test_norm_gradient_is_the_difference_quotient(over, silu):
    r = rng_of(7)
    a = dict(x=r.standard_normal((3, 4)), weight=r.standard_normal(4), bias=r.standard_normal(4))
    dy = r.standard_normal((3, 4))
    dx, dw, db = M.norm_backward(a["x"], dy, a["weight"], a["bias"], over, silu)
    differences(lambda x, weight, bias: (M.norm(x, weight, bias, over, silu)[0] * dy).sum(), a,
                dict(x=dx, weight=dw, bias=db))
