"""Statistics of the group norm over a sequence when some of its tokens are far from the rest, as the first tokens of
a sequence often are: fp32 sums about a shift keep their digits only if the shift is not one of those."""
import pytest
import torch

import test_trained_neural_b200 as tm
from test_mixer import BF, F, Draw

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("B,H,T,d,kind", [(4, 75, 1024, 256, F), (300, 1, 8192, 64, BF), (2, 3, 900, 20, F), (2, 2, 500, 7, F)])
@pytest.mark.parametrize("where", ["value", "token", "every 64th token", "far mean"])
def test_statistics_beside_outliers(B, H, T, d, kind, where):
    """A thread sums 64 values at most, two at a time, about the mean of 16 of them: 32 additions of positive terms, each
    within u of the sum, which comes to at most (1 + 64 / 256) times the squares about the mean when one value, and to
    less when a token, is far from the rest: 40 u of the variance if all err alike, 20 u of 1 / sqrt(variance). Joining
    up to 8 batches and 64 row groups rounds at random, 3 u each: 0.58 * 3 u sqrt(72) / 2 = 7 u. 64 u holds both twice
    over. (Squares about an outlier of a run of 512 values come to 512 times what they are about their mean.)

    The means m_p of the parts are held in fp32, each off by at most e = 3 u |m| after its joins. That moves the variance
    v by (2 / N) sum n_p (m_p - m) e_p + e^2, at most 2 b e + e^2 with b^2 the variance of the parts' means (Cauchy and
    Schwarz). A part is 8 values or more: b = sqrt(v / 8) for random ones. So 1 / sqrt(v) is off by up to
    b e / v = 1.06 u |m| / sqrt(v) of itself, beside the same u |m| / sqrt(v) by which the mean's rounding moves y."""
    r = Draw("outliers", B, H, T, d, where)
    x = r.normal(B, H, T, d)
    if where == "value":
        x[:, :, 0, 0] = 1e4 + 100 * r.normal(B, H)
    elif where == "far mean":
        x += 3e4
    else:
        x[:, :, slice(0, 1) if where == "token" else slice(0, T, 64)] *= 1e4
    x = x.to(kind)
    y, stats = tm.group_norm(x, over="sequence", dtype=F)
    m, v = x.double().mean((2, 3)), x.double().var((2, 3), unbiased=False)
    rstd = (v + 1e-5) ** -0.5
    assert ((stats[..., 1] / rstd - 1).abs() <= U * (64 + 1.1 * m.abs() * rstd)).all(), ((stats[..., 1] / rstd - 1).abs().max() / U).item()
    assert ((stats[..., 0] - m).abs() <= 64 * U * v.sqrt() + 2 * U * m.abs()).all()
    want = (x.double() - m[..., None, None]) * rstd[..., None, None]
    # the mean's error is 64 u of the spread and its rounding, the factor's as above
    far = (m.abs() * rstd)[..., None, None]
    assert ((y - want).abs() <= 64 * U * (2 + want.abs()) + U * far * (2 + 1.1 * want.abs())).all()


@pytest.mark.parametrize("B,H,T,d", [(2, 3, 900, 20), (1, 2, 40, 7)])
def test_squares_past_fp32_do_not_become_a_variance_of_nothing(B, H, T, d):
    """Values of 1e25, whose squares overflow: not a factor of 1 / sqrt(eps) and finite outputs made with it. A NaN
    reaches the statistics and outputs of its own group, and no other."""
    x = Draw("overflow", B, H, T, d).normal(B, H, T, d)
    y, stats = tm.group_norm(x * 1e25, over="sequence")
    assert not (stats[..., 1] > 1e-18).any() and not (y.abs() > 1e6).any()
    want = tm.group_norm(x, over="sequence")
    x[0, 1, T // 2, 3] = float("nan")
    got = tm.group_norm(x, over="sequence")
    for p, q in zip(got, want):
        assert torch.isnan(p[0, 1]).all()
        p[0, 1] = q[0, 1]
        assert torch.equal(p, q)
