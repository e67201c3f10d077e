"""Layer norm of rows beyond the kernels that keep a row on chip (more than
16384 columns, or a few less where 16 bytes do not divide them), where the mean
is far above the spread, against the 64-bit oracle.

Tolerances, u = 2^-24. A term takes part in at most D = 54 + C / 2^19 additions
(8 columns, 16 on each of two levels in a thread, C / 2^19 on the third,
13 over the block and one to spare), so a sum is off by at most D u times its
terms' magnitudes.
With m the first reading's mean, e = (D + 1) u mean|x| its error, d = x - m and
mean|d| <= mean|x - mu| + e:
  rest = mean(d):  er = (D + 3) u mean|d| (u |d| from d itself);
  mean = m + rest: er + u |mean|;
  variance = mean(d^2) - rest^2: dv = (D + 7) u mean(d^2) + 2 e er + u e^2;
  rstd: relative dr = dv / (2 (var + eps)) + 3 u, where dv is small beside var
      + eps (asserted);
  y: |gamma| r (u |d| + er + u |x - mu|) + |gamma h| (dr + 2 u) + u (|y| + |beta|).
Backward, with the statistics given, h = (x - mean) rstd, g = dy gamma, s and t
the means of g and g h:
  h: eh = u rstd |x - mean| + 2 u |h|, g: u |g|;
  s: (D + 2) u mean|g|, t: (D + 4) u mean|g h| + mean(|g| eh);
  dx: rstd (2 u |g| + es + |h| et + |t| eh + 6 u (|g| + |s| + |h t|)) + u |dx|.
Rounding to the output type adds half a step, or half its smallest subnormal.
"""
import numpy as np
import pytest
import torch

from flashattention_attention_backward_gb300 import runner
from oracle import dropout, layer_norm, layer_norm_backward

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = float(np.float32(1e-5))
DEV = torch.device("cuda:0")
BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F4: 2.0 ** -149}


def _np(t):
    return t.double().cpu().numpy()


def _within(name, got, want, tol):
    g = _np(got)
    tol = tol + np.abs(want) * (torch.finfo(got.dtype).eps / 2 * (1 + 1e-6)) + TINY[got.dtype]
    # values beyond the type's range round to infinity
    most = torch.finfo(got.dtype).max
    beyond = np.isinf(g) & (np.sign(g) == np.sign(want)) & (np.abs(want) + tol > most)
    assert not (~np.isinf(g) & (np.abs(want) - tol > most)).any(), name
    err = np.where(beyond, 0.0, np.abs(np.where(beyond, 0.0, g) - want * ~beyond))
    assert not np.isnan(err).any(), name
    w = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), "%s at %s: error %.3e, allowed %.3e" % (name, w, err[w], tol[w])


def _rows(kind, C, dtype, seed=1):
    g = torch.Generator().manual_seed(seed + C)
    noise = torch.randn(C, generator=g)
    ramp = torch.arange(C).float() % 64 / 64
    x = {"constant": torch.stack((torch.full((C,), 1000.3), torch.full((C,), -7.1))),
         "far": torch.stack((1000.3 + 0.01 * noise, -4096 + ramp)),
         "plain": torch.stack((1.5 * noise + 0.25, 1e-4 * noise))}[kind]
    return x.to(dtype).to(DEV)


def _check(x64, ex, gamma, beta, y, mean, rstd):
    """ex: error of the elements before the norm."""
    C = x64.shape[1]
    D = 54 + C / 2 ** 19
    want, m, r = layer_norm(x64, gamma, beta, EPS)
    off = np.abs(x64 - m[:, None])
    e = (D + 1) * U * np.abs(x64).mean(1) + ex.mean(1)
    d = off.mean(1) + e
    er = (D + 3) * U * d + ex.mean(1)
    square = (off ** 2).mean(1) + e ** 2
    dv = (D + 7) * U * square + 2 * e * er + U * e ** 2 + 2 * (off * ex).mean(1) + (ex ** 2).mean(1)
    assert (dv < 0.01 / r ** 2).all()
    dr = dv * r ** 2 / 2 * 1.02 + 3 * U
    _within("mean", mean, m, er + U * np.abs(m))
    _within("rstd", rstd, r, r * dr)
    g = np.ones(C) if gamma is None else np.abs(gamma)
    b = 0.0 if beta is None else np.abs(beta)
    h = off * r[:, None]
    tol = g * r[:, None] * (U * (off + e[:, None]) + er[:, None] + ex + U * off) + \
        g * h * (dr[:, None] + 2 * U) + U * (np.abs(want) + b)
    _within("y", y, want, tol)


@pytest.mark.parametrize("dtype", [F4, HF, BF])
@pytest.mark.parametrize("kind", ["constant", "far", "plain"])
@pytest.mark.parametrize("C", [16383, 16385, 16392, 40000, 131071, 1 << 20])
def test_mean_far_above_the_spread(C, kind, dtype):
    x = _rows(kind, C, dtype)
    y, mean, rstd = runner.layer_norm(x, None, None, EPS)
    _check(_np(x), np.zeros(x.shape), None, None, y, mean, rstd)
    if kind == "constant":
        assert torch.equal(mean, x[:, 0].float()) and (y == 0).all()
    g = torch.Generator().manual_seed(C)
    gamma = (1 + 0.2 * torch.randn(C, generator=g)).to(DEV)
    beta = (0.2 * torch.randn(C, generator=g)).to(DEV)
    y, mean, rstd = runner.layer_norm(x, gamma, beta, EPS)
    _check(_np(x), np.zeros(x.shape), _np(gamma), _np(beta), y, mean, rstd)


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("C", [16385, 131072])
def test_with_a_residual(C, p):
    """The sum's mean is far above its spread by the residual."""
    x, res = _rows("plain", C, F4) * 0.01, _rows("far", C, F4)
    z, y, mean, rstd = runner.dropout_add_norm(x, res, None, None, EPS, (p, 77))
    dropped = dropout(_np(x), p, 77)
    want = dropped + _np(res)
    ex = 2 * U * np.abs(dropped) + U * np.abs(want)
    _within("z", z, want, ex)
    # the statistics are those of the rounded sum, which is z itself in 32 bits
    _check(_np(z), np.zeros(z.shape), None, None, y, mean, rstd)


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_a_bad_row_stays_alone(bad):
    x = _rows("plain", 20000, BF).repeat(3, 1)
    good, m, r = runner.layer_norm(x)
    x2 = x.clone()
    x2[2, 19999] = bad
    y, mean, rstd = runner.layer_norm(x2)
    fine = [0, 1, 3, 4, 5]
    assert torch.equal(y[fine], good[fine]) and torch.equal(mean[fine], m[fine])
    assert torch.equal(rstd[fine], r[fine]) and torch.isnan(y[2]).all()
    assert torch.isnan(mean[2]) if bad != bad else float(mean[2]) == bad


def test_statistics_of_neighbouring_lengths():
    """A row with one column more goes to other kernels; its mean and its root
    are the same but for both bounds' roundings."""
    x = _rows("far", 16385, F4)
    _, m, r = runner.layer_norm(x[:, :16384].contiguous())
    x2 = x[:, :16384].repeat(1, 2).contiguous()  # the same mean and variance
    _, m2, r2 = runner.layer_norm(x2)
    # one block's tree on chip: at most 16 + 10 additions and four products deep
    size = np.abs(_np(x)).mean(1)
    assert (np.abs(_np(m) - _np(m2)) <= 32 * U * size).all()
    spread = _np(r2) ** -2
    assert (np.abs(_np(r) / _np(r2) - 1) <= 40 * U + (32 * U * size) ** 2 / spread).all()


@pytest.mark.parametrize("dtype", [F4, HF, BF])
@pytest.mark.parametrize("kind", ["constant", "far", "plain"])
@pytest.mark.parametrize("C", [16383, 16385, 40000, 131071, 1 << 20])
def test_gradients_far_from_zero(C, kind, dtype):
    """dy's mean far above its spread: dx is a small difference of its terms."""
    D = 54 + C / 2 ** 19
    dy, x = _rows(kind, C, dtype), _rows("plain", C, dtype, seed=3)
    gen = torch.Generator().manual_seed(C)
    gamma = (1 + 0.2 * torch.randn(C, generator=gen)).to(DEV)
    _, mean, rstd = runner.layer_norm(x, None, None, EPS)
    for w in (None, gamma):
        dx, dgamma, dbeta = runner.layer_norm_backward(dy, x, w, mean, rstd)
        w64 = np.ones(C) if w is None else _np(w)
        want, dg, db = layer_norm_backward(_np(dy), _np(x), w64, _np(mean), _np(rstd))
        r = _np(rstd)[:, None]
        off = np.abs(_np(x) - _np(mean)[:, None])
        h, g = off * r, np.abs(_np(dy) * w64)
        signed = (_np(x) - _np(mean)[:, None]) * r
        s = np.abs((_np(dy) * w64).mean(1, keepdims=True))
        t = np.abs((_np(dy) * w64 * signed).mean(1, keepdims=True))
        eh = U * r * off + 2 * U * h
        es = (D + 2) * U * g.mean(1, keepdims=True)
        et = (D + 4) * U * (g * h).mean(1, keepdims=True) + (g * eh).mean(1, keepdims=True)
        tol = r * (2 * U * g + es + h * et + t * eh + 6 * U * (g + s + h * t)) + U * np.abs(want)
        _within("dx", dx, want, tol)
        # two rows: a column's sum is two terms
        terms = np.abs(_np(dy)) * (h + eh)
        _within("dgamma", dgamma, dg, 8 * U * terms.sum(0))
        _within("dbeta", dbeta, db, 2 * U * np.abs(_np(dy)).sum(0))


def test_offsets_past_32_bits():
    """33 rows of 2^26 columns: the last begins 2^31 elements behind the first."""
    rows, C = 33, 1 << 26
    x = torch.empty(rows, C, dtype=BF, device=DEV)
    ramp = (torch.arange(4096, device=DEV) % 256).to(BF).repeat(C // 4096)
    x[:] = ramp
    x[-1] = -2 * ramp
    y, mean, rstd = runner.layer_norm(x)
    # 256 values of equal number: mean 127.5, variance (256^2 - 1) / 12
    D = 54 + C / 2 ** 19
    for row, f in ((0, 1), (17, 1), (32, -2)):
        sd = np.sqrt(f * f * (256 ** 2 - 1) / 12 + EPS)
        assert abs(float(mean[row]) - f * 127.5) <= 2 * U * abs(f) * 127.5 + (D + 3) * U * sd
        assert abs(float(rstd[row]) * sd - 1) <= (D + 12) * U
        want = f * (np.arange(256) - 127.5) / sd
        _within("y", y[row, -256:], want, (D + 16) * U * np.abs(want) + 4 * U)
    dx, _, _ = runner.layer_norm_backward(y, x, None, mean, rstd, weight_grads=False)
    # dy = y is h: g - mean(g) - h mean(g h) = 0 but for y's rounding to bf16
    h = np.abs(_np(y[-1, :256]))
    assert (np.abs(_np(dx[-1, -256:])) <= 2 * float(rstd[-1]) * 2.0 ** -8 * (h + h.max())).all()
