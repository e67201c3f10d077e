"""Layer norm, dropout with a residual and the two together, forward and
backward, against the 64-bit oracle.

Tolerances, per element, u = 2^-24, C columns. A sum over a row is a tree over
threads of serial sums: at most D = C / 32 + 24 additions deep, so its error
is at most D u times the sum of magnitudes. Then
  mean:  dm = (D + 2) u mean|x|;
  rstd:  the sum of squares is off by (D + 4) u of itself, and by dm^2 for
         the mean: relative dr = ((D + 4) / 2 + 4) u + dm^2 / (2 (var + eps));
  y:     |gamma| r (dm + 2 u |x - mu|) + |gamma h| (dr + 4 u) + u |y|.
The dropped sum x / (1 - p) + residual is off by 3 u of its terms, which goes
into x's error above. Backward, with the statistics given:
  h:  3 u |h| + u r |mu|,  g: u |g|,
  dz: r (2 u |g| + (D + 4) u mean|g| + |h| (D + 8) u mean|g h|)
      + 8 u r (|g| + |mean g| + |h mean(g h)|) + r eh (|mean(g h)| + |h| mean|g|) + u |dz|,
  with eh = u r |mu| + 3 u |h| from h's error;
  weights: a column's sum over rows is at most 1100 additions deep (one
      thread's rows, then at most 1024 partial sums, or fewer rows than that):
      (min(rows, 1100) + 8) u sum|dy h|.
Rounding to the output type adds half a step of the value, or half its
smallest subnormal.
"""

import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from oracle import dropout, element_keep_mask, layer_norm, layer_norm_backward

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
DEV = torch.device("cuda:0")


def _np(t):
    return t.double().cpu().numpy()


def _within(name, got, want, tol):
    g = _np(got)
    assert g.shape == want.shape
    tol = tol + np.abs(want) * (torch.finfo(got.dtype).eps / 2 * (1 + 1e-6)) + TINY[got.dtype]
    err = np.abs(g - want)
    assert not np.isnan(err).any(), name
    w = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), "%s at %s: error %.3e, allowed %.3e" % (name, w, err[w], tol[w])


def _check_forward(x64, ex, gamma, beta, eps, y, mean, rstd):
    """ex: error of the row's elements before the norm."""
    C = x64.shape[1]
    D = C / 32 + 24
    g = 1.0 if gamma is None else _np(gamma)
    b = 0.0 if beta is None else _np(beta)
    want, m, r = layer_norm(x64, g, b, eps)
    var = 1 / r ** 2 - eps
    dm = (D + 2) * U * np.abs(x64).mean(1) + ex.mean(1)
    off = x64 - m[:, None]
    # an error ex of the elements moves the squares' mean by 2 mean(|off| ex) + mean(ex^2)
    dv = dm ** 2 + 2 * (np.abs(off) * ex).mean(1) + (ex ** 2).mean(1)
    dr = ((D + 4) / 2 + 4) * U + dv / (2 * (var + eps))
    _within("mean", mean, m, dm)
    _within("rstd", rstd, r, r * dr)
    h = off * r[:, None]
    tol = np.abs(g) * r[:, None] * (dm[:, None] + ex + 2 * U * np.abs(off)) + \
        np.abs(g * h) * (dr[:, None] + 4 * U) + U * (np.abs(want) + np.abs(b))
    _within("y", y, want, tol)


def _make(rows, C, dtype, wdtype, seed, shift=0.25):
    g = torch.Generator().manual_seed(seed)
    x = (1.5 * torch.randn(rows, C, generator=g) + shift).to(dtype).to(DEV)
    other = torch.randn(rows, C, generator=g).to(dtype).to(DEV)
    gamma = (1 + 0.2 * torch.randn(C, generator=g)).to(wdtype).to(DEV)
    beta = (0.2 * torch.randn(C, generator=g)).to(wdtype).to(DEV)
    return x, other, gamma, beta


BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
SHAPES = [
    # rows, C, dtype, weight type
    (1, 1, F4, F4), (3, 2, BF, BF), (5, 7, HF, F4), (1, 64, BF, F4), (1000, 64, BF, BF),
    (333, 128, BF, F4), (700, 128, F4, F4), (129, 256, HF, HF), (77, 100, BF, BF),
    (64, 520, BF, F4), (33, 1001, HF, F4), (17, 1024, F4, F4), (40, 1536, BF, BF),
    (2, 4096, BF, BF), (301, 4096, BF, F4), (31, 4095, BF, BF), (9, 5000, F4, F4),
    (170, 8192, BF, BF), (5, 8192, F4, BF), (7, 12288, HF, F4), (160, 16384, BF, BF),
    (3, 16384, F4, F4), (2, 16385, BF, BF), (2, 40000, BF, F4), (1, 70001, F4, F4),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_layer_norm(shape):
    rows, C, dtype, wdtype = shape
    x, _, gamma, beta = _make(rows, C, dtype, wdtype, rows + C)
    for g, b in ((gamma, beta), (gamma, None), (None, None)):
        y, mean, rstd = runner.layer_norm(x, g, b, 1e-5)
        _check_forward(_np(x), np.zeros((rows, C)), g, b, float(np.float32(1e-5)), y, mean, rstd)
    # in place, without the statistics
    z = x.clone()
    code, wcode = runner._DTYPES[dtype], runner._DTYPES[wdtype]
    y, _, _ = runner.layer_norm(x, gamma, beta, 1e-5)
    attn.check(attn.attn_layer_norm(z, gamma, beta, z, None, None, rows, C, 1e-5, code, wcode,
                                    torch.cuda.current_stream()))
    assert torch.equal(z, y)


def _check_weights(h, dy64, dgamma, dbeta):
    D = min(h.shape[0], 1100) + 8
    _within("dgamma", dgamma, (dy64 * h).sum(0), D * U * np.abs(dy64 * h).sum(0))
    _within("dbeta", dbeta, dy64.sum(0), D * U * np.abs(dy64).sum(0))


def _dz_tolerance(dy64, z64, gamma, mean, rstd, want):
    C = z64.shape[1]
    D = C / 32 + 24
    r = rstd[:, None]
    h = (z64 - mean[:, None]) * r
    g = dy64 if gamma is None else dy64 * _np(gamma)
    eh = U * r * np.abs(mean)[:, None] + 3 * U * np.abs(h)
    s, t = g.mean(1, keepdims=True), (g * h).mean(1, keepdims=True)
    sa, ta = np.abs(g).mean(1, keepdims=True), np.abs(g * h).mean(1, keepdims=True)
    ga = np.abs(g)
    et = (ga * eh).mean(1, keepdims=True)
    tol = r * (2 * U * ga + (D + 4) * U * sa + np.abs(h) * ((D + 8) * U * ta + et)) + \
        8 * U * r * (ga + np.abs(s) + np.abs(h * t)) + r * eh * np.abs(t) + U * np.abs(want)
    return h, tol


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_layer_norm_backward(shape):
    rows, C, dtype, wdtype = shape
    x, dy, gamma, beta = _make(rows, C, dtype, wdtype, rows * 3 + C)
    for g in (gamma, None):
        _, mean, rstd = runner.layer_norm(x, g, None, 1e-5)
        dx, dgamma, dbeta = runner.layer_norm_backward(dy, x, g, mean, rstd)
        assert dgamma.dtype == dbeta.dtype == (dtype if g is None else wdtype)
        g64 = 1.0 if g is None else _np(g)
        want, _, _ = layer_norm_backward(_np(dy), _np(x), g64, _np(mean), _np(rstd))
        h, tol = _dz_tolerance(_np(dy), _np(x), g, _np(mean), _np(rstd), want)
        _within("dx", dx, want, tol)
        _check_weights(h, _np(dy), dgamma, dbeta)
    # the same bits again; without weight gradients; in place of dy
    again = runner.layer_norm_backward(dy, x, None, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dgamma, dbeta)))
    alone = runner.layer_norm_backward(dy, x, None, mean, rstd, weight_grads=False)
    assert torch.equal(alone[0], dx) and alone[1] is alone[2] is None
    code = runner._DTYPES[dtype]
    ws = torch.empty(attn.attn_layer_norm_bwd_workspace_bytes(rows, C) // 4, device=DEV)
    one = torch.empty(C, dtype=wdtype, device=DEV)
    d2 = dy.clone()
    attn.check(attn.attn_layer_norm_bwd(d2, x, None, mean, rstd, d2, None, one, ws, rows, C, code,
                                        runner._DTYPES[wdtype], torch.cuda.current_stream()))
    assert torch.equal(d2, dx)
    _within("dbeta alone", one, _np(dy).sum(0),
            (min(rows, 1100) + 8) * U * np.abs(_np(dy)).sum(0))


def test_backward_against_differences():
    """The gradients of both operators against central differences of the
    GPU's own fp32 forward. The loss is summed in 64 bits; its terms carry the
    forward's fp32 rounding, so a difference over a step of 2^-7 of values of
    size 2 is good to about sqrt(n) 2^-22 2^7 for n = 39 terms, and to the
    third derivative's step^2 / 6: 1e-3 covers both several times."""
    rows, C, p, seed, step = 3, 13, 0.4, 99, 2.0 ** -7
    x, res, gamma, beta = _make(rows, C, F4, F4, 1)
    dy = torch.randn(rows, C, generator=torch.Generator().manual_seed(8)).to(DEV)
    dz = torch.randn(rows, C, generator=torch.Generator().manual_seed(9)).to(DEV)

    def loss(x, res, gamma, beta):
        z, y, _, _ = runner.dropout_add_norm(x, res, gamma, beta, 1e-3, (p, seed))
        return float((y.double() * dy).sum() + (z.double() * dz).sum())

    z, y, mean, rstd = runner.dropout_add_norm(x, res, gamma, beta, 1e-3, (p, seed))
    grads = runner.dropout_add_norm_backward(dy, dz, z, gamma, mean, rstd, (p, seed))
    inputs = [x, res, gamma, beta]
    for which in range(4):
        flat = grads[which].reshape(-1)
        for i in range(0, flat.numel(), 5):
            plus, minus = ([t.clone() for t in inputs] for _ in range(2))
            plus[which].reshape(-1)[i] += step
            minus[which].reshape(-1)[i] -= step
            width = float(plus[which].reshape(-1)[i].double() - minus[which].reshape(-1)[i].double())
            d = (loss(*plus) - loss(*minus)) / width
            assert abs(d - float(flat[i])) <= 1e-3 * max(1.0, abs(d)), (which, i)


@pytest.mark.parametrize("dtype", [BF, HF, F4])
@pytest.mark.parametrize("n", [1, 3, 4, 7, 8, 31, 1000, 4096, 100001, 2345678])
def test_dropout_add(n, dtype):
    g = torch.Generator().manual_seed(n)
    x = torch.randn(n, generator=g).to(dtype).to(DEV)
    res = torch.randn(n, generator=g).to(dtype).to(DEV)
    for p, seed in ((0.1, 5), (0.5, (1 << 63) + 77), (0.9, 1 << 40)):
        keep = element_keep_mask(n, seed, p)
        y = runner.dropout_add(x, None, (p, seed))
        # mask equal element by element (an x of 0 is the same either way)
        kept = _np(y) != 0
        assert np.array_equal(kept[_np(x) != 0], keep[_np(x) != 0])
        want = dropout(_np(x), p, seed)
        _within("y", y, want, 2 * U * np.abs(want))
        y = runner.dropout_add(x, res, (p, seed))
        _within("y + residual", y, want + _np(res), 3 * U * (np.abs(want) + np.abs(_np(res))))
        z = x.clone()  # in place
        attn.check(attn.attn_dropout_add(z, res, z, n, p, seed, runner._DTYPES[dtype],
                                         torch.cuda.current_stream()))
        assert torch.equal(z, y)
    assert torch.equal(runner.dropout_add(x), x)
    _within("sum", runner.dropout_add(x, res), _np(x) + _np(res), 0.0 * _np(x) + U * 4)


def test_dropout_drops_infinities_and_nan():
    n, p, seed = 4096, 0.5, 3
    keep = torch.from_numpy(element_keep_mask(n, seed, p)).to(DEV)
    for bad in (float("inf"), float("nan")):
        x = torch.full((n,), bad, dtype=BF, device=DEV)
        y = runner.dropout_add(x, torch.ones_like(x), (p, seed))
        assert (y[~keep] == 1).all() and not torch.isfinite(y[keep]).any()


def test_dropout_writes_nothing_behind_the_end():
    for n in (1, 5, 9, 4095, 100003):
        buf = torch.full((n + 64,), 7.0, dtype=BF, device=DEV)
        x = torch.ones(n + 64, dtype=BF, device=DEV)
        attn.check(attn.attn_dropout_add(x, None, buf, n, 0.5, 1, attn.ATTN_BF16,
                                         torch.cuda.current_stream()))
        assert (buf[n:] == 7).all() and (buf[:n] != 7).all()


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_dropout_add_norm(shape, p):
    rows, C, dtype, wdtype = shape
    x, res, gamma, beta = _make(rows, C, dtype, wdtype, rows * 5 + C)
    seed = 1234567 + C
    z, y, mean, rstd = runner.dropout_add_norm(x, res, gamma, beta, 1e-5, (p, seed))
    dropped = dropout(_np(x), p, seed)
    want = dropped + _np(res)
    ex = 3 * U * (np.abs(dropped) + np.abs(_np(res)))
    _within("z", z, want, ex)
    _check_forward(want, ex, gamma, beta, float(np.float32(1e-5)), y, mean, rstd)
    # in place: z over the residual, y over x
    x2, res2 = x.clone(), res.clone()
    attn.check(attn.attn_dropout_add_norm(
        x2, res2, gamma, beta, res2, x2, None, None, rows, C, 1e-5, p, seed,
        runner._DTYPES[dtype], runner._DTYPES[wdtype], torch.cuda.current_stream()))
    assert torch.equal(res2, z) and torch.equal(x2, y)


@pytest.mark.parametrize("p", [0.0, 0.2])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_dropout_add_norm_backward(shape, p):
    rows, C, dtype, wdtype = shape
    z, dy, gamma, _ = _make(rows, C, dtype, wdtype, rows * 7 + C)
    dz_in = torch.randn(rows, C, generator=torch.Generator().manual_seed(C)).to(dtype).to(DEV)
    seed = (1 << 50) + C
    _, mean, rstd = runner.layer_norm(z, gamma, None, 1e-5)
    for extra in (dz_in, None):
        dx, dres, dgamma, dbeta = runner.dropout_add_norm_backward(dy, extra, z, gamma, mean, rstd,
                                                                   (p, seed))
        want, _, _ = layer_norm_backward(_np(dy), _np(z), _np(gamma), _np(mean), _np(rstd))
        h, tol = _dz_tolerance(_np(dy), _np(z), gamma, _np(mean), _np(rstd), want)
        if extra is not None:
            want = want + _np(extra)
            tol = tol + U * (np.abs(want) + np.abs(_np(extra)))
        _within("dresidual", dres, want, tol)
        _check_weights(h, _np(dy), dgamma, dbeta)
        if p == 0:
            assert dx is dres
        else:
            keep = element_keep_mask(rows * C, seed, p).reshape(rows, C)
            inv = 1 / (1 - float(np.float32(p)))
            _within("dx", dx, np.where(keep, want * inv, 0.0),
                    np.where(keep, tol * inv + 2 * U * np.abs(want * inv), 0.0))
    # in place: dx over dy, dresidual over dz
    a, b = dy.clone(), dz_in.clone()
    ref = runner.dropout_add_norm_backward(dy, dz_in, z, gamma, mean, rstd, (p, seed))
    g2, b2 = torch.empty_like(gamma), torch.empty_like(gamma)
    ws = torch.empty(attn.attn_layer_norm_bwd_workspace_bytes(rows, C) // 4, device=DEV)
    attn.check(attn.attn_dropout_add_norm_bwd(
        a, b, z, gamma, mean, rstd, a, b, g2, b2, ws, rows, C, p, seed, runner._DTYPES[dtype],
        runner._DTYPES[wdtype], torch.cuda.current_stream()))
    for got, r in zip((a, b, g2, b2), ref):
        assert torch.equal(got, r)


def test_rows_of_extreme_values():
    """Constant rows, a mean far above the spread, and large magnitudes."""
    C = 256
    x = torch.ones(4, C, device=DEV)
    x[0] = 5.0
    x[1] = 4096.0 + torch.arange(C, device=DEV) / 64.0
    x[2] = torch.randn(C, device=DEV) * 1e15
    x[3] = torch.randn(C, device=DEV) * 1e-15
    y, mean, rstd = runner.layer_norm(x, None, None, 1e-5)
    assert (y[0] == 0).all() and float(mean[0]) == 5.0
    _check_forward(_np(x), np.zeros((4, C)), None, None, float(np.float32(1e-5)), y, mean, rstd)


def test_a_bad_row_stays_alone():
    """Infinities and NaN spoil their own rows (and the weights' sums) only."""
    rows, C = 9, 200
    x, dy, gamma, beta = _make(rows, C, BF, F4, 3)
    good, _, _ = runner.layer_norm(x, gamma, beta)
    x2 = x.clone()
    x2[4, 7], x2[6, 0] = float("inf"), float("nan")
    y, mean, rstd = runner.layer_norm(x2, gamma, beta)
    fine = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(y[fine], good[fine]) and torch.isnan(y[[4, 6]]).all()
    _, m, r = runner.layer_norm(x, gamma, beta)
    ref, _, _ = runner.layer_norm_backward(dy, x, gamma, m, r)
    dx, _, _ = runner.layer_norm_backward(dy, x2, gamma, mean, rstd)
    assert torch.equal(dx[fine], ref[fine]) and torch.isnan(dx[[4, 6]]).all()


@pytest.mark.parametrize("rows,C", [(40000, 64), (20000, 100), (3000, 1024), (700, 4096),
                                    (700, 3001), (400, 9000)])
def test_bad_rows_among_many(rows, C):
    """The same where threads take several rows, some of them together."""
    x, dy, gamma, beta = _make(rows, C, BF, F4, 5)
    good, m, r = runner.layer_norm(x, gamma, beta)
    ref, _, _ = runner.layer_norm_backward(dy, x, gamma, m, r)
    bad = torch.arange(3, rows, 7, device=DEV)
    fine = torch.ones(rows, dtype=torch.bool, device=DEV)
    fine[bad] = False
    x2 = x.clone()
    x2[bad, (bad * 5) % C] = float("nan")
    y, mean, rstd = runner.layer_norm(x2, gamma, beta)
    assert torch.equal(y[fine], good[fine]) and torch.isnan(y[bad]).all()
    assert torch.equal(mean[fine], m[fine]) and torch.equal(rstd[fine], r[fine])
    dx, _, _ = runner.layer_norm_backward(dy, x2, gamma, mean, rstd)
    assert torch.equal(dx[fine], ref[fine]) and torch.isnan(dx[bad]).all()


@pytest.mark.parametrize("C", [64, 1001, 4096, 20000])
def test_nothing_outside_is_written(C):
    rows = 5
    x, dy, gamma, beta = _make(rows, C, BF, BF, 4)
    n = rows * C
    bufs = [torch.full((n + 64,), 7.0, dtype=BF, device=DEV) for _ in range(4)]
    stats = [torch.full((rows + 16,), 7.0, device=DEV) for _ in range(2)]
    weights = [torch.full((C + 16,), 7.0, dtype=BF, device=DEV) for _ in range(2)]
    nbytes = attn.attn_layer_norm_bwd_workspace_bytes(rows, C)
    ws = torch.full((nbytes // 4 + 64,), 7.0, device=DEV)
    s = torch.cuda.current_stream()
    attn.check(attn.attn_dropout_add_norm(x, dy, gamma, beta, bufs[0], bufs[1], stats[0], stats[1],
                                          rows, C, 1e-5, 0.3, 8, attn.ATTN_BF16, attn.ATTN_BF16,
                                          s))
    attn.check(attn.attn_dropout_add_norm_bwd(
        dy, None, bufs[0], gamma, stats[0], stats[1], bufs[2], bufs[3], weights[0], weights[1], ws,
        rows, C, 0.3, 8, attn.ATTN_BF16, attn.ATTN_BF16, s))
    torch.cuda.synchronize()
    assert all((b[n:] == 7).all() for b in bufs) and all((t[rows:] == 7).all() for t in stats)
    assert all((w[C:] == 7).all() for w in weights) and (ws[nbytes // 4:] == 7).all()


def test_no_rows():
    x = torch.empty(0, 48, dtype=BF, device=DEV)
    w = torch.ones(48, dtype=BF, device=DEV)
    y, mean, rstd = runner.layer_norm(x, w, w)
    assert y.shape == (0, 48) and mean.shape == (0,)
    dx, dgamma, dbeta = runner.layer_norm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 48) and (dgamma == 0).all() and (dbeta == 0).all()
    assert runner.dropout_add(x, x, (0.1, 1)).shape == (0, 48)


def test_many_rows():
    """More rows than any grid has blocks, offsets past 2^31 elements."""
    rows, C = 17_000_000, 128
    x = torch.empty(rows, C, dtype=BF, device=DEV)
    x[:] = torch.arange(C, device=DEV, dtype=torch.float32).to(BF)
    x[-1] = -x[-1]
    y, mean, rstd = runner.layer_norm(x, None, None)
    want, m, r = layer_norm(_np(x[-2:]), None, None, float(np.float32(1e-5)))
    _within("last rows", y[-2:], want, 1e-5)
    assert torch.equal(y[:4], y[-5:-1]) and torch.equal(y[rows // 2], y[0])
    del y
    seed, p = 5, 0.5
    z = runner.dropout_add(x, None, (p, seed))
    tail = element_keep_mask(C, seed, p, first=(rows - 1) * C).astype(np.float64)
    assert np.array_equal(_np(z[-1]), _np(x[-1]) * 2 * tail)
    del z
    dy = torch.ones_like(x)
    dx, dgamma, dbeta = runner.layer_norm_backward(dy, x, None, mean, rstd)
    # dy = 1: g - mean(g) = 0 and mean(g h) = mean(h), itself a rounding
    assert float(dx.abs().max()) <= 1e-5
    assert (dbeta == torch.tensor(float(rows), dtype=BF, device=DEV)).all()


def test_streams_and_graphs():
    """Two streams with a workspace each, and captured graphs replayed on new
    contents beside eager calls."""
    rows, C = 700, 1024
    x, dy, gamma, beta = _make(rows, C, BF, BF, 21)
    _, mean, rstd = runner.layer_norm(x, gamma, beta)
    want = runner.layer_norm_backward(dy, x, gamma, mean, rstd)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [runner.layer_norm_backward(dy, x, gamma, mean, rstd, stream=s) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))
    sx, sdy = x.clone(), dy.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z, y, m, r = runner.dropout_add_norm(sx, sdy, gamma, beta, 1e-5, (0.1, 5))
        back = runner.dropout_add_norm_backward(sdy, None, z, gamma, m, r, (0.1, 5))
    for scale in (1.0, 0.5):
        sx.copy_(x * scale)
        sdy.copy_(dy * scale)
        graph.replay()
        torch.cuda.synchronize()
        z2, y2, m2, r2 = runner.dropout_add_norm(sx, sdy, gamma, beta, 1e-5, (0.1, 5))
        eager = runner.dropout_add_norm_backward(sdy, None, z2, gamma, m2, r2, (0.1, 5))
        assert torch.equal(z, z2) and torch.equal(y, y2)
        assert all(torch.equal(a, b) for a, b in zip(back, eager))
