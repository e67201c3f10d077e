"""Layer norm at every kind of row that its kernels tell apart (lanes or warps a
row, odd lengths, rows over two blocks), held to the depth of their own sums.
(test_gpu_norm_wide.py has the rows beyond them.)

Tolerances, per element, u = 2^-24, for rows on chip. A thread has at most 16
columns of a row, added in pairs: 8 additions, 5 over the lanes of a warp. Over at
most 32 warps come 2 products and sums a lane and 5 over lanes.
  A warp's mean is off by a = 14 u of its mean |x| (13 additions, a quotient).
  mean: dm = 23 u mean|x| (8 roundings more, and one to spare).
  The squares about the warps' means, joined with n_w (mu_w - mean)^2, add up with
  25 u of themselves (d and its square 2, 14 + 5 additions, 4 in the join). The
  means' own errors move them by
      2 mean_w(|mu_w - mean| (a_w + dm)) + mean_w(a_w^2 + (a_w + dm)^2).
  rstd: between those of var + eps + dv and max(var + eps - dv, eps), and 5 u of
      itself (a sum rounded, rsqrtf 2 units in the last place): dr relative.
  y: |gamma| r (dm + 2 u |x - mean|) + |gamma h| (dr + 2 u) + u (|y| + |beta|).
Backward, with the statistics given: h = (z - mean) rstd: eh = u r |z - mean| + 2 u
|h|; the sums of g and of g h over the row: 8 + 6 additions in a warp, 4 + 3 over
the warps, and the products with 1 / C and rstd: (24 + 4) u of mean|g|, (24 + 6) u
of mean|g h| + mean(|g| eh);
  dx: r (3 u |g| + es + |h| et + |t| eh + 6 u (|g| + |s| + |h t|)) + u |dx|.
  Weights: a thread adds its own rows, at most rows / (152 K) + 1 of them where a
  block has K rows of threads side by side (152 blocks at least are resident), then
  K <= 32, at most 32 and 32 more: rows / (152 K) + 97, and 4 roundings a term.
Rounding to the output type adds half a step of the value, or half its smallest
subnormal.
"""
import numpy as np
import pytest
import torch

from flashattention_attention_backward_gb300 import runner
from oracle import dropout, layer_norm, layer_norm_backward

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24
EPS = float(np.float32(1e-5))
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F4: 2.0 ** -149}
HALF = {BF: 2.0 ** -8, HF: 2.0 ** -11, F4: 2.0 ** -24}


def _np(t):
    return t.double().cpu().numpy()


def _within(name, got, want, tol):
    g = _np(got)
    tol = tol + np.abs(want) * HALF[got.dtype] * (1 + 1e-6) + TINY[got.dtype]
    # values beyond the type's range round to infinity
    most = torch.finfo(got.dtype).max
    beyond = np.isinf(g) & (np.sign(g) == np.sign(want)) & (np.abs(want) + tol > most)
    assert not (~np.isinf(g) & (np.abs(want) - tol > most)).any(), name
    err = np.where(beyond, 0.0, np.abs(np.where(beyond, 0.0, g) - want * ~beyond))
    assert not np.isnan(err).any(), name
    w = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), "%s at %s: error %.3e, allowed %.3e" % (name, w, err[w], tol[w])


def _warps(rows, C, dtype):
    """[rows, C]: the warp of its row that each column belongs to. Vectors of 16
    bytes go round the row's threads (of one block, or of the first and then the
    second); where they do not divide a row it begins inside its first vector."""
    E = 4 if dtype == F4 else 8
    n = C if C % E == 0 else C + 2 * E - 2
    threads = next((t for most, t in ((512, 32), (1024, 64), (2048, 128), (4096, 256))
                    if n <= most), 512)
    shift = (np.arange(rows)[:, None] * C) % E if C % E else np.zeros((rows, 1), int)
    vector = (np.arange(C)[None] + shift) // E
    block = vector // (threads * 16 // E)
    return block * 16 + vector % threads // 32


def _check_forward(x64, gamma, beta, y, mean, rstd, dtype):
    rows, C = x64.shape
    want, m, r = layer_norm(x64, gamma, beta, EPS)
    size = np.abs(x64).mean(1)
    dm = 23 * U * size
    off = np.abs(x64 - m[:, None])
    warp = _warps(rows, C, dtype)
    moved, squares = np.zeros(rows), np.zeros(rows)
    for w in range(warp.max() + 1):
        mine = warp == w
        n = np.maximum(mine.sum(1), 1)
        a = 14 * U * (np.abs(x64) * mine).sum(1) / n
        gap = np.abs((x64 * mine).sum(1) / n - m)
        moved += mine.sum(1) / C * 2 * gap * (a + dm)
        squares += mine.sum(1) / C * (a ** 2 + (a + dm) ** 2)
    dv = 25 * U * ((off ** 2).mean(1) + squares) + moved + squares
    total = 1 / r ** 2  # var + eps
    least = np.maximum(total - dv, EPS)
    dr = np.maximum(np.sqrt(total / least) - 1, 1 - np.sqrt(total / (total + dv))) + 5 * U
    _within("mean", mean, m, dm)
    _within("rstd", rstd, r, r * dr)
    g = np.abs(gamma)
    tol = g * r[:, None] * (1 + dr[:, None]) * (dm[:, None] + 2 * U * off) + \
        g * off * r[:, None] * (dr[:, None] + 2 * U) + U * (np.abs(want) + np.abs(beta))
    _within("y", y, want, tol)


def _rows(C, dtype):
    """Plain rows, rows far above their spread, a ramp, magnitudes from end to end."""
    g = torch.Generator().manual_seed(C)
    noise = torch.randn(5, C, generator=g)
    ramp = torch.arange(C).float() % 64 / 64
    big, small = (1e15, 1e-15) if dtype != HF else (300.0, 1e-4)
    x = torch.stack((1.5 * noise[0] + 0.25, 1000.3 + 0.01 * noise[1], -4096 + ramp,
                     noise[2] * big, noise[3] * small, 64 + noise[4]))
    return x.to(dtype).to(DEV)


def _weights(C, dtype):
    g = torch.Generator().manual_seed(C + 1)
    return ((1 + 0.2 * torch.randn(C, generator=g)).to(dtype).to(DEV),
            (0.2 * torch.randn(C, generator=g)).to(dtype).to(DEV))


ON_CHIP = [1, 7, 64, 100, 128, 200, 256, 333, 512, 520, 1001, 1024, 2047, 2104, 4095, 4096, 5000,
           8184, 8192, 8200, 9001, 12288, 16370, 16384]


@pytest.mark.parametrize("dtype", [F4, HF, BF])
@pytest.mark.parametrize("C", ON_CHIP)
def test_rows_of_extreme_values(C, dtype):
    x = _rows(C, dtype)
    for wdtype in (F4, dtype):
        gamma, beta = _weights(C, wdtype)
        y, mean, rstd = runner.layer_norm(x, gamma, beta, EPS)
        _check_forward(_np(x), _np(gamma), _np(beta), y, mean, rstd, dtype)


@pytest.mark.parametrize("dtype", [F4, HF, BF])
@pytest.mark.parametrize("C", ON_CHIP)
def test_gradients_at_extreme_values(C, dtype):
    """dy far from zero, z plain and far above its spread."""
    gamma, _ = _weights(C, F4)
    dy, z = _rows(C, dtype), _rows(C, dtype)[[0, 5, 1, 0, 5, 2]].contiguous()
    _, mean, rstd = runner.layer_norm(z, None, None, EPS)
    dx, dgamma, dbeta = runner.layer_norm_backward(dy, z, gamma, mean, rstd)
    want, dg, db = layer_norm_backward(_np(dy), _np(z), _np(gamma), _np(mean), _np(rstd))
    r = _np(rstd)[:, None]
    off = _np(z) - _np(mean)[:, None]
    h, g = off * r, _np(dy) * _np(gamma)
    eh = U * r * np.abs(off) + 2 * U * np.abs(h)
    means = [np.abs(v.mean(1, keepdims=True)) for v in (g, g * h)]
    es = 28 * U * np.abs(g).mean(1, keepdims=True)
    et = 30 * U * np.abs(g * h).mean(1, keepdims=True) + (np.abs(g) * eh).mean(1, keepdims=True)
    h, g = np.abs(h), np.abs(g)
    tol = r * (3 * U * g + es + h * et + means[1] * eh + 6 * U * (g + means[0] + h * means[1])) + \
        U * np.abs(want)
    _within("dx", dx, want, tol)
    # six rows: a column's sum is six terms
    _within("dgamma", dgamma, dg, 12 * U * (np.abs(_np(dy)) * (h + eh)).sum(0))
    _within("dbeta", dbeta, db, 6 * U * np.abs(_np(dy)).sum(0))


@pytest.mark.parametrize("rows,C,side_by_side", [(6_000_000, 64, 32), (5_000_000, 128, 16),
                                                 (700_000, 1000, 8), (150_000, 4096, 2)])
def test_weight_gradients_of_many_rows(rows, C, side_by_side):
    """Each thread sums many rows. The sums in 64 bits on the GPU, in parts."""
    g = torch.Generator(device=DEV).manual_seed(C)
    x = torch.empty(rows, C, dtype=BF, device=DEV).normal_(generator=g)
    dy = torch.empty(rows, C, dtype=BF, device=DEV).normal_(0.5, 1, generator=g)
    _, mean, rstd = runner.layer_norm(x)
    gamma = torch.ones(C, device=DEV)
    _, dgamma, dbeta = runner.layer_norm_backward(dy, x, gamma, mean, rstd)
    want, size = torch.zeros(2, C, dtype=torch.float64, device=DEV), torch.zeros(
        2, C, dtype=torch.float64, device=DEV)
    part = 1 << 27
    for a in range(0, rows, part // C):
        b = min(rows, a + part // C)
        d = dy[a:b].double()
        h = (x[a:b].double() - mean[a:b, None].double()) * rstd[a:b, None].double()
        want += torch.stack(((d * h).sum(0), d.sum(0)))
        size += torch.stack(((d * h).abs().sum(0), d.abs().sum(0)))
    depth = rows / (152 * side_by_side) + 97
    for name, got, w, s in zip(("dgamma", "dbeta"), (dgamma, dbeta), want, size):
        _within(name, got, _np(w), (depth + 4) * U * _np(s))


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("shift", [0.0, 4.0, 32.0])
@pytest.mark.parametrize("rows,C", [(70, 128), (33, 1001), (9, 4096)])
def test_forward_to_backward_in_16_bits(rows, C, shift, p):
    """dropout_add_norm and its backward behind it, in bf16, against the chain in
    64 bits. The backward reads z rounded to bf16 beside the statistics of the
    unrounded sum: its h is off by r 2^-8 |z|, which costs
      dx: r (|h| mean(|g| eh) + |t| eh),  dgamma: sum |dy| eh;
    everything else is below 64 u of the terms' magnitudes."""
    gen = torch.Generator().manual_seed(rows)
    draw = lambda: torch.randn(rows, C, generator=gen)  # noqa: E731
    x, res = draw().to(BF).to(DEV), (draw() + shift).to(BF).to(DEV)
    dy, dz = draw().to(BF).to(DEV), draw().to(BF).to(DEV)
    gamma, beta = _weights(C, F4)
    drop = (p, 99)
    z, y, mean, rstd = runner.dropout_add_norm(x, res, gamma, beta, EPS, drop)
    dx, dres, dgamma, dbeta = runner.dropout_add_norm_backward(dy, dz, z, gamma, mean, rstd, drop)
    p32 = float(np.float32(p))
    z64 = dropout(_np(x), p32, 99) + _np(res)
    y64, m, r = layer_norm(z64, _np(gamma), _np(beta), EPS)
    back, dg, db = layer_norm_backward(_np(dy), z64, _np(gamma), m, r)
    want = back + _np(dz)
    h, g = (z64 - m[:, None]) * r[:, None], _np(dy) * _np(gamma)
    s, t = (np.abs(v.mean(1, keepdims=True)) for v in (g, g * h))
    size = np.abs(z64).mean(1, keepdims=True)
    eh = r[:, None] * (2.0 ** -8 + 64 * U) * (np.abs(z64) + 2.0 ** -8 * size)
    h, g = np.abs(h), np.abs(g)
    tol = r[:, None] * (h * (g * eh).mean(1, keepdims=True) + t * eh +
                        eh * (g * eh).mean(1, keepdims=True) +
                        64 * U * (g + s + g.mean(1, keepdims=True) +
                                  h * (g * h).mean(1, keepdims=True))) + U * np.abs(want)
    _within("z", z, z64, 3 * U * (np.abs(z64) + 2 * np.abs(_np(res))))
    far = 1 + np.abs(m / z64.std(1))[:, None]
    _within("y", y, y64, np.abs(_np(gamma)) * 64 * U * (r[:, None] * size + h * far) +
            2 * U * (np.abs(y64) + np.abs(_np(beta))))
    _within("dresidual", dres, want, tol)
    keep = dropout(np.ones_like(z64), p32, 99)
    _within("dx", dx, want * keep, tol * keep + 2 * U * np.abs(want * keep))
    _within("dgamma", dgamma, dg, (np.abs(_np(dy)) * eh).sum(0) +
            64 * U * (np.abs(_np(dy)) * h).sum(0))
    _within("dbeta", dbeta, db, 64 * U * np.abs(_np(dy)).sum(0))

# for many of these n, n times the fp32 value of 1 / n is not 1
LENGTHS = [1, 2, 3, 41, 47, 61, 64, 82, 83, 97, 107, 123, 128, 200, 333, 520, 1001, 1021, 1536,
           2047, 2104, 3001, 4093, 4095, 4096, 5000, 6015, 8191, 8192, 8195, 9001, 12287, 16370,
           16383, 16384, 20001]


@pytest.mark.parametrize("dtype", [BF, HF, F4])
@pytest.mark.parametrize("C", LENGTHS)
def test_equal_values(C, dtype):
    """Rows of one value v each. v has at most 8 significant bits and C at most
    15, so every sum of copies of v and its product with a count are exact in 24
    bits; the mean, a quotient rounded once, is v, every difference is 0 and y is
    beta to the last bit."""
    v = torch.tensor([5.0, -1000.0, 0.0703125, 13.25, -255.0, 3.984375], device=DEV).to(dtype)
    x = v[:, None].expand(-1, C).contiguous()
    g = torch.Generator().manual_seed(C)
    gamma = torch.randn(C, generator=g).to(dtype).to(DEV)
    beta = torch.randn(C, generator=g).to(dtype).to(DEV)
    y, mean, rstd = runner.layer_norm(x, gamma, beta, 1e-5)
    assert torch.equal(mean, v.float())
    assert torch.equal(y, beta.expand_as(y))
    # 1 / sqrt(eps) of the fp32 eps: rsqrtf is off by at most 2 units in the last
    # place, 2^-23 of the value each at most
    want = 1 / np.sqrt(float(np.float32(1e-5)))
    assert (np.abs(rstd.double().cpu().numpy() - want) <= 2 * 2.0 ** -23 * want).all()
    # a sum with a residual: 4 more bits
    half = (v * 0.5).to(dtype)[:, None].expand(-1, C).contiguous()
    z, y, mean, _ = runner.dropout_add_norm(half, half, gamma, beta, 1e-5)
    assert torch.equal(z, x) and torch.equal(mean, v.float())
    assert torch.equal(y, beta.expand_as(y))


@pytest.mark.parametrize("dtype", [F4, BF])
@pytest.mark.parametrize("rows,C", [(256, 64), (257, 64), (400, 64), (512, 64), (513, 64),
                                    (129, 128), (300, 1001), (700, 4096)])
def test_weight_gradients_repeat(rows, C, dtype):
    """The same call, the same bits, at row counts where the joined form and the
    plain one choose different grids; between the forms only the order of a
    column's additions differs."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    dy, dz, z = (torch.randn(rows, C, generator=g, device=DEV).to(dtype) for _ in range(3))
    gamma, _ = _weights(C, F4)
    _, mean, rstd = runner.layer_norm(z)
    plain = runner.layer_norm_backward(dy, z, gamma, mean, rstd)
    h = (_np(z) - _np(mean)[:, None]) * _np(rstd)[:, None]
    size = np.stack((np.abs(_np(dy) * h).sum(0), np.abs(_np(dy)).sum(0)))
    for extra, p in ((None, 0.0), (dz, 0.0), (dz, 0.3)):
        args = (dy, extra, z, gamma, mean, rstd, (p, 5))
        one, two = (runner.dropout_add_norm_backward(*args) for _ in range(2))
        assert all(torch.equal(a, b) for a, b in zip(one, two))
        # two orders of at most rows + 4 roundings a term each
        for a, b, s in zip(one[2:], plain[1:], size):
            assert (np.abs(_np(a) - _np(b)) <= 2 * (rows + 4) * U * s).all()
