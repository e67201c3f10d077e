"""Where the attention over a paged cache can lose digits: small weights beside one
large one in fp16, softcaps far above the logits, and rows of a tile that belong to
no query of its sequence.

An error e of every logit moves a weight by at most 2 e of itself and LSE by e. In
fp16 a weight's operand is rounded to half a step of 2^-24 below 2^-14, and a row's
largest operand is 2^9 or more: 2^-34 of the row's largest weight besides half a
step h of each.
"""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from oracle import cache_attention
from test_gpu_cache import BF, HF, U, Case, _half_step

pytestmark = pytest.mark.gpu


def _check(c, o, lse, scale, softcap, e, small=0.0):
    """Against the oracle: e an error of each logit, given each row's X (the largest
    sum of |scale q k|); small: an error of each weight besides half a step of it."""
    q64, k64, v64 = (t.double().cpu().numpy() for t in [c.q] + c.caches)
    O, LSE, A, X = cache_attention(q64, k64, v64, c.starts, c.lengths, c.table, scale, c.causal,
                                   softcap, c.left, c.sinks)
    rows = slice(int(c.starts[0]), int(c.starts[-1]))
    O, LSE, A, e = O[rows], LSE[rows], A[rows], e(X[rows])
    err = np.abs(lse.double().cpu().numpy()[rows] - LSE)
    tol = e + 2.0 ** -18 + 4 * U * np.abs(LSE)
    assert (err <= tol).all(), "LSE %.3e, allowed %.3e" % (err.max(), tol[err > tol].min())
    h = _half_step(c.dtype)
    tol = (h + 2.0 ** -16 + 2.0 ** -20 + 2 * e[..., None]) * A + h * np.abs(O) + 2.0 ** -25 + small
    err = np.abs(o.double().cpu().numpy()[rows] - O)
    assert (err <= tol).all(), "O %.3e, allowed %.3e" % (err.max(), tol[err > tol].min())
    assert attn.attn_device_status(clear=True) == (0, 0)


@pytest.mark.parametrize("a", [8.0, 15.5, 17.25, 20.0, 23.0])
@pytest.mark.parametrize("d,softcap,tokens", [(64, 0.0, 1), (128, 0.0, 1), (256, 0.0, 1),
                                              (128, 0.0, 20), (64, 30.0, 1), (128, 30.0, 1),
                                              (128, 500.0, 20), (64, 500.0, 1),
                                              (128, 500.0, 1)])
def test_small_weights_beside_a_large_one(d, softcap, tokens, a):
    """One key that every row sees with the logit a, thousands with logit 0: what
    the many weigh together is not lost, though each is e^-a of the one. As many
    key/value heads as keep a tile's keys with one CTA."""
    heads, length = 160, 4096
    c = Case([(tokens, length)], heads, heads, d, 64, HF)
    first = int(c.table[0, 0])
    c.q.zero_()
    c.q[:, :, 0] = 1.0
    k, v = c.caches
    k.zero_()
    k[first, 0, :, 0] = a
    v.uniform_(0.5, 1.5)  # one sign
    v[first, 0] = 0.0
    o, lse = c.attend(scale=1.0, softcap=softcap)
    assert attn.attn_device_status(clear=True) == (0, 0)
    z = softcap * np.tanh(a / softcap) if softcap else a
    dense = v[c.pages_d[0, :length // 64].long()].flatten(0, 1).double()  # [length, heads, d]
    p = torch.arange(length - tokens, length, device="cuda")
    total = (p + np.exp(z))[:, None]
    O, LSE = dense.cumsum(0)[p] / total[..., None], total.log()
    # the logits are one product each, off by a rounding, under the cap by 2^-20
    # of themselves
    e = (2 * U + (2.0 ** -20 if softcap else 0.0)) * a
    assert float((lse.double() - LSE).abs().max()) <= e + 2.0 ** -18 + 4 * U * float(LSE.max())
    h = _half_step(HF)
    tol = (2 * h + 2.0 ** -16 + 2.0 ** -20 + 2 * e) * O + 2.0 ** -25 + length * 1.5 * 2.0 ** -34
    err = (o.double() - O).abs()
    assert bool((err <= tol).all()), "O %.3e" % float((err - tol).max())


@pytest.mark.parametrize("softcap", [400.0, 1e4, 1e5, 1e8, 1e30, 3e38])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens", [1, 60])  # tiles of few rows and of many
def test_caps_far_above_the_logits(tokens, d, dtype, softcap):
    """tanh's error shrinks with its argument: a logit far below the cap is off by
    2^-20 of itself, not of the cap."""
    c = Case([(tokens, 300), (1, 900), (2, 70)], 4, 2, d, 16, dtype)
    scale = d ** -0.5
    o, lse = c.attend(softcap=softcap)
    _check(c, o, lse, scale, softcap, lambda x: ((d + 8) * 2 * U + 2.0 ** -20) * x,
           small=900 * 4 * 2.0 ** -34)


@pytest.mark.parametrize("fill", [0.0, 300.0, float("nan"), float("inf")])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, HF), (256, BF)])
def test_rows_behind_change_nothing(d, dtype, fill):
    """Rows of q behind the last sequence, and the next sequence's, stand in a tile
    with the last tokens of a chunk and change no bit of theirs."""
    c = Case([(20, 300), (1, 40), (20, 260)], 2, 1, d, 16, dtype, behind=120)
    for softcap in (0.0, 20.0, 5.0):
        o, lse = c.attend(softcap=softcap)
        q = c.q.clone()
        q[41:] = fill
        o2, lse2 = c.attend(q=q, softcap=softcap)
        assert torch.equal(o2[:41], o[:41]) and torch.equal(lse2[:41], lse[:41]), softcap
        q[20] = fill if fill == fill and abs(fill) < 1e4 else 100.0
        o2, lse2 = c.attend(q=q, softcap=softcap)
        for rows in (slice(0, 20), slice(21, 41)):
            assert torch.equal(o2[rows], o[rows]) and torch.equal(lse2[rows], lse[rows]), softcap
    assert attn.attn_device_status(clear=True) == (0, 0)
