"""attn_cache_append and attn_cache_fwd (a paged key/value cache) against the
64-bit oracle.

Append: rotated elements are held to the rotary tests' bound, 12 u (|a| + |b|)
with u = 2^-24 plus half a step of the output's type; values and columns that do
not turn are copies.

Attention, per element of O: P enters the second product rounded to the cache's
type, half a step h of each weight (2^-8 for bf16, 2^-11 for fp16), so that O is
off by at most h A, A = sum of P |v|; the output's rounding adds h |O|. A logit is
a sum of d products in fp32: off by at most (d + 8) 2 u X, X the largest sum of
|scale q k| (twice u, as tensor cores may drop bits instead of rounding them), and
the exponential adds 2^-20 of itself; a softcap's tanh is off by 2^-20. An error e
of every logit moves a weight by at most 2 e of itself: 2 e A in all, and the
sum over the keys in fp32, added in any order within a tile and split, 2^-16 A.
LSE: e, the logarithm's 2^-22 and a few steps of its size.
"""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from oracle import cache_append, cache_attention

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, HF = torch.bfloat16, torch.float16


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


class Case:
    """Tensors of one batch. seqs: (new tokens, length with them); order: how the
    cache's dimensions lie in memory; hidden slots hold NaN."""

    def __init__(self, seqs, H, H_kv, d, page, dtype, left=-1, sinks=0, causal=True, order="slot",
                 seed=1, before=0, behind=0, sigma=1.0):
        dev = torch.device("cuda:0")
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.H, self.H_kv, self.d, self.page, self.dtype = seqs, H, H_kv, d, page, dtype
        self.left, self.sinks, self.causal, self.before = left, sinks, causal, before
        starts = np.cumsum([before] + [n for n, _ in seqs])
        self.T = int(starts[-1]) + behind
        need = [(L + page - 1) // page for _, L in seqs]
        self.n_pages, self.max_pages = sum(need) + 2, max(need + [1]) + 1
        order_ = torch.randperm(self.n_pages, generator=g).tolist()
        self.table = np.full((len(seqs), self.max_pages), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order_[at:at + n]
            at += n
        self.starts = starts.astype(np.int32)
        self.lengths = np.array([L for _, L in seqs], dtype=np.int32)
        self.pages_d, self.starts_d, self.lengths_d = (
            torch.from_numpy(np.ascontiguousarray(a)).to(dev)
            for a in (self.table, self.starts, self.lengths))

        def normal(*shape):
            return (torch.randn(shape, generator=g) * sigma).to(dtype).to(dev)

        self.qkv = normal(self.T, H + 2 * H_kv, d)  # a packed projection
        self.q, self.k, self.v = (self.qkv[:, :H], self.qkv[:, H:H + H_kv],
                                  self.qkv[:, H + H_kv:])
        if d % 8 != 0:  # pointers are 16-byte aligned
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        shape = (self.n_pages, page, H_kv, d) if order == "slot" else \
            (self.n_pages, H_kv, page, d)
        self.caches = []
        for _ in range(2):
            c = normal(*shape)
            self.caches.append(c if order == "slot" else c.transpose(1, 2))

    def hide(self, value=float("nan")):
        """Fills every slot that no query sees with `value`."""
        seen = np.zeros((self.n_pages, self.page), dtype=bool)
        for b, (n, L) in enumerate(self.seqs):
            if n == 0 or L == 0:
                continue
            j = np.arange(L)
            if self.left >= 0:
                j = j[(j >= L - n - self.left) | (j < self.sinks)]
            seen[self.table[b][j // self.page], j % self.page] = True
        hidden = torch.from_numpy(~seen).cuda()
        for c in self.caches:
            c[hidden] = value
        # pages without a visible slot have been given away
        given = np.flatnonzero(~seen.any(1))
        table = np.where(np.isin(self.table, given), 1 << 30, self.table).astype(np.int32)
        self.pages_d.copy_(torch.from_numpy(table))

    def batch(self):
        return tuple(self.caches) + (self.pages_d, self.starts_d, self.lengths_d)

    def attend(self, q=None, scale=None, softcap=0.0, **kw):
        return runner.cache_attention(self.q if q is None else q, *self.batch(),
                                      self.d ** -0.5 if scale is None else scale, self.causal,
                                      softcap, self.left, self.sinks, **kw)

    def check(self, o, lse, q=None, scale=None, softcap=0.0):
        scale = self.d ** -0.5 if scale is None else scale
        q64, k64, v64 = (t.double().cpu().numpy() for t in (
            [self.q if q is None else q] + self.caches))
        O, LSE, A, X = cache_attention(q64, k64, v64, self.starts, self.lengths, self.table,
                                       scale, self.causal, softcap, self.left, self.sinks)
        rows = slice(int(self.starts[0]), int(self.starts[-1]))
        got, got_lse = o.double().cpu().numpy()[rows], lse.double().cpu().numpy()[rows]
        O, LSE, A, X = O[rows], LSE[rows], A[rows], X[rows]
        e = (self.d + 8) * 2 * U * X + (softcap * 2.0 ** -20 if softcap > 0 else 0.0)
        h = _half_step(self.dtype)
        tol = (h + 2.0 ** -16 + 2.0 ** -20 + 2 * e[..., None]) * A + h * np.abs(O) + 2.0 ** -25
        err = np.abs(got - O)
        assert not np.isnan(got).any()
        worst = np.unravel_index((err - tol).argmax(), err.shape) if err.size else ()
        assert (err <= tol).all(), "O%s %.3e, allowed %.3e" % (worst, err[worst], tol[worst])
        none = np.isneginf(LSE)
        assert (np.isneginf(got_lse) == none).all() and (got[none] == 0).all()
        err = np.abs(got_lse[~none] - LSE[~none])
        tol = e[~none] + 2.0 ** -18 + 4 * U * np.abs(LSE[~none])
        assert (err <= tol).all(), "LSE %.3e" % err.max()
        assert attn.attn_device_status(clear=True) == (0, 0)


# ------------------------------------------------------------------- append
APPEND = [
    # sequences, H, H_kv, d, rot, interleaved, page, dtype, order
    ([(1, 1)], 1, 1, 64, 64, False, 8, BF, "slot"),
    ([(1, 500), (0, 7), (1, 1), (1, 64), (0, 0)], 32, 8, 128, 128, False, 64, BF, "slot"),
    ([(1, 1 + 9 * i) for i in range(150)], 4, 2, 64, 64, True, 16, HF, "head"),
    ([(70, 333), (0, 9), (129, 129), (3, 1000)], 6, 3, 64, 32, True, 16, HF, "slot"),
    ([(257, 300)], 8, 2, 256, 64, False, 32, BF, "head"),
    ([(33, 40), (2, 2)], 5, 5, 128, 0, False, 8, BF, "slot"),
    ([(19, 50)], 3, 1, 72, 24, False, 4, BF, "slot"),   # rot / 2 is no multiple of 8
    ([(19, 50), (4, 9)], 3, 2, 33, 30, True, 5, HF, "head"),  # odd d, odd pages
    ([(5, 5)], 2, 1, 1, 0, False, 1, BF, "slot"),
]


@pytest.mark.parametrize("seqs,H,H_kv,d,rot,interleaved,page,dtype,order", APPEND)
def test_append(seqs, H, H_kv, d, rot, interleaved, page, dtype, order):
    c = Case(seqs, H, H_kv, d, page, dtype, order=order, before=2, behind=3)
    plan = runner.Rotary(rot, c.q.device, scaling="ramp", factor=4.0, original_length=4096,
                         interleaved=interleaved)
    turns = plan.turns.tolist()[:rot // 2]
    before = [t.double().cpu().numpy() for t in [c.q, c.k, c.v] + c.caches]
    out = torch.full(c.q.shape, 7.0, dtype=dtype, device=c.q.device)
    assert runner.cache_append(c.q, c.k, c.v, *c.batch(), plan, out=out) is out
    assert attn.attn_device_status(clear=True) == (0, 0)
    q, kc, vc = cache_append(*before, turns, plan.magnitude, interleaved, c.starts, c.lengths,
                             c.table)
    rows = slice(int(c.starts[0]), int(c.starts[-1]))
    # the largest |a| + |b| of the pairs bounds all
    for got, want, x in ((out[rows], q[rows], before[0][rows]), (c.caches[0], kc, before[1])):
        err = np.abs(got.double().cpu().numpy() - want)
        tol = np.abs(want) * (_half_step(dtype) * (1 + 1e-6)) + 2.0 ** -25 + \
            12 * U * plan.magnitude * 2 * np.abs(x).max()
        assert (err <= tol).all()
    assert np.array_equal(c.caches[1].double().cpu().numpy(), vc)
    # what belongs to no sequence is left as it was
    assert (out[:rows.start] == 7).all() and (out[rows.stop:] == 7).all()
    old = before[3]
    touched = np.abs(kc - old).max((2, 3)) > 0
    assert np.array_equal(c.caches[0].double().cpu().numpy()[~touched], old[~touched])
    # in place, and without q
    fresh = c.caches[0].clone(), c.caches[1].clone()
    q2 = c.q.clone()
    runner.cache_append(q2, c.k, c.v, *fresh, *c.batch()[2:], plan, out=q2)
    assert torch.equal(q2[rows], out[rows]) and torch.equal(fresh[0], c.caches[0])
    assert runner.cache_append(None, c.k, c.v, *fresh, *c.batch()[2:], plan) is None
    assert torch.equal(fresh[0], c.caches[0]) and torch.equal(fresh[1], c.caches[1])


def test_append_keeps_bits():
    """Values of every kind (NaN with its bits, infinities, zeros' signs)."""
    c = Case([(64, 64)], 1, 2, 64, 16, HF)
    bits = torch.randint(-2 ** 15, 2 ** 15, c.v.shape, dtype=torch.int16, device="cuda")
    v = bits.view(torch.float16)
    plan = runner.Rotary(0, "cuda:0")
    runner.cache_append(None, c.k, v, *c.batch(), plan)
    got = torch.cat([c.caches[1][p].view(torch.int16) for p in c.table[0][:4]])
    assert torch.equal(got, bits)


def test_append_far_positions_and_bad_slots():
    """Slots outside the table or the cache are left out and reported; the
    others, and q, are written."""
    c = Case([(4, 40), (3, 10), (2, 30)], 2, 1, 64, 8, BF)
    plan = runner.Rotary(64, "cuda:0")
    good = [t.clone() for t in c.caches]
    q = runner.cache_append(c.q, c.k, c.v, *good, *c.batch()[2:], plan)
    table = c.table.copy()
    table[0, 4] = c.n_pages  # positions 36 .. 39: all of the first one's new tokens
    table[2, 3] = -1         # 28, 29 of the third
    bad = [t.clone() for t in c.caches]
    q2 = runner.cache_append(c.q, c.k, c.v, *bad, torch.from_numpy(table).cuda(), *c.batch()[3:],
                             plan)
    assert attn.attn_device_status(clear=True) == (0, attn.ATTN_ERR_PAGE)
    assert attn.attn_device_status(clear=True) == (0, 0)
    assert torch.equal(q, q2)
    for g, b, old in zip(good, bad, c.caches):
        want = old.clone()
        for j in (7, 8, 9):  # the second sequence's
            want[c.table[1][j // 8], j % 8] = g[c.table[1][j // 8], j % 8]
        assert torch.equal(b, want)
    # lengths past the table's end, and shorter than the new tokens
    for lengths in ((400, 10, 30), (2, 10, 30)):
        b2 = [t.clone() for t in c.caches]
        runner.cache_append(c.q, c.k, c.v, *b2, c.pages_d, c.starts_d,
                            torch.tensor(lengths, dtype=torch.int32, device="cuda"), plan)
        assert attn.attn_device_status(clear=True) == (0, attn.ATTN_ERR_PAGE)


# ---------------------------------------------------------------- attention
ATTEND = [
    # sequences, H, H_kv, d, page, dtype, left, sinks, softcap, causal, order
    ([(1, 1)], 1, 1, 64, 8, BF, -1, 0, 0.0, True, "slot"),
    ([(1, 500)], 32, 8, 128, 64, BF, -1, 0, 0.0, True, "slot"),
    ([(1, n) for n in (1, 2, 15, 16, 17, 127, 128, 129, 255, 256, 257, 1000)], 8, 2, 128, 16, BF,
     -1, 0, 0.0, True, "slot"),
    ([(1, 20000)], 4, 1, 64, 64, HF, -1, 0, 0.0, True, "head"),
    ([(1, 9000), (0, 0), (2, 40), (0, 300)], 8, 1, 256, 32, BF, -1, 0, 0.0, True, "slot"),
    ([(300, 300)], 2, 2, 64, 16, BF, -1, 0, 0.0, True, "slot"),
    ([(129, 700), (1, 333), (64, 64), (0, 12), (7, 130)], 6, 2, 128, 64, BF, -1, 0, 0.0, True,
     "head"),
    ([(40, 300)], 5, 1, 128, 24, HF, -1, 0, 0.0, True, "slot"),
    ([(31, 257), (2, 513)], 7, 1, 64, 48, BF, -1, 0, 0.0, True, "slot"),
    ([(3, 400)], 128, 1, 64, 128, BF, -1, 0, 0.0, True, "slot"),
    ([(3, 400)], 96, 1, 128, 256, HF, -1, 0, 0.0, True, "head"),
    ([(70, 400), (1, 129)], 8, 4, 256, 16, HF, -1, 0, 0.0, True, "slot"),
    ([(200, 900), (1, 2000), (5, 5)], 4, 2, 128, 16, BF, 100, 4, 0.0, True, "slot"),
    ([(200, 900), (1, 2000)], 4, 2, 64, 32, HF, 7, 0, 0.0, True, "slot"),
    ([(1, 5000), (1, 100)], 8, 2, 128, 64, BF, 1023, 300, 0.0, True, "slot"),
    ([(150, 700), (1, 800)], 6, 2, 64, 16, HF, 255, 130, 20.0, True, "head"),
    ([(150, 300), (1, 300)], 4, 4, 128, 16, BF, -1, 0, 5.0, True, "slot"),
    ([(50, 300), (1, 70)], 4, 2, 128, 16, BF, 0, 1, 0.0, True, "slot"),
    ([(90, 300), (1, 70)], 4, 2, 64, 16, BF, -1, 0, 0.0, False, "slot"),
    ([(90, 300), (1, 70)], 4, 2, 128, 16, BF, 30, 9, 0.0, False, "slot"),
    ([(33, 500)], 4, 2, 256, 16, BF, 60, 5, 15.0, True, "slot"),
    # logits far below the cap and near it; tiles of few rows and of many
    ([(60, 300), (1, 700), (2, 40)], 8, 2, 128, 16, BF, -1, 0, 50.0, True, "slot"),
    ([(60, 300), (1, 700), (2, 40)], 6, 2, 64, 16, HF, 90, 3, 400.0, True, "head"),
    ([(1, 3000), (3, 100)], 8, 2, 64, 64, BF, -1, 0, 3.0, True, "slot"),
    ([(1, 2000), (1, 90), (2, 500)], 16, 1, 64, 32, BF, 700, 6, 30.0, True, "slot"),
]


@pytest.mark.parametrize("seqs,H,H_kv,d,page,dtype,left,sinks,softcap,causal,order", ATTEND)
def test_attention(seqs, H, H_kv, d, page, dtype, left, sinks, softcap, causal, order):
    c = Case(seqs, H, H_kv, d, page, dtype, left, sinks, causal, order, before=1, behind=2,
             sigma=2.0 if softcap else 1.0)
    o = torch.full((c.T, H + 1, d), 7.0, dtype=dtype, device="cuda")  # rows of a wider tensor
    lse = torch.full((c.T, H), 7.0, device="cuda")
    clean = c.attend(softcap=softcap, out=(o[:, :H], lse))
    c.check(*clean, softcap=softcap)
    assert (o[:, H] == 7).all()
    for t in (o, lse):  # rows of no sequence
        assert (t[:1] == 7).all() and (t[c.T - 2:] == 7).all()
    # the same bits again, in other tensors, with NaN in every slot that no query sees
    rows = slice(1, c.T - 2)
    c.hide()
    o2, lse2 = c.attend(softcap=softcap)
    assert attn.attn_device_status(clear=True) == (0, 0)
    assert torch.equal(o2[rows], o[rows, :H]) and torch.equal(lse2[rows], lse[rows])
    c.hide(float("inf"))
    o2, lse2 = c.attend(softcap=softcap)
    assert torch.equal(o2[rows], o[rows, :H]) and torch.equal(lse2[rows], lse[rows])


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed):
    """Batches drawn from all that the call takes: chunks and single tokens,
    pages of any multiple of 8, groups of up to 128 heads, windows, sinks."""
    r = np.random.default_rng(100 + seed)
    d = int(r.choice([64, 128, 256]))
    H_kv = int(r.choice([1, 2, 3, 5]))
    G = int(r.choice([1, 2, 3, 4, 7, 8, 16, 33]))
    longest = int(r.choice([40, 400, 3000]))
    seqs = []
    for _ in range(int(r.integers(1, 9))):
        n = int(r.choice([0, 1, 1, r.integers(1, 9), r.integers(1, 150)]))
        seqs.append((n, n + int(r.integers(0, longest))))
    seqs.append((1, 1 + int(r.integers(0, longest))))
    softcap = float(r.choice([0.0, 0.0, 2.0, 30.0, 300.0]))
    c = Case(seqs, H_kv * G, H_kv, d, int(r.choice([8, 16, 24, 40, 64, 104, 128, 192])),
             [BF, HF][seed % 2], int(r.choice([-1, -1, 0, 9, 127, 128, 500])),
             int(r.choice([0, 0, 1, 5, 64, 128, 300])), bool(r.random() < 0.8),
             str(r.choice(["slot", "head"])), seed, int(r.integers(0, 3)), int(r.integers(0, 3)),
             float(r.choice([0.5, 1.0, 2.0])))
    o, lse = c.attend(softcap=softcap)
    c.check(o, lse, softcap=softcap)
    rows = slice(int(c.starts[0]), int(c.starts[-1]))
    c.hide()
    o2, lse2 = c.attend(softcap=softcap)
    assert torch.equal(o2[rows], o[rows]) and torch.equal(lse2[rows], lse[rows])


def test_large_logits():
    """Logits far apart and far from 0: the running maximum moves often, and a
    scale of its own."""
    c = Case([(20, 600), (1, 900)], 4, 2, 128, 16, BF, sigma=4.0)
    o, lse = c.attend(scale=0.4)
    c.check(o, lse, scale=0.4)


def test_rows_that_see_nothing():
    """More new tokens than positions: the first stand before the sequence."""
    c = Case([(5, 2), (1, 40), (3, 0)], 4, 2, 64, 16, BF)
    o, lse = c.attend()
    assert (o[:3] == 0).all() and (o[6:] == 0).all()
    assert torch.isneginf(lse[:3]).all() and torch.isneginf(lse[6:]).all()
    c.check(o, lse)
    # a batch without any key at all
    c = Case([(2, 0), (1, 0)], 4, 2, 64, 16, BF)
    o, lse = c.attend()
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("length", [40, 3000])  # tiles of one CTA and of many
def test_nan_stays_visible(length, d, softcap):
    """NaN in a query, or in a key that a row sees: its O and LSE are NaN, and the
    other rows what they were."""
    c = Case([(1, length), (2, length + 7)], 4, 2, d, 16, BF)
    o, lse = c.attend(softcap=softcap)

    def same(rows, o2, lse2):
        if softcap == 0:
            assert torch.equal(o2[rows], o[rows]) and torch.equal(lse2[rows], lse[rows])
            return
        # rows of one warp share tanh's form, which a NaN among them may change:
        # logits then differ by 20 * 2e-7, LSE by as much and its roundings; every P
        # and O may round to the other side, each a step of 2^-7, and the mean of
        # |v|, weighted, stays below 2
        assert float((lse2[rows] - lse[rows]).abs().max()) <= 1e-5 + 8 * U * 10
        assert float((o2[rows].double() - o[rows].double()).abs().max()) <= 2 * 2 * 2 ** -7

    q = c.q.clone()
    q[0, 1, 5] = float("nan")
    o2, lse2 = c.attend(q=q, softcap=softcap)
    bad = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    bad[0, 1] = True
    assert o2[bad].isnan().all() and lse2[bad].isnan().all()
    same(~bad, o2, lse2)
    # key/value head 0 of the second sequence at its first position
    c.caches[0][int(c.table[1, 0]), 0, 0, 0] = float("nan")
    o3, lse3 = c.attend(softcap=softcap)
    bad.zero_()
    bad[1:, :2] = True
    assert o3[bad].isnan().all() and lse3[bad].isnan().all()
    same(~bad, o3, lse3)


def test_bad_pages_and_long_lengths():
    """A page outside the cache reads as zeros, keys past the table are hidden;
    both are reported."""
    c = Case([(1, 100), (1, 30)], 2, 1, 64, 16, BF)
    table = c.table.copy()
    table[0, 2] = c.n_pages + 5
    table[0, 3] = -7
    o, lse = runner.cache_attention(c.q, *c.caches, torch.from_numpy(table).cuda(), c.starts_d,
                                    c.lengths_d, 0.125)
    assert attn.attn_device_status(clear=True) == (0, attn.ATTN_ERR_PAGE)
    zeroed = [t.clone() for t in c.caches]
    for t in zeroed:
        t[c.table[0, 2:4].tolist()] = 0
    o2, lse2 = runner.cache_attention(c.q, *zeroed, *c.batch()[2:], 0.125)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    lengths = c.lengths_d.clone()
    lengths[1] = 5000
    o3, _ = runner.cache_attention(c.q, *c.batch()[:4], lengths, 0.125, causal=False)
    assert attn.attn_device_status(clear=True)[1] == attn.ATTN_ERR_PAGE
    assert torch.equal(o3[0], runner.cache_attention(c.q, *c.batch(), 0.125)[0][0])
    attn.attn_device_status(clear=True)


def test_counts_past_32_bits():
    """A window and sinks that an int32 cannot hold."""
    c = Case([(3, 130), (1, 300)], 4, 2, 64, 16, BF)
    want, lse = c.attend()
    for left, sinks in ((1 << 32, 0), ((1 << 32) + 5, 0), (5, 1 << 32), (5, (1 << 31) + 1)):
        c.left, c.sinks = left, sinks
        o, lse2 = c.attend()
        assert torch.equal(o, want) and torch.equal(lse, lse2), (left, sinks)


def test_without_lse_and_strides():
    """The C entry point with no place for LSE and contiguous tensors."""
    c = Case([(3, 130), (1, 300)], 4, 2, 128, 16, BF)
    q, o = c.q.contiguous(), torch.empty(c.T, 4, 128, dtype=BF, device="cuda")
    ws = torch.empty(attn.attn_cache_fwd_workspace_bytes(c.T, 2, 4, 2, 128), dtype=torch.uint8,
                     device="cuda")
    attn.check(attn.attn_cache_fwd(q, *c.caches, o, None, c.starts_d, c.lengths_d, c.pages_d, ws,
                                   c.T, 2, 4, 2, 128, 16, c.max_pages, c.n_pages, 0.1, True, 0.0,
                                   -1, 0, attn.ATTN_BF16))
    want, lse = c.attend(scale=0.1)
    assert torch.equal(o, want)
    c.check(o, lse, scale=0.1)


def test_shared_pages():
    """Sequences that begin with the same pages."""
    c = Case([(1, 200), (3, 210), (1, 196)], 4, 2, 64, 16, BF)
    c.table[1:, :12] = c.table[0, :12]
    c.pages_d.copy_(torch.from_numpy(c.table))
    c.check(*c.attend())


def test_many_sequences():
    rng = np.random.default_rng(5)
    c = Case([(int(rng.integers(0, 4)), int(rng.integers(4, 90))) for _ in range(700)], 4, 2, 64, 16,
             BF)
    c.check(*c.attend())


def test_captured_graph_follows_the_lengths():
    """One captured step of append and attention, replayed as the sequences
    grow; a second graph with a workspace of its own between the replays."""
    H, H_kv, d, page, B = 4, 2, 64, 16, 3
    first = [200, 15, 1]
    c = Case([(1, L + 8) for L in first], H, H_kv, d, page, BF)  # room for eight steps
    plan = runner.Rotary(d, "cuda:0")
    nbytes = max(attn.attn_cache_fwd_workspace_bytes(B, B, H, H_kv, d), 16)
    graphs = []
    for _ in range(2):
        caches = [t.clone() for t in c.caches]
        q, ws = torch.empty_like(c.q), torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c.q), torch.empty(B, H, device="cuda")
        lengths = c.lengths_d.clone()

        def step():
            runner.cache_append(c.q, c.k, c.v, *caches, c.pages_d, c.starts_d, lengths, plan,
                                out=q)
            runner.cache_attention(q, *caches, c.pages_d, c.starts_d, lengths, 0.125, out=out,
                                   workspace=ws)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        # the workspace lives as long as the graph that uses it
        graphs.append((graph, caches, q, out, lengths, ws))
    g = torch.Generator().manual_seed(9)
    for n in range(8):
        c.qkv.copy_(torch.randn(c.qkv.shape, generator=g).to(BF))
        for graph, _, _, _, lengths, _ in graphs:
            lengths.copy_(torch.tensor([L + n + 1 for L in first], dtype=torch.int32))
            graph.replay()
        torch.cuda.synchronize()
        (_, caches, q, out, lengths, _), other = graphs[0], graphs[1]
        c.lengths = lengths.cpu().numpy()
        c.caches = caches
        c.check(*out, q=q)
        assert all(torch.equal(a, b) for a, b in zip(out, other[3]))


def test_streams():
    """Calls on two side streams at once, each with a workspace of its own."""
    cases = [Case([(1, 6000), (30, 400)], 8, 2, 128, 64, BF, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for c, s, o in zip(cases, streams, outs):
            o.append(c.attend(stream=s))
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        c.check(*o[0])
        for x in o[1:]:
            assert torch.equal(x[0], o[0][0]) and torch.equal(x[1], o[0][1])


def test_offsets_past_32_bits():
    """A cache of more than 2^32 elements, its last pages in use."""
    page, H_kv, d = 64, 8, 128
    n_pages = (1 << 32) // (page * H_kv * d) + 64
    c = Case([(3, 150), (1, 90)], 16, H_kv, d, page, BF)
    big = [torch.zeros(n_pages, page, H_kv, d, dtype=BF, device="cuda") for _ in range(2)]
    shift = n_pages - c.n_pages
    for b, s in zip(big, c.caches):
        b[shift:] = s
    table = np.where(c.table >= 0, c.table + shift, -1).astype(np.int32)
    plan = runner.Rotary(d, "cuda:0")
    q = runner.cache_append(c.q, c.k, c.v, *c.batch(), plan)
    pages = torch.from_numpy(table).cuda()
    q2 = runner.cache_append(c.q, c.k, c.v, *big, pages, *c.batch()[3:], plan)
    assert torch.equal(q, q2) and all(torch.equal(b[shift:], s) for b, s in zip(big, c.caches))
    o, lse = c.attend(q=q)
    o2, lse2 = runner.cache_attention(q, *big, pages, *c.batch()[3:], c.d ** -0.5)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert attn.attn_device_status(clear=True) == (0, 0)


@pytest.mark.parametrize("left,sinks", [(-1, 0), (200, 5)])
def test_chunks_meet_training(left, sinks):
    """A sequence served in chunks of many lengths gives what the training
    forward gives on the whole of it, to both calls' tolerances."""
    H, H_kv, d, N = 8, 2, 128, 777
    c = Case([(N, N)], H, H_kv, d, 64, BF, left, sinks)
    plan = runner.Rotary(d, "cuda:0")
    o, lse = torch.empty_like(c.q), torch.empty(N, H, device="cuda")
    first = 0
    for n in (1, 1, 7, 128, 129, 1, 400, 110):
        rows = slice(first, first + n)
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        lengths = torch.tensor([first + n], dtype=torch.int32, device="cuda")
        q = runner.cache_append(c.q[rows], c.k[rows], c.v[rows], *c.batch()[:3], starts, lengths,
                                plan)
        o[rows], lse[rows] = runner.cache_attention(q, *c.batch()[:3], starts, lengths, d ** -0.5,
                                                    window_left=left, sinks=sinks)
        first += n
    assert first == N

    def heads(t):
        return t.transpose(0, 1)[None].contiguous()

    q, k = runner.rotary(heads(c.q), heads(c.k), plan)
    o2, lse2 = runner.forward(q, k, heads(c.v), d ** -0.5, True, window=(left, -1), sinks=sinks)
    scale = float(o2.abs().max())
    assert float((heads(o).float() - o2.float()).abs().max()) <= 4e-2 * scale
    assert float((lse.T[None] - lse2).abs().max()) <= 2e-5
