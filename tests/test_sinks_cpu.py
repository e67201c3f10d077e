"""The window with sinks, without a GPU: the oracle's mask against the
definition pair by pair and its gradients against differences, and the
argument checks of the entry points and the torch wrappers."""
import numpy as np
import pytest
import torch

from flashattention_attention_backward_gb300 import runner
from oracle import attention_backward, attention_forward, head_forward

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    from flashattention_attention_backward_gb300.build import build
    import flashattention_attention_backward_gb300 as attn

    build()
    return attn


@pytest.mark.parametrize("causal,window,sinks", [(True, (3, -1), 2), (False, (2, 1), 4),
                                                 (False, (0, 0), 1), (True, (0, -1), 30),
                                                 (False, (-1, 2), 3), (True, (4, -1), 0)])
def test_oracle_mask(causal, window, sinks):
    n, d = 11, 4
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((n, d)) for _ in range(3))
    fw = head_forward(q, k, v, 0.5, causal, window=window, sinks=sinks)
    left = window[0] if window[0] >= 0 else n
    right = 0 if causal else (window[1] if window[1] >= 0 else n)
    for i in range(n):
        seen = [j for j in range(n) if j <= i + right and (j >= i - left or j < sinks)]
        assert set(np.flatnonzero(fw["P"][i])) == set(seen)
        w = np.exp(0.5 * k[seen] @ q[i])
        assert np.allclose(fw["O"][i], (w / w.sum()) @ v[seen], rtol=1e-12, atol=0)
        assert np.isclose(fw["LSE"][i], np.log(w.sum()), rtol=1e-12)


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(4)
    B, H, H_kv, N, d = 1, 2, 1, 9, 3
    x = [rng.standard_normal(s) for s in ((B, H, N, d), (B, H_kv, N, d), (B, H_kv, N, d))]
    do = rng.standard_normal((B, H, N, d))
    kw = dict(causal=True, softcap=1.5, window=(2, -1), sinks=2)
    grads = attention_backward(*x, do, 0.7, **kw)
    step = 1e-5
    for t, g in enumerate(grads):
        for at in np.ndindex(x[t].shape):
            side = []
            for s in (step, -step):
                y = [a.copy() for a in x]
                y[t][at] += s
                side.append((attention_forward(*y, 0.7, **kw)[0] * do).sum())
            # central differences: step^2 times a third derivative, and the
            # sums' rounding over the step
            assert abs((side[0] - side[1]) / (2 * step) - g[at]) <= 1e-8


def test_refusals(lib):
    def fwd(fn, **kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, lse=FAKE, B=1, H=2, H_kv=1, N=8, d=64,
                 scale=0.125, causal=True, softcap=0.0, left=4, right=-1, sinks=1)
        a.update(kw)
        return fn(*a.values())

    def bwd(**kw):
        a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, do=FAKE, lse=FAKE, dq=FAKE, dk=FAKE, dv=FAKE,
                 B=1, H=2, H_kv=1, N=8, d=64, scale=0.125, causal=True, softcap=0.0, dpsum=FAKE,
                 left=4, right=-1, sinks=1)
        a.update(kw)
        return lib.attn_bwd_sinks(*a.values())

    calls = [lambda **kw: fwd(lib.attn_fwd_sinks, **kw),
             lambda **kw: fwd(lib.attn_fwd_ref_sinks, **kw), bwd]
    for call in calls:
        assert call(sinks=-1) == lib.ATTN_ERR_SHAPE
        assert call(q=0) == call(k=0) == call(lse=0) == lib.ATTN_ERR_NULL
        assert call(v=FAKE + 8) == lib.ATTN_ERR_ALIGN
        assert call(d=96) == lib.ATTN_ERR_UNSUPPORTED
        assert call(H=3, H_kv=2) == call(scale=float("nan")) == lib.ATTN_ERR_SHAPE
        assert call(N=0, sinks=7) == lib.ATTN_OK
    assert bwd(dpsum=0) == lib.ATTN_ERR_NULL


def test_runner_refusals():
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 8)
    for call in (lambda **kw: runner.forward(t, t, t, 0.125, True, **kw),
                 lambda **kw: runner.backward(t, t, t, t, t, lse, 0.125, True, **kw)):
        with pytest.raises(ValueError, match="CUDA"):
            call(sinks=1)
    for kw, what in ((dict(sinks=-1), "negative"), (dict(sinks=1, dropout=(0.1, 3)), "dropout"),
                     (dict(sinks=1, deterministic=True), "deterministic")):
        with pytest.raises(ValueError, match=what):
            runner._check_sinks(kw["sinks"], None, kw.get("dropout")) if what != "deterministic" \
                else _refuse_deterministic(kw)


def _refuse_deterministic(kw):
    """backward() meets that check behind the device's; give it tensors that
    pass for CUDA ones."""
    saved = runner._dims, runner._check_lse
    runner._dims, runner._check_lse = (lambda *a: (1, 2, 2, 8, 64)), (lambda *a: None)
    try:
        t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
        runner.backward(t, t, t, t, t, None, 0.125, True, **kw)
    finally:
        runner._dims, runner._check_lse = saved


def test_counts_past_32_bits():
    assert runner._check_sinks(1 << 32, None, None) == ((-1, -1), 1 << 30)
    assert runner._check_sinks(0, (-1 << 33, 1 << 33), None) == ((-1, 1 << 30), 0)
    assert runner._check_sinks(0, None, (0.1, 3)) == (None, 0)
