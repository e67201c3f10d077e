"""The calls over a paged cache, without a GPU: the oracle against attention
written out on one dense sequence, and the argument checks of the entry points
and the torch wrappers."""
import ctypes

import numpy as np
import pytest
import torch

from flashattention_attention_backward_gb300 import runner
from oracle import attention_forward, cache_append, cache_attention, frequencies, rotate

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from flashattention_attention_backward_gb300.build import build
    import flashattention_attention_backward_gb300 as attn

    build()
    return attn


def test_oracle_is_dense_attention():
    """A sequence appended in three chunks attends as the whole one does."""
    rng = np.random.default_rng(2)
    H, H_kv, d, page, N = 4, 2, 8, 4, 23
    q, k, v = (rng.standard_normal((N, h, d)) for h in (H, H_kv, H_kv))
    turns = [int(f / (2 * np.pi) * 2 ** 64) for f in frequencies(d, 1e4, "plain", 1, 0, 1, 32)[0]]
    pages = [rng.permutation(8)]
    kc, vc = np.full((8, page, H_kv, d), np.nan), np.full((8, page, H_kv, d), np.nan)
    o, lse = np.empty((N, H, d)), np.empty((N, H))
    for first, end in ((0, 9), (9, 10), (10, N)):
        starts, lengths = [0, end - first], [end]
        qo, kc, vc = cache_append(q[first:end], k[first:end], v[first:end], kc, vc, turns, 1.0,
                                  False, starts, lengths, pages)
        o[first:end], lse[first:end] = cache_attention(qo, kc, vc, starts, lengths, pages, 0.3,
                                                       left=6, sinks=2)[:2]
    p = np.arange(N)[None]
    qr, kr = (rotate(x.transpose(1, 0, 2)[None], turns, p) for x in (q, k))
    O, LSE = attention_forward(qr, kr, v.transpose(1, 0, 2)[None], 0.3, True, window=(6, -1),
                               sinks=2)
    assert np.allclose(o, O[0].transpose(1, 0, 2), rtol=1e-12, atol=1e-14)
    assert np.allclose(lse, LSE[0].T, rtol=1e-12)


def _append(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, q_out=FAKE, k_cache=FAKE, v_cache=FAKE, turns=FAKE,
             starts=FAKE, lengths=FAKE, pages=FAKE, T=5, B=2, H=4, H_kv=2, d=64, rot=64,
             magnitude=1.0, interleaved=False, page_size=16, max_pages=3, n_pages=9, dtype=0,
             strides=None)
    a.update(kw)
    return lib.attn_cache_append(*a.values())


def _fwd(lib, **kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, o=FAKE, lse=FAKE, starts=FAKE, lengths=FAKE,
             pages=FAKE, workspace=FAKE, T=5, B=2, H=4, H_kv=2, d=64, page_size=16, max_pages=3,
             n_pages=9, scale=0.125, causal=True, softcap=0.0, left=-1, sinks=0, dtype=0,
             strides=None)
    a.update(kw)
    return lib.attn_cache_fwd(*a.values())


def test_append_refusals(lib):
    call = lambda **kw: _append(lib, **kw)  # noqa: E731
    for name in ("q", "k", "v", "q_out", "k_cache", "v_cache", "turns", "starts", "lengths",
                 "pages"):
        assert call(**{name: 0}) == lib.ATTN_ERR_NULL, name
    for name in ("q", "k", "v", "q_out", "k_cache", "v_cache", "turns"):
        assert call(**{name: FAKE + 8}) == lib.ATTN_ERR_ALIGN, name
    for name in ("starts", "lengths", "pages"):
        assert call(**{name: FAKE + 2}) == lib.ATTN_ERR_ALIGN, name
    for kw in (dict(T=-1), dict(B=-1), dict(H=-1), dict(H_kv=0), dict(d=0), dict(rot=3),
               dict(rot=-2), dict(rot=66), dict(magnitude=NAN), dict(page_size=0),
               dict(max_pages=-1), dict(n_pages=-1), dict(dtype=2), dict(dtype=-1),
               dict(strides=[-1] * 14),
               # inputs may be broadcast, outputs not
               dict(strides=[0] * 14), dict(strides=[0] * 6 + [256, 64] + [0, 128, 64] * 2)):
        assert call(**kw) == lib.ATTN_ERR_SHAPE, kw
    assert call(T=1 << 30, H=1 << 10) == call(H=20000, H_kv=1) == lib.ATTN_ERR_TOO_LARGE
    assert call(strides=[1 << 40] * 14) == lib.ATTN_ERR_TOO_LARGE
    with pytest.raises(ValueError, match="strides"):
        call(strides=[1, 2, 3])
    nothing = dict(q=0, k=0, v=0, q_out=0, k_cache=0, v_cache=0, turns=0, starts=0, lengths=0,
                   pages=0)
    assert call(T=0, **nothing) == call(B=0, **nothing) == lib.ATTN_OK


def test_attention_refusals(lib):
    call = lambda **kw: _fwd(lib, **kw)  # noqa: E731
    for name in ("q", "k_cache", "v_cache", "o", "starts", "lengths", "pages", "workspace"):
        assert call(**{name: 0}) == lib.ATTN_ERR_NULL, name
    for name in ("q", "k_cache", "v_cache", "o", "lse", "workspace"):
        assert call(**{name: FAKE + 8}) == lib.ATTN_ERR_ALIGN, name
    for kw in (dict(T=-1), dict(B=-1), dict(H=-1), dict(H_kv=0), dict(H=3), dict(d=0),
               dict(scale=NAN), dict(scale=0.0), dict(scale=-1.0), dict(softcap=NAN),
               dict(sinks=-1), dict(page_size=0), dict(max_pages=-1), dict(n_pages=-1),
               dict(dtype=2), dict(strides=[-8] * 10), dict(strides=[0] * 10)):
        assert call(**kw) == lib.ATTN_ERR_SHAPE, kw
    for kw in (dict(d=96), dict(page_size=12), dict(H=129, H_kv=1)):
        assert call(**kw) == lib.ATTN_ERR_UNSUPPORTED, kw
    # strides of whole 16-byte groups
    good = [256, 64, 256, 64, 2048, 128, 64, 2048, 128, 64]
    for i in range(10):
        assert call(strides=good[:i] + [good[i] + 4] + good[i + 1:]) == lib.ATTN_ERR_ALIGN, i
    assert call(T=1 << 30, H=1 << 10, H_kv=16) == lib.ATTN_ERR_TOO_LARGE
    assert call(T=0, q=0, o=0, workspace=0, starts=0) == call(B=0) == call(H=0, q=0) == lib.ATTN_OK


def test_workspace_sizes(lib):
    f = lib.attn_cache_fwd_workspace_bytes
    assert f(5, 2, 4, 2, 64) >= 0
    assert f(-1, 2, 4, 2, 64) == f(5, 2, 3, 2, 64) == lib.ATTN_ERR_SHAPE
    assert f(5, 2, 4, 2, 80) == lib.ATTN_ERR_UNSUPPORTED
    assert isinstance(lib.library().attn_cache_fwd_workspace_bytes.restype(), ctypes.c_longlong)


def _tensors(**kw):
    bf = torch.bfloat16
    t = dict(q=torch.zeros(5, 4, 64, dtype=bf), k=torch.zeros(5, 2, 64, dtype=bf),
             v=torch.zeros(5, 2, 64, dtype=bf), k_cache=torch.zeros(9, 16, 2, 64, dtype=bf),
             v_cache=torch.zeros(9, 16, 2, 64, dtype=bf),
             pages=torch.zeros(2, 3, dtype=torch.int32),
             starts=torch.zeros(3, dtype=torch.int32), lengths=torch.zeros(2, dtype=torch.int32))
    t.update(kw)
    return t


@pytest.mark.parametrize("kw,what", [
    (dict(), "CUDA"),
    (dict(k_cache=torch.zeros(9, 16, 2, 64)), "bfloat16"),
    (dict(k_cache=torch.zeros(9, 16, 64, dtype=torch.bfloat16)), "4-D"),
    (dict(v_cache=torch.zeros(9, 16, 3, 64, dtype=torch.bfloat16)), "4-D of one shape"),
    (dict(pages=torch.zeros(2, 3)), "int32"),
    (dict(lengths=torch.zeros(2, dtype=torch.int64)), "int32"),
    (dict(starts=torch.zeros(2, dtype=torch.int32)), "starts"),
    (dict(zip(("k_cache", "v_cache"),
              [torch.zeros(1, 8, 2, 64, dtype=torch.bfloat16).expand(1 << 32, 8, 2, 64)] * 2)),
     "2\\^31"),
    (dict(q=torch.zeros(5, 4, 32, dtype=torch.bfloat16)), "rows"),
    (dict(q=torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "contiguous"),
])
def test_runner_refusals(lib, kw, what):
    t = _tensors(**kw)
    plan = type("Plan", (), dict(rot=64, turns=torch.zeros(32, dtype=torch.int64), magnitude=1.0,
                                 interleaved=False))
    rest = [t[n] for n in ("k_cache", "v_cache", "pages", "starts", "lengths")]
    with pytest.raises(ValueError, match=what):
        runner.cache_append(t["q"], t["k"], t["v"], *rest, plan)
    with pytest.raises(ValueError, match=what):
        runner.cache_attention(t["q"], *rest, 0.125)


def test_runner_bounds_counts():
    # what the C calls take is the low 32 bits of an int
    assert [runner._bound(n) for n in (-(1 << 40), -1, 0, 7, 1 << 30, 1 << 32, (1 << 40) + 1)] == \
        [-1, -1, 0, 7, 1 << 30, 1 << 30, 1 << 30]
