"""Argument checks of the rotary, layer-norm and dropout entry points and of
their torch wrappers, and the host-side frequencies: no GPU needed, nothing
is launched."""
import math

import numpy as np
import pytest
import torch

from oracle import frequencies

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from flashattention_attention_backward_gb300.build import build
    import flashattention_attention_backward_gb300 as attn

    build()
    return attn


@pytest.mark.parametrize("rot", [0, 2, 32, 64, 128, 256])
@pytest.mark.parametrize("scaling", ["plain", "linear", "base", "ramp"])
def test_frequencies(lib, rot, scaling):
    code = {"plain": 0, "linear": 1, "base": 2, "ramp": 3}[scaling]
    rc, turns, m = lib.attn_rotary_frequencies(rot, 500000.0, code, 8.0, 8192, 1.0, 32.0)
    assert rc == lib.ATTN_OK and len(turns) == rot // 2
    w, mag = frequencies(rot, 500000.0, scaling, 8.0, 8192, 1.0, 32.0)
    assert abs(m - mag) <= 2.0 ** -24 * mag
    for t, x in zip(turns, w):
        want = x / (2 * math.pi) * 2.0 ** 64
        # a handful of 64-bit roundings (pow, divisions, the ramp), and half a unit
        assert abs(t - want) <= 64 * 2.0 ** -53 * want + 0.5


def test_frequencies_refusals(lib):
    f = lib.attn_rotary_frequencies
    assert f(63)[0] == f(-2)[0] == lib.ATTN_ERR_SHAPE
    assert f(64, 0.5)[0] == f(64, NAN)[0] == f(64, INF)[0] == lib.ATTN_ERR_SHAPE
    assert f(64, 1e4, 4)[0] == f(64, 1e4, -1)[0] == lib.ATTN_ERR_SHAPE
    for code in (1, 2, 3):
        assert f(64, 1e4, code, 0.5, 4096)[0] == f(64, 1e4, code, NAN, 4096)[0] == \
            lib.ATTN_ERR_SHAPE
    assert f(64, 1e4, 3, 2.0, 0)[0] == lib.ATTN_ERR_SHAPE
    assert f(64, 1e4, 3, 2.0, 4096, 32.0, 32.0)[0] == lib.ATTN_ERR_SHAPE
    assert f(64, 1e4, 3, 2.0, 4096, -1.0, 32.0)[0] == lib.ATTN_ERR_SHAPE
    assert f(64, 1e4, 0, NAN)[0] == lib.ATTN_OK  # the plain kind ignores the factor
    assert lib.library().attn_rotary_frequencies(None, None, 64, 1e4, 0, 1.0, 0, 1.0, 32.0) == \
        lib.ATTN_ERR_NULL


def _rotary_args(lib, **kw):
    a = dict(q=FAKE, k=FAKE, q_out=FAKE, k_out=FAKE, turns=FAKE, positions=FAKE, pos_stride=0, B=1,
             H=2, H_kv=1, N=8, d=64, rot=64, magnitude=1.0, interleaved=False, adjoint=False,
             dtype=0, strides=None)
    a.update(kw)
    return lib.attn_rotary(*a.values())


def test_rotary_refusals(lib):
    call = lambda **kw: _rotary_args(lib, **kw)  # noqa: E731
    for name in ("q", "k", "q_out", "k_out", "turns"):
        assert call(**{name: 0}) == lib.ATTN_ERR_NULL, name
        assert call(**{name: FAKE + 8}) == lib.ATTN_ERR_ALIGN, name
    assert call(positions=FAKE + 4) == lib.ATTN_ERR_ALIGN
    for kw in (dict(B=-1), dict(H=-1), dict(H_kv=-1), dict(N=-1), dict(d=0), dict(rot=-2),
               dict(rot=63), dict(rot=66), dict(pos_stride=-1), dict(magnitude=NAN),
               dict(strides=[0] * 11 + [-1]),
               # inputs may be broadcast, outputs not
               dict(strides=[0] * 12), dict(strides=[0] * 6 + [1024, 512, 64, 512, 64, 0])):
        assert call(**kw) == lib.ATTN_ERR_SHAPE, kw
    assert call(dtype=3) == call(dtype=-1) == lib.ATTN_ERR_SHAPE
    assert call(N=1 << 30, B=1 << 11) == lib.ATTN_ERR_TOO_LARGE
    assert call(strides=[0, 0, 1 << 40] * 4) == lib.ATTN_ERR_TOO_LARGE
    with pytest.raises(ValueError, match="strides"):
        call(strides=[1, 2, 3])
    # empty problems, their pointers NULL
    assert call(B=0, q=0, k=0, q_out=0, k_out=0) == lib.ATTN_OK
    assert call(N=0) == call(H=0, H_kv=0, q=0, k=0, q_out=0, k_out=0) == lib.ATTN_OK


def test_finalize_rotary_refusals(lib):
    def call(**kw):
        a = dict(dq_accum=FAKE, dq=FAKE, dk=FAKE, dk_out=FAKE, scale=0.125, turns=FAKE,
                 positions=0, pos_stride=0, B=1, H=2, H_kv=1, N=8, d=64, rot=64, magnitude=1.0,
                 interleaved=False, strides=None)
        a.update(kw)
        return lib.attn_bwd_finalize_rotary(*a.values())

    for name in ("dq_accum", "dq", "dk", "dk_out", "turns"):
        assert call(**{name: 0}) == lib.ATTN_ERR_NULL, name
        assert call(**{name: FAKE + 8}) == lib.ATTN_ERR_ALIGN, name
    for kw in (dict(B=-1), dict(rot=63), dict(rot=66), dict(scale=NAN), dict(scale=INF),
               dict(strides=[-1] * 6), dict(strides=[0] * 6)):
        assert call(**kw) == lib.ATTN_ERR_SHAPE, kw
    assert call(B=0) == call(N=0) == lib.ATTN_OK


def test_layer_norm_refusals(lib):
    def fwd(**kw):
        a = dict(x=FAKE, gamma=FAKE, beta=FAKE, y=FAKE, mean=FAKE, rstd=FAKE, rows=4, C=64,
                 eps=1e-5, dtype=0, wdtype=2)
        a.update(kw)
        return lib.attn_layer_norm(*a.values())

    def bwd(**kw):
        a = dict(dy=FAKE, x=FAKE, gamma=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE, dgamma=FAKE,
                 dbeta=FAKE, workspace=FAKE, rows=4, C=64, dtype=0, wdtype=2)
        a.update(kw)
        return lib.attn_layer_norm_bwd(*a.values())

    for call, needed, others in ((fwd, "x y", "gamma beta mean rstd"),
                                 (bwd, "dy x mean rstd dx workspace", "gamma dgamma dbeta")):
        for name in needed.split():
            assert call(**{name: 0}) == lib.ATTN_ERR_NULL, name
        for name in (needed + " " + others).split():
            assert call(**{name: FAKE + 4}) == lib.ATTN_ERR_ALIGN, name
        assert call(rows=-1) == call(C=0) == call(C=-5) == lib.ATTN_ERR_SHAPE
        assert call(dtype=3) == call(wdtype=-1) == lib.ATTN_ERR_SHAPE
        assert call(rows=1 << 40) == call(rows=1 << 30, C=1 << 20) == \
            call(rows=1, C=(1 << 29) + 1) == lib.ATTN_ERR_TOO_LARGE
    assert fwd(eps=-1.0) == fwd(eps=NAN) == fwd(eps=INF) == lib.ATTN_ERR_SHAPE
    assert fwd(rows=0, x=0, y=0, mean=0, rstd=0) == lib.ATTN_OK
    assert bwd(rows=0, dgamma=0, dbeta=0, workspace=0, dy=0, x=0, dx=0) == lib.ATTN_OK
    size = lib.attn_layer_norm_bwd_workspace_bytes
    assert size(-1, 64) == size(4, 0) == lib.ATTN_ERR_SHAPE
    assert size(1 << 40, 64) == lib.ATTN_ERR_TOO_LARGE
    # two fp32 sums a column for each of at most 1024 blocks
    for rows, C in ((0, 64), (1, 64), (4096, 1001), (1 << 30, 128)):
        assert 0 < size(rows, C) <= 1024 * 2 * C * 4 and size(rows, C) % (2 * C * 4) == 0


def test_dropout_refusals(lib):
    def add(**kw):
        a = dict(x=FAKE, residual=FAKE, y=FAKE, n=64, p=0.1, seed=1, dtype=0)
        a.update(kw)
        return lib.attn_dropout_add(*a.values())

    def fwd(**kw):
        a = dict(x=FAKE, residual=FAKE, gamma=FAKE, beta=FAKE, z=FAKE, y=2 * FAKE, mean=FAKE,
                 rstd=FAKE, rows=4, C=64, eps=1e-5, p=0.1, seed=1, dtype=0, wdtype=0)
        a.update(kw)
        return lib.attn_dropout_add_norm(*a.values())

    def bwd(**kw):
        a = dict(dy=FAKE, dz=FAKE, z=FAKE, gamma=FAKE, mean=FAKE, rstd=FAKE, dx=FAKE,
                 dresidual=2 * FAKE, dgamma=FAKE, dbeta=FAKE, workspace=FAKE, rows=4, C=64, p=0.1,
                 seed=1, dtype=0, wdtype=0)
        a.update(kw)
        return lib.attn_dropout_add_norm_bwd(*a.values())

    for call, needed in ((add, "x y"), (fwd, "x residual z y"),
                         (bwd, "dy z mean rstd dx dresidual workspace")):
        for name in needed.split():
            assert call(**{name: 0}) == lib.ATTN_ERR_NULL, name
            assert call(**{name: FAKE + 2}) == lib.ATTN_ERR_ALIGN, name
        for p in (-0.1, 1.0, 1.5, NAN, INF):
            assert call(p=p) == lib.ATTN_ERR_SHAPE, p
        assert call(dtype=7) == lib.ATTN_ERR_SHAPE
    assert add(residual=FAKE + 2) == fwd(beta=FAKE + 2) == bwd(dz=FAKE + 2) == lib.ATTN_ERR_ALIGN
    assert add(n=-1) == fwd(rows=-1) == bwd(C=0) == lib.ATTN_ERR_SHAPE
    assert fwd(eps=-1e-5) == lib.ATTN_ERR_SHAPE
    # the two outputs of a call are two buffers
    assert fwd(y=FAKE) == bwd(dresidual=FAKE) == lib.ATTN_ERR_SHAPE
    assert add(n=1 << 40) == lib.ATTN_ERR_TOO_LARGE
    assert add(n=0, x=0, y=0, residual=0) == fwd(rows=0) == lib.ATTN_OK
    assert bwd(rows=0, dgamma=0, dbeta=0, workspace=0) == lib.ATTN_OK


def test_runner_refusals(lib):
    from flashattention_attention_backward_gb300 import runner

    plan = runner.Rotary(64, "cpu")
    assert plan.turns.dtype == torch.int64 and plan.turns.numel() == 32 and plan.magnitude == 1.0
    assert int(plan.turns[0]) == int(round(2.0 ** 64 / (2 * math.pi)))
    with pytest.raises(ValueError, match="scaling"):
        runner.Rotary(64, "cpu", scaling="other")
    with pytest.raises(lib.AttnError):
        runner.Rotary(63, "cpu")
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64)
    for bad, match in (((q[0], k), "4-D"), ((q, k[:, :, :4]), "shape"), ((q, k.half()), "both"),
                       ((q.double(), None), "both"), ((q.transpose(2, 3), None), "contiguous"),
                       ((q, k), "CUDA")):
        with pytest.raises(ValueError, match=match):
            runner.rotary(*bad, runner.Rotary(8, "cpu"))
    x, w = torch.zeros(4, 16), torch.ones(16)
    for args, match in (((x.double(),), "bfloat16"), ((x.t(),), "contiguous"),
                        ((torch.zeros(()),), "C"), ((x, w[:8]), "gamma"),
                        ((x, w, w.half()), "share"), ((x, w, w), "CUDA")):
        with pytest.raises(ValueError, match=match):
            runner.layer_norm(*args)
    with pytest.raises(ValueError, match="residual"):
        runner.dropout_add(x, x[:2])
    with pytest.raises(ValueError, match="CUDA"):
        runner.dropout_add(x)
    with pytest.raises(ValueError, match="CUDA"):
        runner.dropout_add_norm(x, x)
    with pytest.raises(ValueError, match="CUDA"):
        runner.layer_norm_backward(x, x, w, x[:, 0], x[:, 0])
    with pytest.raises(ValueError, match="CUDA"):
        runner.dropout_add_norm_backward(x, None, x, w, x[:, 0], x[:, 0])
