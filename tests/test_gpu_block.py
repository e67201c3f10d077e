"""Norm, rotary positions, attention, dropout + residual + norm run together,
forward and backward, against the 64-bit oracle of the same chain; and the
rotary's adjoint at the end of each form of the attention backward.

Tolerances: attention's gradients and O by the parity bar of the other tests.
In the whole chain a value passes at most 7 roundings to bf16 forward (norm,
rotary, P, O, dropout's sum, and twice more inside the matrix products'
operands) and 7 back, each at most half a step, 2^-8 relative; their
contributions add up in the Frobenius norm to at most 14 * 2^-8 of it.
"""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from flashattention_attention_backward_gb300.inputs import Workload, make_inputs
from oracle import (attention_backward, attention_forward, dropout, layer_norm,
                    layer_norm_backward, rotate)

pytestmark = pytest.mark.gpu

from parity_helpers import check_grad, rel_fro  # noqa: E402

DEV = torch.device("cuda:0")
CHAIN = 14 * 2.0 ** -8


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("form", ["plain", "dropout", "window", "deterministic", "given buffers"])
@pytest.mark.parametrize("d,interleaved", [(64, True), (128, False)])
def test_backward_of_rotated_inputs(form, d, interleaved):
    """runner.backward(rotary=...) gives the gradients of what went into the
    rotation."""
    w = Workload("rot", 2, 4, 2, 200, d, True, seed_base=31)
    x = make_inputs(w)
    q, k, v, do = (x[n].to(DEV) for n in ("q", "k", "v", "do"))
    plan = runner.Rotary(d // 2, DEV, interleaved=interleaved)
    positions = torch.randint(0, 100000, (w.B, 1), generator=torch.Generator().manual_seed(4)) + \
        torch.arange(w.N)
    qr, kr = runner.rotary(q, k, plan, positions.to(DEV))
    kw = {"dropout": {"dropout": (0.25, 9)}, "window": {"window": (64, -1)}}.get(form, {})
    o, lse = runner.forward(qr, kr, v, w.scale, True, **kw)
    if form == "deterministic":
        kw = {"deterministic": True}
    if form == "given buffers":
        kw = {"bufs": runner.BackwardBuffers(qr, kr)}
    dq, dk, dv = runner.backward(qr, kr, v, o, do, lse, w.scale, True, rotary=plan,
                                 positions=positions.to(DEV), **kw)
    oracle_kw = {"dropout": {"dropout": (0.25, 9)}, "window": {"window": (64, -1)}}.get(form, {})
    turns, p = plan.turns.tolist(), positions.numpy()
    # the bf16 values that the attention call saw
    dQ, dK, dV = attention_backward(_np(qr), _np(kr), _np(v), _np(do), w.scale, True, **oracle_kw)
    check_grad("dQ", dq.cpu(), rotate(dQ, turns, p, 1.0, interleaved, adjoint=True))
    check_grad("dK", dk.cpu(), rotate(dK, turns, p, 1.0, interleaved, adjoint=True))
    check_grad("dV", dv.cpu(), dV)


def test_positions_need_a_rotary():
    t = torch.zeros(1, 1, 8, 64, dtype=torch.bfloat16, device=DEV)
    lse = torch.zeros(1, 1, 8, device=DEV)
    with pytest.raises(ValueError, match="rotary"):
        runner.backward(t, t, t, t, t, lse, 0.1, True, positions=torch.arange(8, device=DEV))
    plan = runner.Rotary(64, DEV)
    for bad in (torch.arange(7, device=DEV), torch.arange(8, device=DEV).int(), torch.arange(8)):
        with pytest.raises(ValueError):
            runner.rotary(t, t, plan, bad)
    with pytest.raises(ValueError, match="rot"):
        runner.rotary(t, t, runner.Rotary(128, DEV))


class _Chain:
    """x -> norm -> packed q, k, v -> rotary -> attention with dropout ->
    dropout + residual -> norm."""
    B, N, H, H_kv, d = 2, 150, 4, 2, 64
    p, seed = 0.1, 2024

    def __init__(self, seed):
        g = torch.Generator().manual_seed(seed)
        wide, C = (self.H + 2 * self.H_kv) * self.d, self.H * self.d
        draw = lambda *s: torch.randn(*s, generator=g).bfloat16().to(DEV)  # noqa: E731
        self.x, self.res = draw(self.B, self.N, wide), draw(self.B, self.N, C)
        self.g1, self.b1 = 1 + 0.1 * draw(wide).float(), 0.1 * draw(wide).float()
        self.g2, self.b2 = 1 + 0.1 * draw(C).float(), 0.1 * draw(C).float()
        self.dy, self.dz = draw(self.B, self.N, C), draw(self.B, self.N, C)
        self.plan = runner.Rotary(self.d, DEV)
        self.scale = self.d ** -0.5

    def heads(self, t):
        t = t.view(self.B, self.N, self.H + 2 * self.H_kv, self.d).transpose(1, 2)
        return t[:, :self.H], t[:, self.H:self.H + self.H_kv], t[:, self.H + self.H_kv:]

    def run(self):
        drop = (self.p, self.seed)
        h, m1, r1 = runner.layer_norm(self.x, self.g1, self.b1)
        q, k, v = self.heads(h)
        q, k = runner.rotary(q, k, self.plan)
        v = v.contiguous()
        o, lse = runner.forward(q, k, v, self.scale, True, dropout=drop)
        a = o.transpose(1, 2).reshape(self.B, self.N, -1)
        z, y, m2, r2 = runner.dropout_add_norm(a, self.res, self.g2, self.b2, dropout=drop)
        da, dres, dg2, db2 = runner.dropout_add_norm_backward(self.dy, self.dz, z, self.g2, m2, r2,
                                                              drop)
        do = da.view(self.B, self.N, self.H, self.d).transpose(1, 2).contiguous()
        dq, dk, dv = runner.backward(q, k, v, o, do, lse, self.scale, True, dropout=drop,
                                     rotary=self.plan)
        dh = torch.cat((dq, dk, dv), 1).transpose(1, 2).reshape(self.x.shape)
        dx, dg1, db1 = runner.layer_norm_backward(dh, self.x, self.g1, m1, r1)
        return {"z": z, "y": y, "dx": dx, "dres": dres, "dg1": dg1, "db1": db1, "dg2": dg2,
                "db2": db2}

    def oracle(self):
        drop = (float(np.float32(self.p)), self.seed)
        rows = lambda t: t.reshape(self.B * self.N, -1)  # noqa: E731
        split = lambda t: tuple(np.ascontiguousarray(s) for s in np.split(  # noqa: E731
            t.reshape(self.B, self.N, -1, self.d).transpose(0, 2, 1, 3),
            (self.H, self.H + self.H_kv), 1))
        flat = lambda t: rows(t.transpose(0, 2, 1, 3).reshape(self.B, self.N, -1))  # noqa: E731
        eps, turns = 1e-5, self.plan.turns.tolist()
        pos = np.broadcast_to(np.arange(self.N), (self.B, self.N))
        x, g1, g2 = rows(_np(self.x)), _np(self.g1), _np(self.g2)
        h, m1, r1 = layer_norm(x, g1, _np(self.b1), eps)
        q, k, v = split(h)
        q, k = rotate(q, turns, pos), rotate(k, turns, pos)
        o, _ = attention_forward(q, k, v, self.scale, True, dropout=drop)
        z = rows(_np(self.res)) + dropout(flat(o), *drop)
        y, m2, r2 = layer_norm(z, g2, _np(self.b2), eps)
        dy = rows(_np(self.dy))
        dz, dg2, db2 = layer_norm_backward(dy, z, g2, m2, r2)
        dz = dz + rows(_np(self.dz))
        da = dropout(dz, *drop)
        do = da.reshape(self.B, self.N, self.H, self.d).transpose(0, 2, 1, 3)
        dq, dk, dv = attention_backward(q, k, v, do, self.scale, True, dropout=drop)
        dh = np.concatenate((rotate(dq, turns, pos, adjoint=True),
                             rotate(dk, turns, pos, adjoint=True), dv), 1)
        dx, dg1, db1 = layer_norm_backward(flat(dh), x, g1, m1, r1)
        return {"z": z, "y": y, "dx": dx, "dres": dz, "dg1": dg1, "db1": db1, "dg2": dg2,
                "db2": db2}


def test_chain_against_the_oracle():
    c = _Chain(1)
    got, want = c.run(), c.oracle()
    rc, status = attn.attn_device_status(clear=True)
    assert rc == 0 and status == 0
    for name, ref in want.items():
        g = _np(got[name]).reshape(ref.shape)
        assert np.isfinite(g).all(), name
        assert rel_fro(g, ref) <= CHAIN, "%s: %.3e" % (name, rel_fro(g, ref))


def test_chain_captured():
    """The chain in a graph, replayed on new contents beside eager runs."""
    c, fresh = _Chain(2), _Chain(3)
    c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run()
    for name in ("x", "res", "dy", "dz"):
        getattr(c, name).copy_(getattr(fresh, name))
    for name in ("g1", "b1", "g2", "b2"):
        getattr(c, name).copy_(getattr(fresh, name))
    graph.replay()
    torch.cuda.synchronize()
    want = fresh.run()
    torch.cuda.synchronize()
    for name in ("z", "y", "dres", "dg2", "db2"):  # a fixed order of sums: the same bits
        assert torch.equal(out[name], want[name]), name
    for name in ("dx", "dg1", "db1"):  # behind dQ, whose atomics come in any order
        assert rel_fro(_np(out[name]), _np(want[name])) <= CHAIN, name


class _Mixed:
    """Calls behind one another, behind a fill and a copy, and behind the join of
    two streams: each must find the results of what stands before it."""

    def __init__(self, rows, C):
        g = torch.Generator(device=DEV).manual_seed(rows + C)
        self.src = torch.randint(-8, 8, (rows, C), device=DEV, generator=g).float()
        self.gamma = torch.randn(C, device=DEV, generator=g)
        self.x, self.z, self.out, self.dx = (torch.zeros_like(self.src) for _ in range(4))
        self.dgamma, self.dbeta = (torch.zeros(C, device=DEV) for _ in range(2))

    def run(self, main, other, between=lambda: None):
        x = self.x
        with torch.cuda.stream(main):
            x.zero_()
            x.copy_(self.src)
            between()
            y = runner.dropout_add(x, self.src)
            between()
            forked = torch.cuda.Event()
            forked.record(main)
        with torch.cuda.stream(other):
            other.wait_event(forked)
            side = runner.dropout_add(y)
            between()
            joined = torch.cuda.Event()
            joined.record(other)
        with torch.cuda.stream(main):
            self.out.zero_()
            main.wait_event(joined)
            between()
            z = runner.dropout_add(side, y)
            between()
            norm, mean, rstd = runner.layer_norm(z, self.gamma, self.gamma)
            between()
            dx, dgamma, dbeta = runner.layer_norm_backward(z, norm, self.gamma, mean, rstd)
            between()
            self.dx.copy_(runner.dropout_add(dx, norm))
            self.z.copy_(z)
            self.out.copy_(norm)
            self.dgamma.copy_(dgamma)
            self.dbeta.copy_(dbeta)

    def results(self):
        return [t.clone() for t in (self.z, self.out, self.dx, self.dgamma, self.dbeta)]


@pytest.mark.parametrize("rows,C", [(1, 1), (40, 64), (300, 1001), (64, 10000), (3, 20000)])
def test_calls_wait_for_what_stands_before(rows, C):
    """Back to back and in a graph the same bits as with a wait after each call."""
    m = _Mixed(rows, C)
    main, other = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    m.run(main, other, between=torch.cuda.synchronize)
    torch.cuda.synchronize()
    assert torch.equal(m.z, 4 * m.src)  # sums of small integers: exact
    want = m.results()
    for _ in range(20):
        m.run(main, other)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(m.results(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        m.run(main, other)
    for t in (m.z, m.out, m.dx, m.dgamma, m.dbeta):
        t.fill_(7)
    torch.cuda.synchronize()
    for _ in range(20):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(m.results(), want))
