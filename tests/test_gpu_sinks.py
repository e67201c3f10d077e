"""attn_fwd_sinks, attn_fwd_ref_sinks and attn_bwd_sinks (a local window whose
first keys stay visible) against the fp64 oracle under the same mask, with the
tolerances of the other parity tests (dQ, dK, dV max-rel <= 2e-2 and Frobenius
<= 5e-3; O max-rel <= 2e-2; LSE abs <= 1e-5)."""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from flashattention_attention_backward_gb300.inputs import WORKLOADS, Workload, make_inputs, \
    sample_slices
from oracle import attention_backward, attention_forward
from parity_helpers import O_MAX_REL, check_grad, lse_tol, rel_max

pytestmark = pytest.mark.gpu


def _w(B, H, H_kv, N, d, causal, softcap=0.0, sigma=1.0, seed=77):
    return Workload("sinks", B, H, H_kv, N, d, causal, softcap, sigma, 1.0, seed)


CASES = [
    # workload, window, sinks: sinks inside a block, at its edge, over several
    # blocks, meeting the band, past the sequence; bands far from the sinks
    (_w(1, 1, 1, 1, 64, True), (0, -1), 1),
    (_w(2, 2, 1, 129, 128, True), (0, -1), 1),
    (_w(1, 4, 2, 700, 128, True), (100, -1), 4),
    (_w(1, 2, 2, 640, 64, True), (63, -1), 127),
    (_w(1, 2, 2, 641, 64, True), (200, -1), 128),
    (_w(2, 3, 1, 777, 128, True), (50, -1), 129),
    (_w(1, 2, 1, 900, 256, True), (130, -1), 5),
    (_w(1, 2, 2, 515, 256, False), (40, 70), 300),
    (_w(1, 6, 3, 999, 64, False, 2.0, 2.0), (255, 100), 130),
    (_w(1, 2, 1, 450, 128, True, 5.0, 2.0), (31, -1), 40),
    (_w(1, 2, 2, 400, 128, False), (10, 0), 390),
    (_w(1, 2, 2, 333, 64, True), (5, -1), 5000),
    (_w(16, 8, 4, 300, 128, True), (20, -1), 3),
    (_w(1, 2, 2, 385, 128, False), (-1, 37), 64),
    # key blocks with sinks that clusters of CTAs share, ragged ends, few and
    # many heads a group, all sinks in one block and in several
    (_w(1, 8, 1, 1500, 128, True), (100, -1), 4),
    (_w(1, 3, 3, 2001, 64, True), (64, -1), 200),
    (_w(1, 4, 2, 1300, 64, False, 3.0, 2.0), (70, 30), 257),
    (_w(2, 5, 1, 1111, 256, True), (50, -1), 129),
    (_w(1, 1, 1, 1030, 256, False, 4.0, 2.0), (50, 9), 1),
    (_w(1, 2, 1, 1025, 128, True, 8.0, 2.0), (10, -1), 1025),
    # more clusters than run at once
    (_w(1, 18, 18, 1000, 64, True), (60, -1), 4),
]


def _run(w, win, sinks, x):
    dev = torch.device("cuda:0")
    q, k, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))
    out = {}
    for impl in ("tc", "ref"):
        out["o_" + impl], out["lse_" + impl] = runner.forward(
            q, k, v, w.scale, w.causal, w.softcap, window=win, sinks=sinks, impl=impl)
    out["dq"], out["dk"], out["dv"] = runner.backward(
        q, k, v, out["o_tc"], do, out["lse_tc"], w.scale, w.causal, w.softcap, window=win,
        sinks=sinks)
    torch.cuda.synchronize()
    assert attn.attn_device_status(clear=True) == (0, 0)
    return {n: t.cpu() for n, t in out.items()}


def _check_forward(out, O, LSE, at=(slice(None),)):
    for impl in ("tc", "ref"):
        err = float(np.abs(out["lse_" + impl][at].double().numpy() - LSE).max())
        assert err <= lse_tol(LSE), "LSE %s %.3e" % (impl, err)
        assert rel_max(out["o_" + impl][at].double().numpy(), O) <= O_MAX_REL, impl


@pytest.mark.parametrize("w,win,sinks", CASES,
                         ids=lambda c: "%d-%d-%d" % (c.N, c.d, c.H) if hasattr(c, "N") else str(c))
def test_against_oracle(w, win, sinks):
    x = make_inputs(w)
    out = _run(w, win, sinks, x)
    f64 = {n: x[n].double().numpy() for n in ("q", "k", "v", "do")}
    args = (w.scale, w.causal, w.softcap)
    O, LSE = attention_forward(f64["q"], f64["k"], f64["v"], *args, window=win, sinks=sinks)
    _check_forward(out, O, LSE)
    grads = attention_backward(f64["q"], f64["k"], f64["v"], f64["do"], *args, window=win,
                               sinks=sinks)
    for name, g in zip(("dq", "dk", "dv"), grads):
        check_grad(name, out[name], g)


def test_no_sinks_is_the_local_call():
    """sinks = 0, and any sinks without a left bound: the same bits."""
    w = _w(1, 4, 2, 500, 128, True)
    dev = torch.device("cuda:0")
    x = make_inputs(w)
    q, k, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))
    shape = (w.B, w.H, w.H_kv, w.N, w.d, w.scale, True, 0.0)
    for left, sinks in ((70, 0), (-1, 9), (499, 9), (5000, 600)):
        o, lse = runner.forward(q, k, v, w.scale, True, window=(left, -1))
        dq, dk, dv = runner.backward(q, k, v, o, do, lse, w.scale, True, window=(left, -1))
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        attn.check(attn.attn_fwd_sinks(q, k, v, o2, lse2, *shape, left, -1, sinks))
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        _, dk2, dv2 = runner.backward(q, k, v, o, do, lse, w.scale, True, window=(left, -1),
                                      sinks=sinks)
        torch.cuda.synchronize()
        assert torch.equal(dk, dk2) and torch.equal(dv, dv2)


def test_counts_past_32_bits():
    """Every key a sink: the causal call's values, up to P's and O's roundings."""
    w = _w(1, 4, 2, 300, 64, True)
    x = make_inputs(w)
    f64 = {n: x[n].double().numpy() for n in ("q", "k", "v")}
    O, LSE = attention_forward(f64["q"], f64["k"], f64["v"], w.scale, True, 0.0)
    q, k, v = (x[n].cuda() for n in ("q", "k", "v"))
    for win, sinks in (((70, -1), 1 << 32), ((1 << 32, 1 << 33), 0), ((1 << 32, -1), 3)):
        out = {}
        for impl in ("tc", "ref"):
            out["o_" + impl], out["lse_" + impl] = runner.forward(
                q, k, v, w.scale, True, window=win, sinks=sinks, impl=impl)
        _check_forward({n: t.cpu() for n, t in out.items()}, O, LSE)


def test_captured_and_on_a_stream():
    """A captured step replayed on new inputs, and one on a side stream."""
    w = _w(2, 4, 2, 600, 64, True)
    dev = torch.device("cuda:0")
    x = make_inputs(w)
    q, k, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))

    def step(stream=None):
        o, lse = runner.forward(q, k, v, w.scale, True, window=(90, -1), sinks=6, stream=stream)
        return (o, lse) + tuple(runner.backward(q, k, v, o, do, lse, w.scale, True,
                                                window=(90, -1), sinks=6, stream=stream))[1:]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out[0], want[0])
    q.mul_(-1)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("w,left,sinks", [(_w(1, 8, 1, 1500, 128, True), 100, 4),
                                          (_w(2, 5, 1, 1111, 256, True), 50, 129)],
                         ids=["128", "256"])
def test_captured_with_clusters(w, left, sinks):
    """Both launches of the backward have ended where what follows them begins: a
    captured step, replayed over and over, gives the oracle's gradients."""
    dev = torch.device("cuda:0")
    x = make_inputs(w)
    q, k, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))
    kw = dict(window=(left, -1), sinks=sinks)
    o, lse = runner.forward(q, k, v, w.scale, True, **kw)
    runner.backward(q, k, v, o, do, lse, w.scale, True, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [runner.backward(q, k, v, o, do, lse, w.scale, True, **kw) for _ in range(2)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    f64 = {n: x[n].double().numpy() for n in ("q", "k", "v", "do")}
    grads = attention_backward(f64["q"], f64["k"], f64["v"], f64["do"], w.scale, True, 0.0,
                               window=(left, -1), sinks=sinks)
    for got in out:
        for name, t, g in zip(("dq", "dk", "dv"), got, grads):
            check_grad(name, t.cpu(), g)


def test_rotary_gradients():
    """The finalize step behind a backward with sinks takes the gradients back
    through the rotation."""
    w = _w(1, 4, 2, 300, 128, True)
    dev = torch.device("cuda:0")
    x = make_inputs(w)
    q0, k0, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))
    plan = runner.Rotary(128, dev)
    q, k = runner.rotary(q0, k0, plan)
    kw = dict(window=(40, -1), sinks=3)
    o, lse = runner.forward(q, k, v, w.scale, True, **kw)
    dq, dk, dv = runner.backward(q, k, v, o, do, lse, w.scale, True, rotary=plan, **kw)
    f64 = [t.double().cpu().numpy() for t in (q, k, v, do)]
    gq, gk, gv = attention_backward(*f64, w.scale, True, **kw)
    from oracle import rotate
    turns, p = plan.turns.tolist(), np.arange(w.N)[None]
    check_grad("dq", dq.cpu(), rotate(gq, turns, p, plan.magnitude, False, True))
    check_grad("dk", dk.cpu(), rotate(gk, turns, p, plan.magnitude, False, True))
    check_grad("dv", dv.cpu(), gv)


def test_causal_gqa_sampled():
    """The causal GQA shape under a window of 1024 keys and four sinks, on a
    seeded sample of (batch, KV head) slices."""
    w, win, sinks = WORKLOADS["causal_gqa"], (1023, -1), 4
    x = make_inputs(w)
    out = _run(w, win, sinks, x)
    for (b, g) in sample_slices(w, 2):
        heads = slice(g * w.G, (g + 1) * w.G)
        part = [x[n][b:b + 1, i].double().numpy()
                for n, i in (("q", heads), ("k", slice(g, g + 1)), ("v", slice(g, g + 1)),
                             ("do", heads))]
        O, LSE = attention_forward(*part[:3], w.scale, True, window=win, sinks=sinks)
        _check_forward(out, O[0], LSE[0], (b, heads))
        grads = attention_backward(*part, w.scale, True, window=win, sinks=sinks)
        check_grad("dq", out["dq"][b, heads], grads[0][0])
        check_grad("dk", out["dk"][b, g], grads[1][0, 0])
        check_grad("dv", out["dv"][b, g], grads[2][0, 0])
