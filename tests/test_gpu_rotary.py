"""attn_rotary and attn_bwd_finalize_rotary against the 64-bit oracle.

Tolerance, per element, with u = 2^-24 (half an fp32 step): the reduced angle
is off by at most 3 u of itself (conversion, constant, product; at most
pi / 4) and 2^-32 turn, the Taylor sum of cosine and sine by 2 u: 5 u in all;
the factor m adds a rounding each (6 u), the two products and their sum three
more of |a| + |b|: 9 u (|a| + |b|) m, and the finalize step's scale one more.
12 u covers both. Rounding the output to its type adds half a step of it, or
half the smallest subnormal.
"""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from oracle import rotate

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def _close(got, x, plan, positions, adjoint=False, scale=1.0):
    """got against the oracle's rotation of x (both [B, heads, N, d])."""
    assert not torch.isnan(got).any()
    x64 = x.double().cpu().numpy() * scale
    p = positions.cpu().numpy()
    t = [int(v) for v in plan.turns.tolist()][:plan.rot // 2]
    want = rotate(x64, t, p, plan.magnitude, plan.interleaved, adjoint)
    half = plan.rot // 2
    ia = np.arange(half) * 2 if plan.interleaved else np.arange(half)
    ib = ia + (1 if plan.interleaved else half)
    size = np.abs(x64) * (U / 8 if scale == 1.0 else U)
    pair = (np.abs(x64[..., ia]) + np.abs(x64[..., ib])) * plan.magnitude * 12 * U
    size[..., ia], size[..., ib] = pair, pair
    tol = size + np.abs(want) * (torch.finfo(got.dtype).eps / 2 * (1 + 1e-6)) + TINY[got.dtype]
    err = np.abs(got.double().cpu().numpy() - want)
    worst = np.unravel_index((err - tol).argmax(), err.shape)
    assert (err <= tol).all(), "%s: error %.3e, allowed %.3e" % (worst, err[worst], tol[worst])


def _positions(kind, B, N, dev, seed):
    if kind == "rows":
        return None, torch.arange(N)[None].repeat(B, 1)
    g = torch.Generator().manual_seed(seed)
    if kind == "shared":
        p = torch.randint(0, 4096, (N,), generator=g)
        return p.to(dev), p[None].repeat(B, 1)
    far = {"each": 131072, "far": 1 << 45}[kind]
    p = torch.randint(-far if kind == "far" else 0, far, (B, N), generator=g)
    return p.to(dev), p


CASES = [
    # B, H, H_kv, N, d, rot, interleaved, dtype, positions
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, "rows"),
    (3, 32, 8, 1, 128, 128, False, torch.bfloat16, "far"),
    (2, 4, 2, 67, 128, 128, True, torch.bfloat16, "each"),
    (2, 5, 3, 129, 64, 32, True, torch.float16, "shared"),
    (1, 2, 1, 33, 256, 64, False, torch.float32, "each"),
    (2, 3, 3, 31, 256, 256, True, torch.float32, "rows"),
    (1, 8, 0, 70, 128, 64, False, torch.bfloat16, "rows"),
    (1, 3, 2, 19, 80, 48, False, torch.float16, "rows"),   # groups of 16 bytes, odd number
    (1, 3, 2, 19, 72, 24, False, torch.bfloat16, "rows"),  # rot / 2 is no multiple of 8
    (1, 3, 2, 19, 72, 24, True, torch.bfloat16, "rows"),
    (2, 3, 1, 21, 36, 12, True, torch.float16, "far"),     # rows are no multiple of 16 bytes
    (2, 3, 1, 21, 33, 30, False, torch.bfloat16, "each"),  # odd d
    (1, 2, 2, 7, 2, 2, True, torch.float32, "rows"),
    (1, 2, 2, 7, 1, 0, False, torch.bfloat16, "rows"),     # a copy
    (1, 40, 4, 300, 64, 64, False, torch.bfloat16, "rows"),
]


@pytest.mark.parametrize("adjoint", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_rotary(case, adjoint):
    B, H, H_kv, N, d, rot, interleaved, dtype, kind = case
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(hash(case[:6]) & 0xFFFF)
    q = torch.randn(B, H, N, d, generator=g).to(dtype).to(dev)
    k = torch.randn(B, H_kv, N, d, generator=g).to(dtype).to(dev) if H_kv else None
    plan = runner.Rotary(rot, dev, scaling="ramp", factor=4.0, original_length=4096,
                         interleaved=interleaved)
    p, p_all = _positions(kind, B, N, dev, 5)
    qo, ko = runner.rotary(q, k, plan, p, adjoint=adjoint)
    _close(qo, q, plan, p_all, adjoint)
    if H_kv:
        _close(ko, k, plan, p_all, adjoint)
    # in place
    q2, k2 = q.clone(), None if k is None else k.clone()
    runner.rotary(q2, k2, plan, p, adjoint=adjoint, out=(q2, k2))
    assert torch.equal(q2, qo) and (k is None or torch.equal(k2, ko))


@pytest.mark.parametrize("dtype,d,rot", [(torch.bfloat16, 128, 128), (torch.float16, 40, 8),
                                         (torch.float32, 20, 12)])
def test_rotary_packed(dtype, d, rot):
    """q and k inside a packed projection, outputs inside another whose other
    columns stay as they are."""
    B, N, H, H_kv = 2, 37, 6, 2
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(11)
    qkv = torch.randn(B, N, H + 2 * H_kv, d, generator=g).to(dtype).to(dev)
    # rows of the output packing are longer than what is written
    out = torch.full((B, N, H + 2 * H_kv + 1, d + 8), 7.0, dtype=dtype, device=dev)
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + H_kv].transpose(1, 2)
    qo = out[:, :, :H, :d].transpose(1, 2)
    ko = out[:, :, H:H + H_kv, :d].transpose(1, 2)
    plan = runner.Rotary(rot, dev)
    before = qkv.clone()
    runner.rotary(q, k, plan, out=(qo, ko))
    assert torch.equal(before, qkv)
    p = torch.arange(N)[None].repeat(B, 1)
    _close(qo, q, plan, p)
    _close(ko, k, plan, p)
    assert (out[:, :, H + H_kv:] == 7).all() and (out[..., d:] == 7).all()


def test_rotary_far_strides():
    """Element offsets past 2^32: the last batch lies 5e9 elements behind the first."""
    dev = torch.device("cuda:0")
    step = 5_000_000_000 // 16 * 16
    buf = torch.empty(step + 4096, dtype=torch.bfloat16, device=dev)
    x = torch.as_strided(buf, (2, 2, 3, 64), (step, 192, 64, 1))
    x.copy_(torch.randn(2, 2, 3, 64, generator=torch.Generator().manual_seed(2)))
    plan = runner.Rotary(64, dev)
    y, _ = runner.rotary(x, None, plan)
    _close(y, x.contiguous(), plan, torch.arange(3)[None].repeat(2, 1))
    back, _ = runner.rotary(y, None, plan, adjoint=True, out=(x, None))
    _close(x.contiguous(), y, plan, torch.arange(3)[None].repeat(2, 1), adjoint=True)


def test_rotary_keeps_infinities_in_their_pair():
    dev = torch.device("cuda:0")
    x = torch.ones(1, 1, 5, 64, device=dev)
    x[0, 0, 2, 3] = float("inf")
    x[0, 0, 3, 50] = float("nan")
    y, _ = runner.rotary(x, None, runner.Rotary(32, dev))
    bad = (~torch.isfinite(y)).nonzero().tolist()
    assert bad == [[0, 0, 2, 3], [0, 0, 2, 19], [0, 0, 3, 50]]


FINALIZE = [
    # B, H, H_kv, N, d, rot, interleaved, positions, packed
    (1, 2, 2, 256, 64, 64, False, "rows", False),
    (2, 8, 2, 131, 128, 128, True, "each", True),
    (1, 3, 1, 65, 256, 64, False, "shared", True),
    (1, 4, 0, 1, 128, 128, False, "far", False),
    (2, 2, 1, 9, 36, 20, False, "rows", False),
    (1, 1, 1, 5, 7, 4, True, "rows", False),
]


@pytest.mark.parametrize("case", FINALIZE, ids=lambda c: "-".join(map(str, c)))
def test_finalize_rotary(case):
    B, H, H_kv, N, d, rot, interleaved, kind, packed = case
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(17)
    acc = (10 * torch.randn(B, H, N, d, generator=g)).to(dev)
    dk = torch.randn(B, H_kv, N, d, generator=g).bfloat16().to(dev)
    plan = runner.Rotary(rot, dev, scaling="ramp", factor=8.0, original_length=2048,
                         interleaved=interleaved)
    p, p_all = _positions(kind, B, N, dev, 6)
    scale = d ** -0.5
    if packed:
        whole = torch.full((B, N, H + 2 * H_kv, d), 7.0, dtype=torch.bfloat16, device=dev)
        dq, dko = whole[:, :, :H].transpose(1, 2), whole[:, :, H:H + H_kv].transpose(1, 2)
        strides = list(dq.stride()[:3]) + list(dko.stride()[:3])
    else:
        dq, dko, strides = torch.empty_like(acc, dtype=torch.bfloat16), dk.clone(), None
    ps = 0 if p is None or p.dim() == 1 else p.stride(0)
    attn.check(attn.attn_bwd_finalize_rotary(
        acc, dq, dk if packed else dko, dko, scale, plan.turns, p, ps, B, H, H_kv, N, d, rot,
        plan.magnitude, interleaved, strides, torch.cuda.current_stream()))
    s32 = float(np.float32(scale))
    _close(dq, acc, plan, p_all, True, s32)
    if H_kv:
        _close(dko, dk, plan, p_all, True)
    if packed:
        assert (whole[:, :, H + H_kv:] == 7).all()


def test_rotary_streams_and_graph():
    """Two streams at once, and a captured call replayed on new contents."""
    dev = torch.device("cuda:0")
    plan = runner.Rotary(128, dev)
    xs = [torch.randn(2, 8, 256, 128, device=dev).bfloat16() for _ in range(2)]
    want = [runner.rotary(x, None, plan)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [runner.rotary(x, None, plan, stream=s)[0] for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x, y = xs[0].clone(), torch.empty_like(xs[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        runner.rotary(x, None, plan, out=(y, None))
    x.copy_(xs[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want[1])


def test_empty():
    dev = torch.device("cuda:0")
    plan = runner.Rotary(64, dev)
    q, k = runner.rotary(torch.empty(2, 4, 0, 64, device=dev), torch.empty(2, 1, 0, 64, device=dev),
                         plan)
    assert q.shape == (2, 4, 0, 64) and k.shape == (2, 1, 0, 64)
