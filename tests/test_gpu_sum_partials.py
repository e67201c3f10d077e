"""attn_bwd_sum_partials, and the deterministic backward of rotated inputs: dQ
rounded once."""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from flashattention_attention_backward_gb300.inputs import Workload, make_inputs
from oracle import rotate

FAKE = 0x10000  # a 16-byte aligned non-null address; never dereferenced
U = 2.0 ** -24


def test_refusals():
    from flashattention_attention_backward_gb300.build import build
    build()

    def call(part=FAKE, out=FAKE, B=1, H=2, N=64, d=64):
        return attn.attn_bwd_sum_partials(part, out, B, H, N, d, True)

    assert call(part=0) == call(out=0) == attn.ATTN_ERR_NULL
    assert call(part=FAKE + 8) == call(out=FAKE + 4) == attn.ATTN_ERR_ALIGN
    assert call(B=-1) == call(N=-1) == attn.ATTN_ERR_SHAPE
    assert call(d=96) == attn.ATTN_ERR_UNSUPPORTED
    assert call(B=0) == attn.ATTN_OK


def _summed(partials, B, H, N, d, causal):
    """(sum, sum of magnitudes) [B, H, N, d] of the stored tiles, in 64 bits."""
    M = (N + 127) // 128
    P = M * (M + 1) // 2 if causal else M * M
    t = partials[:B * H * P * 128 * d].double().cpu().numpy().reshape(B, H, P, 128, d)
    out, size = np.zeros((B, H, M * 128, d)), np.zeros((B, H, M * 128, d))
    for m in range(M):
        for n in range(m + 1 if causal else M):
            tile = t[:, :, m * (m + 1) // 2 + n if causal else m * M + n]
            out[:, :, m * 128:(m + 1) * 128] += tile
            size[:, :, m * 128:(m + 1) * 128] += np.abs(tile)
    return out[:, :, :N], size[:, :, :N]


@pytest.mark.gpu
@pytest.mark.parametrize("d,N,causal,interleaved", [
    (64, 200, True, True), (128, 300, True, False), (64, 257, False, False), (256, 130, True, True)])
def test_deterministic_dq_is_rounded_once(d, N, causal, interleaved):
    """dQ against the 64-bit rotation of the call's own partial tiles. A sum over
    M key blocks is off by M u of its terms' magnitudes, the scale and the rotation
    by 12 u (|a| + |b|) as in attn_rotary's tests, and the result is rounded to
    bf16 once: half a step."""
    dev = torch.device("cuda:0")
    w = Workload("sum", 2, 4, 2, N, d, causal, seed_base=57)
    x = make_inputs(w)
    q, k, v, do = (x[n].to(dev) for n in ("q", "k", "v", "do"))
    plan = runner.Rotary(d // 2, dev, interleaved=interleaved)
    q, k = runner.rotary(q, k, plan)
    o, lse = runner.forward(q, k, v, w.scale, causal)
    bufs = runner.BackwardBuffers(q, k)
    dq, dk, dv = (t.clone() for t in runner.backward(
        q, k, v, o, do, lse, w.scale, causal, bufs=bufs, deterministic=True, rotary=plan))
    total, size = _summed(bufs.dq_partials, w.B, w.H, N, d, causal)
    M = (N + 127) // 128
    s = float(np.float32(w.scale))
    turns, pos = plan.turns.tolist(), np.broadcast_to(np.arange(N), (w.B, N))
    want = rotate(total * s, turns, pos, 1.0, interleaved, adjoint=True)
    half = plan.rot // 2
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + (1 if interleaved else half)
    tol = (M + 1) * U * size * s
    pair = 12 * U * (np.abs(total[..., ia]) + np.abs(total[..., ib])) * s + \
        tol[..., ia] + tol[..., ib]
    tol[..., ia], tol[..., ib] = pair, pair
    tol = tol + np.abs(want) * 2.0 ** -8 * (1 + 1e-6) + 2.0 ** -134
    err = np.abs(dq.double().cpu().numpy() - want)
    assert (err <= tol).all(), (err / tol).max()
    # the same bits again, in buffers of its own; dV as without the rotary
    again = runner.backward(q, k, v, o, do, lse, w.scale, causal, deterministic=True, rotary=plan)
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dv)))
    plain = runner.backward(q, k, v, o, do, lse, w.scale, causal, deterministic=True)
    assert torch.equal(plain[2], dv)
    # the sum in 32 bits, rounded, is what attn_bwd_finalize_partials gives
    acc = torch.empty((w.B, w.H, N, d), device=dev)
    stream = torch.cuda.current_stream()
    attn.check(attn.attn_bwd_sum_partials(bufs.dq_partials, acc, w.B, w.H, N, d, causal, stream))
    assert torch.equal((acc * w.scale).bfloat16(), plain[0])
