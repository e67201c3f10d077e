"""Calls over a paged cache as a server makes them: on side streams, with keys and
values of one tensor, replayed while the batch changes its shape."""
import numpy as np
import pytest
import torch

import flashattention_attention_backward_gb300 as attn
from flashattention_attention_backward_gb300 import runner
from test_gpu_cache import BF, HF, Case

pytestmark = pytest.mark.gpu


def test_append_on_side_streams():
    """Append and attention of two batches on two side streams at once: the bits of the
    calls on the current one."""
    cases = [Case([(1, 700), (40, 300), (0, 9)], 8, 2, 128, 16, BF, seed=s) for s in (1, 2)]
    plan = runner.Rotary(128, "cuda:0")
    want = []
    for c in cases:
        caches = [t.clone() for t in c.caches]
        q = runner.cache_append(c.q, c.k, c.v, *caches, *c.batch()[2:], plan)
        want.append((q, *caches, *runner.cache_attention(q, *caches, *c.batch()[2:], 0.1)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                caches = [t.clone() for t in c.caches]
            q = runner.cache_append(c.q, c.k, c.v, *caches, *c.batch()[2:], plan, stream=s)
            got.append((q, *caches,
                        *runner.cache_attention(q, *caches, *c.batch()[2:], 0.1, stream=s)))
    torch.cuda.synchronize()
    assert attn.attn_device_status(clear=True) == (0, 0)
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i % 2])), i


@pytest.mark.parametrize("d,dtype", [(64, HF), (256, BF)])
def test_keys_and_values_of_one_tensor(d, dtype):
    """Each page holds its keys, then its values."""
    c = Case([(3, 150), (1, 700), (60, 60)], 4, 2, d, 32, dtype)
    plan = runner.Rotary(d, "cuda:0")
    both = torch.stack(c.caches, 1)  # [pages, 2, page, heads, d]
    caches = both[:, 0], both[:, 1]
    q = runner.cache_append(c.q, c.k, c.v, *c.batch(), plan)
    q2 = runner.cache_append(c.q, c.k, c.v, *caches, *c.batch()[2:], plan)
    assert torch.equal(q, q2) and all(torch.equal(a, b) for a, b in zip(caches, c.caches))
    o, lse = c.attend(q=q)
    o2, lse2 = runner.cache_attention(q, *caches, *c.batch()[2:], d ** -0.5)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    c.check(o, lse, q=q)


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_replayed_with_other_starts(softcap):
    """A captured step replayed with the batch's rows given to its sequences in other
    ways, some of them to none: those keep what they held."""
    T, H, H_kv, d, page = 64, 4, 2, 64, 16
    splits = [(64, 0, 0), (1, 1, 1), (0, 50, 3), (20, 20, 24), (0, 0, 0)]
    c = Case([(T, 900), (0, 500), (0, 900)], H, H_kv, d, page, BF)
    plan = runner.Rotary(d, "cuda:0")
    ws = torch.empty(attn.attn_cache_fwd_workspace_bytes(T, 3, H, H_kv, d), dtype=torch.uint8,
                     device="cuda")
    caches = [t.clone() for t in c.caches]
    q, out = torch.empty_like(c.q), (torch.empty(T, H, d, dtype=BF, device="cuda"),
                                     torch.empty(T, H, device="cuda"))

    def step():
        runner.cache_append(c.q, c.k, c.v, *caches, c.pages_d, c.starts_d, c.lengths_d, plan,
                            out=q)
        runner.cache_attention(q, *caches, c.pages_d, c.starts_d, c.lengths_d, 0.125,
                               softcap=softcap, out=out, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i, split in enumerate(splits):
        c.starts = np.cumsum([0] + list(split)).astype(np.int32)
        c.lengths = np.array([900, 500, 900 - i], dtype=np.int32)
        c.starts_d.copy_(torch.from_numpy(c.starts))
        c.lengths_d.copy_(torch.from_numpy(c.lengths))
        for t in (q, *out):
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        end = int(c.starts[-1])
        for t in (q, *out):
            assert (t[end:] == 7).all()
        c.caches = caches
        if end:
            c.check(*out, q=q, scale=0.125, softcap=softcap)
