"""The torch wrappers on a stream other than the current one.

Memory that a wrapper allocates has to come from the blocks of the stream that
writes it: a block that the current stream's allocator hands out may still be
read or written by work queued there. On the CPU the wrappers run with torch's
stream functions and the library's calls replaced, and every allocation is
checked for the stream that was current; on the GPU a block is dropped while
queued work still reads it."""
import contextlib

import pytest
import torch

from flashattention_attention_backward_gb300 import runner

BF, F4 = torch.bfloat16, torch.float32


class _Stream:
    def __init__(self, name, device="cpu"):
        self.name, self.cuda_stream, self.device = name, 64, torch.device(device)


@pytest.fixture
def fake(monkeypatch):
    """Records (stream current at an allocation), the stream of each library call
    and (tensor, stream) of each record_stream."""
    seen = {"made": [], "calls": [], "recorded": [], "tensors": []}
    streams = [_Stream("caller's")]

    @contextlib.contextmanager
    def on(stream):
        streams.append(stream)
        yield
        streams.pop()

    monkeypatch.setattr(torch.cuda, "Stream", _Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: streams[-1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    for name in ("empty", "empty_like"):
        def make(*args, _of=getattr(torch, name), **kwargs):
            t = _of(*args, **kwargs)
            seen["made"].append(streams[-1].name)
            seen["tensors"].append(t)
            return t
        monkeypatch.setattr(torch, name, make)
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: seen["recorded"].append((t.data_ptr(), s.name)))
    for name in [n for n in vars(runner) if n.startswith("attn_") and "bytes" not in n]:
        def call(*args):
            seen["calls"].append(args[-1].name)
            return 0
        monkeypatch.setattr(runner, name, call)
    monkeypatch.setattr(runner, "attn_bwd_dq_partials_bytes", lambda *a: 4096)
    monkeypatch.setattr(runner, "attn_layer_norm_bwd_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(runner, "_check_cuda", lambda device, **tensors: None)
    monkeypatch.setattr(runner, "_dims", lambda q, k, *others: (*q.shape[:2], k.shape[1],
                                                                 *q.shape[2:]))
    return seen


def _plan():
    plan = object.__new__(runner.Rotary)
    plan.rot, plan.interleaved, plan.magnitude = 64, False, 1.0
    plan.turns = torch.zeros(32, dtype=torch.int64)
    return plan


def _calls(dev, plan, N=8, C=64):
    """{name: call on a stream}: results of every wrapper that allocates."""
    g = torch.Generator().manual_seed(N)
    draw = lambda *s: torch.randn(*s, generator=g).to(BF).to(dev)  # noqa: E731
    q, o, do = (draw(1, 2, N, 64) for _ in range(3))
    k, v = draw(1, 1, N, 64), draw(1, 1, N, 64)
    lse = torch.zeros(1, 2, N, device=dev) + 5.0
    x, dy, w = draw(N, C), draw(N, C), torch.ones(C, device=dev)
    mean, rstd = torch.zeros(N, device=dev), torch.ones(N, device=dev)
    back = lambda s, **kw: runner.backward(q, k, v, o, do, lse, 0.125, True, stream=s,  # noqa: E731
                                           **kw)
    return {
        "forward": lambda s: runner.forward(q, k, v, 0.125, True, stream=s),
        "forward ref": lambda s: runner.forward(q, k, v, 0.125, True, stream=s, impl="ref"),
        "forward dropout": lambda s: runner.forward(q, k, v, 0.125, True, stream=s,
                                                    dropout=(0.1, 3)),
        "forward window": lambda s: runner.forward(q, k, v, 0.125, True, stream=s,
                                                   window=(4, -1)),
        "backward": back,
        "backward deterministic": lambda s: back(s, deterministic=True),
        "backward dropout": lambda s: back(s, dropout=(0.1, 3)),
        "backward window": lambda s: back(s, window=(4, -1)),
        "backward rotary": lambda s: back(s, rotary=plan),
        "backward deterministic rotary": lambda s: back(s, rotary=plan, deterministic=True),
        "rotary": lambda s: runner.rotary(q, k, plan, stream=s),
        "layer norm": lambda s: runner.layer_norm(x, w, w, stream=s),
        "layer norm backward": lambda s: runner.layer_norm_backward(dy, x, w, mean, rstd,
                                                                    stream=s),
        "dropout add": lambda s: (runner.dropout_add(x, dy, (0.1, 3), stream=s),),
        "dropout add norm": lambda s: runner.dropout_add_norm(x, dy, w, w, 1e-5, (0.1, 3),
                                                              stream=s),
        "dropout add norm backward": lambda s: runner.dropout_add_norm_backward(
            dy, x, x, w, mean, rstd, (0.1, 3), stream=s),
    }


NAMES = ["forward", "forward ref", "forward dropout", "forward window", "backward",
         "backward deterministic", "backward dropout", "backward window", "backward rotary",
         "backward deterministic rotary", "rotary", "layer norm", "layer norm backward",
         "dropout add", "dropout add norm", "dropout add norm backward"]


@pytest.mark.parametrize("name", NAMES)
def test_allocations_belong_to_the_stream_that_writes_them(fake, name):
    side = _Stream("side")
    got = _calls("cpu", _plan())[name](side)
    assert fake["calls"] and set(fake["calls"]) == {"side"}
    assert fake["made"] and set(fake["made"]) == {"side"}
    # the results may be used where the call was made
    assert {(t.data_ptr(), "caller's") for t in got} <= set(fake["recorded"])
    del fake["calls"][:], fake["made"][:], fake["recorded"][:]
    _calls("cpu", _plan())[name](None)
    assert set(fake["calls"]) == set(fake["made"]) == {"caller's"}


def test_buffers_belong_to_their_stream(fake):
    q = torch.zeros(1, 1, 8, 64, dtype=BF)
    runner.BackwardBuffers(q, q, _Stream("side"))
    assert set(fake["made"]) == {"side"}
    # the partials' buffer may be replaced while its last user runs
    bufs = runner.BackwardBuffers(q, q)
    lse = torch.zeros(1, 1, 8)
    runner.backward(q, q, q, q, q, lse, 0.1, True, bufs=bufs, deterministic=True,
                    stream=_Stream("third"))
    assert (bufs.dq_partials.data_ptr(), "third") in fake["recorded"]


def test_given_outputs_are_used_on_the_stream(fake):
    q = torch.zeros(1, 1, 8, 64, dtype=BF)
    out = (torch.zeros_like(q), torch.zeros_like(q))
    runner.rotary(q, q, _plan(), out=out, stream=_Stream("side"))
    assert {(t.data_ptr(), "side") for t in out} <= set(fake["recorded"])


def test_a_stream_of_another_device_is_refused(fake):
    for name, call in _calls("cpu", _plan()).items():
        with pytest.raises(ValueError, match="stream is on"):
            call(_Stream("side", "cuda:1"))
        assert not fake["calls"], name


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_results_beside_queued_work(name):
    """Queued work on the current stream reads blocks that are already dropped,
    of every size that the call allocates; the call on another stream neither
    gets them nor writes them."""
    dev = torch.device("cuda:0")
    call = _calls(dev, runner.Rotary(64, dev), N=512, C=1024)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    sizes = sorted({t.numel() * t.element_size() for t in want} |
                   {2 * 512 * 4, 2 * 512 * 64 * 4, attn_workspace(512, 1024)})
    blocks = [torch.full((n,), 1, dtype=torch.uint8, device=dev) for n in sizes for _ in range(3)]
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)  # about 50 ms
    sums = [b.double().sum() for b in blocks]
    places = {b.data_ptr() for b in blocks}
    total = [b.numel() for b in blocks]
    del blocks
    got = call(side)
    side.synchronize()  # the call has written while the sums still wait
    assert not places & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert [int(s) for s in sums] == total
    for a, b in zip(got, want):
        if name.startswith("backward") and "deterministic" not in name:
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -6, atol=2 ** -10)
        else:
            assert torch.equal(a, b)


def attn_workspace(rows, C):
    from flashattention_attention_backward_gb300 import attn_layer_norm_bwd_workspace_bytes
    return attn_layer_norm_bwd_workspace_bytes(rows, C)


@pytest.mark.gpu
def test_stream_handles():
    """A handle, an object with a handle and the default stream's handle 0."""
    dev = torch.device("cuda:0")
    x = torch.randn(64, 256, device=dev)
    want = runner.layer_norm(x)[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    class Handle:
        cuda_stream = side.cuda_stream

    for stream in (side, side.cuda_stream, Handle(), 0, torch.cuda.default_stream()):
        y = runner.layer_norm(x, stream=stream)[0]
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_captured_on_a_joined_stream():
    """A call on another stream inside a capture that forks to it and joins it
    again; its memory belongs to the graph, and replays follow new contents."""
    dev = torch.device("cuda:0")
    x, dy = (torch.randn(300, 1024, device=dev).to(BF) for _ in range(2))
    w = torch.ones(1024, device=dev)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    runner.layer_norm_backward(dy, x, w, *runner.layer_norm(x, w, w)[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=main):
        t = runner.dropout_add(x, dy)
        side.wait_stream(main)
        y, mean, rstd = runner.layer_norm(t, w, w, stream=side)
        dx, dgamma, dbeta = runner.layer_norm_backward(dy, t, w, mean, rstd, stream=side)
        main.wait_stream(side)
        out = runner.dropout_add(dx, y)
        # dropped inside the capture, used again by what follows it
        del t, dx
        last = runner.dropout_add(out, y)
    for scale in (1.0, 0.5):
        x.mul_(scale)
        graph.replay()
        torch.cuda.synchronize()
        t2 = runner.dropout_add(x, dy)
        y2, m2, r2 = runner.layer_norm(t2, w, w)
        dx2, dg2, db2 = runner.layer_norm_backward(dy, t2, w, m2, r2)
        out2 = runner.dropout_add(dx2, y2)
        for a, b in ((y, y2), (dgamma, dg2), (dbeta, db2), (out, out2),
                     (last, runner.dropout_add(out2, y2))):
            assert torch.equal(a, b)
