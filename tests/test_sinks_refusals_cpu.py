"""What the torch wrappers refuse of sinks, through the calls themselves (these checks
come before those of the tensors, so no GPU is needed)."""
import pytest
import torch

from flashattention_attention_backward_gb300 import runner


def _backward(**kw):
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    return runner.backward(t, t, t, t, t, torch.zeros(1, 2, 8), 0.125, True, **kw)


def _forward(**kw):
    t = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    return runner.forward(t, t, t, 0.125, True, **kw)


@pytest.mark.parametrize("call,kw,what", [
    (_backward, dict(sinks=1, deterministic=True), "sinks have no deterministic"),
    (_backward, dict(sinks=1, window=(4, -1), deterministic=True), "sinks have no deterministic"),
    (_backward, dict(sinks=1, dropout=(0.1, 3)), "sinks have no dropout"),
    (_forward, dict(sinks=1, dropout=(0.1, 3)), "sinks have no dropout"),
    (_backward, dict(sinks=-1), "negative"),
    (_forward, dict(sinks=-1), "negative"),
])
def test_refusals(call, kw, what):
    with pytest.raises(ValueError, match=what):
        call(**kw)
