"""Layer norm at every kind of row that its kernels tell apart (lanes or warps a
row, odd lengths, rows over two blocks, rows read again), held to the depth of
their own sums."""
import numpy as np
import pytest
import torch

from flashattention_attention_backward_gb300 import runner

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF, HF, F4 = torch.bfloat16, torch.float16, torch.float32

# for many of these n, n times the fp32 value of 1 / n is not 1
LENGTHS = [1, 2, 3, 41, 47, 61, 64, 82, 83, 97, 107, 123, 128, 200, 333, 520, 1001, 1021, 1536,
           2047, 2104, 3001, 4093, 4095, 4096, 5000, 6015, 8191, 8192, 8195, 9001, 12287, 16370,
           16383, 16384, 20001]


@pytest.mark.parametrize("dtype", [BF, HF, F4])
@pytest.mark.parametrize("C", LENGTHS)
def test_equal_values(C, dtype):
    """Rows of one value v each. v has at most 8 significant bits and C at most
    15, so every sum of copies of v and its product with a count are exact in 24
    bits; the mean, a quotient rounded once, is v, every difference is 0 and y is
    beta to the last bit."""
    v = torch.tensor([5.0, -1000.0, 0.0703125, 13.25, -255.0, 3.984375], device=DEV).to(dtype)
    x = v[:, None].expand(-1, C).contiguous()
    g = torch.Generator().manual_seed(C)
    gamma = torch.randn(C, generator=g).to(dtype).to(DEV)
    beta = torch.randn(C, generator=g).to(dtype).to(DEV)
    y, mean, rstd = runner.layer_norm(x, gamma, beta, 1e-5)
    assert torch.equal(mean, v.float())
    assert torch.equal(y, beta.expand_as(y))
    # 1 / sqrt(eps) of the fp32 eps: rsqrtf is off by at most 2 units in the last
    # place, 2^-23 of the value each at most
    want = 1 / np.sqrt(float(np.float32(1e-5)))
    assert (np.abs(rstd.double().cpu().numpy() - want) <= 2 * 2.0 ** -23 * want).all()
    # a sum with a residual: 4 more bits
    half = (v * 0.5).to(dtype)[:, None].expand(-1, C).contiguous()
    z, y, mean, _ = runner.dropout_add_norm(half, half, gamma, beta, 1e-5)
    assert torch.equal(z, x) and torch.equal(mean, v.float())
    assert torch.equal(y, beta.expand_as(y))
