"""Further cases of the residual + RMS norm and its backward on the GPU."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(256, 2048), (128, 999), (64, 1032), (1024, 128), (1024, 1000), (512, 333), (2, 7168)])
def test_dw_is_added_up_pairwise(T, d):
    """Equal rows, as many as a power of two and one to a block or wave: sums in pairs only double them, so
    dw is exact, whatever the bits of a row.  (Added one after the other, 3 times a value already rounds.)"""
    dev()
    say(f"  T={T} d={d}")
    g = torch.Generator(device="cuda")
    g.manual_seed(d)
    row = torch.randn(d, generator=g, device="cuda")
    h, one = row.expand(T, d).contiguous(), torch.ones((T, d), device="cuda")
    _, dw = moe.moe_add_rmsnorm_backward(one, h, one[0], torch.ones(T, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(dw, row * T)
