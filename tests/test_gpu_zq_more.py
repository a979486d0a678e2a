"""More refusals of the calls on activations kept in 8 bits."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev

pytestmark = pytest.mark.gpu


def _wgrad_arguments():
    T, K, E, d, I = 40, 2, 4, 128, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    idx = torch.rand((T, E), generator=g, device="cuda").topk(K, 1).indices.int()
    _, go, row_token, slot_row = moe.moe_dispatch(idx, E, include_shared=True)
    R = T * K + T
    z_q, z_scale = moe.fp8_quant_1x128(rand(R, 2 * I))
    return dict(dh=rand(T, d), topk_gate=rand(T, K), slot_row=slot_row, row_token=row_token, z_q=z_q, z_scale=z_scale,
                dh_row=rand(R, I), u=rand(T, d).bfloat16(), group_offset=go, shared_row0=T * K)


def test_weight_gradients_refuse_another_device(monkeypatch):
    """Tensors of a GPU that is not the current one, as the other calls have it: nothing is launched."""
    dev()
    args = _wgrad_arguments()
    moe.moe_wgrad_zq(**args)
    torch.cuda.synchronize()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1 + args["z_q"].get_device())
        with pytest.raises(moe.MoEError, match="expected the current GPU"):
            moe.moe_wgrad_zq(**args)


@pytest.mark.parametrize("name", ["dh", "topk_gate", "slot_row", "row_token", "z_q", "z_scale", "dh_row", "u", "group_offset"])
def test_weight_gradients_refuse(name):
    """Every tensor on the host, of another type, with another number of dimensions, and of a size less."""
    dev()
    args = _wgrad_arguments()
    t = args[name]
    bad = [t.cpu(), t.double(), t.unsqueeze(0), t.reshape(-1) if t.dim() == 2 else t[None]]
    if name != "group_offset":              # its size says how many groups there are
        bad.append(t[:-1])
    for i, b in enumerate(bad):
        with pytest.raises(moe.MoEError):
            moe.moe_wgrad_zq(**{**args, name: b})
            pytest.fail(f"{name}, case {i} was taken")
