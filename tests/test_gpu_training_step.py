"""The training step of examples/training_step.py: its gradients against 64 bits without
quantisation, what the balance loss adds to them, and the step in a graph."""
import os
import sys

import pytest
import torch

from helpers import dev, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import training_step as ts  # noqa: E402

pytestmark = pytest.mark.gpu
F8 = torch.float64
U = 2.0 ** -24


@pytest.mark.parametrize("T,d,E,K,I", [(384, 512, 16, 4, 256), (130, 256, 8, 2, 128), (9, 128, 4, 1, 256)])
def test_gradients(T, d, E, K, I):
    """E4M3 rounds by 2.5% on the average (2^-4 at most), and a path from dout to a gradient takes up to eight
    such operands (dY, W2, z, dz, W13, and u, h or W again): 8% of independent roundings, doubled for what
    SwiGLU's factors make of z's, and half as much again for sums of few terms."""
    dev()
    say(f"  T={T} d={d} E={E} K={K} I={I}")
    block = ts.Block(T, d, E, K, I)
    r = block.forward()
    g = block.backward(r)
    torch.cuda.synchronize()
    ref = block.reference(r["idx"])
    for k, want in ref.items():
        got = (r["out"] if k == "out" else g[k]).to(F8)
        rel = float((got - want).norm() / want.norm())
        say(f"  {k}: {rel:.3f}")
        assert rel < (0.05 if k == "out" else 0.25), (k, rel)


def test_the_balance_loss_in_the_gradients():
    """With its weight a thousand times larger the balance loss moves du and de by its own gradient's products,
    which FP32 gives to 768 terms' roundings; padding's logits get nothing."""
    dev()
    block = ts.Block(384, 512, 16, 4, 256)
    r = block.forward()
    with_loss = block.backward(r)
    alpha = ts.ALPHA
    try:
        ts.ALPHA = 0.0
        without = block.backward(r)
    finally:
        ts.ALPHA = alpha
    torch.cuda.synchronize()
    assert (without["dlogits"] == 0).all() and (with_loss["dlogits"][int(block.starts[-1]):] == 0).all()
    dl, u, e = with_loss["dlogits"].to(F8), r["norm"].y.to(F8), block.centroids.to(F8)
    for got, base, a, b in ((with_loss["du"], without["du"], dl, e),
                            (with_loss["centroids"], without["centroids"], dl.t().contiguous(), u)):
        want = base.to(F8) + a @ b
        size = base.to(F8).abs() + a.abs() @ b.abs()
        assert ((got.to(F8) - want).abs() <= (3 * a.shape[1] + 2) * U * size).all()
    assert (with_loss["centroids"] != without["centroids"]).any()
    # the counts are the choice's own, over the tokens of sequences
    last = int(block.starts[-1])
    assert torch.equal(r["balance"].expert_count, torch.bincount(r["idx"][:last].reshape(-1).long(), minlength=16).int())


def test_step_is_repeatable_and_runs_in_a_graph():
    dev()
    block = ts.Block(200, 256, 8, 2, 128)
    names = ("x", "weight", "shift", "centroids", "w13", "w2")

    def run():
        r = block.forward()
        g = block.backward(r)
        return [r["out"], *r["balance"]] + [g[k] for k in names]

    want = run()
    again = run()
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    for i in range(3):
        block.x.mul_(-0.9)
        block.dout.mul_(1.1)
        graph.replay()
        torch.cuda.synchronize()
        eager = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_bias_update_takes_the_counts():
    dev()
    block = ts.Block(130, 256, 8, 2, 128)
    before = block.bias.clone()
    r, _ = block.step()
    torch.cuda.synchronize()
    c = r["balance"].expert_count.long() * 8
    total = int(block.starts[-1]) * 2
    assert int(r["balance"].expert_count.sum()) == total
    assert torch.equal(block.bias, before + torch.where(c > total, -ts.GAMMA, torch.where(c < total, ts.GAMMA, 0.0)).float())


def test_runs_at_other_sizes():
    dev()
    block = ts.Block(640, 1024, 32, 8, 512)
    r, g = block.step()
    torch.cuda.synchronize()
    assert all(torch.isfinite(t).all() for t in (r["out"], *g.values()))


def test_two_steps_at_once():
    """Forward and backward on two streams at the same time, each with its own scratch: one after the other's bits."""
    dev()
    blocks = [ts.Block(1500, 512, 16, 4, 256, seed=s) for s in (1, 2)]

    def run(block):
        r = block.forward()
        g = block.backward(r)
        return [r["out"], r["zq"], r["zs"], *r["balance"], *(g[k] for k in sorted(g))]

    want = [run(b) for b in blocks]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(4):
        got = [None, None]
        for k in (0, 1):
            with torch.cuda.stream(streams[k]):
                got[k] = run(blocks[k])
        torch.cuda.synchronize()
        for k in (0, 1):
            assert all(torch.equal(a, b) for a, b in zip(got[k], want[k])), (i, k)
