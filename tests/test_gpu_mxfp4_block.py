"""The MXFP4 expert block of examples/mxfp4_block.py, stage by stage against 64
bits on the codes that the stage before it gave, and end to end against the block
without quantisation."""
import os
import sys

import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import mxfp4_block as block  # noqa: E402

pytestmark = pytest.mark.gpu
F8 = torch.float64


@pytest.mark.parametrize("T,d,E,K,I", [(1, 512, 16, 4, 256), (130, 512, 16, 4, 256), (700, 1024, 8, 2, 512)])
def test_block(T, d, E, K, I):
    dev()
    say(f"  T={T} d={d} E={E} K={K} I={I}")
    x, stream, weight, centroids, bias, ex, masters = block.make(T, d, E, K, I)
    r = block.forward(x, stream, weight, centroids, bias, K, ex)
    torch.cuda.synchronize()
    n, off, rows = r["norm"], r["offset"].tolist(), r["row_token"].long()
    val = lambda q, s: moe.mxfp4_dequant_1x32(q, s, dtype=torch.float32).to(F8)  # noqa: E731
    # h: the exact product of the codes, then SwiGLU, then MXFP4: within half of the widest step (1 of 4, at 4
    # to 6) of each value, or of half of the smallest value's step
    u, h = val(r["uq"], r["us"]), val(r["hq"], r["hs"])
    want = torch.empty_like(h)
    for g in range(E + 1):
        a, b = off[g], off[g + 1]
        if a == b:
            continue
        c = (u[rows[a:b]] @ val(ex.w13[g], ex.s13[g]).t()).view(b - a, I // 128, 2, 128)
        want[a:b] = (torch.nn.functional.silu(c[:, :, 0]) * c[:, :, 1]).reshape(b - a, I)
    step = torch.exp2(r["hs"].to(F8) - 127).repeat_interleave(32, 1)
    near = want.abs() / step
    half = torch.where(near < 2, 0.25, torch.where(near < 4, 0.5, 1.0)) + torch.where(near > 6, near - 6, 0.0)
    assert ((h - want).abs() <= (half * (1 + 1e-5) + 1e-5) * step).all()
    # y: bf16 of the exact product of h's codes; K terms of binary32 before it
    y = torch.cat([h[a:b] @ val(ex.w2[g], ex.s2[g]).t() for g, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    size = torch.cat([h[a:b].abs() @ val(ex.w2[g], ex.s2[g]).abs().t() for g, (a, b) in enumerate(zip(off[:-1], off[1:]))])
    assert ((r["y"].to(F8) - y).abs() <= 2.0 ** -8 * y.abs() + I * 2.0 ** -24 * size).all()
    # the combine adds the norm's h
    out = n.h.to(F8) + r["y"][T * K:].to(F8) + (r["gate"].to(F8)[:, :, None] * r["y"].to(F8)[r["slot_row"].long()]).sum(1)
    assert ((r["out"].to(F8) - out).abs() <= 1e-5 * (out.abs() + r["y"].abs().max())).all()
    # end to end: E2M1 rounds by up to 1/4 and on the average by some 12%; three such operands in a row
    tokens = sorted({0, T // 2, T - 1})
    ref = block.unquantised(r, x, stream, weight, masters, tokens, E)
    base = (x.float() + stream.float())[tokens].to(F8).cpu()
    rel = (r["out"][tokens].to(F8).cpu() - ref).norm(dim=1) / (ref - base).norm(dim=1)
    say(f"  experts' sum off by {rel.max():.3f} end to end")
    assert (rel < 0.35).all()


def test_block_in_a_graph():
    dev()
    x, stream, weight, centroids, bias, ex, _ = block.make(64, 512, 16, 4, 256)
    want = block.forward(x, stream, weight, centroids, bias, 4, ex)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block.forward(x, stream, weight, centroids, bias, 4, ex)
    for i in range(3):
        x.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        eager = block.forward(x, stream, weight, centroids, bias, 4, ex)
        torch.cuda.synchronize()
        for k in ("uq", "us", "hq", "hs", "y", "out"):
            assert torch.equal(held[k], eager[k]), (i, k)
    assert not torch.equal(held["out"], want["out"])


def test_norm_feeds_the_fp8_experts():
    """The norm's FP8 copy, handed to the FP8 grouped GEMM, gives what quantising its bf16 output gives."""
    dev()
    T, d, N = 40, 512, 256
    x, stream, weight, *_ = block.make(T, d, 2, 1, 128)
    n = moe.moe_add_rmsnorm(x, weight, block.EPS, residual=stream, quant=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    bq, bs = moe.fp8_quant_128x128(torch.randn((N, d), generator=g, device="cuda"))
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    q, s = moe.fp8_quant_1x128(n.y)
    a = moe.grouped_gemm_fp8_blockscaled(n.q, n.scale, off, T, bq[None], bs[None])
    b = moe.grouped_gemm_fp8_blockscaled(q, s, off, T, bq[None], bs[None])
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_backward_of_the_block():
    dev()
    x, stream, weight, centroids, bias, ex, _ = block.make(50, 512, 8, 2, 256)
    r = block.forward(x, stream, weight, centroids, bias, 2, ex)
    du, ds = torch.randn_like(x), torch.randn_like(x)
    dx, dw = block.backward(r, weight, du, ds)
    torch.cuda.synchronize()
    h = (x.float() + stream.float()).to(F8).requires_grad_()
    w = weight.to(F8).requires_grad_()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + block.EPS) * w
    (y * du.to(F8)).sum().backward()
    want = h.grad + ds.to(F8)
    # the kernel reads h rounded to bf16 (2^-8 of each value and of the row's mean products) and rounds dx once
    assert (dx.to(F8) - want).norm() <= 2.0 ** -7 * want.norm()
    assert (dw.to(F8) - w.grad).norm() <= 2.0 ** -7 * w.grad.norm()
