"""Residual + RMS norm and its backward on the GPU, against the definitions in
64 bits.

Bounds.  U = 2^-24 is binary32's unit roundoff, 2^-8 bf16's.  A row's sum of d
terms is added up as at most 16 terms a thread (32 where d % 8 != 0 never
applies more), 6 wave steps and 16 waves, and every other quantity takes a few
operations: 64 U covers a sum's relative error (terms of one sign) with the
arithmetic around it."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float64

# widths: one value, odd, under and at a wave's vectors, a wave's largest, past it, tiles of 128, the layer's, the limit
WIDTHS = [1, 2, 7, 8, 127, 128, 511, 512, 513, 520, 999, 1000, 1024, 1025, 1032, 2048, 4096, 7168, 16383, 16384]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda") * scale


def _rounded(dtype):
    return BF if dtype == torch.bfloat16 else U


def _inputs(T, d, xt, rt, wt, seed=0):
    g = _gen(seed)
    x = _rand(g, T, d)
    x[torch.rand((T, d), generator=g, device="cuda") < 1e-2] *= 100.0
    res = None if rt is None else _rand(g, T, d, scale=3.0).to(DT[rt])
    return x.to(DT[xt]), res, (1.0 + 0.3 * _rand(g, d)).to(DT[wt])


def _check_forward(x, res, w, quant):
    T, d = x.shape
    r = moe.moe_add_rmsnorm(x, w, EPS, residual=res, quant=quant)
    torch.cuda.synchronize()
    h = x.to(F8) if res is None else x.to(F8) + res.to(F8)
    rstd = 1.0 / torch.sqrt((h * h).sum(1) / d + EPS)
    assert (r.rstd.to(F8) / rstd - 1).abs().max() <= 64 * U
    y = h * rstd[:, None] * w.to(F8)
    assert ((r.y.to(F8) - y).abs() <= (BF + 80 * U) * y.abs() + 2.0 ** -133).all()
    if res is None:
        assert r.h is None
    else:
        want = (x.float() + res.float()).to(res.dtype)
        assert torch.equal(r.h.view(torch.uint8), want.view(torch.uint8))
    if quant:
        q, s = moe.fp8_quant_1x128(r.y)
        assert torch.equal(q, r.q) and torch.equal(s, r.scale)
    else:
        assert r.q is None and r.scale is None


@pytest.mark.parametrize("d", WIDTHS)
def test_forward_widths(d):
    dev()
    for T, rt in ((1, None), (5, "bf16"), (3, "f32")):
        say(f"  T={T} d={d} residual={rt}")
        x, res, w = _inputs(T, d, "bf16" if d % 3 else "f32", rt, "f32" if d % 2 else "bf16", seed=d)
        _check_forward(x, res, w, quant=d % 128 == 0)


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("rt", [None, "bf16", "f32"])
@pytest.mark.parametrize("wt", ["bf16", "f32"])
def test_forward_types(xt, rt, wt):
    dev()
    for T, d in ((33, 640), (33, 1280), (9, 333)):
        _check_forward(*_inputs(T, d, xt, rt, wt), quant=d % 128 == 0)


@pytest.mark.parametrize("T,d", [(2047, 2048), (2049, 2048), (5000, 1152), (8193, 256), (20001, 128)])
def test_forward_more_rows_than_the_grid(T, d):
    dev()
    _check_forward(*_inputs(T, d, "bf16", "bf16", "f32"), quant=True)


def test_forward_rows_that_pass_a_launch():
    """Four rows of 8 values to a block of 256 threads: more than 2^32 threads."""
    dev()
    T, d = (1 << 26) + 5, 8
    say(f"  T={T}")
    x = torch.empty((T, d), dtype=torch.int8, device="cuda").random_(-100, 100, generator=_gen(3)).bfloat16()
    w = torch.linspace(0.5, 2.0, d, device="cuda")
    r = moe.moe_add_rmsnorm(x, w, EPS)
    torch.cuda.synchronize()
    for at in range(0, T, 1 << 23):
        h = x[at:at + (1 << 23)].to(F8)
        rstd = 1.0 / torch.sqrt((h * h).mean(1) + EPS)
        assert (r.rstd[at:at + (1 << 23)].to(F8) / rstd - 1).abs().max() <= 64 * U
        y = h * rstd[:, None] * w.to(F8)
        assert ((r.y[at:at + (1 << 23)].to(F8) - y).abs() <= (BF + 80 * U) * y.abs() + 2.0 ** -133).all()


def test_forward_special_rows():
    """A row of zeros normalises to zeros; NaN and infinity stay in their row; tiny and huge rows
    keep their precision as long as their squares are binary32 numbers."""
    dev()
    d = 1280
    g = _gen(3)
    x = _rand(g, 6, d)
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    x[3] *= 1e-12
    x[4] *= 1e15
    w = 1.0 + 0.1 * _rand(g, d)
    r = moe.moe_add_rmsnorm(x, w, EPS, quant=True)
    torch.cuda.synchronize()
    assert (r.y[0] == 0).all() and (r.rstd[0].to(F8) * EPS ** 0.5 - 1).abs() <= 64 * U
    assert torch.isnan(r.y[1]).all()
    assert torch.isnan(r.y[2, 7]) and (r.y[2][torch.arange(d, device="cuda") != 7] == 0).all()
    good = [3, 4, 5]
    h = x[good].to(F8)
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w.to(F8)
    assert ((r.y[good].to(F8) - y).abs() <= (BF + 80 * U) * y.abs()).all()
    q, s = moe.fp8_quant_1x128(r.y)
    assert torch.equal(q, r.q) and torch.equal(s.view(torch.int32), r.scale.view(torch.int32))


def test_forward_in_place_and_repeatable():
    dev()
    x, res, w = _inputs(300, 1280, "bf16", "bf16", "f32")
    want = moe.moe_add_rmsnorm(x, w, EPS, residual=res, quant=True)
    again = moe.moe_add_rmsnorm(x, w, EPS, residual=res, quant=True)
    assert all(torch.equal(a, b) for a, b in zip(want, again))
    stream = res.clone()
    got = moe.moe_add_rmsnorm(x, w, EPS, residual=stream, h_out=stream, quant=True)
    assert got.h is stream and all(torch.equal(a, b) for a, b in zip(got, want))
    xx = x.clone()
    got = moe.moe_add_rmsnorm(xx, w, EPS, residual=res, y=xx, quant=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_forward_no_rows():
    dev()
    x = torch.empty((0, 256), device="cuda")
    r = moe.moe_add_rmsnorm(x, torch.ones(256, device="cuda"), EPS, residual=x, quant=True)
    assert r.y.shape == (0, 256) and r.scale.shape == (0, 2)


def _gradient(dy, h, w, rstd, dh):
    xh = h.to(F8) * rstd.to(F8)[:, None]
    g = dy.to(F8) * w.to(F8)
    c = (g * xh).mean(1, keepdim=True)
    r = rstd.to(F8)[:, None]
    dx = r * (g - xh * c) + (0.0 if dh is None else dh.to(F8))
    size = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + (0.0 if dh is None else dh.to(F8).abs())
    return dx, size, (dy.to(F8) * xh).sum(0), (dy.to(F8) * xh).abs().sum(0)


def _check_backward(T, d, yt, ht, wt, gt, seed=0):
    g = _gen(seed)
    h, _, w = _inputs(T, d, ht, None, wt, seed)
    dy = _rand(g, T, d, scale=1e-2).to(DT[yt])
    dh = None if gt is None else _rand(g, T, d, scale=1e-2).to(DT[gt])
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    dx, dw = moe.moe_add_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    torch.cuda.synchronize()
    assert dx.dtype == (dy.dtype if dh is None else dh.dtype)
    rx, size, rw, wsize = _gradient(dy, h, w, rstd, dh)
    assert ((dx.to(F8) - rx).abs() <= _rounded(dx.dtype) * rx.abs() + 80 * U * size).all()
    # dw: a block's rows one after the other, at most 2048 partial rows as 16 sums, then those
    terms = -(-T // 512) + 2048 // 16 + 16 + 4
    assert ((dw.to(F8) - rw).abs() <= terms * U * wsize).all()
    return dx, dw


@pytest.mark.parametrize("d", WIDTHS)
def test_backward_widths(d):
    dev()
    for T, gt in ((1, None), (5, "bf16"), (3, "f32")):
        say(f"  T={T} d={d} dh={gt}")
        _check_backward(T, d, "bf16" if d % 3 else "f32", "f32" if d % 5 else "bf16", "f32" if d % 2 else "bf16", gt, d)


@pytest.mark.parametrize("yt", ["bf16", "f32"])
@pytest.mark.parametrize("ht", ["bf16", "f32"])
@pytest.mark.parametrize("gt", [None, "bf16", "f32"])
def test_backward_types(yt, ht, gt):
    dev()
    for T, d, wt in ((33, 640, "bf16"), (33, 1280, "f32"), (9, 333, "f32")):
        _check_backward(T, d, yt, ht, wt, gt)


@pytest.mark.parametrize("T,d", [(511, 2048), (513, 2048), (4099, 1152), (2049, 256), (8195, 128)])
def test_backward_many_rows(T, d):
    dev()
    a = _check_backward(T, d, "bf16", "bf16", "f32", "bf16")
    b = _check_backward(T, d, "bf16", "bf16", "f32", "bf16")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_backward_no_rows_and_in_place():
    dev()
    e = torch.empty((0, 256), device="cuda")
    dx, dw = moe.moe_add_rmsnorm_backward(e, e, torch.ones(256, device="cuda"), torch.empty(0, device="cuda"),
                                          dw=torch.full((256,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and (dw == 0).all()
    g = _gen(5)
    h, dy, dh = (_rand(g, 40, 1280) for _ in range(3))
    w, rstd = torch.ones(1280, device="cuda"), torch.rsqrt(h.square().mean(1) + EPS)
    want = moe.moe_add_rmsnorm_backward(dy, h, w, rstd, dh=dh)
    for i in range(3):
        t = [dy.clone(), h.clone(), dh.clone()]
        got = moe.moe_add_rmsnorm_backward(t[0], t[1], w, rstd, dh=t[2], dx=t[i])
        assert got[0] is t[i] and all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradient_against_differences():
    """The kernels' gradients of L = <dy, y> + <dh, h> against central differences of L in 64 bits along
    random directions of x (residual's are the same) and of the weight."""
    dev()
    for T, d in ((7, 96), (5, 1100)):
        g = _gen(d)
        x, res, dy, dh, w = _rand(g, T, d), _rand(g, T, d), _rand(g, T, d), _rand(g, T, d), 1.0 + 0.3 * _rand(g, d)
        r = moe.moe_add_rmsnorm(x, w, EPS, residual=res)
        dx, dw = moe.moe_add_rmsnorm_backward(dy, r.h, w, r.rstd, dh=dh)

        def loss(x_, w_):
            h = x_ + res.to(F8)
            y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * w_
            return float((dy.to(F8) * y).sum() + (dh.to(F8) * h).sum())

        # the differences' own error: third derivatives times step^2, rounding 2^-53 |L| / step
        step = 1e-4
        for _ in range(4):
            vx, vw = _rand(g, T, d).to(F8), _rand(g, d).to(F8)
            nx = (loss(x.to(F8) + step * vx, w.to(F8)) - loss(x.to(F8) - step * vx, w.to(F8))) / (2 * step)
            nw = (loss(x.to(F8), w.to(F8) + step * vw) - loss(x.to(F8), w.to(F8) - step * vw)) / (2 * step)
            assert abs(nx - float((dx.to(F8) * vx).sum())) <= 1e-5 * float((dx.to(F8) * vx).abs().sum())
            assert abs(nw - float((dw.to(F8) * vw).sum())) <= 1e-5 * float((dw.to(F8) * vw).abs().sum())


def test_on_another_stream_and_in_a_graph():
    dev()
    x, res, w = _inputs(70, 1280, "bf16", "bf16", "f32")
    g = _gen(9)
    dy = _rand(g, 70, 1280).to(torch.bfloat16)

    def step():
        r = moe.moe_add_rmsnorm(x, w, EPS, residual=res, quant=True)
        return (*r, *moe.moe_add_rmsnorm_backward(dy, r.h, w, r.rstd, dh=r.y))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        x.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_binding_refusals():
    dev()
    x, w = torch.zeros((4, 256), device="cuda"), torch.ones(256, device="cuda")
    bad = [
        lambda: moe.moe_add_rmsnorm(x.half(), w, EPS),
        lambda: moe.moe_add_rmsnorm(x, w[:128], EPS),
        lambda: moe.moe_add_rmsnorm(x, w.cpu(), EPS),
        lambda: moe.moe_add_rmsnorm(x[:, ::2], w[:128], EPS),
        lambda: moe.moe_add_rmsnorm(x, w, EPS, residual=x[:2]),
        lambda: moe.moe_add_rmsnorm(x, w, EPS, h_out=x),
        lambda: moe.moe_add_rmsnorm(x, w, -1.0),
        lambda: moe.moe_add_rmsnorm(x[:, :100].contiguous(), w[:100].contiguous(), EPS, quant=True),
        lambda: moe.moe_add_rmsnorm(x[0], w, EPS),
        lambda: moe.moe_add_rmsnorm_backward(x, x[:2], w, x[:, 0].contiguous()),
        lambda: moe.moe_add_rmsnorm_backward(x, x, w, x[:3, 0].contiguous()),
        lambda: moe.moe_add_rmsnorm_backward(x, x, w, x[:, 0].contiguous(), dh=x.bfloat16(), dx_dtype=torch.float32),
        lambda: moe.moe_add_rmsnorm_backward(x, x, w, x[:, 0].contiguous(),
                                             ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            pytest.fail(f"case {i} was taken")
