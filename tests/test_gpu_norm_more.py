"""Further cases of the residual + RMS norm and its backward on the GPU."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say
from test_gpu_norm import DT, EPS, _check_backward, _check_forward, _gen, _inputs, _rand

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


# ------------------------------------------------------------------ variants by size

@pytest.mark.parametrize("T,d", [(4700, 7168), (36000, 999), (36000, 1000), (110000, 333), (280000, 128), (8300, 4095),
                                 (2100, 16384), (33000, 1032)])
def test_backward_past_the_caches(T, d):
    """More than 64 MiB of dx, which is stored past the caches: rows of a wave and of a block, aligned and not."""
    dev()
    say(f"  T={T} d={d}")
    _check_backward(T, d, "bf16", "bf16", "f32", "bf16" if T % 200 else None, seed=T)


@pytest.mark.parametrize("T,d", [(5000, 999), (9001, 1000), (2500, 1025), (9001, 333), (3001, 7), (1500, 16383)])
def test_backward_of_many_odd_rows(T, d):
    """Several rows one after the other in each wave or block, the last ones fewer."""
    dev()
    say(f"  T={T} d={d}")
    a = _check_backward(T, d, "f32", "bf16", "f32", "f32", seed=d)
    b = _check_backward(T, d, "f32", "bf16", "f32", "f32", seed=d)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,d", [(9001, 999), (5000, 4095), (40001, 333), (3000, 16383)])
def test_forward_of_many_odd_rows(T, d):
    dev()
    say(f"  T={T} d={d}")
    _check_forward(*_inputs(T, d, "bf16", "bf16", "f32", seed=d), quant=False)


# ------------------------------------------------------------------ aliases

ALIAS_WIDTHS = [7, 128, 333, 512, 640, 999, 1000, 1032, 4095, 7168]


@pytest.mark.parametrize("d", ALIAS_WIDTHS)
def test_forward_aliases(d):
    """Every overlap that the call allows, against separate outputs, bit for bit."""
    dev()
    T, quant = 77, d % 128 == 0

    def call(x, res, **outs):
        r = moe.moe_add_rmsnorm(x, w, EPS, residual=res, quant=quant, **outs)
        torch.cuda.synchronize()
        return [t for t in r if t is not None]

    for xt, rt in (("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")):
        x, res, w = _inputs(T, d, xt, rt, "f32", seed=d)
        want = call(x, res)
        forms = [("h_out is residual", lambda a, b: dict(h_out=b))]
        if xt == rt:
            forms.append(("h_out is x", lambda a, b: dict(h_out=a)))
        if xt == "bf16":
            forms += [("y is x", lambda a, b: dict(y=a)), ("y is x, h_out is residual", lambda a, b: dict(y=a, h_out=b))]
        if rt == "bf16":
            forms.append(("y is residual", lambda a, b: dict(y=b)))
            if xt == rt:
                forms.append(("y is residual, h_out is x", lambda a, b: dict(y=b, h_out=a)))
        for name, outs in forms:
            say(f"  d={d} {xt} {rt}: {name}")
            a, b = x.clone(), res.clone()
            got = call(a, b, **outs(a, b))
            assert all(torch.equal(p, q) for p, q in zip(got, want)), name
        if xt == "bf16":
            a = x.clone()
            assert all(torch.equal(p, q) for p, q in zip(call(a, None, y=a), call(x, None)))


@pytest.mark.parametrize("d", ALIAS_WIDTHS)
def test_backward_aliases(d):
    dev()
    say(f"  d={d}")
    for T, t in ((77, "bf16"), (77, "f32"), (3000, "f32")):
        g = _gen(d)
        args = [_rand(g, T, d).to(DT[t]) for _ in range(3)]
        w, rstd = 1.0 + 0.3 * _rand(g, d), torch.rsqrt(args[1].float().square().mean(1) + EPS)
        want = moe.moe_add_rmsnorm_backward(args[0], args[1], w, rstd, dh=args[2])
        for i in range(3):
            c = [a.clone() for a in args]
            got = moe.moe_add_rmsnorm_backward(c[0], c[1], w, rstd, dh=c[2], dx=c[i])
            torch.cuda.synchronize()
            assert got[0] is c[i] and all(torch.equal(a, b) for a, b in zip(got, want)), i


# ------------------------------------------------------------------ NaN and infinities

@pytest.mark.parametrize("d", [7, 128, 333, 512, 640, 999, 1024, 1032, 4095, 4096])
def test_special_rows(d):
    """A NaN makes its row NaN; an infinity makes rstd 0, itself NaN and the rest of its row 0; a row of zeros
    stays zeros; their neighbours are as without them."""
    dev()
    say(f"  d={d}")
    at = d // 2
    for xt in ("bf16", "f32"):
        x, _, w = _inputs(9, d, xt, None, "f32", seed=d)
        clean = moe.moe_add_rmsnorm(x, w, EPS, quant=d % 128 == 0)
        bad = x.clone()
        bad[1], bad[3, d - 1], bad[5, at], bad[7, 0] = 0.0, float("nan"), float("inf"), -float("inf")
        r = moe.moe_add_rmsnorm(bad, w, EPS, quant=d % 128 == 0)
        torch.cuda.synchronize()
        same = [0, 2, 4, 6, 8]
        assert torch.equal(r.y[same], clean.y[same]) and torch.equal(r.rstd[same], clean.rstd[same])
        assert (r.y[1] == 0).all() and torch.isnan(r.y[3]).all() and torch.isnan(r.rstd[3])
        for row, col in ((5, at), (7, 0)):
            rest = torch.arange(d, device="cuda") != col
            assert r.rstd[row] == 0 and torch.isnan(r.y[row, col]) and (r.y[row][rest] == 0).all()
        if r.q is not None:
            q, s = moe.fp8_quant_1x128(r.y)
            assert torch.equal(q, r.q) and torch.equal(s.view(torch.int32), r.scale.view(torch.int32))


@pytest.mark.parametrize("d", [7, 128, 333, 512, 640, 999, 1024, 1032, 4095, 4096])
def test_backward_special_rows(d):
    """A NaN in dy or h makes its row of dx NaN and its column of dw; one in dh stays where it is."""
    dev()
    say(f"  d={d}")
    T, at = 9, d // 2
    for t in ("bf16", "f32"):
        g = _gen(d)
        dy, h, dh = (_rand(g, T, d).to(DT[t]) for _ in range(3))
        w, rstd = 1.0 + 0.3 * _rand(g, d), torch.rsqrt(h.float().square().mean(1) + EPS)
        want = moe.moe_add_rmsnorm_backward(dy, h, w, rstd, dh=dh)
        dy[2, at], h[4, d - 1], dh[6, 0] = float("nan"), float("nan"), float("nan")
        dx, dw = moe.moe_add_rmsnorm_backward(dy, h, w, rstd, dh=dh)
        torch.cuda.synchronize()
        nan = torch.zeros((T, d), dtype=torch.bool, device="cuda")
        nan[2], nan[4], nan[6, 0] = True, True, True
        cols = torch.zeros(d, dtype=torch.bool, device="cuda")
        cols[[at, d - 1]] = True
        assert torch.equal(torch.isnan(dx), nan) and torch.equal(dx[~nan], want[0][~nan])
        assert torch.equal(torch.isnan(dw), cols) and torch.equal(dw[~cols], want[1][~cols])
