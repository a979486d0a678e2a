"""Residual + layer norm and its backward on the GPU, against the definitions in
64 bits.

Bounds.  U = 2^-24 is binary32's unit roundoff, 2^-8 bf16's.  A sum over a row's d
terms is added up as at most 16 terms a thread, 6 wave steps and 16 waves: with the
arithmetic around it 64 U of the sum of the terms' sizes covers it.  So the mean is
off by 64 U mean|h| at most, and by U |h| more an element where x + residual was
rounded; the centred row c carries that error, which in rstd shows relative to
1 / rstd, and 48 U for its own sum, division and root."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF = 2.0 ** -8
EPS = 1e-5
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


def _inputs(T, d, xt, rt, wt, seed=0, offset=0.7):
    g = _gen(seed)
    x = _rand(g, T, d) + offset
    x[torch.rand((T, d), generator=g, device="cuda") < 1e-2] *= 100.0
    res = None if rt is None else (_rand(g, T, d, scale=3.0) - 0.4).to(DT[rt])
    return x.to(DT[xt]), res, (1.0 + 0.3 * _rand(g, d)).to(DT[wt]), (0.3 * _rand(g, d)).to(DT[wt])


def _reference(x, res, w, b, eps):
    """h, mean, rstd, y in 64 bits, and how far each of the last three may be off (y before its rounding)."""
    h = x.to(F8) if res is None else x.to(F8) + res.to(F8)
    mean = h.mean(1, keepdim=True)
    c = h - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + eps)
    off_mean = 65 * U * h.abs().mean(1, keepdim=True)
    off_c = off_mean + U * (h.abs() + c.abs())
    off_rstd = torch.sqrt((off_c * off_c).mean(1, keepdim=True)) * rstd + 48 * U       # relative
    y = c * rstd * w.to(F8)
    off_y = off_c * rstd * w.to(F8).abs() + y.abs() * (off_rstd + 4 * U)
    if b is not None:
        y = y + b.to(F8)
        off_y = off_y + U * y.abs()
    return mean[:, 0], rstd[:, 0], y, off_mean[:, 0], off_rstd[:, 0], off_y


def _check_forward(x, res, w, b, quant, eps=EPS):
    r = moe.moe_add_layernorm(x, w, eps, bias=b, residual=res, quant=quant)
    torch.cuda.synchronize()
    mean, rstd, y, off_mean, off_rstd, off_y = _reference(x, res, w, b, eps)
    assert ((r.mean.to(F8) - mean).abs() <= off_mean).all()
    assert ((r.rstd.to(F8) / rstd - 1).abs() <= off_rstd).all()
    assert ((r.y.to(F8) - y).abs() <= BF * y.abs() + 1.01 * off_y + 2.0 ** -133).all()
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
    return r


@pytest.mark.parametrize("d", WIDTHS)
def test_forward_widths(d):
    dev()
    for T, rt in ((1, None), (5, "bf16"), (3, "f32")):
        say(f"  T={T} d={d} residual={rt}")
        x, res, w, b = _inputs(T, d, "bf16" if d % 3 else "f32", rt, "f32" if d % 2 else "bf16", seed=d)
        _check_forward(x, res, w, None if T == 3 else b, quant=d % 128 == 0)


# every start of a row in its 16 bytes; lanes to a row 16, 32, 64 and a block, up to the last width of each; many turns
SHIFTED = [(1, 1), (1, 7), (7, 1), (2, 3), (3, 5), (37, 9), (100, 57), (5000, 61), (9, 121), (9, 122), (2001, 127), (20011, 65),
           (300, 129), (70, 249), (70, 250), (9001, 255), (70, 505), (70, 506), (3001, 511), (50, 1017), (50, 1018), (2500, 1023),
           (30, 2041), (1203, 2047), (20, 8185), (20, 8186), (700, 8191), (9, 16377), (9, 16378), (600, 16383), (131072 + 5, 67)]


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("T,d", SHIFTED)
def test_rows_of_no_multiple_of_8(T, d, xt):
    """Forward and backward, the operands between NaN, the outputs between guards."""
    dev()
    say(f"  T={T} d={d} {xt}")
    pad = 1024

    def inside(t):
        big = torch.full((t.numel() + 2 * pad,), float("nan"), dtype=t.dtype, device="cuda")
        big[pad:pad + t.numel()] = t.reshape(-1)
        return big, big[pad:pad + t.numel()].view(t.shape)

    def guarded(want, call):
        outs = [inside(torch.zeros_like(t)) for t in want]
        call([view for _, view in outs])
        torch.cuda.synchronize()
        for (big, view), t in zip(outs, want):
            assert torch.equal(view, t) and torch.isnan(big[:pad]).all() and torch.isnan(big[pad + t.numel():]).all()

    x, res, w, b = _inputs(T, d, xt, xt, "f32", seed=T + d)
    want = _check_forward(x, res, w, b, quant=False)
    hx, hres, hw, hb = (inside(t)[1] for t in (x, res, w, b))
    guarded((want.h, want.y, want.mean, want.rstd), lambda o: moe.moe_add_layernorm(
        hx, hw, EPS, bias=hb, residual=hres, h_out=o[0], y=o[1], mean=o[2], rstd=o[3]))
    _check_backward(T, d, xt, xt, "f32", xt, seed=T + d)
    dy, dh = _inputs(T, d, xt, xt, "f32", seed=1)[:2]
    grads = moe.moe_add_layernorm_backward(dy, x, w, want.mean, want.rstd, dh=dh)
    hdy, hx, hw, hm, hr, hdh = (inside(t)[1] for t in (dy, x, w, want.mean, want.rstd, dh))
    guarded(grads, lambda o: moe.moe_add_layernorm_backward(hdy, hx, hw, hm, hr, dh=hdh, dx=o[0], dw=o[1], db=o[2]))


@pytest.mark.parametrize("xt", ["bf16", "f32"])
@pytest.mark.parametrize("rt", [None, "bf16", "f32"])
@pytest.mark.parametrize("wt", ["bf16", "f32"])
def test_forward_types(xt, rt, wt):
    dev()
    for T, d in ((33, 640), (33, 1280), (9, 333)):
        _check_forward(*_inputs(T, d, xt, rt, wt), quant=d % 128 == 0)


@pytest.mark.parametrize("T,d", [(2049, 2048), (5000, 1152), (8193, 256), (20001, 128), (9001, 999), (40001, 333)])
def test_forward_many_rows(T, d):
    dev()
    say(f"  T={T} d={d}")
    _check_forward(*_inputs(T, d, "bf16", "bf16", "f32"), quant=d % 128 == 0)


def test_forward_rows_that_pass_a_launch():
    """Four rows of 8 values to a block of 256 threads: more than 2^32 threads."""
    dev()
    T, d = (1 << 26) + 5, 8
    say(f"  T={T}")
    x = torch.empty((T, d), dtype=torch.int8, device="cuda").random_(-100, 100, generator=_gen(3)).bfloat16()
    w, b = torch.linspace(0.5, 2.0, d, device="cuda"), torch.linspace(-1.0, 1.0, d, device="cuda")
    r = moe.moe_add_layernorm(x, w, EPS, bias=b)
    torch.cuda.synchronize()
    for at in range(0, T, 1 << 23):
        part = slice(at, at + (1 << 23))
        mean, rstd, y, off_mean, off_rstd, off_y = _reference(x[part], None, w, b, EPS)
        assert ((r.mean[part].to(F8) - mean).abs() <= off_mean).all()
        assert ((r.rstd[part].to(F8) / rstd - 1).abs() <= off_rstd).all()
        assert ((r.y[part].to(F8) - y).abs() <= BF * y.abs() + 1.01 * off_y + 2.0 ** -133).all()


@pytest.mark.parametrize("offset", [1e3, -1e5, 1e6])
def test_rows_far_from_zero_keep_their_variance(offset):
    """Squares summed about the mean: a mean many times the spread costs its rounding in h - mean and no more
    (as sum(h^2) - d mean^2 the variance would be rounding alone)."""
    dev()
    for d in (128, 333, 1280, 7168):
        x, _, w, b = _inputs(17, d, "f32", None, "f32", seed=d, offset=offset)
        _check_forward(x, None, w, b, quant=False)


@pytest.mark.parametrize("d", [7, 128, 333, 512, 640, 999, 1024, 1032, 4095, 4096])
def test_forward_special_rows(d):
    """A row of equal values gives the bias; a NaN or an infinity makes its row NaN; neighbours are as without them."""
    dev()
    say(f"  d={d}")
    for xt in ("bf16", "f32"):
        x, _, w, b = _inputs(9, d, xt, None, "f32", seed=d)
        clean = moe.moe_add_layernorm(x, w, EPS, bias=b, quant=d % 128 == 0)
        bad = x.clone()
        bad[0], bad[1] = 0.0, 3.0
        bad[3, d - 1], bad[5, d // 2], bad[7, 0] = float("nan"), float("inf"), -float("inf")
        r = moe.moe_add_layernorm(bad, w, EPS, bias=b, quant=d % 128 == 0)
        torch.cuda.synchronize()
        same = [2, 4, 6, 8]
        assert torch.equal(r.y[same], clean.y[same]) and torch.equal(r.rstd[same], clean.rstd[same])
        assert torch.equal(r.y[0], b.bfloat16()) and r.mean[0] == 0
        # 3 d adds up exactly, so the mean is 3 and the row is its bias
        assert torch.equal(r.y[1], b.bfloat16()) and r.mean[1] == 3
        for row in (3, 5, 7):
            assert torch.isnan(r.y[row]).all() and torch.isnan(r.rstd[row])
        if r.q is not None:
            q, s = moe.fp8_quant_1x128(r.y)
            assert torch.equal(q, r.q) and torch.equal(s.view(torch.int32), r.scale.view(torch.int32))


def test_forward_no_rows_and_repeatable():
    dev()
    e = torch.empty((0, 256), device="cuda")
    r = moe.moe_add_layernorm(e, torch.ones(256, device="cuda"), EPS, residual=e, quant=True)
    assert r.y.shape == (0, 256) and r.scale.shape == (0, 2)
    x, res, w, b = _inputs(300, 1280, "bf16", "bf16", "f32")
    want = moe.moe_add_layernorm(x, w, EPS, bias=b, residual=res, quant=True)
    again = moe.moe_add_layernorm(x, w, EPS, bias=b, residual=res, quant=True)
    assert all(torch.equal(p, q) for p, q in zip(want, again))


ALIAS_WIDTHS = [7, 128, 333, 512, 640, 999, 1000, 1032, 4095, 7168]


@pytest.mark.parametrize("d", ALIAS_WIDTHS)
def test_forward_aliases(d):
    """Every overlap that the call allows, against separate outputs, bit for bit."""
    dev()
    T, quant = 77, d % 128 == 0

    def call(x, res, **outs):
        r = moe.moe_add_layernorm(x, w, EPS, bias=b, residual=res, quant=quant, **outs)
        torch.cuda.synchronize()
        return [t for t in r if t is not None]

    for xt, rt in (("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f32")):
        x, res, w, b = _inputs(T, d, xt, rt, "f32", seed=d)
        want = call(x, res)
        forms = [("h_out is residual", lambda p, q: dict(h_out=q))]
        if xt == rt:
            forms.append(("h_out is x", lambda p, q: dict(h_out=p)))
        if xt == "bf16":
            forms += [("y is x", lambda p, q: dict(y=p)), ("y is x, h_out is residual", lambda p, q: dict(y=p, h_out=q))]
        if rt == "bf16":
            forms.append(("y is residual", lambda p, q: dict(y=q)))
            if xt == rt:
                forms.append(("y is residual, h_out is x", lambda p, q: dict(y=q, h_out=p)))
        for name, outs in forms:
            say(f"  d={d} {xt} {rt}: {name}")
            p, q = x.clone(), res.clone()
            got = call(p, q, **outs(p, q))
            assert all(torch.equal(s, t) for s, t in zip(got, want)), name
        if xt == "bf16":
            p = x.clone()
            assert all(torch.equal(s, t) for s, t in zip(call(p, None, y=p), call(x, None)))


# ------------------------------------------------------------------ backward

def _statistics(h):
    """mean and rstd FP32 of the rows as they are."""
    m = h.to(F8).mean(1)
    return m.float(), (1.0 / torch.sqrt(h.to(F8).var(1, correction=0) + EPS)).float()


def _gradient(dy, h, w, mean, rstd, dh):
    r = rstd.to(F8)[:, None]
    xh = (h.to(F8) - mean.to(F8)[:, None]) * r
    g = dy.to(F8) * w.to(F8)
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    size = r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, size = dx + dh.to(F8), size + dh.to(F8).abs()
    return dx, size, (dy.to(F8) * xh).sum(0), (dy.to(F8) * xh).abs().sum(0), dy.to(F8).sum(0), dy.to(F8).abs().sum(0)


def _check_backward(T, d, yt, ht, wt, gt, seed=0):
    g = _gen(seed)
    h, _, w, _ = _inputs(T, d, ht, None, wt, seed)
    dy = _rand(g, T, d, scale=1e-2).to(DT[yt])
    dh = None if gt is None else _rand(g, T, d, scale=1e-2).to(DT[gt])
    mean, rstd = _statistics(h)
    dx, dw, db = moe.moe_add_layernorm_backward(dy, h, w, mean, rstd, dh=dh)
    torch.cuda.synchronize()
    assert dx.dtype == (dy.dtype if dh is None else dh.dtype)
    rx, size, rw, wsize, rb, bsize = _gradient(dy, h, w, mean, rstd, dh)
    rounded = BF if dx.dtype == torch.bfloat16 else U
    assert ((dx.to(F8) - rx).abs() <= rounded * rx.abs() + 80 * U * size).all()
    # dw, db: a block's rows one after the other, at most 2048 partial rows as 16 sums, then those
    terms = -(-T // 256) + 2048 // 16 + 16 + 6
    assert ((dw.to(F8) - rw).abs() <= terms * U * wsize).all()
    assert ((db.to(F8) - rb).abs() <= terms * U * bsize).all()
    again = moe.moe_add_layernorm_backward(dy, h, w, mean, rstd, dh=dh, bias_grad=False)
    assert again[2] is None and torch.equal(again[0], dx) and torch.equal(again[1], dw)
    return dx, dw, db


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


@pytest.mark.parametrize("T,d", [(511, 2048), (513, 2048), (4099, 1152), (2049, 256), (8195, 128), (5000, 999),
                                 (2500, 1025), (9001, 333), (3001, 7), (1500, 16383), (1300, 7168)])
def test_backward_many_rows(T, d):
    dev()
    say(f"  T={T} d={d}")
    a = _check_backward(T, d, "bf16", "bf16", "f32", "bf16")
    b = _check_backward(T, d, "bf16", "bf16", "f32", "bf16")
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("T,d", [(4700, 7168), (36000, 999), (110000, 333), (280000, 128), (2100, 16384), (33000, 1032)])
def test_backward_past_the_caches(T, d):
    """More than 64 MiB of dx, which is stored past the caches."""
    dev()
    say(f"  T={T} d={d}")
    _check_backward(T, d, "bf16", "bf16", "f32", "bf16" if T % 200 else None, seed=T)


@pytest.mark.parametrize("T,d", [(256, 2048), (128, 999), (64, 1032), (1024, 128), (1024, 1000), (512, 333), (2, 7168)])
def test_weight_gradients_are_added_up_pairwise(T, d):
    """Equal rows, as many as a power of two and one to a block or wave: sums in pairs only double them, so
    dw and db are exact, whatever the bits of a row."""
    dev()
    say(f"  T={T} d={d}")
    row = _rand(_gen(d), d)
    h, one = row.expand(T, d).contiguous(), torch.ones((T, d), device="cuda")
    _, dw, db = moe.moe_add_layernorm_backward(one, h, one[0], torch.zeros(T, device="cuda"), torch.ones(T, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(dw, row * T) and (db == T).all()


def test_backward_no_rows():
    dev()
    e = torch.empty((0, 256), device="cuda")
    n = torch.empty(0, device="cuda")
    full = [torch.full((256,), 7.0, device="cuda") for _ in range(2)]
    dx, dw, db = moe.moe_add_layernorm_backward(e, e, torch.ones(256, device="cuda"), n, n, dw=full[0], db=full[1])
    torch.cuda.synchronize()
    assert dx.shape == (0, 256) and (dw == 0).all() and (db == 0).all()


@pytest.mark.parametrize("d", ALIAS_WIDTHS)
def test_backward_aliases(d):
    dev()
    say(f"  d={d}")
    for T, t in ((77, "bf16"), (77, "f32"), (3000, "f32")):
        g = _gen(d)
        args = [_rand(g, T, d).to(DT[t]) for _ in range(3)]
        w, (mean, rstd) = 1.0 + 0.3 * _rand(g, d), _statistics(args[1])
        want = moe.moe_add_layernorm_backward(args[0], args[1], w, mean, rstd, dh=args[2])
        for i in range(3):
            c = [a.clone() for a in args]
            got = moe.moe_add_layernorm_backward(c[0], c[1], w, mean, rstd, dh=c[2], dx=c[i])
            torch.cuda.synchronize()
            assert got[0] is c[i] and all(torch.equal(a, b) for a, b in zip(got, want)), i


@pytest.mark.parametrize("d", [7, 128, 333, 512, 640, 999, 1024, 1032, 4095, 4096])
def test_backward_special_rows(d):
    """A NaN in dy or h makes its row of dx NaN and its column of dw (and of db for dy); one in dh stays where it is."""
    dev()
    say(f"  d={d}")
    T, at = 9, d // 2
    for t in ("bf16", "f32"):
        g = _gen(d)
        dy, h, dh = (_rand(g, T, d).to(DT[t]) for _ in range(3))
        w, (mean, rstd) = 1.0 + 0.3 * _rand(g, d), _statistics(h)
        want = moe.moe_add_layernorm_backward(dy, h, w, mean, rstd, dh=dh)
        dy[2, at], h[4, d - 1], dh[6, 0] = float("nan"), float("nan"), float("nan")
        dx, dw, db = moe.moe_add_layernorm_backward(dy, h, w, mean, rstd, dh=dh)
        torch.cuda.synchronize()
        nan = torch.zeros((T, d), dtype=torch.bool, device="cuda")
        nan[2], nan[4], nan[6, 0] = True, True, True
        wcols, bcols = (torch.zeros(d, dtype=torch.bool, device="cuda") for _ in range(2))
        wcols[[at, d - 1]] = True
        bcols[at] = True
        assert torch.equal(torch.isnan(dx), nan) and torch.equal(dx[~nan], want[0][~nan])
        assert torch.equal(torch.isnan(dw), wcols) and torch.equal(dw[~wcols], want[1][~wcols])
        assert torch.equal(torch.isnan(db), bcols) and torch.equal(db[~bcols], want[2][~bcols])


def test_gradient_against_differences():
    """The kernels' gradients of L = <dy, y> + <dh, h> against central differences of L in 64 bits along
    random directions of x (residual's are the same), of the weight and of the bias."""
    dev()
    for T, d in ((7, 96), (5, 1100)):
        g = _gen(d)
        x, res, dy, dh, w, b = (_rand(g, T, d), _rand(g, T, d), _rand(g, T, d), _rand(g, T, d), 1.0 + 0.3 * _rand(g, d),
                                _rand(g, d))
        r = moe.moe_add_layernorm(x, w, EPS, bias=b, residual=res)
        grads = [t.to(F8) for t in moe.moe_add_layernorm_backward(dy, r.h, w, r.mean, r.rstd, dh=dh)]

        def loss(x_, w_, b_):
            h = x_ + res.to(F8)
            c = h - h.mean(1, keepdim=True)
            y = c / torch.sqrt((c * c).mean(1, keepdim=True) + EPS) * w_ + b_
            return float((dy.to(F8) * y).sum() + (dh.to(F8) * h).sum())

        # the differences' own error: third derivatives times step^2, rounding 2^-53 |L| / step
        step, at = 1e-4, [x.to(F8), w.to(F8), b.to(F8)]
        for i, grad in enumerate(grads):
            for _ in range(4):
                v = _rand(g, *grad.shape).to(F8)
                up, down = list(at), list(at)
                up[i], down[i] = at[i] + step * v, at[i] - step * v
                assert abs((loss(*up) - loss(*down)) / (2 * step) - float((grad * v).sum())) <= 1e-5 * float((grad * v).abs().sum())


def test_on_another_stream_and_in_a_graph():
    dev()
    x, res, w, b = _inputs(70, 1280, "bf16", "bf16", "f32")
    dy = _rand(_gen(9), 70, 1280).to(torch.bfloat16)

    def step():
        r = moe.moe_add_layernorm(x, w, EPS, bias=b, residual=res, quant=True)
        return (*r, *moe.moe_add_layernorm_backward(dy, r.h, w, r.mean, r.rstd, dh=r.y))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
        graph = torch.cuda.CUDAGraph()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        x.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(held, eager)), i


def test_binding_refusals():
    dev()
    x, w = torch.zeros((4, 256), device="cuda"), torch.ones(256, device="cuda")
    n = x[:, 0].contiguous()
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: moe.moe_add_layernorm(x.half(), w, EPS),
        lambda: moe.moe_add_layernorm(x, w[:128], EPS),
        lambda: moe.moe_add_layernorm(x, w.cpu(), EPS),
        lambda: moe.moe_add_layernorm(x, w, EPS, bias=w.bfloat16()),
        lambda: moe.moe_add_layernorm(x, w, EPS, bias=w[:128]),
        lambda: moe.moe_add_layernorm(x[:, ::2], w[:128], EPS),
        lambda: moe.moe_add_layernorm(x, w, EPS, residual=x[:2]),
        lambda: moe.moe_add_layernorm(x, w, EPS, h_out=x),
        lambda: moe.moe_add_layernorm(x, w, EPS, scale=w),
        lambda: moe.moe_add_layernorm(x, w, -1.0),
        lambda: moe.moe_add_layernorm(x[:, :100].contiguous(), w[:100].contiguous(), EPS, quant=True),
        lambda: moe.moe_add_layernorm(x[0], w, EPS),
        lambda: moe.moe_add_layernorm_backward(x, x[:2], w, n, n),
        lambda: moe.moe_add_layernorm_backward(x, x, w, n[:3], n),
        lambda: moe.moe_add_layernorm_backward(x, x, w, n, n.double()),
        lambda: moe.moe_add_layernorm_backward(x, x, w, n, n, dh=x.bfloat16(), dx_dtype=torch.float32),
        lambda: moe.moe_add_layernorm_backward(x, x, w, n, n, bias_grad=False, db=w),
        lambda: moe.moe_add_layernorm_backward(x, x, w, n, n, ws=small),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            pytest.fail(f"case {i} was taken")
