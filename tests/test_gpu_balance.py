"""The balance loss over packed sequences, its gradient, and the router's backward
from all logits, on the GPU, against the definitions in 64 bits.

Bounds.  U = 2^-24.  p = s / sum s: a sum of at most 256 terms as 4 a lane and 6 wave
steps, and a division, 12 U.  P adds one sign's terms: a run's tokens 16 waves at a
time, the 16 waves, then a sequence's records four at a time."""
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float64
ALPHA = 1e-2


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _inputs(T, E, K, seed=0):
    g = _gen(seed)
    scores = torch.sigmoid(2.0 * _rand(g, T, E) + _rand(g, E))
    return scores, torch.topk(scores, K, dim=1).indices.to(torch.int32) if T else scores.new_empty((0, K), dtype=torch.int32)


def _starts(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _reference(scores, idx, starts, dloss, dlogits_in):
    T, E = scores.shape
    K = idx.shape[1]
    s = scores.to(F8)
    total = s.sum(1, keepdim=True)
    p = torch.where(total == 0, 0.0, s / torch.where(total == 0, 1.0, total))
    loss, count, size = [], [], torch.zeros((T, E), dtype=F8, device="cuda")
    grad = torch.zeros((T, E), dtype=F8, device="cuda")
    for q, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
        ids = idx[a:b].long().reshape(-1)
        n = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E)
        count.append(n)
        if a == b:
            loss.append(torch.zeros((), dtype=F8, device="cuda"))
            continue
        f = n.to(F8) * E / (K * (b - a))
        loss.append(ALPHA * (f * p[a:b].mean(0)).sum())
        dl = 1.0 if dloss is None else float(dloss[q])
        coef = dl * ALPHA / (b - a) * p[a:b] * (1.0 - s[a:b])
        fp = p[a:b] @ f
        grad[a:b] = coef * (f - fp[:, None])
        size[a:b] = coef.abs() * (f + fp[:, None])
    if dlogits_in is not None:
        grad, size = grad + dlogits_in.to(F8), size + dlogits_in.to(F8).abs()
    return torch.stack(loss), torch.stack(count).to(torch.int32), grad, size


def _check(scores, idx, starts, dloss=None, dlogits_in=None, device_starts=None):
    T, E = scores.shape
    K = idx.shape[1]
    start = _starts(starts) if device_starts is None else device_starts
    r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start)
    grad = moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA, seq_start=start, dloss=dloss, dlogits_in=dlogits_in)
    torch.cuda.synchronize()
    loss, count, want, size = _reference(scores, idx, starts, dloss, dlogits_in)
    assert torch.equal(r.seq_count, count)
    assert torch.equal(r.expert_count, count.sum(0, dtype=torch.int32))
    terms = 12 + -(-T // (256 * 16)) + 4 + 16 + 256 // 4 + 4 + 8 + 8
    if T <= 4096:                 # perhaps one block to a sequence: a lane adds up every 16th (64th) token of 1024 (4096)
        terms += min(-(-T // 16), 64)
    assert ((r.loss.to(F8) - loss).abs() <= terms * U * loss).all()
    # coef p (1 - s): 18 U of the gradient; f - sum f p: 10 U of f and 24 U of the sum; the addition
    assert ((grad.to(F8) - want).abs() <= 48 * U * size + 2.0 ** -149).all()
    return r, grad


@pytest.mark.parametrize("E,K", [(1, 1), (2, 2), (3, 1), (16, 4), (61, 7), (64, 8), (65, 16), (128, 8), (200, 16), (255, 8), (256, 8)])
def test_experts(E, K):
    dev()
    for T in (1, 2, 63, 64, 65, 300, 1000, 5000):
        say(f"  E={E} K={K} T={T}")
        scores, idx = _inputs(T, E, K, seed=T)
        _check(scores, idx, [0, T])
        _check(scores, idx, [0, T // 3, T // 3, T], dloss=_rand(_gen(1), 3), dlogits_in=1e-4 * _rand(_gen(2), T, E))


@pytest.mark.parametrize("T,starts", [
    (500, [0, 0, 0, 500, 500, 500]),                       # empty ones in front, behind
    (500, [17, 17, 40, 40, 40, 41, 300, 483]),             # gaps at both ends
    (64, [0, 0]), (64, [64, 64]), (64, [10, 10, 10]),      # nothing at all
    (1, [0, 1]), (1, [0, 0, 1, 1]),
    (1000, list(range(0, 1001, 8))),                       # sequences shorter than a chunk
    (1000, list(range(1001))),                             # of one token each
    (700, [0] * 3000 + [333] * 3000 + [700]),              # thousands of empty ones
    (9000, list(range(0, 9001, 8))), (9000, list(range(9001))), (9000, [17, 17, 40, 40, 41, 300, 8983]),
    (9000, [0] * 3000 + [333] * 3000 + [700]), (4096, [0, 4000] + list(range(4000, 4096, 6))),
    (40000, [0, 39999, 40000]), (40000, [1, 2, 39000]), (70000, [0, 17, 16400, 69999]),
])
def test_sequences(T, starts):
    dev()
    say(f"  T={T} sequences={len(starts) - 1}")
    scores, idx = _inputs(T, 40, 5, seed=T)
    _check(scores, idx, starts, dloss=1.0 + _rand(_gen(3), len(starts) - 1).abs())


@pytest.mark.parametrize("T,E,K", [(131072, 256, 8), (262145, 33, 3), (16384, 256, 8)])
def test_long(T, E, K):
    dev()
    say(f"  T={T} E={E}")
    scores, idx = _inputs(T, E, K, seed=T)
    _check(scores, idx, [0, T])
    r, _ = _check(scores, idx, [0, 5, T // 2 + 1, T - 7, T - 1])
    again = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=_starts([0, 5, T // 2 + 1, T - 7, T - 1]))
    assert all(torch.equal(a, b) for a, b in zip(r, again))


def test_past_32_bit_offsets():
    """The last tokens of 8 GiB of scores: their counts and gradients as of those tokens alone, bit for bit."""
    dev()
    T, E, K, last = 2 ** 23 + 77, 256, 2, 100
    block, picks = _inputs(4096, E, K, seed=5)
    scores = block.repeat(-(-T // 4096), 1)[:T]
    idx = picks.repeat(-(-T // 4096), 1)[:T].contiguous()
    say("  inputs made")
    scores[T - last:], idx[T - last:] = _inputs(last, E, K, seed=6)
    r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=_starts([0, T - last, T]))
    grad = moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA, seq_start=_starts([0, T - last, T]))
    tail, tail_idx = scores[T - last:].clone(), idx[T - last:].clone()
    one = moe.moe_balance_loss(tail, tail_idx, ALPHA)
    want = moe.moe_balance_loss_backward(tail, one.seq_count, K, ALPHA)
    torch.cuda.synchronize()
    assert torch.equal(r.seq_count[1], one.seq_count[0]) and torch.equal(grad[T - last:], want)
    # other chunks, so another order of the sums: 117 roundings as _check counts them, on both sides
    assert ((r.loss[1] - one.loss[0]).abs() <= 2 * 117 * U * one.loss[0]).all()
    assert int(r.seq_count[0].sum()) == K * (T - last) and int(r.expert_count.sum()) == K * T
    f = r.seq_count[0].to(F8) * E / (K * (T - last))
    s = scores[T - last - 50:T - last].to(F8)
    p = s / s.sum(1, keepdim=True)
    coef, fp = ALPHA / (T - last) * p * (1.0 - s), (p @ f)[:, None]
    assert ((grad[T - last - 50:T - last].to(F8) - coef * (f - fp)).abs() <= 48 * U * coef * (f + fp)).all()


def test_whole_batch_and_equal_lengths():
    """No starts: one sequence of all tokens.  Equal lengths: moe_seq_balance_loss but for the order of the sums."""
    dev()
    T, E, K = 4096, 256, 8
    scores, idx = _inputs(T, E, K)
    whole = moe.moe_balance_loss(scores, idx, ALPHA)
    one = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=_starts([0, T]))
    assert all(torch.equal(a, b) for a, b in zip(whole, one))
    g = moe.moe_balance_loss_backward(scores, whole.seq_count, K, ALPHA)
    assert torch.equal(g, moe.moe_balance_loss_backward(scores, whole.seq_count, K, ALPHA, seq_start=_starts([0, T])))
    for L in (64, 1024):
        r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=_starts(list(range(0, T + 1, L))))
        old = moe.moe_seq_balance_loss(scores, idx, L, ALPHA)
        assert ((r.loss.to(F8) - old.to(F8)).abs() <= 2 * (64 + L) * U * old.to(F8)).all()


def test_no_tokens():
    dev()
    scores, idx = _inputs(0, 16, 4)
    for start in (None, _starts([0, 0, 0])):
        r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start)
        torch.cuda.synchronize()
        assert (r.loss == 0).all() and (r.seq_count == 0).all() and (r.expert_count == 0).all()
        assert moe.moe_balance_loss_backward(scores, r.seq_count, 4, ALPHA, seq_start=start).shape == (0, 16)


def test_closed_forms():
    """Uniform use gives alpha; all tokens on the same K experts with all their score there alpha E / K."""
    dev()
    T, E, K = 512, 64, 4
    scores = torch.full((T, E), 0.25, device="cuda")
    idx = (torch.arange(T * K, device="cuda").view(T, K) % E).to(torch.int32)
    r = moe.moe_balance_loss(scores, idx, ALPHA)
    assert abs(float(r.loss) / ALPHA - 1) <= 4e-6
    assert (moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA).abs() <= 1e-12).all()
    scores = torch.zeros((T, E), device="cuda")
    scores[:, :K] = 0.5
    r = moe.moe_balance_loss(scores, torch.arange(K, device="cuda", dtype=torch.int32).expand(T, K).contiguous(), ALPHA)
    assert abs(float(r.loss) / (ALPHA * E / K) - 1) <= 4e-6


@pytest.mark.parametrize("T", [300, 5000])
def test_odd_values(T):
    """Rows of zeros add nothing and get nothing; indices outside [0, E) are not counted; tiny scores keep
    their shares; a NaN stays in its sequence and, in padding, nowhere."""
    dev()
    E, K = 40, 4
    scores, idx = _inputs(T, E, K)
    scores[5] = 0.0
    scores[40:60] = 0.0
    scores[70] *= 1e-37
    idx[7, 1], idx[8, 0], idx[9] = -1, E, 2 ** 30
    starts = [0, 40, 60, 250]
    r, g = _check(scores, idx, starts)
    assert (g[5] == 0).all() and (g[40:60] == 0).all() and r.loss[1] == 0 and (g[250:] == 0).all()
    bad = scores.clone()
    bad[100, 3], bad[270] = float("nan"), float("nan")
    start = _starts(starts)
    r2 = moe.moe_balance_loss(bad, idx, ALPHA, seq_start=start)
    g2 = moe.moe_balance_loss_backward(bad, r2.seq_count, K, ALPHA, seq_start=start)
    torch.cuda.synchronize()
    assert torch.equal(r2.loss[:2], r.loss[:2]) and torch.isnan(r2.loss[2]) and torch.equal(r2.seq_count, r.seq_count)
    rest = torch.arange(T, device="cuda") != 100
    assert torch.isnan(g2[100]).all() and torch.equal(g2[rest], g[rest])


@pytest.mark.parametrize("T", [200, 5000])
def test_starts_outside_the_batch_are_held_inside(T):
    dev()
    scores, idx = _inputs(T, 30, 3)
    _check(scores, idx, [0, 50, T], device_starts=_starts([-7, 50, 1 << 30]))


def test_in_place_and_against_differences():
    dev()
    T, E, K, starts = 60, 24, 3, [0, 25, 25, 55]
    g = _gen(4)
    x = _rand(g, T, E)
    scores = torch.sigmoid(x)
    idx = torch.topk(scores, K, dim=1).indices.to(torch.int32)
    dloss, add = _rand(g, 3), _rand(g, T, E)
    start = _starts(starts)
    r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start)
    want = moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA, seq_start=start, dloss=dloss, dlogits_in=add)
    held = add.clone()
    got = moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA, seq_start=start, dloss=dloss, dlogits_in=held,
                                        dlogits=held)
    assert got is held and torch.equal(got, want)
    grad = moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA, seq_start=start, dloss=dloss).to(F8)

    def loss(x_):
        total, s = 0.0, torch.sigmoid(x_)
        for q, (a, b) in enumerate(zip(starts[:-1], starts[1:])):
            if b > a:
                f = r.seq_count[q].to(F8) * E / (K * (b - a))
                total += float(dloss[q]) * ALPHA * float((f * (s[a:b] / s[a:b].sum(1, keepdim=True)).mean(0)).sum())
        return total

    step = 1e-4        # scores rounded to 32 bits move the gradient by 2^-23 of itself or so
    for _ in range(4):
        v = _rand(g, T, E).to(F8)
        n = (loss(x.to(F8) + step * v) - loss(x.to(F8) - step * v)) / (2 * step)
        assert abs(n - float((grad * v).sum())) <= 1e-5 * float((grad * v).abs().sum())


@pytest.mark.parametrize("T", [900, 9000])
def test_balance_on_another_stream_and_in_a_graph(T):
    """Captured with its starts on the device: replays follow what they hold then."""
    dev()
    E, K = 61, 4
    scores, idx = _inputs(T, E, K)
    start = _starts([0, 100, 100, 650])

    def step():
        r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start)
        return (*r, moe.moe_balance_loss_backward(scores, r.seq_count, K, ALPHA, seq_start=start))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i, starts in enumerate(([0, 1, 2, 3], [5, 300, 800, 900], [0, 0, 900, 900])):
        start.copy_(_starts(starts))
        scores.mul_(0.9)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


# ------------------------------------------------------------------ the router's backward from all logits

def _operands(T, d, E, seed=0):
    g = _gen(seed)
    dl = 1e-3 * _rand(g, T, E) * torch.exp(2.0 * _rand(g, T, E))
    return dl, _rand(g, T, d).bfloat16(), _rand(g, E, d).bfloat16()


def _check_logits(dl, u, e, du_in=None, de_in=None):
    T, E = dl.shape
    du, de = moe.moe_router_logits_backward(dl, u, e, du_in=du_in, de_in=de_in)
    torch.cuda.synchronize()
    x, uu, ee = dl.to(F8), u.to(F8), e.to(F8)
    for got, a, b, add in ((du, x, ee, du_in), (de, x.t().contiguous(), uu, de_in)):
        ref, size = a @ b, a.abs() @ b.abs()
        if add is not None:
            ref, size = ref + add.to(F8), size + add.to(F8).abs()
        # exact products, three for each of K terms, added up one after the other at worst
        worst = (3 * a.shape[1] + 2) * U
        assert ((got.to(F8) - ref).abs() <= worst * size + 2.0 ** -120).all()
        # roundings of random sign: the error of all outputs together
        if ref.numel() > 1000:
            assert float((got.to(F8) - ref).norm()) <= 1.5 * (3 * a.shape[1]) ** 0.5 * U * float(size.norm())
    return du, de


@pytest.mark.parametrize("E", [1, 2, 15, 16, 17, 31, 32, 33, 61, 64, 65, 96, 127, 128, 129, 200, 255, 256])
def test_logits_experts(E):
    dev()
    for T, d in ((1, 128), (33, 128), (130, 384)):
        say(f"  E={E} T={T} d={d}")
        _check_logits(*_operands(T, d, E, seed=E))


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, 1031, 2049])
def test_logits_tokens(T):
    dev()
    for E, d in ((8, 128), (61, 640), (256, 256)):
        say(f"  T={T} E={E} d={d}")
        dl, u, e = _operands(T, d, E, seed=T)
        _check_logits(dl, u, e, du_in=_rand(_gen(1), T, d), de_in=_rand(_gen(2), E, d))


@pytest.mark.parametrize("T", [4095, 4096, 4097, 4111, 4127, 4128, 4129, 4223, 4225, 5003])
def test_logits_many_tokens(T):
    """About the number of tokens from which on planes of x are written and the tokens split in parts."""
    dev()
    for E, d in ((1, 128), (8, 256), (61, 640), (64, 128), (65, 384), (128, 128), (129, 384), (256, 256), (200, 1280)):
        say(f"  T={T} E={E} d={d}")
        dl, u, e = _operands(T, d, E, seed=T)
        _check_logits(dl, u, e, du_in=_rand(_gen(1), T, d), de_in=_rand(_gen(2), E, d))


@pytest.mark.parametrize("T,d,E", [(33, 65536, 5), (584, 7168, 40), (586, 7168, 40), (2049, 2048, 30), (128, 32896, 3)])
def test_logits_wide(T, d, E):
    dev()
    _check_logits(*_operands(T, d, E, seed=d))


@pytest.mark.parametrize("T,d,E", [(4096, 7168, 256), (5003, 1152, 160), (300, 16384, 7), (20001, 256, 64), (70001, 128, 33)])
def test_logits_large(T, d, E):
    dev()
    say(f"  T={T} d={d} E={E}")
    dl, u, e = _operands(T, d, E)
    a = _check_logits(dl, u, e)
    b = moe.moe_router_logits_backward(dl, u, e)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_logits_past_32_bit_offsets():
    dev()
    T, d, E = 160001, 7168, 20
    dl, u, e = _operands(T, d, E, seed=9)
    du_in = _rand(_gen(1), T, d)
    say("  inputs made")
    du, de = moe.moe_router_logits_backward(dl, u, e, du_in=du_in)
    torch.cuda.synchronize()
    x = dl.to(F8)
    for rows in (slice(0, 40), slice(149790, 149840), slice(T - 70, T)):      # 149797 rows of du are 2^32 bytes
        ref, size = x[rows] @ e.to(F8) + du_in[rows].to(F8), x[rows].abs() @ e.to(F8).abs() + du_in[rows].to(F8).abs()
        assert ((du[rows].to(F8) - ref).abs() <= (3 * E + 2) * U * size).all()
    cols = slice(d - 130, d)
    xt, uu = x.t().contiguous(), u[:, cols].to(F8)
    assert ((de[:, cols].to(F8) - xt @ uu).abs() <= (3 * T + 2) * U * (xt.abs() @ uu.abs())).all()
    # roundings of random sign
    assert float((de[:, cols].to(F8) - xt @ uu).norm()) <= 1.5 * (3 * T) ** 0.5 * U * float((xt.abs() @ uu.abs()).norm())


@pytest.mark.parametrize("T,d,E", [(300, 384, 61), (513, 256, 256), (64, 128, 16), (4300, 128, 61), (4300, 384, 200)])
def test_logits_keep_all_bits(T, d, E):
    """One product to an output: the 32-bit logits come through with all their bits."""
    dev()
    g = _gen(T)
    dl = _rand(g, T, E) * torch.exp(8.0 * _rand(g, T, E))
    e = torch.zeros((E, d), device="cuda")
    pick = torch.randint(0, E, (d,), generator=g, device="cuda")
    e[pick, torch.arange(d, device="cuda")] = 0.5
    u = torch.zeros((T, d), device="cuda")
    row = torch.randint(0, T, (d,), generator=g, device="cuda")
    u[row, torch.arange(d, device="cuda")] = -2.0
    du, de = moe.moe_router_logits_backward(dl, u.bfloat16(), e.bfloat16())
    torch.cuda.synchronize()
    assert torch.equal(du, 0.5 * dl[:, pick])
    assert torch.equal(de, -2.0 * dl[row].t())


@pytest.mark.parametrize("T,d,E", [(700, 256, 100), (3000, 128, 256), (4500, 128, 256), (9000, 256, 60)])
def test_logits_whole_numbers(T, d, E):
    """Sums of whole numbers under 2^24 are exact in any order."""
    dev()
    g = _gen(T)
    dl = torch.randint(-40, 41, (T, E), generator=g, device="cuda").float()
    u, e = (torch.randint(-8, 9, s, generator=g, device="cuda").bfloat16() for s in ((T, d), (E, d)))
    du, de = moe.moe_router_logits_backward(dl, u, e)
    torch.cuda.synchronize()
    assert torch.equal(du.to(F8), dl.to(F8) @ e.to(F8)) and torch.equal(de.to(F8), dl.to(F8).t().contiguous() @ u.to(F8))


@pytest.mark.parametrize("T", [200, 4200])
def test_logits_special_values(T):
    """NaN and infinite logits reach their row of du and their row of de, and nothing else."""
    dev()
    d, E = 256, 70
    dl, u, e = _operands(T, d, E)
    want = moe.moe_router_logits_backward(dl, u, e)
    bad = dl.clone()
    bad[5, 3], bad[77, 69], bad[199, 0] = float("nan"), float("inf"), -float("inf")
    du, de = moe.moe_router_logits_backward(bad, u, e)
    torch.cuda.synchronize()
    rows, cols = torch.ones(T, dtype=torch.bool, device="cuda"), torch.ones(E, dtype=torch.bool, device="cuda")
    rows[[5, 77, 199]], cols[[3, 69, 0]] = False, False
    assert torch.equal(du[rows], want[0][rows]) and torch.equal(de[cols], want[1][cols])
    assert torch.isnan(du[5]).all() and torch.isnan(de[3]).all()
    sign = torch.sign(e[69].float())
    assert torch.equal(du[77][sign != 0], (sign * float("inf"))[sign != 0]) and torch.isnan(du[77][sign == 0]).all()
    assert not torch.isfinite(de[69]).any() and not torch.isfinite(de[0]).any()
    # a denormal's products are under the smallest normal number: at most lost
    tiny = torch.full((T, E), 1e-40, device="cuda")
    du, _ = moe.moe_router_logits_backward(tiny, u, e)
    assert (du.abs() <= 1e-36).all()


@pytest.mark.parametrize("T", [300, 4300])
def test_logits_no_tokens_one_output_and_in_place(T):
    dev()
    d, E = 256, 20
    dl, u, e = _operands(0, d, E)
    add = _rand(_gen(1), E, d)
    du, de = moe.moe_router_logits_backward(dl, u, e)
    assert du.shape == (0, d) and (de == 0).all()
    assert torch.equal(moe.moe_router_logits_backward(dl, u, e, de_in=add)[1], add)
    dl, u, e = _operands(T, d, E)
    du_in = _rand(_gen(2), T, d)
    want = moe.moe_router_logits_backward(dl, u, e, du_in=du_in, de_in=add)
    only = moe.moe_router_logits_backward(dl, u, e, du_in=du_in, want_de=False)
    assert only[1] is None and torch.equal(only[0], want[0])
    only = moe.moe_router_logits_backward(dl, u, e, de_in=add, want_du=False)
    assert only[0] is None and torch.equal(only[1], want[1])
    a, b = du_in.clone(), add.clone()
    got = moe.moe_router_logits_backward(dl, u, e, du_in=a, de_in=b, du=a, de=b)
    torch.cuda.synchronize()
    assert got[0] is a and got[1] is b and torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("T,d,E", [(1, 128, 1), (45, 256, 33), (97, 384, 70), (130, 128, 129), (161, 256, 200),
                                   (4097, 128, 1), (4129, 256, 33), (4225, 384, 70), (4131, 128, 129), (4161, 256, 200)])
def test_logits_operands_inside_a_buffer(T, d, E):
    """Nothing around the operands is read (there are NaN) and nothing around the outputs written."""
    dev()
    pad = 1 << 16                                    # values, on each side

    def inside(x):
        big = torch.full((x.numel() + 2 * pad,), float("nan"), dtype=x.dtype, device="cuda")
        view = big[pad:pad + x.numel()].view(x.shape)
        view.copy_(x)
        return big, view

    dl, u, e = _operands(T, d, E, seed=T)
    add = _rand(_gen(1), T, d), _rand(_gen(2), E, d)
    want = moe.moe_router_logits_backward(dl, u, e, du_in=add[0], de_in=add[1])
    (_, dl), (_, u), (_, e), (_, du_in), (_, de_in) = (inside(x) for x in (dl, u, e, *add))
    outs = [inside(torch.zeros_like(x)) for x in want]
    ws_bytes = moe.load_library().moe_router_logits_backward_workspace_bytes(T, d, E)
    room, ws = inside(torch.zeros(ws_bytes // 4 + 1, device="cuda"))
    moe.moe_router_logits_backward(dl, u, e, du_in=du_in, de_in=de_in, du=outs[0][1], de=outs[1][1],
                                   ws=ws.view(torch.uint8).view(-1))
    torch.cuda.synchronize()
    for (big, view), x in zip([*outs, (room, ws)], [*want, None]):
        assert x is None or torch.equal(view, x)
        assert torch.isnan(big[:pad]).all() and torch.isnan(big[pad + view.numel():]).all()


def test_logits_against_differences():
    """L = <g, u . e^T> is linear in u and in e: its differences are its gradient."""
    dev()
    T, d, E = 40, 128, 12
    dl, u, e = _operands(T, d, E)
    du, de = moe.moe_router_logits_backward(dl, u, e)
    g = _gen(8)
    for _ in range(4):
        vu, ve = _rand(g, T, d).to(F8), _rand(g, E, d).to(F8)
        logits = lambda a, b: float((dl.to(F8) * (a @ b.t().contiguous())).sum())  # noqa: E731
        nu = (logits(u.to(F8) + vu, e.to(F8)) - logits(u.to(F8) - vu, e.to(F8))) / 2
        ne = (logits(u.to(F8), e.to(F8) + ve) - logits(u.to(F8), e.to(F8) - ve)) / 2
        assert abs(nu - float((du.to(F8) * vu).sum())) <= 1e-6 * float((du.to(F8) * vu).abs().sum())
        assert abs(ne - float((de.to(F8) * ve).sum())) <= 1e-6 * float((de.to(F8) * ve).abs().sum())


@pytest.mark.parametrize("T", [700, 4700])
def test_logits_on_another_stream_and_in_a_graph(T):
    dev()
    d, E = 384, 61
    dl, u, e = _operands(T, d, E)
    du_in, de_in = _rand(_gen(1), T, d), _rand(_gen(2), E, d)

    def step():
        return moe.moe_router_logits_backward(dl, u, e, du_in=du_in, de_in=de_in)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        dl.mul_(-1.5)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_binding_refusals():
    dev()
    scores, idx = _inputs(64, 16, 4)
    start = _starts([0, 64])
    r = moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start)
    dl, u, e = _operands(64, 256, 16)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    bad = [
        lambda: moe.moe_balance_loss(scores.half(), idx, ALPHA),
        lambda: moe.moe_balance_loss(scores, idx.long(), ALPHA),
        lambda: moe.moe_balance_loss(scores, idx[:60], ALPHA),
        lambda: moe.moe_balance_loss(scores.cpu(), idx, ALPHA),
        lambda: moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start.long()),
        lambda: moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start[:1]),
        lambda: moe.moe_balance_loss(scores, idx, ALPHA, seq_start=start.cpu()),
        lambda: moe.moe_balance_loss(scores[:, ::2], idx, ALPHA),
        lambda: moe.moe_balance_loss(scores.repeat(64, 1), idx.repeat(64, 1), ALPHA, ws=small),
        lambda: moe.moe_balance_loss(scores[:, :3].contiguous(), idx, ALPHA),           # K above E
        lambda: moe.moe_balance_loss(torch.zeros((4, 257), device="cuda"), idx[:4], ALPHA),
        lambda: moe.moe_balance_loss_backward(scores, r.seq_count, 0, ALPHA),
        lambda: moe.moe_balance_loss_backward(scores, r.seq_count, 17, ALPHA),
        lambda: moe.moe_balance_loss_backward(scores, r.seq_count[:, :8], 4, ALPHA),
        lambda: moe.moe_balance_loss_backward(scores, r.seq_count, 4, ALPHA, seq_start=_starts([0, 5, 64])),
        lambda: moe.moe_balance_loss_backward(scores, r.seq_count, 4, ALPHA, dloss=torch.ones(2, device="cuda")),
        lambda: moe.moe_balance_loss_backward(scores, r.seq_count, 4, ALPHA, dlogits_in=scores[:60]),
        lambda: moe.moe_router_logits_backward(dl.bfloat16(), u, e),
        lambda: moe.moe_router_logits_backward(dl, u.float(), e),
        lambda: moe.moe_router_logits_backward(dl, u[:60], e),
        lambda: moe.moe_router_logits_backward(dl, u, e[:, :128]),
        lambda: moe.moe_router_logits_backward(dl, u, e.cpu()),
        lambda: moe.moe_router_logits_backward(dl, u[:, :100].contiguous(), e[:, :100].contiguous()),
        lambda: moe.moe_router_logits_backward(dl, u, e, want_du=False, want_de=False),
        lambda: moe.moe_router_logits_backward(dl, u, e, want_du=False, du_in=u.float()),
        lambda: moe.moe_router_logits_backward(dl, u, e, want_de=False, de_in=e.float()),
        lambda: moe.moe_router_logits_backward(dl, u, e, du_in=u),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            pytest.fail(f"case {i} was taken")
