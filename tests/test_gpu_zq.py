"""Activations kept in 8 bits: the expert product that writes z's codes, and the
SwiGLU backward and weight gradients that read them.

What is kept is fp8_quant_1x128 of the FP32 z, bit for bit, and the backward of the
kept z is the FP32 path's backward of the values that the codes stand for, bit for
bit: those comparisons need no tolerance.  Against the formula in 64 bits a code may
be half an E4M3 step off (relative 2^-4, or half a subnormal step 2^-10 of the scale),
besides FP32 arithmetic (1e-5 of the terms' size covers the exponential)."""
import numpy as np
import pytest
import torch

import sigmoid_top_routing_02_amd as moe
from helpers import dev, say

pytestmark = pytest.mark.gpu

F8 = torch.float64


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rand(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device="cuda")


def _operands(sizes, N, K, T=None, seed=0):
    g = _gen(seed)
    M, G = sum(sizes), len(sizes)
    a = _rand(g, T or M, K)
    a[torch.rand(a.shape, generator=g, device="cuda") < 1e-3] *= 100.0
    aq, a_s = moe.fp8_quant_1x128(a)
    bq, bs = moe.fp8_quant_128x128(_rand(g, G * N, K) * K ** -0.5)
    idx = None if T is None else torch.randint(0, T, (M,), generator=g, device="cuda", dtype=torch.int32)
    return aq, a_s, _offsets(sizes), bq.view(G, N, K), bs.view(G, N // 128, K // 128), idx


# 32-row tiles (few rows to a group), 128-row tiles, the shapes that the FP32 forms take through the ring kernel
@pytest.mark.parametrize("sizes,N,K,T", [
    ([1], 256, 128, None), ([3, 0, 5, 1], 512, 256, None), ([31, 32, 33, 64], 768, 384, 40),
    ([0, 0, 17], 256, 2048, None), ([200, 129, 0, 128, 1], 512, 640, 300), ([300, 127], 256, 128, None),
    ([1000], 1024, 2304, None), ([400, 700, 1], 512, 1024, 256), ([5] * 40, 256, 896, 64),
    ([700, 2, 0, 900], 4096, 7168, 512),
])
def test_product_keeps_z(sizes, N, K, T):
    dev()
    say(f"  sizes={sizes[:8]} N={N} K={K}")
    aq, a_s, off, bq, bs, idx = _operands(sizes, N, K, T)
    M = sum(sizes)
    hq, hs, zq, zs = moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, M, bq, bs, a_row_index=idx)
    fq, fs, z = moe.grouped_gemm_fp8_blockscaled(aq, a_s, off, M, bq, bs, epi=moe.MOE_EPI_SWIGLU_QUANT_Z, a_row_index=idx)
    q, s = moe.fp8_quant_1x128(z)
    torch.cuda.synchronize()
    assert torch.equal(hq, fq) and torch.equal(hs, fs)
    assert torch.equal(zq, q) and torch.equal(zs, s)


def test_product_many_tiles_and_repeats():
    """Several tiles to a CU, so that tiles hand over to each other; the same call gives the same bits."""
    dev()
    g = np.random.default_rng(3)
    sizes = g.integers(0, 900, 40).tolist()
    aq, a_s, off, bq, bs, idx = _operands(sizes, 1024, 384, 1000)
    M = sum(sizes)
    a = moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, M, bq, bs, a_row_index=idx)
    b = moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, M, bq, bs, a_row_index=idx)
    z = moe.grouped_gemm_fp8_blockscaled(aq, a_s, off, M, bq, bs, epi=moe.MOE_EPI_SWIGLU_QUANT_Z, a_row_index=idx)
    q, s = moe.fp8_quant_1x128(z[2])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert torch.equal(a[0], z[0]) and torch.equal(a[1], z[1]) and torch.equal(a[2], q) and torch.equal(a[3], s)


@pytest.mark.parametrize("M", [40, 300])
def test_product_special_values(M):
    """NaN, infinities, zeros and the largest and smallest values in z: the codes that the quantiser gives them."""
    dev()
    aq, a_s, off, bq, bs, _ = _operands([M], 512, 384)
    a_s[3, 1], a_s[4, 0], a_s[5], a_s[6], a_s[7] = float("nan"), float("inf"), 3e38, 1e-38, 0.0
    bs[0, 3, 2] = -float("inf")                       # gate and up columns 384 to 511, of every row
    aq[8, 130], aq[9, 5], aq[10] = 0x7F, 0xFF, 0x80
    hq, hs, zq, zs = moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, M, bq, bs)
    fq, fs, z = moe.grouped_gemm_fp8_blockscaled(aq, a_s, off, M, bq, bs, epi=moe.MOE_EPI_SWIGLU_QUANT_Z)
    q, s = moe.fp8_quant_1x128(z)
    torch.cuda.synchronize()
    assert torch.isnan(z[3]).all() and torch.isinf(z[4, :384]).any() and torch.isnan(z[8, :384]).all() and torch.isfinite(z[11, :384]).all()
    assert torch.equal(zs.view(torch.int32), s.view(torch.int32)) and torch.equal(zq, q)
    assert torch.equal(hs.view(torch.int32), fs.view(torch.int32)) and torch.equal(hq, fq)


def test_product_leaves_other_rows():
    """Rows behind the last group's are not written; no rows at all is a call that does nothing."""
    dev()
    aq, a_s, off, bq, bs, _ = _operands([40, 30], 256, 256)
    rows = 70
    full = [torch.full((rows + 9, c), 7, dtype=t, device="cuda") for c, t in
            ((128, torch.uint8), (1, torch.float32), (256, torch.uint8), (2, torch.float32))]
    outs = [t[:rows] for t in full]
    moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, rows, bq, bs, h_q=outs[0], h_scale=outs[1], z_q=outs[2], z_scale=outs[3])
    torch.cuda.synchronize()
    assert all((t[rows:] == 7).all() for t in full) and not (outs[2] == 7).all()
    none = moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, _offsets([0, 0]), 0, bq, bs)
    assert [tuple(t.shape) for t in none] == [(0, 128), (0, 1), (0, 256), (0, 2)]


def _kept(R, I, seed=0, scale=1.3):
    g = _gen(seed)
    zq, zs = moe.fp8_quant_1x128(scale * _rand(g, R, 2 * I))
    return zq, zs, 1e-3 * _rand(g, R, I)


@pytest.mark.parametrize("R,I", [(1, 128), (2, 384), (7, 1024), (129, 256), (777, 384), (1000, 2048), (40001, 128),
                                 (3, 65536), (33000, 2048)])
def test_swiglu_backward(R, I):
    dev()
    say(f"  R={R} I={I}")
    zq, zs, dh = _kept(R, I, seed=R)
    q, s = moe.moe_swiglu_backward_zq(zq, zs, dh)
    z = moe.fp8_dequant_1x128(zq, zs, dtype=torch.float32)
    fq, fs = moe.moe_swiglu_backward(z, dh)
    torch.cuda.synchronize()
    assert torch.equal(q, fq) and torch.equal(s, fs)
    if R * I > 1 << 22:
        return
    zz = z.to(F8).view(R, I // 128, 2, 128)
    gate, up, g = zz[:, :, 0], zz[:, :, 1], dh.to(F8).view(R, I // 128, 128)
    sg = torch.sigmoid(gate)
    want = torch.stack((g * up * sg * (1 + gate * (1 - sg)), g * gate * sg), 2)
    size = torch.stack(((g * up).abs() * sg * (1 + gate.abs() * (1 - sg)), (g * gate).abs() * sg), 2)
    sc = s.to(F8).view(R, I // 128, 2, 1)
    top = want.abs().amax(3, keepdim=True)
    assert ((sc * 448.0 - top).abs() <= 1e-5 * size.amax(3, keepdim=True) + 2.0 ** -23 * top)[top > 0].all()
    got = q.view(torch.float8_e4m3fn).to(F8).view_as(want) * sc
    assert ((got - want).abs() <= torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * sc) * (1 + 1e-5) + 1e-5 * size).all()


def test_swiglu_backward_odd_values():
    """Tiles of zeros, gates that saturate either way, codes of NaN, tiny and huge scales."""
    dev()
    R, I = 12, 256
    zq, zs, dh = _kept(R, I)
    zq[0] = 0
    dh[1] = 0.0
    zs[2] *= 100.0          # gates of hundreds: the sigmoid is 0 or 1
    zq[3, 5], zq[4, 130] = 0x7F, 0xFF
    zs[5], zs[6] = 1e-38, 1e30
    dh[7, 3], dh[8, 4] = float("nan"), float("inf")
    q, s = moe.moe_swiglu_backward_zq(zq, zs, dh)
    fq, fs = moe.moe_swiglu_backward(moe.fp8_dequant_1x128(zq, zs, dtype=torch.float32), dh)
    torch.cuda.synchronize()
    nan = lambda t: (t & 0x7F) == 0x7F  # noqa: E731  (a NaN's sign is not fixed)
    assert torch.equal(nan(q), nan(fq)) and torch.equal(q[~nan(q)], fq[~nan(q)])
    assert torch.equal(s.view(torch.int32), fs.view(torch.int32))
    v = q.view(torch.float8_e4m3fn).float()
    assert (v[0] == 0).all() and (v[1] == 0).all() and torch.isfinite(v[2]).all()
    assert torch.isnan(v[3, 5]) and torch.isnan(v[3, 133]) and not torch.isnan(v[3, :5]).any()


def test_swiglu_backward_in_place_and_no_rows():
    dev()
    zq, zs, dh = _kept(500, 384)
    want = moe.moe_swiglu_backward_zq(zq, zs, dh)
    a, b = zq.clone(), zs.clone()
    got = moe.moe_swiglu_backward_zq(a, b, dh, dz_q=a, dz_scale=b)
    torch.cuda.synchronize()
    assert got[0] is a and torch.equal(a, want[0]) and torch.equal(b, want[1])
    q, s = moe.moe_swiglu_backward_zq(zq[:0], zs[:0], dh[:0])
    assert q.shape == (0, 768) and s.shape == (0, 6)


def test_swiglu_backward_past_32_bit_offsets():
    """More than 2^32 bytes of z: the last rows are the last rows' own."""
    dev()
    R, I = (1 << 32) // (2 * 16384) + 3, 16384
    say(f"  R={R} I={I}")
    zq = torch.zeros((R, 2 * I), dtype=torch.uint8, device="cuda")
    zs = torch.ones((R, 2 * I // 128), device="cuda")
    dh = torch.zeros((R, I), device="cuda")
    zq[-4:], zs[-4:], dh[-4:] = _kept(4, I)
    q, s = moe.moe_swiglu_backward_zq(zq, zs, dh)
    want = moe.moe_swiglu_backward_zq(zq[-4:].contiguous(), zs[-4:].contiguous(), dh[-4:].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(q[-4:], want[0]) and torch.equal(s[-4:], want[1])
    assert int(q[:-4].max()) == 0


def _routing(T, K, E, seed=0):
    g = np.random.default_rng(seed)
    idx = np.stack([g.permutation(E)[:K] for _ in range(T)]).astype(np.int32)
    idx[idx == 1] = 2 if K == 1 else idx[idx == 1]
    count, go, row_token, slot_row = moe.moe_dispatch(torch.from_numpy(idx).cuda(), E, include_shared=True)
    return go, row_token, slot_row


@pytest.mark.parametrize("T,K,E,d,I", [(300, 2, 6, 256, 128), (5, 1, 4, 128, 384), (1000, 4, 9, 640, 256)])
def test_weight_gradients(T, K, E, d, I):
    """moe_wgrad_zq equals moe_wgrad of the values that the codes stand for, operands and gradients."""
    dev()
    say(f"  T={T} K={K} E={E} d={d} I={I}")
    go, row_token, slot_row = _routing(T, K, E)
    R = T * K + T
    g = _gen(T)
    zq, zs, dh_row = _kept(R, I)
    dh, gate, u = _rand(g, T, d), torch.rand((T, K), generator=g, device="cuda"), _rand(g, T, d).bfloat16()
    a13, a2, abufs, akb = moe.moe_wgrad_zq(dh, gate, slot_row, row_token, zq, zs, dh_row, u, go, shared_row0=T * K)
    z = moe.fp8_dequant_1x128(zq, zs, dtype=torch.float32)
    b13, b2, bbufs, bkb = moe.moe_wgrad(dh, gate, slot_row, row_token, z, dh_row, u, go, shared_row0=T * K)
    torch.cuda.synchronize()
    assert torch.equal(a13, b13) and torch.equal(a2, b2) and torch.equal(akb, bkb)
    n = int(akb[-1])
    assert torch.equal(abufs["hT_q"][:I * 128 * n], bbufs["hT_q"][:I * 128 * n])
    assert torch.equal(abufs["dzT_q"][:2 * I * 128 * n], bbufs["dzT_q"][:2 * I * 128 * n])
    assert torch.equal(abufs["dzT_s"][:2 * I * n], bbufs["dzT_s"][:2 * I * n])


def test_gradient_against_differences():
    """dz's values against central differences of <dh, h(z)> in 64 bits, within its codes' half steps."""
    dev()
    R, I = 6, 256
    zq, zs, dh = _kept(R, I)
    q, s = moe.moe_swiglu_backward_zq(zq, zs, dh)
    grad = moe.fp8_dequant_1x128(q, s, dtype=torch.float32).to(F8)
    z = moe.fp8_dequant_1x128(zq, zs, dtype=torch.float32).to(F8)

    def loss(z_):
        t = z_.view(R, I // 128, 2, 128)
        return float((dh.to(F8) * (t[:, :, 0] * torch.sigmoid(t[:, :, 0]) * t[:, :, 1]).reshape(R, I)).sum())

    g, step = _gen(2), 1e-5
    half = torch.maximum(grad.abs() * 2.0 ** -4 / (1 - 2.0 ** -4), s.to(F8).repeat_interleave(128, 1) * 2.0 ** -10)
    for _ in range(4):
        v = _rand(g, R, 2 * I).to(F8)
        n = (loss(z + step * v) - loss(z - step * v)) / (2 * step)
        assert abs(n - float((grad * v).sum())) <= float((half * v.abs()).sum())


def test_on_another_stream_and_in_a_graph():
    dev()
    sizes = [100, 0, 61, 200]
    aq, a_s, off, bq, bs, idx = _operands(sizes, 512, 256, 90)
    M = sum(sizes)
    dh = 1e-3 * _rand(_gen(4), M, 256)

    def step():
        r = moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, M, bq, bs, a_row_index=idx)
        return (*r, *moe.moe_swiglu_backward_zq(r[2], r[3], dh))

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
        a_s.mul_(1.5)
        dh.mul_(-0.7)
        graph.replay()
        torch.cuda.synchronize()
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, eager)), i


def test_binding_refusals():
    dev()
    aq, a_s, off, bq, bs, _ = _operands([40, 30], 256, 256)
    zq, zs, dh = _kept(70, 128)
    bad = [
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, 71, bq, bs),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq.float(), a_s, off, 70, bq, bs),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off[:2], 70, bq, bs),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off.long(), 70, bq, bs),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, 70, bq, bs, a_row_index=off[:2]),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, 70, bq[:, :128].contiguous(), bs[:, :1].contiguous()),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, 70, bq, bs.cpu()),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, 70, bq, bs, z_q=zq[:69]),
        lambda: moe.grouped_gemm_fp8_swiglu_zq(aq, a_s, off, 70, bq, bs, ws=torch.empty(64, dtype=torch.uint8, device="cuda")),
        lambda: moe.moe_swiglu_backward_zq(zq[:, :200], zs, dh),
        lambda: moe.moe_swiglu_backward_zq(zq, zs[:, :1], dh),
        lambda: moe.moe_swiglu_backward_zq(zq, zs, dh.bfloat16()),
        lambda: moe.moe_swiglu_backward_zq(zq, zs, dh[:69]),
        lambda: moe.moe_swiglu_backward_zq(zq.cpu(), zs.cpu(), dh.cpu()),
        lambda: moe.moe_swiglu_backward_zq(zq, zs, dh, dz_q=zq[:1]),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(moe.MoEError):
            f()
            pytest.fail(f"case {i} was taken")
