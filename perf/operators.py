"""Cases of the residual + RMS norm (forward with an FP8 copy, backward), the
MXFP4 quantiser and the MXFP4 product grouped by expert, at the sizes of the
layer this library serves (d = 7168, I = 2048, top-8 of 256 experts, 32 of them
on one GPU) and at small, odd and ragged ones.

Each case is computed two ways: `run` with own = False in elementary torch
operations in 32 bits, with own = True by the library's calls; `exact` is the
definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # One token being decoded: the norm before a layer, latency alone.
        dict(name="norm_token", op="norm", T=1, d=7168, x="bf16", res="bf16", fp8=True),
        # A prompt of 16384 tokens: the norm's two outputs for router and FP8 experts.
        dict(name="norm_prompt", op="norm", T=16384, d=7168, x="bf16", res="bf16", fp8=True),
        # A width that no vector divides, FP32 rows and no residual: a small model's final norm.
        dict(name="norm_odd", op="norm", T=1023, d=999, x="f32", res="none", fp8=False),
        # A training step's backward at the layer's width, gradient of the residual stream added.
        dict(name="norm_grad", op="norm_grad", T=8192, d=7168, dy="bf16", h="bf16", dh="bf16"),
        # The backward of the odd one, FP32 throughout, no gradient of the stream.
        dict(name="norm_grad_odd", op="norm_grad", T=517, d=999, dy="f32", h="f32", dh="none"),
        # The activations of a decode step of 256 tokens.
        dict(name="quant_decode", op="quant", rows=256, cols=7168, x="bf16"),
        # FP32 masters of eight experts' gate and up projections.
        dict(name="quant_weights", op="quant", rows=32768, cols=7168, x="f32"),
        # One token: eight experts with one row each, gate and up projections.
        dict(name="mx_token", op="mx", G=32, busy=8, T=1, M=8, N=4096, K=7168, epi="swiglu", skew=0.0),
        # A decode step: 256 tokens' rows on this GPU's 32 experts, about eight each.
        dict(name="mx_decode", op="mx", G=32, busy=32, T=256, M=256, N=4096, K=7168, epi="swiglu", skew=0.0),
        # A prompt: 16384 rows, the busiest expert with about four times the mean.
        dict(name="mx_prompt", op="mx", G=32, busy=32, T=16384, M=16384, N=4096, K=7168, epi="swiglu", skew=1.1),
        # The benchmark's dense product, one group.
        dict(name="mx_dense", op="mx", G=1, busy=1, T=8192, M=8192, N=7168, K=16384, epi="f32", skew=0.0),
        # Ragged rows, two empty groups, an N that no tile divides, K of 33 blocks of 32.
        dict(name="mx_odd", op="mx", G=7, busy=5, T=300, M=777, N=1000, K=1056, epi="bf16", skew=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm_grad", "quant", "mx", "mx"))
    if op == "norm":
        d = _log(rng, 64, 16384)
        fp8 = rng.random() < 0.5
        if fp8:
            d = max(128, d // 128 * 128)
        T = _log(rng, 1, min(32768, 16384 * 7168 // d))
        return dict(op=op, T=T, d=d, x=rng.choice(("bf16", "f32")), res=rng.choice(("bf16", "f32", "none")), fp8=fp8)
    if op == "norm_grad":
        d = _log(rng, 64, 16384)
        T = _log(rng, 1, min(32768, 8192 * 7168 // d))
        return dict(op=op, T=T, d=d, dy=rng.choice(("bf16", "f32")), h=rng.choice(("bf16", "f32")),
                    dh=rng.choice(("bf16", "f32", "none")))
    if op == "quant":
        cols = 32 * _log(rng, 1, 512)
        return dict(op=op, rows=_log(rng, 1, min(65536, 32768 * 7168 // cols)), cols=cols, x=rng.choice(("bf16", "f32")))
    epi = rng.choice(("f32", "bf16", "swiglu"))
    N = _log(rng, 16, 7168)
    if epi == "swiglu":
        N = max(256, N // 256 * 256)
    K = 32 * _log(rng, 1, 512)
    G = _log(rng, 1, min(48, max(1, 32 * 4096 * 7168 // (N * K))))
    M = _log(rng, 1, min(16384, int(8192 * 7168 * 16384 / (N * K))))
    busy = rng.randint(1, min(G, M))
    return dict(op=op, G=G, busy=busy, T=max(1, min(M, rng.choice((M, M // 2 + 1)))), M=M, N=N, K=K, epi=epi,
                skew=round(rng.uniform(0.0, 1.2), 2))


def work(case):
    b = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "norm":
        n = case["T"] * case["d"]
        res = b[case["res"]]
        by = n * (b[case["x"]] + 2 * res + 2) + 4 * case["d"] + 4 * case["T"]
        if case["fp8"]:       # codes and scales written, read and returned as bf16 values
            by += n * (1 + 1 + 2) + 2 * n // 128 * 4
        return {"bytes": by, "flops": 6 * n}
    if case["op"] == "norm_grad":
        n = case["T"] * case["d"]
        dx = 2 if case["dh"] == "none" else b[case["dh"]]
        return {"bytes": n * (b[case["dy"]] + b[case["h"]] + b[case["dh"]] + dx) + 8 * case["d"] + 4 * case["T"],
                "flops": 10 * n}
    if case["op"] == "quant":
        n = case["rows"] * case["cols"]
        return {"bytes": n * 2 * b[case["x"]] + 2 * (n // 2 + n // 32), "flops": 4 * n}
    M, N, K = case["M"], case["N"], case["K"]
    mx = K // 2 + K // 32     # bytes of a row of codes and scales
    out = {"f32": 4 * N, "bf16": 2 * N, "swiglu": N}[case["epi"]]
    return {"bytes": case["busy"] * N * mx + min(case["T"], M) * mx + M * (out + 4), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Unit normals with one entry in a thousand a hundred times larger."""
    x = _normal(g, rows, cols)
    big = torch.rand((rows, cols), generator=g, device="cuda") < 1e-3
    return torch.where(big, x * 100.0, x)


def _group_sizes(case, seed):
    """Rows of each group: `busy` groups, one row each at least, the others by a
    power law of exponent `skew` over the groups in a random order."""
    rng = np.random.default_rng([seed, 17])
    G, busy, M = case["G"], case["busy"], case["M"]
    chosen = rng.permutation(G)[:busy]
    p = (np.arange(busy) + 4.0) ** -case["skew"]
    sizes = np.zeros(G, np.int64)
    sizes[chosen] = 1 + rng.multinomial(M - busy, p / p.sum())
    return sizes


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "norm":
        T, d = case["T"], case["d"]
        s["x"] = _activations(g, T, d).to(DT[case["x"]])
        s["res"] = None if case["res"] == "none" else _activations(g, T, d).to(DT[case["res"]])
        s["w"] = 1.0 + 0.2 * _normal(g, d)
    elif case["op"] == "norm_grad":
        T, d = case["T"], case["d"]
        h = _activations(g, T, d).to(DT[case["h"]])
        s["h"] = h
        s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
        s["w"] = 1.0 + 0.2 * _normal(g, d)
        s["dy"] = (_normal(g, T, d) * 1e-2).to(DT[case["dy"]])
        s["dh"] = None if case["dh"] == "none" else (_normal(g, T, d) * 1e-2).to(DT[case["dh"]])
    elif case["op"] == "quant":
        x = _activations(g, case["rows"], case["cols"])
        s["x"] = (x * case["cols"] ** -0.5 if case["x"] == "f32" else x).to(DT[case["x"]])
    else:
        G, N, K, T, M = (case[k] for k in ("G", "N", "K", "T", "M"))
        s["aq"], s["as"] = _quantise(_activations(g, T, K))
        s["bq"] = torch.empty((G, N, K // 2), dtype=torch.uint8, device="cuda")
        s["bs"] = torch.empty((G, N, K // 32), dtype=torch.uint8, device="cuda")
        for i in range(G):
            s["bq"][i], s["bs"][i] = _quantise(_normal(g, N, K) * K ** -0.5)
        s["sizes"] = _group_sizes(case, seed).tolist()
        off = np.concatenate([[0], np.cumsum(s["sizes"])]).astype(np.int32)
        s["off"] = torch.from_numpy(off).cuda()
        s["idx"] = torch.randint(0, T, (M,), generator=g, device="cuda", dtype=torch.int32)
    return s


# ------------------------------------------------------------------ MXFP4 in elementary operations

def _exponent(amax):
    """floor(log2(amax)) - 2, held in an E8M0 byte's range (bias 127)."""
    _, e = torch.frexp(amax)               # amax = m 2^e, 1/2 <= m < 1
    return torch.where(amax == 0, -127, (e - 3).clamp(-127, 125))


def _codes(x):
    """(4-bit codes one to a byte [rows, cols], exponents [rows, cols/32]) of FP32 rows."""
    rows, cols = x.shape
    t = x.view(rows, cols // 32, 32)
    e = _exponent(t.abs().amax(2))
    v = torch.ldexp(t, -e[:, :, None])
    a = v.abs()
    c = torch.zeros_like(a, dtype=torch.uint8)
    for at, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        c += (a >= at) if tie_up else (a > at)
    return (c + 8 * torch.signbit(v)).view(rows, cols), e


def _quantise(x):
    c, e = _codes(x)
    return (c[:, 0::2] | (c[:, 1::2] << 4)).to(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, e, dtype):
    """The values of codes [.., cols] (one to a byte) under exponents [.., cols/32]."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=codes.device)
    v = lut[codes.int()]
    return torch.ldexp(v.view(*e.shape, 32), e[..., None]).view(v.shape)


def _unpacked(q, s, dtype):
    """The values of packed codes [rows, cols/2] and E8M0 bytes [rows, cols/32]."""
    c = torch.stack((q & 15, q >> 4), -1).flatten(-2)
    return _values(c, s.int() - 127, dtype)


# ------------------------------------------------------------------ one pass

def run(s):
    return (_own if own else _plain)(s)


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        h = s["x"].float()
        out = {}
        if s["res"] is not None:
            h = h + s["res"].float()
            out["h"] = h.to(s["res"].dtype)
        r = torch.rsqrt(h.square().mean(1) + EPS)
        y = (h * r[:, None] * s["w"]).to(torch.bfloat16)
        out.update(y=y, rstd=r)
        if case["fp8"]:
            t = y.float().view(y.shape[0], -1, 128)
            amax = t.abs().amax(2, keepdim=True)
            inv = torch.where(amax == 0, 1.0, 448.0 / amax)
            scale = torch.where(amax == 0, 1.0, amax / 448.0)
            q = (t * inv).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
            out["values"] = (q.float() * scale).view(y.shape).to(torch.bfloat16)
        return out
    if case["op"] == "norm_grad":
        dy, xh = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        gw = dy * s["w"]
        dx = (gw - xh * (gw * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["dh"] is not None:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(torch.bfloat16 if s["dh"] is None else s["dh"].dtype), "dw": (dy * xh).sum(0)}
    if case["op"] == "quant":
        c, e = _codes(s["x"].float())
        return {"values": _values(c, e, torch.float32).to(s["x"].dtype), "scale": (e + 127).to(torch.uint8)}
    # One matrix product per expert: the groups are ragged, and a product over
    # padded groups would multiply several times the rows.
    a = _unpacked(s["aq"], s["as"], torch.float32)[s["idx"].long()]
    outs, m = [], 0
    for i, n in enumerate(s["sizes"]):
        if n:
            outs.append(a[m:m + n] @ _unpacked(s["bq"][i], s["bs"][i], torch.float32).t())
            m += n
    c = torch.cat(outs)
    if case["epi"] == "swiglu":
        t = c.view(c.shape[0], -1, 2, 128)
        gate, up = t[:, :, 0], t[:, :, 1]
        c = (gate / (1.0 + torch.exp(-gate)) * up).reshape(c.shape[0], -1)
    return c if case["epi"] == "f32" else c.to(torch.bfloat16)


def _own(s):
    import sigmoid_top_routing_02_amd as moe
    case = s["case"]
    if case["op"] == "norm":
        r = moe.moe_add_rmsnorm(s["x"], s["w"], EPS, residual=s["res"], quant=case["fp8"])
        out = {"y": r.y, "rstd": r.rstd}
        if s["res"] is not None:
            out["h"] = r.h
        if case["fp8"]:
            out["values"] = moe.fp8_dequant_1x128(r.q, r.scale, dtype=torch.bfloat16)
        return out
    if case["op"] == "norm_grad":
        dx, dw = moe.moe_add_rmsnorm_backward(s["dy"], s["h"], s["w"], s["rstd"], dh=s["dh"],
                                              dx_dtype=torch.bfloat16 if s["dh"] is None else s["dh"].dtype)
        return {"dx": dx, "dw": dw}
    if case["op"] == "quant":
        q, scale = moe.mxfp4_quant_1x32(s["x"])
        return {"values": moe.mxfp4_dequant_1x32(q, scale, dtype=s["x"].dtype), "scale": scale}
    epi = {"f32": moe.MOE_MX_STORE_F32, "bf16": moe.MOE_MX_STORE_BF16, "swiglu": moe.MOE_MX_SWIGLU_BF16}[case["epi"]]
    return moe.grouped_gemm_mxfp4(s["aq"], s["as"], s["off"], case["M"], s["bq"], s["bs"], epi=epi, a_row_index=s["idx"])


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(f8) + (0.0 if s["res"] is None else s["res"].to(f8))
        ms = (h * h).sum(1) / case["d"]
        y = h / torch.sqrt(ms + EPS)[:, None] * s["w"].to(f8)
        out = {"y": y, "rstd": 1.0 / torch.sqrt(ms + EPS)}
        if s["res"] is not None:
            out["h"] = h
        if case["fp8"]:
            # E4M3 rounding by the step of each value's binade (subnormals below 2^-6)
            t = y.to(torch.bfloat16).to(f8).view(y.shape[0], -1, 128)
            scale = t.abs().amax(2, keepdim=True) / 448.0
            v = t / torch.where(scale == 0, 1.0, scale)
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
            out["values"] = (torch.round(v / step) * step * scale).view(y.shape)
        return out
    if case["op"] == "norm_grad":
        h, r, w, dy = s["h"].to(f8), s["rstd"].to(f8)[:, None], s["w"].to(f8), s["dy"].to(f8)
        dot = (dy * w * h).sum(1, keepdim=True)
        dx = r * dy * w - r ** 3 * h * dot / case["d"]
        return {"dx": dx if s["dh"] is None else dx + s["dh"].to(f8), "dw": torch.einsum("td,td->d", dy, h * r)}
    if case["op"] == "quant":
        t = s["x"].to(f8).view(case["rows"], -1, 32)
        e = torch.floor(torch.log2(t.abs().amax(2, keepdim=True).clamp_min(2.0 ** -125))) - 2
        v = t * torch.exp2(-e)
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).to(f8)
        v = (torch.round(v / step) * step).clamp(-6.0, 6.0)
        return {"values": (v * torch.exp2(e)).view(case["rows"], -1), "scale": None}
    a = _unpacked(s["aq"], s["as"], f8)
    outs, m = [], 0
    for i, n in enumerate(s["sizes"]):
        rows = s["idx"][m:m + n].long()
        m += n
        c = a.index_select(0, rows) @ _unpacked(s["bq"][i], s["bs"][i], f8).t()
        if case["epi"] == "swiglu":
            t = c.view(n, case["N"] // 256, 256)
            c = (torch.nn.functional.silu(t[:, :, :128]) * t[:, :, 128:]).reshape(n, case["N"] // 2)
        outs.append(c)
    return torch.cat(outs)
