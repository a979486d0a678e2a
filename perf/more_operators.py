"""Cases of the operators that a training step of the layer uses next to its
products: the balance loss over packed sequences with its gradient, that gradient's
way through the router's logits, the SwiGLU backward from activations kept in 8 bits,
and the residual layer norm, forward and backward.  Sizes are the layer's
(d = 7168, I = 2048, top-8 of 256 experts) and small, odd and ragged ones.

Each case is computed two ways: `run` with own = False in elementary torch
operations in 32 bits (the balance loss's long sums in 64), with own = True by the
library's calls; `exact` is the definition in 64 bits.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
ALPHA = 1e-3
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------ cases

def listed():
    return [
        # A training step's batch: four sequences of 4096 tokens, loss and gradient.
        dict(name="balance_step", op="balance", T=16384, seqs=4, even=True, pad=0, E=256, K=8),
        # A small fine-tuning batch of ragged sequences, one of them empty, padding behind the last; odd E.
        dict(name="balance_ragged", op="balance", T=300, seqs=7, even=False, pad=13, E=61, K=4),
        # Documents packed into a long batch.
        dict(name="balance_packed", op="balance", T=131072, seqs=96, even=False, pad=1000, E=256, K=8),
        # The same batch's gradient through the router, added to what the experts' backward gave.
        dict(name="logits_step", op="logits", T=16384, d=7168, E=256, add=True),
        # A small model's router: odd numbers of tokens and experts, nothing to add to.
        dict(name="logits_odd", op="logits", T=1031, d=640, E=61, add=False),
        # SwiGLU backward of every routed and shared row of a training step, from z kept in 8 bits.
        dict(name="swiglu_step", op="swiglu", R=147456, I=2048),
        # The rows of one small expert.
        dict(name="swiglu_odd", op="swiglu", R=777, I=384),
        # One token's norm in front of the layer: latency alone.
        dict(name="norm_token", op="norm", T=1, d=7168, x="bf16", res="bf16", bias=True, fp8=True),
        # The batch's: outputs for the router (bf16) and the experts (FP8).
        dict(name="norm_step", op="norm", T=16384, d=7168, x="bf16", res="bf16", bias=True, fp8=True),
        # A small model's final norm in FP32, a width that no vector divides, no bias.
        dict(name="norm_odd", op="norm", T=1023, d=999, x="f32", res="none", bias=False, fp8=False),
        # The norm's backward at the layer's width with the residual stream's gradient added.
        dict(name="norm_grad", op="norm_grad", T=8192, d=7168, dy="bf16", h="bf16", dh="bf16"),
        # The backward of the odd one, FP32 throughout.
        dict(name="norm_grad_odd", op="norm_grad", T=517, d=999, dy="f32", h="f32", dh="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "logits", "swiglu", "norm", "norm_grad"))
    if op == "balance":
        E = _log(rng, 2, 256)
        T = _log(rng, 1, 131072)
        return dict(op=op, T=T, seqs=_log(rng, 1, min(T, 512)), even=rng.random() < 0.3,
                    pad=rng.choice((0, T // 10)), E=E, K=rng.randint(1, min(E, 8)))
    if op == "logits":
        return dict(op=op, T=_log(rng, 1, 16384), d=128 * _log(rng, 1, 56), E=_log(rng, 1, 256), add=rng.random() < 0.5)
    if op == "swiglu":
        return dict(op=op, R=_log(rng, 1, 147456), I=128 * _log(rng, 1, 16))
    d = _log(rng, 64, 16384)
    if op == "norm":
        fp8 = rng.random() < 0.5
        if fp8:
            d = max(128, d // 128 * 128)
        return dict(op=op, T=_log(rng, 1, min(32768, 16384 * 7168 // d)), d=d, x=rng.choice(("bf16", "f32")),
                    res=rng.choice(("bf16", "f32", "none")), bias=rng.random() < 0.7, fp8=fp8)
    return dict(op=op, T=_log(rng, 1, min(32768, 8192 * 7168 // d)), d=d, dy=rng.choice(("bf16", "f32")),
                h=rng.choice(("bf16", "f32")), dh=rng.choice(("bf16", "f32", "none")))


def work(case):
    b = {"bf16": 2, "f32": 4, "none": 0}
    if case["op"] == "balance":
        T, E, K, S = case["T"], case["E"], case["K"], case["seqs"]
        return {"bytes": 8 * T * E + 4 * T * K + S * (4 * E + 12) + 4 * E, "flops": 9 * T * E}
    if case["op"] == "logits":
        T, d, E = case["T"], case["d"], case["E"]
        add = 1 if case["add"] else 0
        return {"bytes": 4 * T * E + 2 * T * d + 2 * E * d + (4 + 4 * add) * (T * d + E * d), "flops": 4 * T * d * E}
    if case["op"] == "swiglu":
        n = case["R"] * case["I"]
        return {"bytes": n * (2 + 4 + 2) + 4 * n // 128 * 4, "flops": 16 * n}
    n = case["T"] * case["d"]
    if case["op"] == "norm":
        by = n * (b[case["x"]] + 2 * b[case["res"]] + 2) + 8 * case["d"] + 8 * case["T"]
        if case["fp8"]:       # codes and scales written, read and returned as bf16 values
            by += n * (1 + 1 + 2) + 2 * n // 128 * 4
        return {"bytes": by, "flops": 8 * n}
    dx = 2 if case["dh"] == "none" else b[case["dh"]]
    return {"bytes": n * (b[case["dy"]] + b[case["h"]] + b[case["dh"]] + dx) + 12 * case["d"] + 8 * case["T"],
            "flops": 14 * n}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, cols):
    """Normals around a mean of their own for each row, one entry in a thousand a hundred times larger."""
    x = _normal(g, rows, cols) + 0.5 * _normal(g, rows, 1) + 0.5
    big = torch.rand((rows, cols), generator=g, device="cuda") < 1e-3
    return torch.where(big, x * 100.0, x)


def _starts(case, seed):
    """The first token of each sequence, and one past the last one's last."""
    S, n = case["seqs"], case["T"] - case["pad"]
    if case["even"]:
        return (np.arange(S + 1, dtype=np.int64) * n // S).astype(np.int32)
    rng = np.random.default_rng([seed, 23])
    sizes = rng.multinomial(n, rng.dirichlet(np.full(S, 0.7)))
    if S > 2:
        sizes[0] += sizes[S // 2]
        sizes[S // 2] = 0
    return np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "balance":
        T, E, K = case["T"], case["E"], case["K"]
        # sigmoid scores with popular and unpopular experts, and the chosen ones under a small bias
        s["scores"] = torch.sigmoid(1.5 * _normal(g, T, E) + 0.7 * _normal(g, E))
        s["idx"] = torch.topk(s["scores"] + 0.05 * _normal(g, E), K, dim=1).indices.to(torch.int32)
        s["start"] = torch.from_numpy(_starts(case, seed)).cuda()
        s["dloss"] = 1.0 + 0.1 * _normal(g, case["seqs"])
    elif case["op"] == "logits":
        T, d, E = case["T"], case["d"], case["E"]
        s["dlogits"] = 1e-4 * _normal(g, T, E) * torch.exp(_normal(g, T, E))
        s["u"] = _activations(g, T, d).to(torch.bfloat16)
        s["e"] = (_normal(g, E, d) * d ** -0.5).to(torch.bfloat16)
        s["du"] = 1e-3 * _normal(g, T, d) if case["add"] else None
        s["de"] = 1e-2 * _normal(g, E, d) if case["add"] else None
    elif case["op"] == "swiglu":
        R, I = case["R"], case["I"]
        q, scale = _tiles(1.3 * _normal(g, R, 2 * I).view(R, -1, 128))
        s["zq"], s["zs"] = q.view(torch.uint8).view(R, 2 * I), scale.view(R, -1)
        s["dh"] = 1e-3 * _normal(g, R, I)
    elif case["op"] == "norm":
        T, d = case["T"], case["d"]
        s["x"] = _activations(g, T, d).to(DT[case["x"]])
        s["res"] = None if case["res"] == "none" else _activations(g, T, d).to(DT[case["res"]])
        s["w"] = 1.0 + 0.2 * _normal(g, d)
        s["b"] = 0.2 * _normal(g, d) if case["bias"] else None
    else:
        T, d = case["T"], case["d"]
        h = _activations(g, T, d).to(DT[case["h"]])
        s["h"] = h
        s["mean"] = h.double().mean(1).float()
        s["rstd"] = (1.0 / torch.sqrt(h.double().var(1, correction=0) + EPS)).float()
        s["w"] = 1.0 + 0.2 * _normal(g, d)
        s["dy"] = (_normal(g, T, d) * 1e-2).to(DT[case["dy"]])
        s["dh"] = None if case["dh"] == "none" else (_normal(g, T, d) * 1e-2).to(DT[case["dh"]])
    return s


# ------------------------------------------------------------------ plain forms

def _tiles(t):
    """E4M3 codes and FP32 scales of tiles of 128 values (the last dimension)."""
    amax = t.abs().amax(-1, keepdim=True)
    none = amax == 0
    q = (t * torch.where(none, 1.0, 448.0 / amax)).clamp(-448.0, 448.0).to(E4M3)
    return q, torch.where(none, 1.0, amax / 448.0)


def _sequence_of(start, T):
    """The sequence of each token, and whether it has one."""
    t = torch.arange(T, device=start.device)
    q = torch.searchsorted(start.long(), t, right=True) - 1
    inside = (q >= 0) & (q < start.numel() - 1)
    return q.clamp(0, start.numel() - 2), inside


def run(s):
    return (_own if own else _plain)(s)


def _plain(s):
    case = s["case"]
    if case["op"] == "balance":
        E, K, start = case["E"], case["K"], s["start"].long()
        q, inside = _sequence_of(start, case["T"])
        total = s["scores"].sum(1, keepdim=True)
        p = torch.where(total == 0, 0.0, s["scores"] / torch.where(total == 0, 1.0, total))
        chose = torch.zeros_like(s["scores"]).scatter_(1, s["idx"].long(), 1.0)
        # sums over each sequence as products with its tokens' indicator, 1024 tokens at a time
        member = ((torch.arange(case["seqs"], device=q.device) == q[:, None]) & inside[:, None]).double()
        blocks = -(-case["T"] // 1024)
        member, pc = (torch.cat((x, x.new_zeros(blocks * 1024 - case["T"], x.shape[1]))).view(blocks, 1024, -1)
                      for x in (member, torch.cat((p, chose), 1).double()))
        P, n = torch.bmm(member.transpose(1, 2).contiguous(), pc).sum(0).split(E, 1)
        length = (start[1:] - start[:-1]).double()[:, None]
        some = length.clamp_min(1.0)
        f = E * n / (K * some)
        loss = ALPHA * (f * P / some).sum(1)
        coef = (ALPHA * s["dloss"].double()[:, None] / some).float()[q]
        ft = f.float()[q]
        grad = coef * p * (1.0 - s["scores"]) * (ft - (ft * p).sum(1, keepdim=True))
        count = n.to(torch.int32)
        return {"loss": loss.float(), "seq_count": count, "expert_count": count.sum(0, dtype=torch.int32),
                "dlogits": torch.where(inside[:, None], grad, 0.0)}
    if case["op"] == "logits":
        du, de = s["dlogits"] @ s["e"].float(), s["dlogits"].t() @ s["u"].float()
        return {"du": du if s["du"] is None else s["du"] + du, "de": de if s["de"] is None else s["de"] + de}
    if case["op"] == "swiglu":
        R, I = case["R"], case["I"]
        z = (s["zq"].view(E4M3).float().view(R, -1, 128) * s["zs"][:, :, None]).view(R, I // 128, 2, 128)
        gate, up, dh = z[:, :, 0], z[:, :, 1], s["dh"].view(R, I // 128, 128)
        sg = 1.0 / (1.0 + torch.exp(-gate))
        dz = torch.stack((dh * up * sg * (1.0 + gate * (1.0 - sg)), dh * gate * sg), 2)
        q, scale = _tiles(dz)
        return {"dz": q.view(R, 2 * I), "scale": scale.view(R, -1)}
    if case["op"] == "norm":
        h = s["x"].float()
        out = {}
        if s["res"] is not None:
            h = h + s["res"].float()
            out["h"] = h.to(s["res"].dtype)
        mean = h.mean(1)
        c = h - mean[:, None]
        rstd = 1.0 / torch.sqrt(c.square().mean(1) + EPS)
        y = c * rstd[:, None] * s["w"]
        y = (y if s["b"] is None else y + s["b"]).to(torch.bfloat16)
        out.update(y=y, mean=mean, rstd=rstd)
        if case["fp8"]:
            q, scale = _tiles(y.float().view(y.shape[0], -1, 128))
            out["values"] = (q.float() * scale).view(y.shape).to(torch.bfloat16)
        return out
    dy, xh = s["dy"].float(), (s["h"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    gw = dy * s["w"]
    dx = (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(torch.bfloat16 if s["dh"] is None else s["dh"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0)}


# ------------------------------------------------------------------ the library's calls

def _own(s):
    import sigmoid_top_routing_02_amd as moe
    case = s["case"]
    if case["op"] == "balance":
        r = moe.moe_balance_loss(s["scores"], s["idx"], ALPHA, seq_start=s["start"])
        dlogits = moe.moe_balance_loss_backward(s["scores"], r.seq_count, case["K"], ALPHA, seq_start=s["start"],
                                                dloss=s["dloss"])
        return {"loss": r.loss, "seq_count": r.seq_count, "expert_count": r.expert_count, "dlogits": dlogits}
    if case["op"] == "logits":
        du, de = moe.moe_router_logits_backward(s["dlogits"], s["u"], s["e"], du_in=s["du"], de_in=s["de"])
        return {"du": du, "de": de}
    if case["op"] == "swiglu":
        q, scale = moe.moe_swiglu_backward_zq(s["zq"], s["zs"], s["dh"])
        return {"dz": q.view(E4M3), "scale": scale}
    if case["op"] == "norm":
        r = moe.moe_add_layernorm(s["x"], s["w"], EPS, bias=s["b"], residual=s["res"], quant=case["fp8"])
        out = {"y": r.y, "mean": r.mean, "rstd": r.rstd}
        if s["res"] is not None:
            out["h"] = r.h
        if case["fp8"]:
            out["values"] = moe.fp8_dequant_1x128(r.q, r.scale, dtype=torch.bfloat16)
        return out
    dx, dw, db = moe.moe_add_layernorm_backward(s["dy"], s["h"], s["w"], s["mean"], s["rstd"], dh=s["dh"],
                                                dx_dtype=torch.bfloat16 if s["dh"] is None else s["dh"].dtype)
    return {"dx": dx, "dw": dw, "db": db}


# ------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(v):
    """Rounded to E4M3 by the step of each value's binade (subnormals below 2^-6)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def exact(case, seed):
    s = prepare(case, seed)
    f8 = torch.float64
    if case["op"] == "balance":
        sc, start = s["scores"].to(f8), s["start"].tolist()
        E, K = case["E"], case["K"]
        loss, grad = [], torch.zeros_like(sc)
        for q, (a, b) in enumerate(zip(start[:-1], start[1:])):
            if a == b:
                loss.append(0.0)
                continue
            f = torch.bincount(s["idx"][a:b].long().view(-1), minlength=E).to(f8) * (E / (K * (b - a)))
            norm = sc[a:b].sum(1)
            norm = torch.where(norm == 0, torch.inf, norm)
            loss.append(ALPHA * float((f * (sc[a:b] / norm[:, None]).mean(0)).sum()))
            # d/ds of s_i / sum s, then of the sigmoid
            ds = (f - (sc[a:b] @ f / norm)[:, None]) / norm[:, None]
            grad[a:b] = ds * (sc[a:b] - sc[a:b] ** 2) * (float(s["dloss"][q]) * ALPHA / (b - a))
        return {"loss": torch.tensor(loss, dtype=f8), "seq_count": None, "expert_count": None, "dlogits": grad}
    if case["op"] == "logits":
        dl = s["dlogits"].to(f8)
        du, de = torch.mm(dl, s["e"].to(f8)), torch.mm(dl.t().contiguous(), s["u"].to(f8))
        return {"du": du + (0.0 if s["du"] is None else s["du"].to(f8)), "de": de + (0.0 if s["de"] is None else s["de"].to(f8))}
    if case["op"] == "swiglu":
        R, I = case["R"], case["I"]
        q, scale = [], []
        for a in range(0, R, 16384):
            rows = slice(a, min(R, a + 16384))
            z = s["zq"][rows].view(E4M3).to(f8) * s["zs"][rows].to(f8).repeat_interleave(128, 1)
            gate, up = z.view(-1, I // 128, 256).split(128, 2)
            dh = s["dh"][rows].to(f8).view(-1, I // 128, 128)
            sg = torch.sigmoid(gate)
            dz = torch.cat((dh * up * (sg + gate * sg * torch.sigmoid(-gate)), dh * gate * sg), 2).view(-1, 2 * I // 128, 128)
            sc = dz.abs().amax(2) / 448.0
            sc = torch.where(sc == 0, 1.0, sc)
            q.append(_e4m3(dz / sc[:, :, None]).view(-1, 2 * I))
            scale.append(sc)
        return {"dz": torch.cat(q), "scale": torch.cat(scale)}
    if case["op"] == "norm":
        h = s["x"].to(f8) + (0.0 if s["res"] is None else s["res"].to(f8))
        var, mean = torch.var_mean(h, 1, correction=0)
        y = (h - mean[:, None]) / torch.sqrt(var + EPS)[:, None] * s["w"].to(f8)
        if s["b"] is not None:
            y = y + s["b"].to(f8)
        out = {"y": y, "mean": mean, "rstd": 1.0 / torch.sqrt(var + EPS)}
        if s["res"] is not None:
            out["h"] = h
        if case["fp8"]:
            t = y.to(torch.bfloat16).to(f8).view(y.shape[0], -1, 128)
            scale = t.abs().amax(2, keepdim=True) / 448.0
            out["values"] = (_e4m3(t / torch.where(scale == 0, 1.0, scale)) * scale).view(y.shape)
        return out
    r, w, dy = s["rstd"].to(f8)[:, None], s["w"].to(f8), s["dy"].to(f8)
    c = s["h"].to(f8) - s["mean"].to(f8)[:, None]
    d = case["d"]
    dx = r * (dy * w - (dy @ w)[:, None] / d) - r ** 3 * c * ((dy * c) @ w)[:, None] / d
    return {"dx": dx if s["dh"] is None else dx + s["dh"].to(f8), "dw": (dy * c * r).sum(0), "db": dy.sum(0)}
