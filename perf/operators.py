"""Cases of the operators around the latent MoE layer: the block's RMSNorm, dense linear layers
with a fused epilogue, and the whole layer for a few tokens.

  norm          total = x + residual;  y = gamma * total / sqrt(mean(total^2) + eps), as bf16 or as
                e4m3 codes with one fp32 scale per row (s = amax / 448, code = e4m3(y / s))
  norm_bwd      gradients of that: dx (which x and the residual share) and dgamma
  linear        y = act(x W^T + bias) + residual, bf16 or e4m3 operands (per-row scales);
                act: none, silu, gelu, or situ, the layer's gated activation over 2N rows of W
  linear_bwd    dx, dW and dbias of it
  few           the Stable Latent MoE layer on at most 8 tokens, routed against given thresholds

``own`` chooses who computes: False, plain torch operations in fp32 (below); True, the framework.
"""
import math

import torch

own = False

BF = torch.bfloat16
E4M3 = torch.float8_e4m3fn
EPS = 1e-6
CAP = 100.0  # SiTU-GLU cap

# the layer's sizes: hidden d, latent L, E routed experts of which K per token, routed width I,
# S shared experts of width Is
LAYERS = {
    "k3": dict(d=7168, L=3584, E=896, K=16, I=512, S=2, Is=2048),
    "pool448": dict(d=7168, L=3584, E=448, K=8, I=512, S=2, Is=2048),
    "e64": dict(d=7168, L=3584, E=64, K=4, I=512, S=2, Is=2048),
    "mid": dict(d=1024, L=512, E=64, K=8, I=256, S=2, Is=512),
}


def listed():
    return [
        # one token's hidden state at decode: latency
        {"name": "norm_1", "op": "norm", "rows": 1, "cols": 7168, "fp8": False},
        # a prefill batch, a row short of whole, quantised for an e4m3 linear layer
        {"name": "norm_e4m3_8191", "op": "norm", "rows": 8191, "cols": 7168, "fp8": True},
        # the same block's norm in a training step
        {"name": "norm_bwd_8192", "op": "norm_bwd", "rows": 8192, "cols": 7168},
        # a dense feed-forward's down-projection with bias and residual, two tokens at decode
        {"name": "linear_2", "op": "linear", "M": 2, "N": 7168, "K": 4096, "act": "none",
         "bias": True, "resid": True, "fp8": False},
        # a small mixed batch through a projection into the latent width
        {"name": "linear_77", "op": "linear", "M": 77, "N": 3584, "K": 7168, "act": "gelu",
         "bias": True, "resid": False, "fp8": False},
        # a dense feed-forward's gate/value projection at prefill
        {"name": "linear_situ_8192", "op": "linear", "M": 8192, "N": 4096, "K": 7168,
         "act": "situ", "bias": False, "resid": False, "fp8": False},
        # its e4m3 down-projection for a prefill chunk
        {"name": "linear_e4m3_2048", "op": "linear", "M": 2048, "N": 7168, "K": 4096,
         "act": "none", "bias": False, "resid": True, "fp8": True},
        # a training step of the gated projection, gradients in the weights' type
        {"name": "linear_bwd_4096", "op": "linear_bwd", "M": 4096, "N": 4096, "K": 7168,
         "act": "situ", "bias": True, "dw": "bf16"},
        # a ragged micro-batch through a plain projection, fp32 weight gradient
        {"name": "linear_bwd_333", "op": "linear_bwd", "M": 333, "N": 3584, "K": 7168,
         "act": "none", "bias": True, "dw": "fp32"},
        # decode: one stream, eight streams, and four with e4m3 experts
        {"name": "few_1", "op": "few", "layer": "k3", "T": 1, "fp8": False},
        {"name": "few_8", "op": "few", "layer": "k3", "T": 8, "fp8": False},
        {"name": "few_e4m3_4", "op": "few", "layer": "k3", "T": 4, "fp8": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("norm", "norm_bwd", "linear", "linear", "linear_bwd", "few"))
    if op in ("norm", "norm_bwd"):
        c = {"op": op, "rows": _log(rng, 1, 8192), "cols": _log(rng, 256, 7168, 16)}
        if op == "norm":
            c["fp8"] = rng.random() < 0.5
        return c
    if op == "few":
        layer = rng.choice(tuple(LAYERS))
        return {"op": op, "layer": layer, "T": rng.randint(1, 8), "fp8": rng.random() < 0.3}
    act = rng.choice(("none", "silu", "gelu", "situ"))
    c = {"op": op, "M": _log(rng, 1, 8192 if op == "linear" else 4096),
         "N": _log(rng, 128, 4096 if act == "situ" else 7168, 16),
         "K": _log(rng, 128, 7168, 16), "act": act, "bias": rng.random() < 0.5}
    if op == "linear":
        c["resid"] = rng.random() < 0.5
        c["fp8"] = rng.random() < 0.35
    else:
        c["dw"] = "fp32" if act == "none" else "bf16"
    return c


# ------------------------------------------------------------------------------------ inputs
class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)

    def normal(self, *shape, std=1.0, dtype=BF):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=self.g)
        return t if std == 1.0 else t.mul_(std)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=self.g)


def _codes(x):
    """e4m3 codes (one byte) and fp32 row scales of x [..., rows, cols]; both divisions are
    fp32's own (a division by a number would multiply by its rounded inverse)."""
    v = x.float()
    s = v.abs().amax(-1, keepdim=True)
    s = s / torch.full_like(s, 448.0)
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (v / s).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8), s.squeeze(-1).contiguous()


def _linear_inputs(case, r):
    M, N, K = case["M"], case["N"], case["K"]
    rows = 2 * N if case["act"] == "situ" else N
    s = {"x": r.normal(M, K), "w": r.normal(rows, K, std=K ** -0.5),
         "bias": r.normal(rows, std=0.3, dtype=torch.float32) if case["bias"] else None}
    return s, rows


def _layer_weights(z, r):
    d, L, E, I, S, Is = z["d"], z["L"], z["E"], z["I"], z["S"], z["Is"]
    return {"w_down": r.normal(L, d, std=d ** -0.5), "w_router": r.normal(E, L, std=L ** -0.5),
            "w_gate": r.normal(E, I, L, std=L ** -0.5), "w_value": r.normal(E, I, L, std=L ** -0.5),
            "w_edown": r.normal(E, L, I, std=I ** -0.5),
            "gamma": r.uniform(L, lo=0.5, hi=1.5), "w_up": r.normal(d, L, std=L ** -0.5),
            "w_sgate": r.normal(S, Is, d, std=d ** -0.5),
            "w_svalue": r.normal(S, Is, d, std=d ** -0.5),
            "w_sdown": r.normal(S, d, Is, std=Is ** -0.5)}


def _raw(case, seed):
    """The inputs of a case, alike for whoever computes."""
    r = _Draws(seed)
    if case["op"] in ("norm", "norm_bwd"):
        n, c = case["rows"], case["cols"]
        s = {"x": r.normal(n, c), "residual": r.normal(n, c, std=2.0),
             "gamma": r.uniform(c, lo=0.5, hi=1.5)}
        if case["op"] == "norm_bwd":
            total = s["residual"]
            s = {"total": total, "gamma": s["gamma"], "dy": s["x"], "dtotal": r.normal(n, c),
                 "rstd": (total.double().square().mean(1) + EPS).rsqrt().float()}
        return s
    if case["op"] == "linear":
        s, rows = _linear_inputs(case, r)
        s["residual"] = r.normal(case["M"], case["N"]) if case["resid"] else None
        s["xs"] = s["ws"] = None
        if case["fp8"]:
            s["x"], s["xs"] = _codes(s["x"])
            s["w"], s["ws"] = _codes(s["w"])
        return s
    if case["op"] == "linear_bwd":
        s, rows = _linear_inputs(case, r)
        s["dy"] = r.normal(case["M"], case["N"])
        # the pre-activations that the forward pass kept
        s["pre"] = r.normal(case["M"], rows) if case["act"] != "none" else None
        return s
    z = LAYERS[case["layer"]]
    s = {"w": _layer_weights(z, r), "x": r.normal(case["T"], z["d"])}
    # thresholds near the scores' upper K/E quantile, as a balanced router has them
    q = -torch.special.ndtri(torch.tensor(z["K"] / z["E"], dtype=torch.float64)).item()
    s["tau"] = torch.sigmoid(q + 0.1 * r.normal(z["E"], dtype=torch.float32))
    return s


class _Shape:
    def __init__(self, z, T):
        self.T, self.c, self.eps = T, CAP, EPS
        self.__dict__.update(z)


def prepare(case, seed):
    s = _raw(case, seed)
    s["case"] = case
    if not own:
        if case["op"] == "few" and case["fp8"]:  # the experts' weights as such a program keeps them
            for n in ("w_gate", "w_value", "w_edown"):
                w = s["w"].pop(n)
                parts = [_codes(p) for p in w.split(32)]
                s["w"][n] = torch.cat([p[0] for p in parts])
                s["w"][n + "_s"] = torch.cat([p[1] for p in parts])
                del w, parts
        return s
    from latent_compressed_expert_gb300 import lmoe
    s["lmoe"] = lmoe
    if case["op"] in ("linear", "linear_bwd"):
        s["linear"] = lmoe.Linear(s["w"], s["bias"], act=case["act"], w_scales=s.get("ws"))
    if case["op"] == "few":
        s["layer"] = lmoe.Layer(_Shape(LAYERS[case["layer"]], case["T"]), s.pop("w"),
                                expert_fp8=case["fp8"])
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c, lmoe = s["case"], s["lmoe"]
    if c["op"] == "norm":
        if c["fp8"]:
            codes, scales, total = lmoe.add_rmsnorm_e4m3(s["x"], s["gamma"], s["residual"], EPS)
            return {"y": codes.view(E4M3), "scales": scales, "total": total}
        y, total = lmoe.add_rmsnorm(s["x"], s["gamma"], s["residual"], EPS)
        return {"y": y, "total": total}
    if c["op"] == "norm_bwd":
        dx, dgamma = lmoe.add_rmsnorm_backward(s["dy"], s["total"], s["gamma"], s["rstd"],
                                               s["dtotal"])
        return {"dx": dx, "dgamma": dgamma}
    if c["op"] == "linear":
        return {"y": s["linear"].forward(s["x"], s["residual"], x_scales=s["xs"])}
    if c["op"] == "linear_bwd":
        g = s["linear"].backward(s["x"], s["dy"], pre=s["pre"],
                                 dw_dtype=torch.float32 if c["dw"] == "fp32" else BF)
        return {"dx": g["dx"], "dw": g["dw"], **({"dbias": g["dbias"]} if c["bias"] else {})}
    return {"y": s["layer"].forward_few(s["x"], residual=s["x"], tau=s["tau"])}


def _situ(g, v):
    gc, vc = CAP * torch.tanh(g / CAP), CAP * torch.tanh(v / CAP)
    return gc * torch.sigmoid(gc) * vc


def _cdf(p):
    return 0.5 * (1.0 + torch.erf(p * 0.7071067811865476))


def _act(p, act):
    if act == "situ":
        return _situ(*p.chunk(2, -1))
    if act == "silu":
        return p * torch.sigmoid(p)
    return p * _cdf(p) if act == "gelu" else p


def _act_grad(p, dy, act):
    if act == "situ":
        g, v = p.chunk(2, -1)
        tg, tv = torch.tanh(g / CAP), torch.tanh(v / CAP)
        gc, vc = CAP * tg, CAP * tv
        sg = torch.sigmoid(gc)
        return torch.cat([dy * vc * sg * (1 + gc * (1 - sg)) * (1 - tg * tg),
                          dy * gc * sg * (1 - tv * tv)], -1)
    if act == "silu":
        sg = torch.sigmoid(p)
        return dy * sg * (1 + p * (1 - sg))
    if act == "gelu":
        return dy * (_cdf(p) + p * torch.exp(-0.5 * p * p) * 0.3989422804014327)
    return dy


def _quant(v):
    """v [..., cols] fp32 as the values that its e4m3 codes and row scale stand for."""
    codes, s = _codes(v)
    return codes.view(E4M3).float() * s.unsqueeze(-1)


def _run_plain(s):
    c = s["case"]
    if c["op"] == "norm":
        t = s["x"].float() + s["residual"].float()
        y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["gamma"]
        if not c["fp8"]:
            return {"y": y.to(BF), "total": t.to(BF)}
        codes, scales = _codes(y)
        return {"y": codes.view(E4M3), "scales": scales, "total": t.to(BF)}
    if c["op"] == "norm_bwd":
        dy, xh = s["dy"].float(), s["total"].float() * s["rstd"].unsqueeze(1)
        g = dy * s["gamma"]
        dx = (g - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"].unsqueeze(1)
        return {"dx": (dx + s["dtotal"].float()).to(BF), "dgamma": (dy * xh).sum(0)}
    if c["op"] == "linear":
        if c["fp8"]:
            p = s["x"].view(E4M3).float() @ s["w"].view(E4M3).float().T
            p = p * s["xs"].unsqueeze(1) * s["ws"]
        else:
            p = s["x"].float() @ s["w"].float().T
        y = _act(p if s["bias"] is None else p + s["bias"], c["act"])
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(BF)}
    if c["op"] == "linear_bwd":
        dy = s["dy"].float()
        dp = dy if s["pre"] is None else _act_grad(s["pre"].float(), dy, c["act"])
        dw = dp.T @ s["x"].float()
        out = {"dx": (dp @ s["w"].float()).to(BF), "dw": dw if c["dw"] == "fp32" else dw.to(BF)}
        if c["bias"]:
            out["dbias"] = dp.sum(0)
        return out
    return {"y": _few_plain(s, LAYERS[c["layer"]], c)}


def _few_plain(s, z, c):
    w, x = s["w"], s["x"].float()
    # the latent and the logits in 64 bits: a token's K-th and K+1-th scores can lie close
    lat64 = s["x"].double() @ w["w_down"].double().T
    scores = torch.sigmoid(lat64 @ w["w_router"].double().T)
    idx = torch.sort(scores - s["tau"], dim=1, descending=True, stable=True).indices[:, :z["K"]]
    picked = torch.gather(scores, 1, idx)
    gates = (picked / picked.sum(1, keepdim=True)).float()
    lat = lat64.float()

    def experts(name):  # [T, K, out, in]
        if c["fp8"]:
            return w[name][idx].view(E4M3).float() * w[name + "_s"][idx].unsqueeze(-1)
        return w[name][idx].float()

    a = (_quant(lat) if c["fp8"] else lat)[:, None, :, None]
    h = _situ((experts("w_gate") @ a).squeeze(-1), (experts("w_value") @ a).squeeze(-1))
    h = _quant(h) if c["fp8"] else h
    u = ((experts("w_edown") @ h.unsqueeze(-1)).squeeze(-1) * gates.unsqueeze(-1)).sum(1)
    zn = u * torch.rsqrt(u.square().mean(1, keepdim=True) + EPS) * w["gamma"]
    sw = z["S"] * z["Is"]
    hs = _situ(x @ w["w_sgate"].view(sw, -1).float().T, x @ w["w_svalue"].view(sw, -1).float().T)
    ys = hs @ w["w_sdown"].permute(1, 0, 2).reshape(z["d"], sw).float().T
    return (x + zn @ w["w_up"].float().T + ys).to(BF)


# ------------------------------------------------------------------------------------ floors
def work(case):
    if case["op"] == "norm":
        n, c = case["rows"], case["cols"]
        return {"bytes": n * c * (2 + 2 + 2 + (1 if case["fp8"] else 2)) + 4 * c
                + (4 * n if case["fp8"] else 0), "flops": 6 * n * c}
    if case["op"] == "norm_bwd":
        n, c = case["rows"], case["cols"]
        return {"bytes": n * c * 8 + 8 * c + 4 * n, "flops": 12 * n * c}
    if case["op"] in ("linear", "linear_bwd"):
        M, N, K = case["M"], case["N"], case["K"]
        rows = 2 * N if case["act"] == "situ" else N
        if case["op"] == "linear":
            b = 1 if case["fp8"] else 2
            return {"bytes": b * (M + rows) * K + 2 * M * N * (2 if case["resid"] else 1)
                    + (4 * rows if case["bias"] else 0) + (4 * (M + rows) if case["fp8"] else 0),
                    "flops": 2 * M * rows * K}
        return {"bytes": 2 * (M + rows) * K + 2 * M * N + (2 * M * rows if case["act"] != "none" else 0)
                + 2 * M * K + (4 if case["dw"] == "fp32" else 2) * rows * K
                + (4 * rows if case["bias"] else 0), "flops": 4 * M * rows * K}
    z, T = LAYERS[case["layer"]], case["T"]
    sw = z["S"] * z["Is"]
    experts = z["E"] * (1 - (1 - z["K"] / z["E"]) ** T)  # expected distinct ones
    dense = (2 * z["L"] + 3 * sw) * z["d"] + z["E"] * z["L"]
    routed = 3 * z["I"] * z["L"]
    return {"bytes": 2 * dense + experts * routed * (1 if case["fp8"] else 2) + 6 * T * z["d"],
            "flops": 2 * T * (dense + z["K"] * routed)}


# ------------------------------------------------------------------------------------ 64 bits
def _e4m3_64(v):
    """(values of the e4m3 codes of v / s, s) per row: nearest, ties to even.  The recipe's scale
    and quotient are fp32 numbers: bf16 weights often lie on a tie, which only that decides."""
    s = (v.abs().max(dim=-1, keepdim=True).values / 448).float().double()
    s[s == 0] = 1
    q = (v / s).float().double()
    exp = torch.frexp(q.abs().clamp_min(2.0 ** -6)).exponent - 1  # 2^exp <= |q|, at least 2^-6
    step = torch.pow(2.0, (exp - 3).double())
    return (torch.round(q / step) * step).clamp(-448, 448), s


def _gated64(g, v):
    g, v = CAP * (g / CAP).tanh(), CAP * (v / CAP).tanh()
    return v * g / (1 + (-g).exp())


def _few64(s, z, fp8):
    w, K = s["w"], z["K"]
    x = s["x"].double()
    lat = torch.einsum("td,ld->tl", x, w["w_down"].double())
    score = 1 / (1 + torch.exp(-torch.einsum("tl,el->te", lat, w["w_router"].double())))
    key = score - s["tau"].double()
    rank = (key.unsqueeze(2) < key.unsqueeze(1)).sum(2)  # how many experts stand before
    z_out = torch.empty_like(lat)
    for t in range(x.shape[0]):
        chosen = torch.nonzero(rank[t] < K).flatten()
        g = score[t, chosen] / score[t, chosen].sum()
        a = lat[t]
        wg, wv, wd = (w[n][chosen].double() for n in ("w_gate", "w_value", "w_edown"))
        if fp8:
            wg, wv, wd = (q * sc for q, sc in map(_e4m3_64, (wg, wv, wd)))
            a = torch.mul(*_e4m3_64(a))
        h = _gated64(torch.einsum("kil,l->ki", wg, a), torch.einsum("kil,l->ki", wv, a))
        if fp8:
            h = torch.mul(*_e4m3_64(h))
        u = torch.einsum("k,kli,ki->l", g, wd, h)
        z_out[t] = w["gamma"].double() * u / torch.sqrt((u * u).mean() + EPS)
    y = x + torch.einsum("tl,dl->td", z_out, w["w_up"].double())
    for e in range(z["S"]):
        h = _gated64(torch.einsum("td,id->ti", x, w["w_sgate"][e].double()),
                     torch.einsum("td,id->ti", x, w["w_svalue"][e].double()))
        y += torch.einsum("ti,di->td", h, w["w_sdown"][e].double())
    return y


def exact(case, seed):
    s = _raw(case, seed)
    if case["op"] == "norm":
        t = s["x"].double() + s["residual"].double()
        y = s["gamma"].double() * t / torch.sqrt((t * t).sum(1, keepdim=True) / case["cols"] + EPS)
        if not case["fp8"]:
            return {"y": y, "total": t}
        q, sc = _e4m3_64(y)
        return {"y": q, "scales": sc.squeeze(1), "total": t}
    if case["op"] == "norm_bwd":
        t, dy, g = s["total"].double(), s["dy"].double(), s["gamma"].double()
        r = s["rstd"].double().unsqueeze(1)
        dot = (dy * g * t).sum(1, keepdim=True) / case["cols"]
        return {"dx": s["dtotal"].double() + r * dy * g - r ** 3 * t * dot,
                "dgamma": (dy * t * r).sum(0)}
    if case["op"] in ("linear", "linear_bwd"):
        act = case["act"]
        x, w = (s[n].view(E4M3).double() if case.get("fp8") else s[n].double() for n in ("x", "w"))
        if case["op"] == "linear":
            if case["fp8"]:
                x, w = x * s["xs"].double()[:, None], w * s["ws"].double()[:, None]
            p = torch.einsum("mk,nk->mn", x, w)
            if s["bias"] is not None:
                p += s["bias"].double()
            if act == "situ":
                p = _gated64(p[:, :case["N"]], p[:, case["N"]:])
            elif act == "silu":
                p = p / (1 + torch.exp(-p))
            elif act == "gelu":
                p = p * torch.special.ndtr(p)
            return {"y": p if s["residual"] is None else p + s["residual"].double()}
        d = s["dy"].double()
        if act != "none":  # the activation's slope by automatic differentiation
            p = s["pre"].double().requires_grad_(True)
            if act == "situ":
                f = _gated64(p[:, :case["N"]], p[:, case["N"]:])
            else:
                f = p / (1 + torch.exp(-p)) if act == "silu" else p * torch.special.ndtr(p)
            (d,) = torch.autograd.grad(f, p, d)
        out = {"dx": torch.einsum("mn,nk->mk", d, w), "dw": torch.einsum("mn,mk->nk", d, x)}
        if case["bias"]:
            out["dbias"] = torch.einsum("mn->n", d)
        return out
    return {"y": _few64(s, LAYERS[case["layer"]], case["fp8"])}
