"""Cases of the operators that close a training step around the layer: the loss over a vocabulary
at its end, and the update of the weights from their gradients.

  xent          softmax cross entropy of a linear head, without its logits in memory: with
                l = x W^T over V tokens, lse = log sum exp l, loss = lse - l[target]; rows whose
                target is outside 0 .. V-1 have loss 0
  xent_bwd      its gradients for a weight g of each row's loss: with
                d = g (softmax(l) - onehot(target)), and 0 for rows without a target,
                dx = d W and dW = d^T x
  ortho         Newton-Schulz orthogonalisation of matrices [batch, rows, cols]:
                X = G / (|G|_F + eps), then `steps` times X = a X + (b A + c A^2) X, A = X X^T
  muon          momentum, orthogonalisation and update of weights in one call:
                m = beta m + g,  u = g + beta m,  w = w (1 - rate decay) - rate scale ortho(u)

``own`` chooses who computes: False, plain torch operations in fp32 (below); True, the framework.
"""
import math

import torch

own = False

BF = torch.bfloat16
IGNORED = -100
STEPS, EPS = 5, 1e-7
A, B, C = 3.4445, -4.7750, 2.0315  # of the quintic that Muon iterates
BETA, DECAY = 0.95, 0.1


def listed():
    return [
        # the log-probability of one sampled token: latency of reading a large head once
        {"name": "xent_1", "op": "xent", "M": 1, "V": 131072, "K": 7168, "ignored": 0.0},
        # scoring a short prompt with a small head and an odd vocabulary
        {"name": "xent_77", "op": "xent", "M": 77, "V": 32003, "K": 3584, "ignored": 0.1},
        # the loss of a training batch
        {"name": "xent_4096", "op": "xent", "M": 4096, "V": 65536, "K": 7168, "ignored": 0.1},
        # a fine-tuning micro-batch: most rows are a prompt's, without a target
        {"name": "xent_bwd_300", "op": "xent_bwd", "M": 300, "V": 50257, "K": 1024,
         "ignored": 0.6},
        # the gradients of the training batch
        {"name": "xent_bwd_4096", "op": "xent_bwd", "M": 4096, "V": 65536, "K": 7168,
         "ignored": 0.1},
        # one head's projection: latency
        {"name": "ortho_128", "op": "ortho", "batch": 1, "rows": 128, "cols": 1024, "fp32": False},
        # the gate weights of 64 routed experts, gradients as the layer's backward leaves them
        {"name": "ortho_experts", "op": "ortho", "batch": 64, "rows": 512, "cols": 3584,
         "fp32": True},
        # the up-projection, taller than wide
        {"name": "ortho_up", "op": "ortho", "batch": 1, "rows": 7168, "cols": 3584, "fp32": True},
        # a few odd matrices
        {"name": "ortho_odd", "op": "ortho", "batch": 7, "rows": 1001, "cols": 333, "fp32": False},
        # the router's weights
        {"name": "muon_router", "op": "muon", "batch": 1, "rows": 896, "cols": 3584, "fp32": True},
        # a dense feed-forward's projection
        {"name": "muon_dense", "op": "muon", "batch": 1, "rows": 4096, "cols": 7168,
         "fp32": False},
        # the value weights of the experts of a smaller layer
        {"name": "muon_mid", "op": "muon", "batch": 64, "rows": 256, "cols": 512, "fp32": True},
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(("xent", "xent_bwd", "ortho", "ortho", "muon"))
    if op in ("xent", "xent_bwd"):
        return {"op": op, "M": _log(rng, 1, 4096), "V": _log(rng, 1000, 65536),
                "K": _log(rng, 256, 7168, 8), "ignored": rng.choice((0.0, 0.1, 0.6))}
    rows, cols = _log(rng, 32, 4096), _log(rng, 32, 4096)
    most = max(1, int(6e8 / (rows * cols * min(rows, cols) / 64)))  # no more work than listed
    return {"op": op, "batch": _log(rng, 1, min(64, most)), "rows": rows, "cols": cols,
            "fp32": rng.random() < 0.5}


# ------------------------------------------------------------------------------------ inputs
class _Draws:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(int(seed) * 6007 + 29)

    def normal(self, *shape, std=1.0, dtype=BF):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=self.g)
        return t if std == 1.0 else t.mul_(std)

    def uniform(self, *shape, lo=0.0, hi=1.0):
        return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=self.g)


def _raw(case, seed):
    """The inputs of a case, alike for whoever computes."""
    r = _Draws(seed)
    if case["op"] in ("xent", "xent_bwd"):
        M, V, K = case["M"], case["V"], case["K"]
        w = r.normal(V, K, std=K ** -0.5)
        target = torch.empty(M, dtype=torch.int64, device="cuda").random_(0, V, generator=r.g)
        # tokens that the model expects to any degree: their logit stands out by up to 12
        x = r.normal(M, K, dtype=torch.float32)
        x = (x + r.uniform(M, 1, lo=0.0, hi=12.0) * w[target].float()).to(BF)
        target = torch.where(r.uniform(M) < case["ignored"], IGNORED, target)
        s = {"x": x, "w": w, "target": target}
        if case["op"] == "xent_bwd":
            s["dloss"] = r.uniform(M, lo=0.5, hi=1.5) / M
            logits = x.float() @ w.float().T  # the forward pass's
            s["lse"] = torch.logsumexp(logits, 1)
        return s
    n, rows, cols = case["batch"], case["rows"], case["cols"]
    # gradients: noise over a part of low rank, as a batch of few directions leaves them
    g = r.normal(n, rows, cols, std=1e-3, dtype=torch.float32)
    rank = 1 + min(rows, cols) // 8
    low = r.normal(n, rows, rank, dtype=torch.float32) @ r.normal(n, rank, cols, dtype=torch.float32)
    g.add_(low, alpha=2e-3 * rank ** -0.5)
    s = {"g": g if case["fp32"] else g.to(BF)}
    if case["op"] == "muon":
        s["m"] = r.normal(n, rows, cols, std=5e-3, dtype=torch.float32)
        s["w"] = r.normal(n, rows, cols, std=cols ** -0.5)
    return s


def _rates(case):
    """(rate, scale): a step of 0.2 in the root mean square of an orthogonal matrix's entries."""
    return 5e-3, 0.2 * max(case["rows"], case["cols"]) ** 0.5


def prepare(case, seed):
    s = _raw(case, seed)
    s["case"] = case
    if own:
        from latent_compressed_expert_gb300 import lmoe
        if case["op"] in ("xent", "xent_bwd"):
            s["head"] = lmoe.LinearCrossEntropy(s["w"])
        else:
            s["muon"] = lmoe.Muon(beta=BETA, nesterov=True, weight_decay=DECAY, steps=STEPS,
                                  coeffs=(A, B, C), eps=EPS)
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    c = s["case"]
    if c["op"] == "xent":
        loss, lse = s["head"].forward(s["x"], s["target"])
        return {"loss": loss, "lse": lse}
    if c["op"] == "xent_bwd":
        g = s["head"].backward(s["x"], s["target"], s["lse"], s["dloss"], dw_dtype=BF)
        return {"dx": g["dx"], "dw": g["dw"]}
    if c["op"] == "ortho":
        return {"o": s["muon"].orthogonalize(s["g"])}
    rate, scale = _rates(c)
    s["muon"].update(s["w"], s["g"], s["m"], rate, scale=scale)
    return {"w": s["w"], "m": s["m"]}


def _ortho(g):
    """g fp32 [batch, rows, cols]; the smaller side's products."""
    x = g / (g.square().sum((1, 2), keepdim=True).sqrt() + EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.mT
    for _ in range(STEPS):
        p = x @ x.mT
        x = A * x + (B * p + C * (p @ p)) @ x
    return x.mT.contiguous() if tall else x


def _run_plain(s):
    c = s["case"]
    if c["op"] in ("xent", "xent_bwd"):
        x, w, V = s["x"].float(), s["w"].float(), c["V"]
        logits = x @ w.T
        t = s["target"]
        on = (t >= 0) & (t < V)
        if c["op"] == "xent":
            top = logits.amax(1, keepdim=True)
            lse = (logits - top).exp().sum(1).log() + top.squeeze(1)
            picked = logits.gather(1, torch.where(on, t, 0).unsqueeze(1)).squeeze(1)
            return {"loss": torch.where(on, lse - picked, 0.0), "lse": lse}
        d = (logits - s["lse"].unsqueeze(1)).exp()
        hot = torch.arange(V, device=d.device) == t.unsqueeze(1)
        d = torch.where(on.unsqueeze(1), (d - hot.float()) * s["dloss"].unsqueeze(1), 0.0)
        return {"dx": (d @ w).to(BF), "dw": (d.T @ x).to(BF)}
    g = s["g"].float()
    if c["op"] == "ortho":
        return {"o": _ortho(g).to(BF)}
    rate, scale = _rates(c)
    s["m"] = BETA * s["m"] + g
    o = _ortho(g + BETA * s["m"])
    s["w"] = (s["w"].float() * (1 - rate * DECAY) - rate * scale * o).to(BF)
    return {"w": s["w"], "m": s["m"]}


# ------------------------------------------------------------------------------------ floors
def work(case):
    if case["op"] in ("xent", "xent_bwd"):
        M, V, K = case["M"], case["V"], case["K"]
        if case["op"] == "xent":
            return {"bytes": 2 * (M + V) * K + 16 * M, "flops": 2 * M * V * K}
        # the logits once more, and the two products of their gradient
        return {"bytes": 4 * (M + V) * K + 16 * M, "flops": 6 * M * V * K}
    n, size = case["batch"], case["rows"] * case["cols"]
    small = min(case["rows"], case["cols"])
    # A and A^2 are symmetric: half of each
    flops = n * STEPS * (3 * small * size + small ** 3)
    grad = 4 if case["fp32"] else 2
    if case["op"] == "ortho":
        return {"bytes": n * size * (grad + 2), "flops": flops}
    return {"bytes": n * size * (grad + 8 + 4), "flops": flops}


# ------------------------------------------------------------------------------------ 64 bits
def _ortho64(g):
    """Each power of the matrix by itself, from the left."""
    x = g / (torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True) + EPS)
    wide = g.shape[1] <= g.shape[2]
    for _ in range(STEPS):
        if wide:
            gram = torch.einsum("bij,bkj->bik", x, x)
            cube = torch.einsum("bik,bkj->bij", gram, x)
            fifth = torch.einsum("bik,bkj->bij", gram, cube)
        else:
            gram = torch.einsum("bji,bjk->bik", x, x)
            cube = torch.einsum("bij,bjk->bik", x, gram)
            fifth = torch.einsum("bij,bjk->bik", cube, gram)
        x = A * x + B * cube + C * fifth
    return x


def exact(case, seed):
    s = _raw(case, seed)
    if case["op"] in ("xent", "xent_bwd"):
        x, w, t = s["x"].double(), s["w"].double(), s["target"]
        on = (t >= 0) & (t < case["V"])
        logits = torch.einsum("mk,vk->mv", x, w)
        if case["op"] == "xent":
            lse = torch.logsumexp(logits, dim=1)
            loss = torch.zeros_like(lse)
            rows = torch.nonzero(on).flatten()
            loss[rows] = lse[rows] - logits[rows, t[rows]]
            return {"loss": loss, "lse": lse}
        # softmax by the lse that the call is given, an fp32 number
        d = logits.sub_(s["lse"].double()[:, None]).exp_()
        rows = torch.nonzero(on).flatten()
        d[rows, t[rows]] -= 1
        d *= (s["dloss"].double() * on)[:, None]
        return {"dx": torch.einsum("mv,vk->mk", d, w), "dw": torch.einsum("mv,mk->vk", d, x)}
    g = s["g"].double()
    if case["op"] == "ortho":
        return {"o": _ortho64(g)}
    rate, scale = _rates(case)
    m = BETA * s["m"].double() + g
    w = s["w"].double()
    return {"w": w - rate * DECAY * w - rate * scale * _ortho64(g + BETA * m), "m": m}
