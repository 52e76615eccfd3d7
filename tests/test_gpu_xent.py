"""Softmax cross entropy of a linear head and its gradients against plain 64-bit arithmetic.

Tolerances, derived.  A logit is K products, exact in fp32, added in fp32: off by at most
e = K 2^-23 sum|x||w| (the tensor cores may truncate).  exp2 of (l - base) log2(e): two roundings of an
argument of at most 128 (what is further below the maximum is zero next to it), and exp2's own 2 ulp:
relative 128 * 2^-22 + 2^-21.  A row's sum: at most 128 + V / 1024 additions one after the other,
2^-24 each (columns of a tile in four chains, tiles over 32 warps, warps).  log: 2^-22 of its value.
In the backward pass d is rounded to bf16, half a step being 2^-8 of it, or to two bf16 terms, which
leaves 2^-8 of 2^-8 (up to 128 rows); the products' sums are as above, over V and M terms (twice that
with two), and dx and a bf16 dw are rounded once more.  Beyond 128 rows dx takes the target's element of
d without its rounding."""
import pytest
import torch

from latent_compressed_expert_gb300 import lmoe

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HALF, ULP = 2.0 ** -8, 2.0 ** -23
EXP = 128 * 2.0 ** -22 + 2.0 ** -21


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    lmoe.load()
    return torch.device("cuda:0")


def _draw(dev, rows, cols, seed, std=1.0, ld=None):
    g = torch.Generator(device=dev).manual_seed(seed)
    ld = cols if ld is None else ld
    return (torch.randn(rows, ld, generator=g, device=dev) * std).to(BF)[:, :cols]


def _targets(dev, M, V, seed, ignored=0.2, dtype=torch.int64):
    g = torch.Generator(device=dev).manual_seed(seed)
    t = torch.randint(0, V, (M,), generator=g, device=dev)
    off = torch.rand(M, generator=g, device=dev) < ignored
    return torch.where(off, torch.tensor(-100, device=dev), t).to(dtype)


def _logits(x, w):
    x, w = x.double(), w.double()
    return x @ w.T, x.shape[1] * ULP * (x.abs() @ w.abs().T)


def _within(got, want, bound, tag):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), tag
    assert (err <= bound + 1e-35).all(), (tag, float((err / (bound + 1e-35)).max()))


def _check_forward(head, x, t, tag=""):
    V = head.V
    loss, lse = head.forward(x, t)
    l, e = _logits(x, head.w)
    want = torch.logsumexp(l, 1)
    bound = e.amax(1) + EXP + (128 + V / 1024) * 2.0 ** -24 + 2.0 ** -21 * want.abs() + 2.0 ** -22
    _within(lse, want, bound, (tag, "lse"))
    on = (t >= 0) & (t < V)
    at = torch.where(on, t, torch.zeros_like(t)).long().unsqueeze(1)
    picked = l.gather(1, at).squeeze(1)
    assert (loss[~on] == 0).all(), tag
    both = bound + e.gather(1, at).squeeze(1) + ULP * (want.abs() + picked.abs())
    _within(loss[on], (want - picked)[on], both[on], (tag, "loss"))
    torch.cuda.synchronize()
    assert head.device_error() == lmoe.LMOE_OK
    return loss, lse


def _check_backward(head, x, t, lse, g, tag="", **kw):
    V, w = head.V, head.w
    l, e = _logits(x, w)
    on = ((t >= 0) & (t < V)).unsqueeze(1)
    p = (l - lse.double().unsqueeze(1)).exp()
    hot = torch.arange(V, device=x.device) == t.unsqueeze(1)
    gd = g.double().unsqueeze(1)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    d = torch.where(on, gd * (p - hot.double()), zero)
    few = x.shape[0] <= 128
    half, sums = (HALF * HALF, 2) if few else (HALF, 1)
    near = torch.where(on, gd.abs() * p * (1.01 * e + EXP) + 4 * ULP * d.abs(), zero)
    ed = near + half * d.abs()
    x64, w64 = x.double(), w.double()
    dx, dw = d @ w64, d.T @ x64
    edx = ed if few else near + half * torch.where(hot, zero, d.abs())
    ex = edx @ w64.abs() + 1.01 * sums * V * ULP * (d.abs() @ w64.abs()) + HALF * dx.abs()
    ew = ed.T @ x64.abs() + 1.01 * sums * x.shape[0] * ULP * (d.abs().T @ x64.abs())
    out = head.backward(x, t, lse, g, **kw)
    if out["dx"] is not None:
        _within(out["dx"], dx, 1.01 * ex, (tag, "dx"))
    if out["dw"] is not None:
        half = HALF if out["dw"].dtype is BF else ULP
        _within(out["dw"], dw, 1.01 * (ew + half * dw.abs()), (tag, "dw"))
    torch.cuda.synchronize()
    assert head.device_error() == lmoe.LMOE_OK
    return out


def _weights_of_rows(dev, M, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.rand(M, generator=g, device=dev) - 0.25


# one row and one token; a chunk and its edge; tiles of one SM of several widths and their edges;
# SM pairs; many tiles of the vocabulary
SIZES = [(1, 1, 8), (1, 31, 8), (1, 33, 64), (3, 65, 72), (1, 1000, 512), (2, 70001, 136),
         (77, 1003, 1000), (128, 4099, 264), (129, 257, 136), (255, 96, 64), (300, 5000, 1024),
         (1000, 8200, 512), (257, 513, 7168), (2049, 300, 128)]


@pytest.mark.parametrize("M,V,K", SIZES)
def test_forward(dev, M, V, K):
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, V + K, 3 * K ** -0.5))
    _check_forward(head, _draw(dev, M, K, M), _targets(dev, M, V, 5), (M, V, K))


@pytest.mark.parametrize("M,V,K", SIZES)
@pytest.mark.parametrize("dw", [torch.float32, BF])
def test_backward(dev, M, V, K, dw):
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, V + K, 3 * K ** -0.5))
    x, t = _draw(dev, M, K, M), _targets(dev, M, V, 5)
    _, lse = head.forward(x, t)
    _check_backward(head, x, t, lse, _weights_of_rows(dev, M, 9), (M, V, K), dw_dtype=dw)


def test_several_pieces(dev):
    """A vocabulary of two whole pieces and a part of one, with a target in each."""
    M, V, K = 33000, 9001, 64
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.5))
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3)
    t[:3] = torch.tensor([4095, 4096, 9000], device=dev)
    _, lse = _check_forward(head, x, t)
    a = head.backward(x, t, lse, _weights_of_rows(dev, M, 4))
    for part in (slice(0, 500), slice(32500, M)):  # rows of dx by themselves
        sub = _check_backward(head, x[part], t[part], lse[part],
                              _weights_of_rows(dev, M, 4)[part], want_dw=False)
        # the pieces' order of adding differs from the smaller call's: both within their bounds
        big = a["dx"][part].double()
        assert (big - sub["dx"].double()).abs().max() <= 2 * HALF * big.abs().max()
    # dw over all rows, in 64 bits
    l = x.double() @ head.w.double().T
    p = (l - lse.double().unsqueeze(1)).exp_()
    p[torch.arange(M, device=dev)[t >= 0], t[t >= 0]] -= 1
    p *= (_weights_of_rows(dev, M, 4).double() * (t >= 0)).unsqueeze(1)
    want = p.T @ x.double()
    bound = (HALF + 2 * EXP + M * ULP) * (p.abs().T @ x.double().abs())
    _within(a["dw"], want, 1.01 * bound, "dw")


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_target_types_and_strides(dev, dtype):
    M, V, K = 50, 777, 128
    w = _draw(dev, V, K, 1, 0.3, ld=K + 40)
    x = _draw(dev, M, K, 2, ld=K + 8)
    head = lmoe.LinearCrossEntropy(w)
    t = _targets(dev, M, V, 3, dtype=dtype)
    t[0], t[1], t[2] = V, V - 1, torch.iinfo(dtype).min
    _, lse = _check_forward(head, x, t, dtype)
    _check_backward(head, x, t, lse, _weights_of_rows(dev, M, 4), dtype)


def test_no_targets_at_all(dev):
    M, V, K = 40, 600, 64
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1))
    x, t = _draw(dev, M, K, 2), torch.full((M,), -1, device=dev)
    x[3] = float("nan")
    loss, lse = head.forward(x, t)
    assert (loss == 0).all() and torch.isnan(lse[3]) and torch.isfinite(lse[4:]).all()
    x[3] = 1.0
    out = head.backward(x, t, lse, torch.ones(M, device=dev))
    assert not out["dx"].any() and not out["dw"].any()  # also where lse is NaN


def test_rows_that_are_not_finite(dev):
    """Each row's infinities and NaN stay in its own loss, lse and dx."""
    M, V, K = 140, 700, 64
    w = _draw(dev, V, K, 1, 0.2)
    w[:, 0] = 1.0
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3, ignored=0.0)
    head = lmoe.LinearCrossEntropy(w)
    clean = head.forward(x, t)
    xx = x.clone()
    xx[5, 3] = float("nan")
    xx[6, 0] = float("inf")       # all logits +inf
    xx[7, 0] = float("-inf")      # all logits -inf
    loss, lse = head.forward(xx, t)
    assert torch.isnan(lse[5]) and lse[6] == float("inf") and lse[7] == float("-inf")
    assert torch.isnan(loss[5:8]).all()  # inf - inf
    others = [i for i in range(M) if i not in (5, 6, 7)]
    assert torch.equal(loss[others], clean[0][others]) and torch.equal(lse[others], clean[1][others])
    # one token of weight zero probability: w row -> logit -inf for every row with x[0] > 0
    w2 = w.clone()
    w2[9, 0] = float("-inf")
    x2 = x.clone()
    x2[:, 0] = 1.0
    t2 = torch.where(t == 9, 10, t)
    h2 = lmoe.LinearCrossEntropy(w2)
    loss2, lse2 = h2.forward(x2, t2)
    keep = [i for i in range(V) if i != 9]
    want = torch.logsumexp(x2.double() @ w2[keep].double().T, 1)
    _within(lse2, want, 1e-4 + 0 * want, "lse without a token")
    assert torch.isfinite(loss2).all()


def test_large_logits(dev):
    """A row's maximum far from zero on either side; probabilities of one and zero."""
    M, V, K = 130, 1200, 64
    w = _draw(dev, V, K, 1, 1.0)
    x = _draw(dev, M, K, 2)
    w[:, 0], x[:, 0] = 8.0, 0.0
    x[:40, 0], x[40:80, 0] = 400.0, -400.0
    x[80:, 1:] *= 30
    head = lmoe.LinearCrossEntropy(w)
    t = _targets(dev, M, V, 3)
    _, lse = _check_forward(head, x, t)
    _check_backward(head, x, t, lse, _weights_of_rows(dev, M, 4))


def test_against_differences(dev):
    """dx and dw against central differences of the loss along directions that bf16 holds exactly:
    values in steps of 2^-5 up to 1, moved by 2^-5.  With logits z(h) = z + h u and |u| <= U, the
    third derivative of the loss is at most 2 U^3: h^2 U^3 / 3 in the difference quotient."""
    M, V, K, h = 8, 40, 16, 2.0 ** -5
    gen = torch.Generator(device=dev).manual_seed(7)
    grid = lambda *s: torch.randint(-30, 31, s, generator=gen, device=dev).to(BF) * h
    x, w = grid(M, K).to(BF), grid(V, K).to(BF)
    t = _targets(dev, M, V, 3, ignored=0.1)
    g = torch.rand(M, generator=gen, device=dev)
    head = lmoe.LinearCrossEntropy(w)
    _, lse = head.forward(x, t)
    out = head.backward(x, t, lse, g)
    sign = lambda *s: (torch.randint(0, 2, s, generator=gen, device=dev) * 2 - 1).to(BF)
    total = lambda xx, ww: float((lmoe.LinearCrossEntropy(ww).forward(xx, t)[0].double() * g).sum())
    for _ in range(4):
        ux, uw = sign(M, K), sign(V, K)
        for grad, u, f in ((out["dx"], ux, lambda s: total(x + s * h * ux, w)),
                           (out["dw"], uw, lambda s: total(x, w + s * h * uw))):
            diff = (f(1) - f(-1)) / (2 * h)
            got = float((grad.double() * u.double()).sum())
            U = float((x if u is uw else w).double().abs().sum(1).max())
            tol = h * h * U ** 3 / 3 * float(g.sum()) + 2 * HALF * float(grad.double().abs().sum()) \
                + 1e-5 / h
            assert abs(diff - got) <= tol, (diff, got, tol)


def test_same_bits_every_time_and_in_any_batch(dev):
    """Sums are added in a fixed order, and rows do not see their neighbours."""
    M, V, K = 100, 3000, 256
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.2))
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3)
    loss, lse = head.forward(x, t)
    g = _weights_of_rows(dev, M, 4)
    out = head.backward(x, t, lse, g)
    for _ in range(3):
        again = head.forward(x, t)
        assert torch.equal(again[0], loss) and torch.equal(again[1], lse)
        o = head.backward(x, t, lse, g)
        assert torch.equal(o["dx"], out["dx"]) and torch.equal(o["dw"], out["dw"])
    one = head.forward(x[17:18], t[17:18])
    assert torch.equal(one[1], lse[17:18])


def test_parts_of_the_gradients(dev):
    M, V, K = 60, 500, 128
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.2))
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3)
    _, lse = head.forward(x, t)
    g = _weights_of_rows(dev, M, 4)
    both = head.backward(x, t, lse, g)
    a, b = head.backward(x, t, lse, g, want_dw=False), head.backward(x, t, lse, g, want_dx=False)
    assert a["dw"] is None and b["dx"] is None
    assert torch.equal(a["dx"], both["dx"]) and torch.equal(b["dw"], both["dw"])


def test_no_rows(dev):
    head = lmoe.LinearCrossEntropy(_draw(dev, 300, 64, 1))
    x, t = torch.empty(0, 64, dtype=BF, device=dev), torch.empty(0, dtype=torch.int64, device=dev)
    loss, lse = head.forward(x, t)
    assert loss.numel() == lse.numel() == 0
    out = head.backward(x, t, lse, torch.empty(0, device=dev))
    assert out["dx"].shape == (0, 64) and not out["dw"].any()


def test_streams_and_graphs(dev):
    """On a stream of its own, from two streams at once, and captured: the same bits; a graph's replay
    takes the inputs as they are then."""
    M, V, K = 200, 5000, 512
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.1))
    xs = [_draw(dev, M, K, s) for s in (2, 3)]
    t, g = _targets(dev, M, V, 4), _weights_of_rows(dev, M, 5)

    def step(x, stream=None):
        loss, lse = head.forward(x, t, stream=stream)
        out = head.backward(x, t, lse, g, stream=stream)
        return loss, lse, out["dx"], out["dw"]

    want = [step(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = [step(x, s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step(x)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(kept, want[i]))


def test_weights_are_looked_at_each_call(dev):
    head = lmoe.LinearCrossEntropy(_draw(dev, 300, 64, 1))
    x, t = _draw(dev, 9, 64, 2), _targets(dev, 9, 300, 3)
    head.w = _draw(dev, 300, 64, 8)
    _check_forward(head, x, t)
    head.w.mul_(0.5)
    _check_forward(head, x, t)


def test_refusals(dev):
    head = lmoe.LinearCrossEntropy(_draw(dev, 300, 64, 1))
    x, t = _draw(dev, 9, 64, 2), _targets(dev, 9, 300, 3)
    with pytest.raises(ValueError):
        head.forward(x.float(), t)
    with pytest.raises(ValueError):
        head.forward(x, t.float())
    with pytest.raises(ValueError):
        head.forward(x, t[:8])
    with pytest.raises(ValueError):
        head.forward(x, t.cpu())
    with pytest.raises(ValueError):
        head.forward(x, torch.stack([t, t], 1)[:, 0])
    with pytest.raises(ValueError):
        head.forward(x.cpu(), t)
    lse = torch.zeros(9, device=dev)
    with pytest.raises(ValueError):
        head.backward(x, t, lse, lse, dw_dtype=torch.float16)
    with pytest.raises(ValueError):
        head.backward(x, t, lse[:8], lse)
    with pytest.raises(ValueError):
        head.backward(x, t, lse, lse.double())
    with pytest.raises(lmoe.LmoeError):
        lmoe.LinearCrossEntropy(_draw(dev, 300, 60, 1)).forward(_draw(dev, 9, 60, 2), t)
    with pytest.raises(lmoe.LmoeError):   # rows at 8-byte steps
        head.forward(_draw(dev, 9, 64, 2, ld=68), t)


@pytest.mark.parametrize("M", [16, 300])
def test_stalled_wait_is_reported(dev, monkeypatch, M):
    """A wait that runs out ends the call with an error status; the next call is right again."""
    V, K = 2000, 128
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.2))
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3)
    want = head.forward(x, t)
    g = _weights_of_rows(dev, M, 4)
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "50")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    for call in (lambda: head.forward(x, t), lambda: head.backward(x, t, want[1], g)):
        call()
        torch.cuda.synchronize()
        assert head.device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    again = head.forward(x, t)
    torch.cuda.synchronize()
    assert head.device_error() == lmoe.LMOE_OK
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("M", [129, 300, 1000])
@pytest.mark.parametrize("weight", [1 + 2.0 ** -8, 1 / 300, -3e-30])
def test_one_weight_for_all_rows(dev, M, weight):
    """A mean's 1 / rows, and rows without weight before them: what rounding the weight to bf16 would take
    from every target's element (half a step, 2^-8 of it, for the first weight) is not lost.  In units of
    the weight the target's element is p - 1, which for p < 2^-9 rounds to -1: off by p; the others, p,
    by 2^-8 of p.  So both gradients are off by at most weight p |x| or |w| a row, the logits' errors, and
    the products' sums (and the weight's unit taken out and put back, two roundings)."""
    V, K = 20000, 64
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.05))
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3)
    g = torch.full((M,), weight, device=dev)
    g[: M // 2] = 0.0
    _, lse = head.forward(x, t)
    out = head.backward(x, t, lse, g, dw_dtype=torch.float32)
    l, e = _logits(x, head.w)
    on = ((t >= 0) & (t < V)).unsqueeze(1)
    p = (l - lse.double().unsqueeze(1)).exp()
    assert float(p.max()) < 2.0 ** -9
    gd = torch.where(on, g.double().unsqueeze(1), 0.0)
    d = gd * (p - (torch.arange(V, device=dev) == t.unsqueeze(1)).double())
    ed = gd.abs() * p * (1 + 1.01 * e + EXP) + 4 * ULP * d.abs()
    x64, w64 = x.double(), head.w.double()
    ew = ed.T @ x64.abs() + 1.01 * (M + 1) * ULP * (d.abs().T @ x64.abs())
    _within(out["dw"], d.T @ x64, 1.01 * ew, "dw")
    ex = ed @ w64.abs() + 1.01 * (V + 1) * ULP * (d.abs() @ w64.abs())
    want = d @ w64
    _within(out["dx"], want, 1.01 * (ex + HALF * want.abs()), "dx")


def _check_one_weight(head, x, t, g):
    """Rows of one weight, or none: the bounds derived at test_one_weight_for_all_rows."""
    M, V = x.shape[0], head.V
    _, lse = head.forward(x, t)
    out = head.backward(x, t, lse, g, dw_dtype=torch.float32)
    l, e = _logits(x, head.w)
    on = ((t >= 0) & (t < V)).unsqueeze(1)
    p = (l - lse.double().unsqueeze(1)).exp()
    assert float(p.max()) < 2.0 ** -9
    gd = torch.where(on, g.double().unsqueeze(1), 0.0)
    d = gd * (p - (torch.arange(V, device=x.device) == t.unsqueeze(1)).double())
    ed = gd.abs() * p * (1 + 1.01 * e + EXP) + 4 * ULP * d.abs()
    x64, w64 = x.double(), head.w.double()
    live = int((gd != 0).sum())  # the others add zeros
    ew = ed.T @ x64.abs() + 1.01 * (live + 1) * ULP * (d.abs().T @ x64.abs())
    _within(out["dw"], d.T @ x64, 1.01 * ew, "dw")
    ex = ed @ w64.abs() + 1.01 * (V + 1) * ULP * (d.abs() @ w64.abs())
    want = d @ w64
    _within(out["dx"], want, 1.01 * (ex + HALF * want.abs()), "dx")


@pytest.mark.parametrize("other", [1.0, float("nan"), float("inf"), 0.0])
@pytest.mark.parametrize("M", [129, 300, 3000])
def test_weights_of_rows_without_a_target_do_not_count(dev, M, other):
    """The one weight of the rows that have a target is not rounded, whatever the others' is."""
    head = lmoe.LinearCrossEntropy(_draw(dev, 8000, 64, 1, 0.05))
    x, t = _draw(dev, M, 64, 2), _targets(dev, M, 8000, 3, ignored=0.5)
    t[0] = -100
    weight = torch.full((M,), 1 / 300, device=dev)
    weight[t < 0] = other
    got = head.forward(x, t)
    clean = head.backward(x, t, got[1], torch.full((M,), 1 / 300, device=dev))
    out = head.backward(x, t, got[1], weight)
    assert torch.equal(out["dx"], clean["dx"]) and torch.equal(out["dw"], clean["dw"])
    if other == 1.0:
        _check_one_weight(head, x, t, weight)


@pytest.mark.parametrize("M,rows", [(4096, range(5, 4096, 200)), (4096, [4095]), (1000, [999]),
                                    (70000, [3, 69999])])
def test_few_rows_of_one_weight_among_many_without(dev, M, rows):
    """Wherever they lie."""
    V = 8000 if M < 10000 else 3000
    head = lmoe.LinearCrossEntropy(_draw(dev, V, 64, 1, 0.02))
    x, t = _draw(dev, M, 64, 2), _targets(dev, M, V, 3, ignored=0.0)
    g = torch.zeros(M, device=dev)
    g[list(rows)] = 1 / 300
    _check_one_weight(head, x, t, g)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("M,K", [(1, 8), (40, 64), (128, 1032), (300, 64), (1100, 200)])
def test_rows_without_a_target_take_no_part(dev, M, K, bad):
    """Whatever is in them (a padded batch): the other rows' gradients and dw keep their bits, their own
    dx is 0; with weights that are not finite too, for which the formulas give the others NaN."""
    V = 700
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.2))
    x, t, g = _draw(dev, M, K, 2), _targets(dev, M, V, 3, ignored=0.3), _weights_of_rows(dev, M, 4)
    t[0] = -100
    off = t < 0
    _, lse = head.forward(x, t)
    xx, gg = x.clone(), g.clone()
    xx[off] = bad
    xx[0, 1:] = 1.0
    gg[off] = bad
    _, lse2 = head.forward(xx, t)
    assert torch.equal(lse2[~off], lse[~off])
    for dw in (torch.float32, BF):
        want = head.backward(x, t, lse, g, dw_dtype=dw)
        out = head.backward(xx, t, lse2, gg, dw_dtype=dw)
        assert torch.equal(out["dx"], want["dx"]) and torch.equal(out["dw"], want["dw"])
        assert not out["dx"][off].any()
        alone = head.backward(xx, t, lse2, gg, dw_dtype=dw, want_dx=False)
        assert torch.equal(alone["dw"], want["dw"])
    head.w = head.w.clone()
    head.w[5, 3] = bad
    assert not head.backward(x, t, lse, g)["dx"][off].any()


@pytest.mark.parametrize("M", [1, 100, 300, 2049])
@pytest.mark.parametrize("dw", [torch.float32, BF])
def test_rows_that_are_nearly_certain(dev, M, dw):
    """Targets of probability 1 - 1e-3 down to 1 - 1e-9, whose gradient is what is left of it.  A target's
    logit here is a sum of 7168 terms of one sign, which the tensor cores may make 1e-4 too small and
    more; lse is made of the same number, so that p - 1 is only off by lse's own rounding, 2^-20 (lse is
    below 32), the additions to the sum behind it, 2^-24 each, and what the logits' errors e change
    in the other tokens' probabilities.  e: sums within one accumulator are cut off by 2^-23 at most for
    each of 64 products of 16 features, then added in fp32."""
    V, K = 2500, 7168
    gen = torch.Generator(device=dev).manual_seed(3)
    x = _draw(dev, M, K, 2)
    t = torch.randperm(V, generator=gen, device=dev)[:M]
    size = 14 + 16 * torch.rand(M, 1, generator=gen, device=dev)
    w = _draw(dev, V, K, 1, 0.3 * K ** -0.5)
    w[t] = (size / x.float().square().sum(1, keepdim=True) * x.float()).to(BF)
    head = lmoe.LinearCrossEntropy(w)
    g = 0.5 + torch.rand(M, generator=gen, device=dev)
    _, lse = head.forward(x, t)
    out = head.backward(x, t, lse, g, dw_dtype=dw)
    x64, w64 = x.double(), w.double()
    l = x64 @ w64.T
    p = torch.softmax(l, 1)
    hot = torch.arange(V, device=dev) == t.unsqueeze(1)
    gd = g.double().unsqueeze(1)
    left = torch.where(hot, 0.0, p).sum(1, keepdim=True)  # 1 - p of the target
    d = gd * torch.where(hot, -left, p)
    e = (64 + 7) * ULP * (x64.abs() @ w64.abs().T).amax(1, keepdim=True)
    off = 2.0 ** -20 + (128 + V / 1024) * 2.0 ** -24
    ed = gd * torch.where(hot, off + (2 * e + 2.0 ** -20) * left, (2 * e + off + EXP) * p)
    half = HALF * HALF if M <= 128 else HALF
    sums = 2 if M <= 128 else 1
    ew = (ed + half * d.abs()).T @ x64.abs() + 1.01 * sums * M * ULP * (d.abs().T @ x64.abs())
    want = d.T @ x64
    _within(out["dw"], want, 1.01 * (ew + (HALF if dw is BF else ULP) * want.abs()), (M, "dw"))
    ex = (ed + half * torch.where(hot, 0.0, d).abs()) @ w64.abs() + \
        1.01 * sums * V * ULP * (d.abs() @ w64.abs())
    want = d @ w64
    _within(out["dx"], want, 1.01 * (ex + HALF * want.abs()), (M, "dx"))


@pytest.mark.parametrize("base", [0.0, 12.0, 200.0, -3008.0])
@pytest.mark.parametrize("M", [5, 300, 1100])
def test_small_losses_have_no_steps_of_lse(dev, M, base):
    """Logits that fp32 holds exactly, all shifted by `base`: the loss does not see it.  The sum of 40
    tokens' exponentials takes at most 8 + 4 additions, 2^-24 of 1 or so each, and exponentials 2^-21 of
    themselves and 2^-24 of their argument (at most 30); the logarithm 2^-22 of its value."""
    V, K = 40, 8
    w = torch.zeros(V, K, device=dev)
    w[:, 0] = 1.0
    w[:, 1] = -torch.arange(V, device=dev) / 2.0   # tokens' distances from the first
    w[0, 1] = 4.0
    x = torch.zeros(M, K, device=dev)
    x[:, 0] = base
    x[:, 1] = (1 + torch.arange(M, device=dev) % 6) / 2.0
    l = (x.double() @ w.double().T)
    t = torch.arange(M, device=dev) // 6 % 5  # the likely one, and others
    t = torch.where(t > 1, 0, t)
    head = lmoe.LinearCrossEntropy(w.to(BF))
    loss, lse = head.forward(x.to(BF), t)
    want = -torch.log_softmax(l, 1).gather(1, t.unsqueeze(1)).squeeze(1)
    rest = torch.expm1(-torch.log_softmax(l, 1).amax(1)).abs()
    bound = 12 * 2.0 ** -24 * (1 + rest) + rest * (2.0 ** -21 + 30 * 2.0 ** -22) + \
        2.0 ** -22 * want + 2.0 ** -23 * want
    _within(loss, want, 1.01 * bound, "loss")
    _within(lse, torch.logsumexp(l, 1), 1.01 * bound + ULP * l.abs().amax(1), "lse")


@pytest.mark.parametrize("M,K", [(300, 136), (70000, 8), (65536, 264)])
def test_fp32_dw_of_many_rows(dev, M, K):
    """A head of zeros over 128 tokens: d is 2^-7, or that less 1, for all rows, which bf16 holds, and x is
    positive.  The tensor cores cut off less than 2^-23 of what has been summed in each step of 16 rows; over
    the 512 rows that stay in TMEM that is 32 * 2^-23, and their sums are added in fp32, 2^-24 each (a sum of
    both signs: of the larger part).  Multiplying by the unit, 1, changes nothing."""
    V = 128
    head = lmoe.LinearCrossEntropy(torch.zeros(V, K, dtype=BF, device=dev))
    gen = torch.Generator(device=dev).manual_seed(1)
    x = torch.exp2(-8 * torch.rand(M, K, generator=gen, device=dev)).to(BF)
    t = torch.arange(M, device=dev) % 64
    _, lse = head.forward(x, t)
    out = head.backward(x, t, lse, torch.ones(M, device=dev), want_dx=False)
    sums = torch.zeros(V, K, dtype=torch.float64, device=dev).index_add_(0, t, x.double())
    all_rows = x.double().sum(0) / V
    bound = (32 * 2.0 ** -23 + (M // 512 + 1) * 2.0 ** -24 + 2.0 ** -23) * (sums + all_rows)
    _within(out["dw"], all_rows - sums, bound, (M, K))


@pytest.mark.parametrize("M,V,K", [(300, 447232 + 100, 64), (1000, 200000, 256), (128, (1 << 19) + 70, 8),
                                   (5, 300001, 16), (129, (1 << 20) + 40, 8)])
def test_pieces_and_slices(dev, M, V, K):
    """Vocabularies of several pieces whose dx is summed in slices: a last piece of fewer K-blocks than
    slices, and (up to 128 rows) two terms of d.  Targets on both sides of the pieces' edges."""
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, V + K, 3 * K ** -0.5))
    x, t = _draw(dev, M, K, M), _targets(dev, M, V, 5)
    edges = torch.tensor([V - 1, V - 41, 447231, 447232, 134143, 134144, 262144, 524287], device=dev)
    t[:min(M, 8)] = edges[:M].clamp(max=V - 1)
    _, lse = _check_forward(head, x, t, (M, V, K))
    _check_backward(head, x, t, lse, _weights_of_rows(dev, M, 9), (M, V, K))


def test_gradients_of_rows_that_are_not_finite(dev):
    """Each row's infinities and NaN stay in its own dx; dw, which sums over the rows, is NaN as the formulas
    give it."""
    M, V, K = 140, 700, 64
    w = _draw(dev, V, K, 1, 0.2)
    w[:, 0] = 1.0
    x, t = _draw(dev, M, K, 2), _targets(dev, M, V, 3, ignored=0.0)
    head, g = lmoe.LinearCrossEntropy(w), _weights_of_rows(dev, M, 4)
    for rows in (M, 100):
        x0, t0, g0 = x[:rows], t[:rows], g[:rows]
        clean = head.backward(x0, t0, head.forward(x0, t0)[1], g0)
        xx = x0.clone()
        xx[5, 3], xx[6, 0], xx[7, 0] = float("nan"), float("inf"), float("-inf")
        out = head.backward(xx, t0, head.forward(xx, t0)[1], g0)
        others = [i for i in range(rows) if i not in (5, 6, 7)]
        assert torch.equal(out["dx"][others], clean["dx"][others])
        assert torch.isnan(out["dx"][5:8]).all() and torch.isnan(out["dw"]).all()


@pytest.mark.parametrize("M", [100, 129, 700])
def test_certain_of_a_wrong_token(dev, M):
    """The element of the token that has the probability is then as large as the target's; its rounding to
    bf16 counts in dx (beyond 128 rows) as the bounds say."""
    V, K = 900, 512
    x = _draw(dev, M, K, 2)
    w = _draw(dev, V, K, 1, 0.02)
    sure = torch.arange(M, device=dev)
    w[sure] = (12 / K * x.float()).to(BF)
    head, t = lmoe.LinearCrossEntropy(w), (sure + 7) % V
    _, lse = _check_forward(head, x, t, M)
    for dw in (torch.float32, BF):
        _check_backward(head, x, t, lse, _weights_of_rows(dev, M, 4), M, dw_dtype=dw)


@pytest.mark.parametrize("M", [1, 128])
def test_logits_do_not_depend_on_the_tiles(dev, M):
    """Tiles are as wide as the vocabulary asks for, and the backward's pieces have widths of their own.  With
    all other tokens' probability 0, lse is the remaining token's logit, to the last bit."""
    K = 7168
    x = _draw(dev, M, K, 2)
    x[:, 0] = 3e4
    one = _draw(dev, 1, K, 3, 5 * K ** -0.5)
    one[:, 0] = 0.0
    want = None
    for V in (1, 70, 4000, 12000, 22000, 40000):  # 64 to 256 columns
        for at in (0, V // 2, V - 1):
            w = torch.zeros(V, K, dtype=BF, device=dev)
            w[:, 0] = -3e4
            w[at] = one
            _, lse = lmoe.LinearCrossEntropy(w).forward(x, torch.full((M,), at, device=dev))
            want = lse if want is None else want
            assert torch.equal(lse, want), (V, at)
    l, e = _logits(x, one)
    _within(want, l.squeeze(1), e.squeeze(1), "logit")


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("parts", ["both", "dx", "dw"])
def test_rows_of_dx_at_a_distance(dev, M, parts):
    """Through the C entry: dx with gaps between its rows, which stay as they were, and rows behind the last."""
    V, K, ld = 700, 72, 104
    head = lmoe.LinearCrossEntropy(_draw(dev, V, K, 1, 0.2))
    x, t, g = _draw(dev, M, K, 2, ld=K + 16), _targets(dev, M, V, 3), _weights_of_rows(dev, M, 4)
    _, lse = head.forward(x, t)
    want = head.backward(x, t, lse, g)
    dx = torch.full((M + 2, ld), 7.0, dtype=BF, device=dev)
    dw = torch.full((V + 2, K), 7.0, device=dev)
    lib, d = lmoe.load(), head._desc(x, t, None, lse.data_ptr())
    nb = lib.lmoe_linear_xent_backward_workspace_bytes(d)
    ws = torch.full((nb + 256,), 0xA5, dtype=torch.uint8, device=dev)
    rc = lib.lmoe_linear_xent_backward(
        d, g.data_ptr(), None if parts == "dw" else dx.data_ptr(), ld,
        None if parts == "dx" else dw.data_ptr(), lmoe.F32, ws.data_ptr(), nb,
        torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == lmoe.LMOE_OK and head.device_error() == lmoe.LMOE_OK
    assert (ws[nb:] == 0xA5).all() and (dx[:, K:] == 7).all() and (dx[M:] == 7).all()
    assert (dw[V:] == 7).all()
    assert torch.equal(dx[:M, :K], want["dx"]) if parts != "dw" else (dx == 7).all()
    assert torch.equal(dw[:V], want["dw"]) if parts != "dx" else (dw == 7).all()
