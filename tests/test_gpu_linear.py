"""Linear layers with fused epilogues and their gradients against plain 64-bit arithmetic.

Tolerances, derived.  Products of two bf16 (or e4m3) values are exact in fp32; D of them added in
fp32 are off by at most D * 2^-23 * sum|a||b| (the tensor cores may truncate).  bf16 rounding is
off by half a step, 2^-8 of the value.  The activations' slopes are at most 1.13, and their own
arithmetic (exponential, reciprocal, normal distribution function) is within 2^-17 of the terms
they add.  In the backward pass dp is rounded to bf16 before the products: 2^-8 of its terms."""
import pytest
import torch

from latent_compressed_expert_gb300 import lmoe

pytestmark = pytest.mark.gpu
BF, E4M3 = torch.bfloat16, torch.float8_e4m3fn
HALF, FN = 2.0 ** -8, 2.0 ** -17


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    lmoe.load()
    return torch.device("cuda:0")


def _draw(dev, rows, cols, seed, std=1.0, ld=None, off=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    ld = cols if ld is None else ld
    buf = (torch.randn(off + rows * ld, generator=g, device=dev) * std).to(BF)
    return buf[off:].view(rows, ld)[:, :cols]


def _cap(x, c):
    return c * torch.tanh(x / c)


def _act64(p, act, c):
    """(value, error per unit of error in p) of the activation."""
    if act == "situ":
        g, v = p.chunk(2, 1)
        gc, vc = _cap(g, c), _cap(v, c)
        f = gc * torch.sigmoid(gc)
        return f * vc, (1.13 * vc.abs(), f.abs())
    if act == "silu":
        return p * torch.sigmoid(p), 1.13
    if act == "gelu":
        return p * torch.special.ndtr(p), 1.13
    return p, 1.0


def _slope64(pre, dy, act, c):
    """(dp, sum of the magnitudes of its terms)."""
    if act == "situ":
        g, v = pre.chunk(2, 1)
        gc, vc = _cap(g, c), _cap(v, c)
        s = torch.sigmoid(gc)
        kg, kv = s * (1 - (gc / c) ** 2), 1 - (vc / c) ** 2
        dp = torch.cat([dy * vc * kg * (1 + gc * (1 - s)), dy * gc * s * kv], 1)
        # near the cap 1 - t^2 subtracts nearly equal terms: its error is relative to 1
        mag = torch.cat([(dy * vc * s).abs() * (1 + gc.abs() * (1 - s)), (dy * gc * s).abs()], 1)
        return dp, mag
    if act == "silu":
        s = torch.sigmoid(pre)
        return dy * s * (1 + pre * (1 - s)), dy.abs() * s * (1 + pre.abs() * (1 - s))
    if act == "gelu":
        pdf = torch.exp(-0.5 * pre * pre) / (2 * torch.pi) ** 0.5
        return dy * (torch.special.ndtr(pre) + pre * pdf), \
            dy.abs() * (torch.special.ndtr(pre) + pre.abs() * pdf)
    return dy, 0 * dy


def _within(got, want, bound, tag):
    err = (got.double() - want).abs()
    assert torch.isfinite(got.double()).all(), tag
    assert (err <= bound + 1e-35).all(), (tag, float((err / (bound + 1e-35)).max()))


def _check_forward(lin, x, res=None, xs=None, c=100.0, tag="", **kw):
    x64 = x.view(E4M3).double() * xs.double()[:, None] if lin.fp8 else x.double()
    w64 = lin.w.view(E4M3).double() * lin.w_scales.double()[:, None] if lin.fp8 else lin.w.double()
    p = x64 @ w64.T
    ep = lin.K * 2.0 ** -23 * (x64.abs() @ w64.abs().T) + 2.0 ** -22 * p.abs()
    if lin.bias is not None:
        p = p + lin.bias.double()
        ep = ep + 2.0 ** -23 * p.abs()
    y64, k = _act64(p, lin.act, c)
    if lin.act == "situ":
        eg, ev = ep.chunk(2, 1)
        e = k[0] * eg + k[1] * ev
    else:
        e = k * ep
    e = e + FN * y64.abs()
    if res is not None:
        y64 = y64 + res.double()
    y, pre = lin.forward(x, res, x_scales=xs, train=True, **kw)
    _within(y, y64, HALF * y64.abs() + 1.01 * e, (tag, "y"))
    if pre is not None:
        _within(pre, p, HALF * p.abs() + 1.01 * ep, (tag, "pre"))
    assert torch.equal(lin.forward(x, res, x_scales=xs), y)     # the same bits without pre
    torch.cuda.synchronize()
    assert lin.device_error() == lmoe.LMOE_OK
    return y, pre


# M x N x K: one row and one feature group; split reductions at few rows; ragged last tiles in
# every dimension; the one-SM tiles of both widths; SM pairs of both widths
SIZES = [(1, 8, 8), (1, 512, 7168), (3, 3584, 72), (2, 7168, 4096), (77, 3584, 1024),
         (128, 64, 64), (129, 136, 200), (200, 1000, 4104), (513, 72, 3584), (1000, 264, 136),
         (2050, 2056, 520), (4096, 3584, 512), (8200, 1032, 264), (777, 7168, 1032)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward_plain(dev, M, N, K):
    lin = lmoe.Linear(_draw(dev, N, K, N + K, K ** -0.5))
    _check_forward(lin, _draw(dev, M, K, M), tag=(M, N, K))


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu", "situ"])
def test_forward_fused(dev, M, N, K, act):
    rows = 2 * N if act == "situ" else N
    lin = lmoe.Linear(_draw(dev, rows, K, N + K, K ** -0.5), torch.randn(rows, device=dev), act)
    _check_forward(lin, 2 * _draw(dev, M, K, M), _draw(dev, M, N, 7), tag=(M, N, K, act))


def _codes(x):
    return lmoe.quantize_e4m3(x.contiguous())


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (2, 7168, 4096), (77, 3584, 1008), (129, 136, 208),
                                   (2050, 2056, 528), (8200, 1032, 272), (777, 7168, 1024)])
@pytest.mark.parametrize("act", ["none", "situ"])
def test_forward_e4m3(dev, M, N, K, act):
    rows = 2 * N if act == "situ" else N
    w, ws = _codes(_draw(dev, rows, K, N + K, K ** -0.5))
    x, xs = _codes(_draw(dev, M, K, M))
    lin = lmoe.Linear(w, torch.randn(rows, device=dev), act, w_scales=ws)
    _check_forward(lin, x, _draw(dev, M, N, 7), xs=xs, tag=(M, N, K, act))


def test_situ_cap(dev):
    """Pre-activations far past the cap, and a small cap."""
    for c, std in ((100.0, 300.0), (2.0, 3.0)):
        lin = lmoe.Linear(_draw(dev, 128, 64, 1, 64 ** -0.5), act="situ", c=c)
        y, pre = _check_forward(lin, _draw(dev, 40, 64, 2, std), c=c, tag=c)
        dy = _draw(dev, 40, 64, 3)
        _check_backward(lin, _draw(dev, 40, 64, 2, std), dy, pre, c=c, tag=c)


@pytest.mark.parametrize("M", [5, 700, 9000])
def test_strides_and_in_place(dev, M):
    """Row strides and offsets of whole 16 bytes on every operand give the packed bits and touch
    nothing beside the outputs; y may be the residual."""
    N, K = 1032, 520
    w = _draw(dev, N, K, 1, K ** -0.5, ld=K + 24, off=8)
    x, res = _draw(dev, M, K, 2, ld=K + 8, off=16), _draw(dev, M, N, 3, ld=N + 40)
    want = lmoe.Linear(w.contiguous(), act="silu").forward(x.contiguous(), res.contiguous())
    lin = lmoe.Linear(w, act="silu")
    buf = torch.full((M, N + 16), 5.0, dtype=BF, device=dev)
    y = lin.forward(x, res, y=buf[:, 8:N + 8])
    assert torch.equal(y, want)
    assert (buf[:, :8] == 5.0).all() and (buf[:, N + 8:] == 5.0).all()
    inplace = res.contiguous()
    assert torch.equal(lin.forward(x, inplace, y=inplace), want)


def _check_backward(lin, x, dy, pre=None, c=100.0, tag="", **kw):
    d64 = dy.double()
    dp, mag = _slope64(pre.double(), d64, lin.act, c) if lin.act != "none" else (d64, 0 * d64)
    # the operand's error: the slope's arithmetic, then its rounding to bf16
    ed = FN * mag
    edp = ed + (HALF * dp.abs() if lin.act != "none" else 0)
    x64, w64 = x.double(), lin.w.double()
    g = lin.backward(x, dy, pre, **kw)
    again = lin.backward(x, dy, pre, **kw)
    dx64, dw64 = dp @ w64, dp.T @ x64
    ex = edp @ w64.abs() + lin.rows * 2.0 ** -23 * (dp.abs() @ w64.abs())
    ew = edp.T @ x64.abs() + x.shape[0] * 2.0 ** -23 * (dp.abs().T @ x64.abs())
    _within(g["dx"], dx64, HALF * dx64.abs() + 1.02 * ex, (tag, "dx"))
    half = HALF if g["dw"].dtype == BF else 2.0 ** -24
    _within(g["dw"], dw64, half * dw64.abs() + 1.02 * ew, (tag, "dw"))
    if lin.bias is None:
        assert g["dbias"] is None
    else:
        # at most 2 * 128 terms in a chain, then at most 256 parts
        _within(g["dbias"], dp.sum(0), ed.sum(0) + 512 * 2.0 ** -24 * dp.abs().sum(0),
                (tag, "dbias"))
    for n in g:  # a fixed order everywhere
        assert g[n] is None or torch.equal(g[n], again[n]), n
    torch.cuda.synchronize()
    assert lin.device_error() == lmoe.LMOE_OK
    return g


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dw", [torch.float32, BF])
def test_backward_plain(dev, M, N, K, dw):
    lin = lmoe.Linear(_draw(dev, N, K, N + K, K ** -0.5), torch.randn(N, device=dev))
    _check_backward(lin, _draw(dev, M, K, M), _draw(dev, M, N, 3), tag=(M, N, K), dw_dtype=dw)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu", "situ"])
def test_backward_fused(dev, M, N, K, act):
    rows = 2 * N if act == "situ" else N
    lin = lmoe.Linear(_draw(dev, rows, K, N + K, K ** -0.5), torch.randn(rows, device=dev), act)
    x = 2 * _draw(dev, M, K, M)
    _, pre = lin.forward(x, train=True)
    _check_backward(lin, x, _draw(dev, M, N, 3), pre, tag=(M, N, K, act), dw_dtype=BF)


def test_backward_strided_and_partial(dev):
    """Strided dy, x, w and pre give the packed bits; unwanted gradients change nothing."""
    M, N, K = 300, 264, 136
    w = _draw(dev, N, K, 1, K ** -0.5, ld=K + 8)
    x, dy = _draw(dev, M, K, 2, ld=K + 16), _draw(dev, M, N, 3, ld=N + 24, off=8)
    pre = _draw(dev, M, N, 4, ld=N + 8)
    bias = torch.zeros(N, device=dev)
    want = lmoe.Linear(w.contiguous(), bias, "gelu").backward(x.contiguous(), dy.contiguous(),
                                                              pre.contiguous())
    lin = lmoe.Linear(w, bias, "gelu")
    got = lin.backward(x, dy, pre)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    g = lin.backward(x, dy, pre, want_dx=False)
    assert g["dx"] is None and torch.equal(g["dw"], want["dw"])
    g = lin.backward(x, dy, pre, want_dw=False)
    assert g["dw"] is None and torch.equal(g["dx"], want["dx"])
    g = lmoe.Linear(w).backward(x, dy)
    assert g["dbias"] is None


def test_backward_is_the_slope_of_the_forward(dev):
    """Gradients against central differences of the formula in 64 bits along random directions."""
    M, N, K, h = 6, 16, 24, 1e-4
    for act in ("none", "silu", "gelu", "situ"):
        rows = 2 * N if act == "situ" else N
        w, x, dy = _draw(dev, rows, K, 1, K ** -0.5), _draw(dev, M, K, 2), _draw(dev, M, N, 3)
        b = torch.randn(rows, device=dev)
        lin = lmoe.Linear(w, b, act)
        _, pre = lin.forward(x, train=True)
        g = lin.backward(x, dy, pre)

        def loss(x64, w64, b64):
            return float((dy.double() * _act64(x64 @ w64.T + b64, act, 100.0)[0]).sum())

        at = [x.double(), w.double(), b.double()]
        for i, n in enumerate(("dx", "dw", "dbias")):
            gen = torch.Generator(device=dev).manual_seed(i)
            v = torch.randn(at[i].shape, generator=gen, device=dev, dtype=torch.float64)
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + h * v, at[i] - h * v
            num = (loss(*up) - loss(*down)) / (2 * h)
            ana = float((g[n].double() * v).sum())
            # pre was rounded to bf16 (its slopes move by at most ~0.8 * 2^-8 |pre| each), dp and
            # dx again: 4 * 2^-8 of the terms' magnitudes covers the sums at these sizes
            mag = float((g[n].double() * v).abs().sum())
            assert abs(num - ana) <= 4 * HALF * mag + 1e-6, (act, n, num, ana, mag)


def test_no_rows(dev):
    lin = lmoe.Linear(_draw(dev, 16, 8, 1), torch.zeros(16, device=dev), "silu")
    x = torch.empty(0, 8, dtype=BF, device=dev)
    y, pre = lin.forward(x, train=True)
    assert y.shape == (0, 16)
    g = lin.backward(x, y, pre)
    assert g["dx"].shape == (0, 8) and (g["dw"] == 0).all() and (g["dbias"] == 0).all()


def test_other_stream_and_graph(dev):
    """On a caller's stream; and forward and backward captured into a graph, replayed on new data
    while an eager layer on the same weights lives."""
    lin = lmoe.Linear(_draw(dev, 512, 256, 1, 1 / 16), torch.randn(512, device=dev), "situ")
    x, dy = _draw(dev, 300, 256, 2), _draw(dev, 300, 256, 3)
    y, pre = lin.forward(x, train=True)
    want = lin.backward(x, dy, pre)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ys = lin.forward(x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(ys, y)
    xs = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        yg, pg = lin.forward(xs, train=True)
        gg = lin.backward(xs, dy, pg)
    xs.copy_(x)
    graph.replay()
    assert torch.equal(yg, y) and all(torch.equal(gg[n], want[n]) for n in want)


def test_weights_updated_in_place(dev):
    lin = lmoe.Linear(_draw(dev, 64, 64, 1), None)
    x = _draw(dev, 9, 64, 2)
    lin.forward(x)
    lin.w.copy_(_draw(dev, 64, 64, 5))
    assert torch.equal(lin.forward(x), lmoe.Linear(lin.w.clone()).forward(x))


def test_infinities_stay_in_their_rows(dev):
    """A row with infinities and NaN spoils its own output row only (tile rows are separate
    lanes), and a padded tile's rows past M are never stored."""
    lin = lmoe.Linear(_draw(dev, 64, 128, 1, 1 / 11))
    x = _draw(dev, 130, 128, 2).clone()
    want = lin.forward(x)
    x[3, 5], x[129, 0] = float("inf"), float("nan")
    y = lin.forward(x)
    keep = [i for i in range(130) if i not in (3, 129)]
    assert torch.equal(y[keep], want[keep])
    assert not torch.isfinite(y[3].float()).any() and torch.isnan(y[129].float()).all()


def test_stalled_wait_reports_timeout_and_recovers(dev, monkeypatch):
    """A device-side wait that runs out (a barrier nothing arrives on) in both kernels: the call
    ends, the layer reports it, and the next call is correct."""
    for M in (40, 9000):
        lin = lmoe.Linear(_draw(dev, 2048, 2048, 1, 1 / 45))
        x = _draw(dev, M, 2048, 2)
        want = lin.forward(x)
        monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "100")
        monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
        lin.forward(x)
        torch.cuda.synchronize()
        assert lin.device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
        assert lin.device_error() == lmoe.LMOE_OK
        monkeypatch.delenv("LMOE_FAULT_INJECT")
        monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
        assert torch.equal(lin.forward(x), want)


def test_refusals(dev):
    w, x = _draw(dev, 64, 64, 1), _draw(dev, 4, 64, 2)
    b = torch.zeros(64, device=dev)
    for bad in (lambda: lmoe.Linear(w, act="tanh"), lambda: lmoe.Linear(w.float()),
                lambda: lmoe.Linear(w, b[:32]), lambda: lmoe.Linear(w, b.to(BF)),
                lambda: lmoe.Linear(w[:63], act="situ"),
                lambda: lmoe.Linear(w.view(torch.uint8)),
                lambda: lmoe.Linear(w).forward(x[:, :32]), lambda: lmoe.Linear(w).forward(x.cpu()),
                lambda: lmoe.Linear(w).forward(x, x[:2]),
                lambda: lmoe.Linear(w).forward(x, x_scales=torch.ones(4, device=dev)),
                lambda: lmoe.Linear(w, act="silu").backward(x, x),
                lambda: lmoe.Linear(w).backward(x, x, dw_dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lmoe.Linear(_draw(dev, 64, 60, 1)).forward(_draw(dev, 4, 60, 1)),   # K
                lambda: lmoe.Linear(_draw(dev, 12, 64, 1)).forward(x),                      # N
                lambda: lmoe.Linear(w).forward(_draw(dev, 4, 64, 1, ld=68)),                # stride
                lambda: lmoe.Linear(w).forward(_draw(dev, 4, 64, 1, off=1)),                # address
                lambda: lmoe.Linear(*[t for t in (_codes(w)[0],)], None, "none",
                                    _codes(w)[1]).backward(x, x)):
        with pytest.raises(lmoe.LmoeError):
            bad()


def test_weight_gradient_of_many_rows(dev):
    """An fp32 dw does not lose precision with the number of rows.  The MMA adds 16 rows at a time and
    cuts off less than 2^-23 of what has been summed, 2^-24 on average; over the 512 rows that stay in
    one accumulator, whose partial sums grow like the root of their number, that is
    32 * 2/3 * 2^-24 = 1.3e-6 of the sum, to which the fp32 additions of the parts bring at most
    8 * 2^-24.  2e-6 bounds both; 4096 rows in one accumulator would be 4e-6 off."""
    M, N, K = 4096, 2048, 1024
    x, dy = _draw(dev, M, K, 1), _draw(dev, M, N, 2)
    lin = lmoe.Linear(_draw(dev, N, K, 3, K ** -0.5))
    want = dy.double().T @ x.double()
    for g in (lin.backward(x, dy), lin.backward(x, dy, want_dx=False)):
        assert (g["dw"].double() - want).norm() <= 2e-6 * want.norm()


def _within_or_nan(got, want, bound, tag):
    """_within, and NaN exactly where the formula gives it."""
    nan = want.isnan()
    assert torch.equal(got.isnan(), nan), (tag, int(got.isnan().sum()), int(nan.sum()))
    ok = want.isinf() & (got.double() == want) | nan
    _within(got.double().masked_fill(ok, 0), want.masked_fill(ok, 0), bound.masked_fill(ok, 0), tag)


@pytest.mark.parametrize("M", [5, 2050])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "situ"])
@pytest.mark.parametrize("fp8", [False, True])
def test_forward_of_nan_and_infinities(dev, M, act, fp8):
    """Rows with a NaN or an infinity give what the formulas give, others are not touched."""
    N, K = 264, 272
    rows = 2 * N if act == "situ" else N
    w, x, xs, ws = _draw(dev, rows, K, 1, K ** -0.5).contiguous(), _draw(dev, M, K, 2).clone(), None, None
    clean = x.clone()
    if fp8:  # codes have a NaN and no infinity
        (w, ws), (x, xs) = _codes(w), _codes(x)
        clean = x.clone()
        x[1, 3] = 0x7f
    else:
        x[1, 3], x[2, 0], x[3, K - 1] = float("nan"), float("inf"), -float("inf")
    lin = lmoe.Linear(w, torch.randn(rows, device=dev), act, w_scales=ws)
    w64 = w.view(E4M3).double() * ws.double()[:, None] if fp8 else w.double()
    x64 = x.view(E4M3).double() * xs.double()[:, None] if fp8 else x.double()
    p = (x64[1:4, None] * w64).sum(2) + lin.bias.double()
    y64, _ = _act64(p, act, 100.0)
    y, pre = lin.forward(x, x_scales=xs, train=True)
    want = lin.forward(clean, x_scales=xs)
    keep = [i for i in range(M) if i not in (1, 2, 3)]
    assert torch.equal(y[keep], want[keep])
    # finite results here: capped gates and values, 2^-8 of themselves; and, of e4m3 rows, sums as at
    # the head of this file
    e = K * 2.0 ** -23 * (x64[1:4].nan_to_num(0, 0, 0).abs() @ w64.abs().T)
    if act == "situ":
        e = (e[:, :N] + e[:, N:]) * 113.0
    _within_or_nan(y[1:4], y64, (HALF + 2 * FN) * y64.abs() + 1.2 * e, ("y", act))
    if pre is not None:
        e = K * 2.0 ** -23 * (x64[1:4].nan_to_num(0, 0, 0).abs() @ w64.abs().T)
        _within_or_nan(pre[1:4], p, HALF * p.abs() + 1.01 * e, ("pre", act))


@pytest.mark.parametrize("M", [40, 300])
@pytest.mark.parametrize("act", ["silu", "gelu", "situ"])
def test_backward_of_nan_and_infinities(dev, M, act):
    """NaN, infinite and huge pre-activations: gradients as the formulas give them, in the rows and
    features that they belong to."""
    N, K = 64, 72
    rows = 2 * N if act == "situ" else N
    lin = lmoe.Linear(_draw(dev, rows, K, 1, K ** -0.5), torch.zeros(rows, device=dev), act)
    x, dy, pre = _draw(dev, M, K, 2), _draw(dev, M, N, 3), _draw(dev, M, rows, 4).clone()
    pre[7, 5], pre[9, 11], pre[12, 13] = float("nan"), float("inf"), -float("inf")
    pre[20, 3], pre[21, 4] = 1e38, -1e38
    if act == "situ":
        pre[15, N + 20], pre[16, N + 21] = float("nan"), -float("inf")
    dp, mag = _slope64(pre.double(), dy.double(), act, 100.0)
    assert dp.isnan().any() and not dp.isinf().any()
    ed = FN * mag
    edp = ed + HALF * dp.abs()
    x64, w64 = x.double(), lin.w.double()
    g = lin.backward(x, dy, pre)
    dx64, dw64 = dp @ w64, dp.T @ x64
    _within_or_nan(g["dx"], dx64, HALF * dx64.abs() + 1.02 * (
        edp @ w64.abs() + rows * 2.0 ** -23 * (dp.abs() @ w64.abs())), ("dx", act))
    _within_or_nan(g["dw"], dw64, 2.0 ** -24 * dw64.abs() + 1.02 * (
        edp.T @ x64.abs() + M * 2.0 ** -23 * (dp.abs().T @ x64.abs())), ("dw", act))
    _within_or_nan(g["dbias"], dp.sum(0), ed.sum(0) + 512 * 2.0 ** -24 * dp.abs().sum(0),
                   ("dbias", act))


@pytest.mark.parametrize("act", ["silu", "situ"])
def test_far_below_zero(dev, act):
    """Finite pre-activations far below zero, where the logistic function is nothing: identity
    weights bring them through the product exactly."""
    N = 64
    rows = 2 * N if act == "situ" else N
    values = torch.tensor([-1e38, -3e36, -1e30, -1e5, -200.0, -120.0, -90.0, -60.0, 90.0, 1e38])
    x = torch.ones(10, 64, dtype=BF, device=dev)
    x[:, 1] = values.to(dev)
    w = torch.zeros(rows, 64, dtype=BF, device=dev)
    w[0, 1] = 1.0
    if act == "situ":
        w[N, 0] = 1.0
    lin = lmoe.Linear(w, act=act)
    y, pre = _check_forward(lin, x, tag=act)
    dy = torch.ones(10, N, dtype=BF, device=dev)
    dp, mag = _slope64(pre.double(), dy.double(), act, 100.0)
    edp = FN * mag + HALF * dp.abs()
    x64, w64 = x.double(), w.double()
    g = lin.backward(x, dy, pre)
    _within_or_nan(g["dx"], dp @ w64, HALF * (dp @ w64).abs() + 1.02 * (
        edp @ w64.abs() + rows * 2.0 ** -23 * (dp.abs() @ w64.abs())), ("dx", act))
    # some products of gradients and 1e38 pass fp32's range: infinities of their sign
    dw64 = (dp.T @ x64).float().double()
    _within_or_nan(g["dw"], dw64, 2.0 ** -24 * dw64.abs() + 1.02 * (
        edp.T @ x64.abs() + 10 * 2.0 ** -23 * (dp.abs().T @ x64.abs())), ("dw", act))


def _pair(dev, rows, K, seed, fp8=False, ld=None):
    """Weights (e4m3: with scales) and a bias."""
    w = _draw(dev, rows, K, seed, K ** -0.5, ld=ld)
    w, ws = _codes(w) if fp8 else (w, None)
    return w, torch.randn(rows, device=dev), ws


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_and_bias_replaced(dev, fp8):
    """Tensors assigned to a layer, and storage that a tensor of it was given, are what the next call
    computes with; what does not fit the layer is refused."""
    N, K, M = 64, 80, 9
    x, xs = (_codes(_draw(dev, M, K, 2)) if fp8 else (_draw(dev, M, K, 2), None))
    w, b, ws = _pair(dev, N, K, 1, fp8)
    lin = lmoe.Linear(w, b, "silu", w_scales=ws)
    kept = [w, b, ws]

    def fresh():
        return lmoe.Linear(lin.w.clone(), None if lin.bias is None else lin.bias.clone(), "silu",
                           w_scales=None if ws is None else lin.w_scales.clone())

    def check():
        y, pre = lin.forward(x, x_scales=xs, train=True)
        want, _ = fresh().forward(x, x_scales=xs, train=True)
        assert torch.equal(y, want)
        if not fp8:
            dy = _draw(dev, M, N, 5)
            got, want = lin.backward(x, dy, pre), fresh().backward(x, dy, pre)
            assert all((got[n] is None) == (want[n] is None) and
                       (got[n] is None or torch.equal(got[n], want[n])) for n in want)

    check()
    lin.w, lin.bias, lin.w_scales = _pair(dev, N, K, 3, fp8, ld=None if fp8 else K + 16)
    check()
    kept += [lin.w, lin.bias, lin.w_scales]
    new = _pair(dev, N, K, 4, fp8)
    kept += [lin.w.data, lin.bias.data]
    lin.w.data, lin.bias.data = new[0], new[1]
    if fp8:
        kept.append(lin.w_scales.data)
        lin.w_scales.data = new[2]
    check()
    lin.bias = None
    check()
    lin.bias = new[1]
    check()
    for bad in (dict(w=new[0][:32]), dict(w=new[0].float()), dict(w=new[0].cpu()),
                dict(bias=new[1][:32]), dict(bias=new[1].to(BF)),
                dict(w_scales=None if fp8 else new[1]), dict(w_scales=new[1][:32])):
        was = {n: getattr(lin, n) for n in bad}
        for n, t in bad.items():
            setattr(lin, n, t)
        with pytest.raises(ValueError):
            lin.forward(x, x_scales=xs)
        for n, t in was.items():
            setattr(lin, n, t)
    check()


def test_cap_changed_and_activation_fixed(dev):
    lin = lmoe.Linear(_draw(dev, 128, 64, 1, 1 / 8), act="situ", c=100.0)
    x = _draw(dev, 9, 64, 2, 30.0)
    lin.c = 2.0
    assert torch.equal(lin.forward(x), lmoe.Linear(lin.w, act="situ", c=2.0).forward(x))
    with pytest.raises(AttributeError):
        lin.act = "none"


# Root-mean-square checks, which the worst-case bounds above leave room under.  A bf16 output that is
# an fp32 sum rounded once is as far from the 64-bit value, in the norm, as that value's own rounding:
# the sum's error (2^-24 of what has been added at each of K / 16 steps: 2e-5 of it at 7168) is two
# orders below the rounding (2^-9), and turns it only near a midpoint, where both neighbours are as
# far.  Partial sums rounded to bf16 would come out at 1.4 times.  ONCE allows 2 %.  dp, rounded to
# bf16, takes the neighbouring value in about 2^-17 / 2^-9 of its elements, one step off: another
# 2.4 % of the square; 5 % in all where the reference rounds dp in its place.
ONCE, ONCE_DP = 1.02, 1.05
LONG = [(1, 512, 7168), (2, 7168, 4096), (8, 512, 7168), (77, 3584, 7168), (300, 1024, 7168),
        (2050, 2056, 7168)]


def _once(got, want, slack, tag):
    err = float((got.double() - want).norm())
    once = float((want.to(BF).double() - want).norm())
    assert err <= slack * once, (tag, err / once)


@pytest.mark.parametrize("M,N,K", LONG)
@pytest.mark.parametrize("act", ["none", "gelu", "situ"])
@pytest.mark.parametrize("fp8", [False, True])
def test_forward_rounds_once(dev, M, N, K, act, fp8):
    rows = 2 * N if act == "situ" else N
    w, b, ws = _pair(dev, rows, K, N + K, fp8)
    x, xs = _codes(_draw(dev, M, K, M)) if fp8 else (_draw(dev, M, K, M), None)
    lin = lmoe.Linear(w, b, act, w_scales=ws)
    res = _draw(dev, M, N, 7)
    w64 = w.view(E4M3).double() * ws.double()[:, None] if fp8 else w.double()
    x64 = x.view(E4M3).double() * xs.double()[:, None] if fp8 else x.double()
    p = x64 @ w64.T + b.double()
    y, pre = lin.forward(x, res, x_scales=xs, train=True)
    _once(y, _act64(p, act, 100.0)[0] + res.double(), ONCE, "y")
    if pre is not None:
        _once(pre, p, ONCE, "pre")


@pytest.mark.parametrize("M,N,K", [(8, 7168, 512), (77, 7168, 3584), (300, 7168, 1024),
                                   (2050, 7168, 1024)])
@pytest.mark.parametrize("act", ["none", "silu", "situ"])
def test_gradients_round_once(dev, M, N, K, act):
    rows = 2 * N if act == "situ" else N
    lin = lmoe.Linear(_draw(dev, rows, K, N + K, K ** -0.5), torch.zeros(rows, device=dev), act)
    x, dy = _draw(dev, M, K, 1), _draw(dev, M, N, 3)
    pre = _draw(dev, M, rows, 4) if act != "none" else None
    dp = dy.double()
    if pre is not None:
        dp = _slope64(pre.double(), dp, act, 100.0)[0].to(BF).double()
    slack = ONCE if act == "none" else ONCE_DP
    g = lin.backward(x, dy, pre, dw_dtype=BF)
    _once(g["dx"], dp @ lin.w.double(), slack, "dx")
    _once(g["dw"], dp.T @ x.double(), slack, "dw")


@pytest.mark.parametrize("M", [40, 3000])
@pytest.mark.parametrize("wants", [(True, True), (True, False), (False, True)])
def test_stalled_backward_reports_timeout_and_recovers(dev, monkeypatch, M, wants):
    """As for the forward, in the kernels of both gradients, together and one by one."""
    lin = lmoe.Linear(_draw(dev, 2048, 2048, 1, 1 / 45))
    x, dy = _draw(dev, M, 2048, 2), _draw(dev, M, 2048, 3)
    run = lambda: lin.backward(x, dy, want_dx=wants[0], want_dw=wants[1])
    want = run()
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "100")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    run()
    torch.cuda.synchronize()
    assert lin.device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    assert lin.device_error() == lmoe.LMOE_OK
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    got = run()
    assert all(want[n] is None or torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("M", [40, 9000])
def test_stalled_wait_of_e4m3_products(dev, monkeypatch, M):
    w, ws = _codes(_draw(dev, 2048, 2048, 1, 1 / 45))
    x, xs = _codes(_draw(dev, M, 2048, 2))
    lin = lmoe.Linear(w, w_scales=ws)
    want = lin.forward(x, x_scales=xs)
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "100")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    lin.forward(x, x_scales=xs)
    torch.cuda.synchronize()
    assert lin.device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    assert torch.equal(lin.forward(x, x_scales=xs), want)
