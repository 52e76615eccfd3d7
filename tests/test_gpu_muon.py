"""Newton-Schulz orthogonalisation and the weight update against plain 64-bit arithmetic.

Tolerances, derived.  What the kernels round, beside sums in fp32 (2^-23 of their terms), are the
fp16 operands of the products: half a step, 2^-11 of a value.  How far that moves the result depends on
the singular values, so the bound is computed for each input: ``_rounded`` runs the iteration in 64 bits
with exactly these roundings (of hi, lo but for the last step, and of A and B off their diagonals), and its distance from the
iteration without them is what the rounding costs.  The kernels' sums put some values on the other side
of a rounding, which gives an error of the same size and, at most, in the same direction: twice the
cost, in the norm and for the largest element, and 1e-5 of the result for the fp32 sums.  The result's
own rounding to bf16 adds 2^-8 of an element, and 2^-9 in the norm (half a step, spread evenly:
2^-8 / sqrt 3 of values that are on average 0.72 of the way to the top of their binade or more)."""
import pytest
import torch

from latent_compressed_expert_gb300 import lmoe

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
HALF = 2.0 ** -8
MUON = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    lmoe.load()
    return torch.device("cuda:0")


def _draw(dev, *shape, seed=0, dtype=F, std=1.0):
    g = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=dev) * std).to(dtype)


def _steps(coeffs, steps):
    c = torch.as_tensor(coeffs, dtype=F)  # as the call rounds them
    return c.expand(steps, 3).double().tolist()


def _exact(u, coeffs=MUON, steps=5, eps=1e-7):
    x = u.double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    for a, b, c in _steps(coeffs, steps):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def _rounded(u, coeffs=MUON, steps=5, eps=1e-7):
    def half(v, scale):
        return (v * scale).to(torch.float16).double() / scale

    x = u.double()
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + eps)
    tall = x.shape[-2] > x.shape[-1]
    x = x.mT if tall else x
    for k, (a, b, c) in enumerate(_steps(coeffs, steps)):
        hi = half(x, 2048.0)
        x = hi + half(x - hi, 2048.0) if k + 1 < steps else hi
        p = hi @ hi.mT
        d = torch.diag_embed(p.diagonal(dim1=-2, dim2=-1))
        o = half(p - d, 1024.0)
        full = b * (o + d) + c * (d @ d + d @ o + o @ d + o @ o)
        bd = torch.diag_embed(full.diagonal(dim1=-2, dim2=-1))
        x = a * x + half(full - bd, 256.0) @ hi + bd @ (x if k + 2 >= steps else hi)
    return x.mT if tall else x


def _norm(t):
    return torch.linalg.matrix_norm(t.double())


def _check(got, u, coeffs=MUON, steps=5, eps=1e-7, tag="", worst=None):
    """got (bf16) against the orthogonalisation of u."""
    want, near = _exact(u, coeffs, steps, eps), _rounded(u, coeffs, steps, eps)
    assert torch.isfinite(got.double()).all(), tag
    size, cost = _norm(want), _norm(near - want)
    if worst is not None:  # what the header promises
        assert (cost <= worst * size).all(), (tag, float((cost / size).max()))
    off = _norm(got.double() - want)
    assert (off <= 2 * cost + (2.0 ** -9 + 1e-5) * size).all(), \
        (tag, float((off / size).max()), float((cost / size).max()))
    most = (near - want).abs().amax((-2, -1), keepdim=True)
    rms = (size / (want.shape[-1] * want.shape[-2]) ** 0.5)[..., None, None]
    err = (got.double() - want).abs()
    assert (err <= HALF * want.abs() + 2 * most + 1e-4 * rms).all(), tag


# one element, row and column; a tile's edge; tall and wide; one SM's tiles and SM pairs
SIZES = [(1, 1), (1, 7), (7, 1), (8, 8), (33, 65), (65, 33), (1, 5000), (5000, 1), (128, 1024),
         (129, 130), (300, 257), (512, 768), (1000, 333), (257, 2000), (2050, 136), (1536, 1600)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("dtype", [F, BF])
def test_orthogonalize(dev, rows, cols, dtype):
    m = lmoe.Muon()
    g = _draw(dev, rows, cols, seed=rows + cols, dtype=dtype)
    # Roundings of a few elements do not average out: with one singular value s in 0.67 .. 1.12, where
    # five steps keep it, A is off by up to 2 * 2^-11 of itself, which moves s by at most
    # |b s^2 + 2 c s^4| = 1.4 times that in a step, and the steps after it by |a + 3 b s^2 + 5 c s^4|
    # = 1.3 times each: 2^-10 * 1.4 * (1 + 1.3 + 1.7 + 2.2 + 2.9) = 1.3e-2.
    _check(m.orthogonalize(g), g, tag=(rows, cols), worst=3e-3 if rows * cols >= 64 else 1.3e-2)
    torch.cuda.synchronize()
    assert m.device_error() == lmoe.LMOE_OK


@pytest.mark.parametrize("batch,rows,cols", [(3, 40, 24), (7, 130, 260), (40, 64, 512), (5, 700, 300),
                                             (2, 512, 1024)])
def test_batches(dev, batch, rows, cols):
    m = lmoe.Muon()
    g = _draw(dev, batch, rows, cols, seed=batch) * torch.logspace(-3, 2, batch, device=dev)[:, None, None]
    out = m.orthogonalize(g)
    _check(out, g, tag=(batch, rows, cols), worst=3e-3)
    # a matrix by itself: the same up to the order of sums that its tiles give
    _check(m.orthogonalize(g[1]), g[1], tag="alone")


@pytest.mark.parametrize("rows,cols", [(256, 512), (512, 256), (200, 200)])
def test_spectra(dev, rows, cols):
    """Gradients whose singular values lie far apart."""
    m, side = lmoe.Muon(), min(rows, cols)
    q = torch.linalg.qr(_draw(dev, rows, side, seed=1).double())[0]
    r = torch.linalg.qr(_draw(dev, cols, side, seed=2).double())[0]
    low = _draw(dev, rows, 8, seed=3) @ _draw(dev, 8, cols, seed=4)
    for name, g in (("five decades", q @ torch.diag(torch.logspace(0, -5, side, device=dev).double()) @ r.T),
                    ("rank 8 and noise", low + 1e-3 * _draw(dev, rows, cols, seed=5)),
                    ("rank 8", low), ("orthogonal", q @ r.T),
                    ("rows of all sizes", torch.logspace(0, -3, rows, device=dev)[:, None] *
                     _draw(dev, rows, cols, seed=6)),
                    ("columns of all sizes", torch.logspace(0, -3, cols, device=dev) *
                     _draw(dev, rows, cols, seed=7)),
                    ("constant", torch.full((rows, cols), 0.3, device=dev))):
        g = g.float()
        # equal elements are rounded alike: the bound of one singular value, derived above
        _check(m.orthogonalize(g), g, tag=name, worst=1.3e-2 if name == "constant" else 3e-3)


@pytest.mark.parametrize("steps,coeffs", [(1, MUON), (2, MUON), (8, MUON), (14, (1.5, -0.5, 0.0)),
                                          (3, [(4.0, -6.0, 3.0), (3.0, -3.2, 1.2), (1.875, -1.25, 0.375)])])
def test_steps_and_coefficients(dev, steps, coeffs):
    m = lmoe.Muon(steps=steps, coeffs=coeffs)
    for rows, cols in ((96, 160), (160, 96)):
        g = _draw(dev, rows, cols, seed=steps)
        _check(m.orthogonalize(g), g, coeffs, steps, tag=(steps, rows))


def test_a_convergent_iteration_gives_orthogonal_rows(dev):
    m = lmoe.Muon(steps=20, coeffs=(1.5, -0.5, 0.0))
    o = m.orthogonalize(_draw(dev, 64, 256, seed=1)).double()
    eye = torch.eye(64, device=dev, dtype=torch.float64)
    # entries of rows of length 1, each off by 2^-8 of itself: their products' sums by 2^-8 at most
    assert ((o @ o.T - eye).abs() <= 2 * HALF + 2e-3).all()


@pytest.mark.parametrize("power", [-120, -80, -41, -20, 20, 39, 60, 100])
def test_scale_of_the_gradient(dev, power):
    """A gradient times a power of two gives the same bits, eps aside, at the ends of fp32 too."""
    m = lmoe.Muon(eps=1e-45)
    g = _draw(dev, 100, 60, seed=2).to(BF).float()
    want = m.orthogonalize(g)
    if power < -100:  # keep the smallest values out of fp32's denormals
        g = torch.where(g.abs() < 2.0 ** -5, torch.zeros_like(g), g)
        want = m.orthogonalize(g)
    assert torch.equal(m.orthogonalize(g * 2.0 ** power), want)


def test_zero_and_small_gradients(dev):
    m = lmoe.Muon()
    g = torch.zeros(3, 50, 40, device=dev)
    g[1] = _draw(dev, 50, 40, seed=1) * 1e-9     # eps is of its size
    g[2, 0, 0] = 1e-3
    out = m.orthogonalize(g)
    assert not out[0].any()
    _check(out[1], g[1])
    _check(out[2], g[2])


def test_matrices_that_are_not_finite_stay_alone(dev):
    m = lmoe.Muon()
    for rows, cols in ((60, 90), (90, 60), (300, 500)):
        g = _draw(dev, 5, rows, cols, seed=1)
        want = m.orthogonalize(g)
        bad = g.clone()
        bad[1, 3, 4], bad[3, 0, 0] = float("nan"), float("inf")
        out = m.orthogonalize(bad)
        assert torch.isnan(out[[1, 3]]).all()
        assert torch.equal(out[[0, 2, 4]], want[[0, 2, 4]])


def test_strides_and_views(dev):
    """Gradients as the layer's backward leaves them: halves of rows, interleaved matrices."""
    m = lmoe.Muon()
    both = _draw(dev, 6, 96, 72, seed=1)
    for v in (both[:, :48], both[:, 48:], both[:, :, 8:40], both[:, :, 3:40],
              both.view(6, 96, 9, 8)[:, :, 0], both[::2], both.transpose(0, 1)[:, :, :50],
              both[2], both[2][:, 5:18], both[:, 7:8]):
        _check(m.orthogonalize(v), v, tag=(v.shape, v.stride()))
        assert torch.equal(m.orthogonalize(v), m.orthogonalize(v.contiguous()))
    b = both.to(BF)
    out = torch.zeros(6, 96, 100, dtype=BF, device=dev)
    m.orthogonalize(b, out=out[:, :, 1:73])
    assert torch.equal(out[:, :, 1:73], m.orthogonalize(b))
    assert not out[:, :, 0].any() and not out[:, :, 73:].any()  # nothing beside it
    want = m.orthogonalize(b)
    assert m.orthogonalize(b, out=b) is b and torch.equal(b, want)


def _update64(m, w, g, mom, rate, scale):
    """(momentum, u, w) in 64 bits; the fp32 values of the call's numbers."""
    f = lambda v: float(torch.tensor(v, dtype=F))
    beta = f(m.beta)
    mom = beta * mom.double() + g.double()
    u = g.double() + beta * mom if m.nesterov else mom
    keep, step = 1 - f(rate) * f(m.weight_decay), f(rate) * f(scale)
    o = _exact(u)
    return mom, u, keep * w.double() - step * o, step


@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("shape", [(1, 1), (40, 24), (3, 130, 70), (4, 64, 256), (2, 300, 333),
                                   (512, 1024)])
@pytest.mark.parametrize("kind", ["bf16", "master", "both"])
def test_update(dev, shape, nesterov, kind):
    m = lmoe.Muon(beta=0.9, nesterov=nesterov, weight_decay=0.1)
    dtype = BF if shape[-1] % 3 else F
    master = _draw(dev, *shape, seed=1, std=0.05)
    w = master.to(BF) if kind != "master" else None
    master = None if kind == "bf16" else master
    g, mom = _draw(dev, *shape, seed=2, dtype=dtype), _draw(dev, *shape, seed=3)
    rate, scale = 0.02, 0.2 * max(shape[-2:]) ** 0.5
    for _ in range(2):
        start = w if master is None else master
        mom64, u, w64, step = _update64(m, start, g, mom, rate, scale)
        near, want = _rounded(u), _exact(u)
        m.update(w, g, mom, rate, scale=scale, master=master)
        assert ((mom.double() - mom64).abs() <= 2.0 ** -23 * (mom64.abs() + g.double().abs())).all()
        most = (near - want).abs().amax((-2, -1), keepdim=True)
        rms = want.square().mean((-2, -1), keepdim=True).sqrt()
        e = step * (2 * most + 1e-4 * rms) + 2.0 ** -22 * (w64.abs() + step * want.abs())
        if master is not None:
            assert ((master.double() - w64).abs() <= e).all()
            if w is not None:
                assert torch.equal(w, master.to(BF))
        else:
            assert ((w.double() - w64).abs() <= e + HALF * w64.abs()).all()
    torch.cuda.synchronize()
    assert m.device_error() == lmoe.LMOE_OK


def test_update_of_views(dev):
    m = lmoe.Muon()
    big = {n: _draw(dev, 4, 80, 96, seed=i, std=0.1) for i, n in enumerate(("g", "m", "master"))}
    w = big["master"].to(BF)
    part = lambda t: t[:, 8:72, 16:80]
    before = {n: t.clone() for n, t in big.items()}
    ref = {n: part(t).contiguous() for n, t in big.items()}
    rw = part(w).contiguous()
    m.update(part(w), part(big["g"]), part(big["m"]), 0.1, master=part(big["master"]))
    m.update(rw, ref["g"], ref["m"], 0.1, master=ref["master"])
    assert torch.equal(part(w), rw) and all(torch.equal(part(big[n]), ref[n]) for n in ref)
    for n, t in big.items():  # nothing beside the views
        part(before[n]).copy_(part(t))
        assert torch.equal(before[n], t)


def test_no_elements(dev):
    m = lmoe.Muon()
    for shape in ((0, 5), (5, 0), (0, 3, 4), (2, 0, 4)):
        assert m.orthogonalize(torch.empty(shape, device=dev)).shape == shape


def test_same_bits_streams_and_graphs(dev):
    m = lmoe.Muon(weight_decay=0.05)
    shapes = [(300, 500), (3, 96, 64)]
    gs = [_draw(dev, *s, seed=i) for i, s in enumerate(shapes)]

    def fresh():
        return [(0.1 * torch.ones(s, device=dev)).to(BF) for s in shapes], \
            [torch.zeros(s, device=dev) for s in shapes]

    def step(ws, ms, streams=(None, None)):
        for w, mo, g, s in zip(ws, ms, gs, streams):
            m.update(w, g, mo, 0.1, stream=s)

    ws, ms = fresh()
    for _ in range(3):
        step(ws, ms)
    streams = [torch.cuda.Stream() for _ in shapes]
    w2, m2 = fresh()
    torch.cuda.synchronize()
    for _ in range(3):
        step(w2, m2, streams)
    torch.cuda.synchronize()
    w3, m3 = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(w3, m3)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for got in ((w2, m2), (w3, m3)):
        assert all(torch.equal(a, b) for a, b in zip(ws + ms, got[0] + got[1]))


def test_refusals(dev):
    m = lmoe.Muon()
    g = _draw(dev, 8, 16)
    for bad in (g.half(), g[0], g.t(), g.cpu(), g[None, None]):
        with pytest.raises(ValueError):
            m.orthogonalize(bad)
    with pytest.raises(ValueError):
        m.orthogonalize(g, out=torch.empty(8, 16, device=dev))
    w, mom = g.to(BF), torch.zeros_like(g)
    with pytest.raises(ValueError):
        m.update(None, g, mom, 0.1)
    with pytest.raises(ValueError):
        m.update(w, g, mom.to(BF), 0.1)
    with pytest.raises(ValueError):
        m.update(w[:4], g, mom, 0.1)
    with pytest.raises(lmoe.LmoeError):
        m.update(w, g, g, 0.1)                 # momentum over the gradient
    with pytest.raises(lmoe.LmoeError):
        m.update(w, g, mom, 0.1, master=mom)
    with pytest.raises(lmoe.LmoeError):
        m.update(w, g, mom, float("nan"))
    with pytest.raises(lmoe.LmoeError):
        m.orthogonalize(torch.zeros(1, 16, device=dev).expand(8, 16))  # rows over each other
    for kw in (dict(steps=0), dict(steps=65), dict(coeffs=(1.0, 2.0)), dict(steps=2, coeffs=[MUON] * 3)):
        with pytest.raises(ValueError):
            lmoe.Muon(**kw)
    for kw in (dict(eps=0.0), dict(eps=float("inf")), dict(coeffs=(1.0, float("nan"), 0.0))):
        with pytest.raises(lmoe.LmoeError):
            lmoe.Muon(**kw).orthogonalize(g)


@pytest.mark.parametrize("shape", [(40, 64), (1024, 1100)])
def test_stalled_wait_is_reported(dev, monkeypatch, shape):
    m = lmoe.Muon()
    g = _draw(dev, *shape, seed=1)
    want = m.orthogonalize(g)
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "50")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    m.orthogonalize(g)
    torch.cuda.synchronize()
    assert m.device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    assert torch.equal(m.orthogonalize(g), want)
    torch.cuda.synchronize()
    assert m.device_error() == lmoe.LMOE_OK


@pytest.mark.parametrize("steps,coeffs,worst", [(5, MUON, 1e-3), (8, MUON, 3e-3), (12, MUON, 5e-3),
                                                (14, (1.5, -0.5, 0.0), 4e-4)])
def test_accuracy_that_the_header_names(dev, steps, coeffs, worst):
    """Well-conditioned matrices (their smaller side's singular values within a factor of ten), by either
    form, tall and wide.  "Or so" is a quarter."""
    m = lmoe.Muon(steps=steps, coeffs=coeffs)
    for rows, cols in ((96, 160), (160, 96), (128, 1024), (512, 768), (1000, 333)):
        g = _draw(dev, rows, cols, seed=steps + rows)
        _check(m.orthogonalize(g), g, coeffs, steps, tag=(steps, rows, cols), worst=1.25 * worst)


@pytest.mark.parametrize("rows,cols", [(2, 16), (16, 2), (200, 300), (300, 200)])
def test_singular_values_up_to_eight(dev, rows, cols):
    """What the header calls safe: one singular value, brought to 8, of two equal rows (or columns), where A
    has 32 off its diagonal, and by 8 (1 - 1/2 + 1/4) to 6."""
    coeffs = [(8.0, 0.0, 0.0), (1.0, -1 / 128, 1 / 16384)]
    m = lmoe.Muon(steps=2, coeffs=coeffs)
    g = torch.zeros(rows, cols, device=dev)
    (g if rows < cols else g.mT)[:2] = _draw(dev, 1, max(rows, cols), seed=rows)
    out = m.orthogonalize(g)
    _check(out, g, coeffs, 2, tag=(rows, cols), worst=1.3e-2)
    assert abs(float(_norm(out)) - 6) <= 6 * (HALF + 1.3e-2)
