"""Residual addition with RMSNorm and its gradients against plain 64-bit arithmetic.

Tolerances, derived: an output rounded to bf16 is off by at most half a step, 2^-8 of its value.
Before that rounding the fp32 arithmetic is off by at most REL of the value: the sum of squares
is added in chains of at most 79 terms per thread and a tree (relative error below 90 * 2^-24,
half of it in rstd), and a handful of further operations at 2^-24 each; 64 * 2^-24 = 2^-18 covers
them.  The gradients subtract two terms, so their bound is REL times the sum of the terms'
magnitudes.  An e4m3 code is compared through what it stands for: half an e4m3 step, 2^-4 of the
value (2^-10 of the scale for subnormals), plus REL."""
import numpy as np
import pytest
import torch

from latent_compressed_expert_gb300 import lmoe

pytestmark = pytest.mark.gpu
BF, REL, HALF = torch.bfloat16, 2.0 ** -18, 2.0 ** -8


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    lmoe.load()
    return torch.device("cuda:0")


def _draw(dev, rows, cols, seed, ld=None, off=0):
    """[rows, cols] bf16 normal values, as a view with row stride ld that starts at element off."""
    g = torch.Generator(device=dev).manual_seed(seed)
    ld = cols if ld is None else ld
    buf = torch.randn(off + rows * ld, generator=g, device=dev).to(BF)
    return buf[off:].view(rows, ld)[:, :cols]


def _ref(x, res, gamma, eps):
    t = x.double() if res is None else x.double() + res.double()
    r = (t.square().mean(1, keepdim=True) + eps).rsqrt()
    return t, r, t * r * gamma.double()


def _close(got, want, extra=None, tag=""):
    err = (got.double() - want).abs()
    bound = (HALF + REL) * want.abs() + (0 if extra is None else extra) + 1e-38
    assert torch.isfinite(got.double()).all(), tag
    assert (err <= bound).all(), (tag, float((err / bound).max()))


# rows x cols: one token, the widths of the layer, several rows per block, short rows, both
# ends of the whole-row kernels, wider than they take, and widths that are no multiple of 8
SHAPES = [(1, 7168), (3, 7168), (305, 7168), (700, 3584), (1000, 256), (65, 8), (7, 16384),
          (310, 16384), (2, 16392), (40, 20000), (5, 1001), (400, 1001), (2, 1), (33, 9)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("with_res", [True, False])
def test_forward(dev, rows, cols, with_res):
    x = _draw(dev, rows, cols, rows + cols)
    res = 3.0 * _draw(dev, rows, cols, rows + cols + 1) if with_res else None
    gamma = torch.rand(cols, device=dev) + 0.5
    t, r, y64 = _ref(x, res, gamma, 1e-6)
    y, total, rstd = lmoe.add_rmsnorm(x, gamma, res, train=True)
    _close(y, y64, tag="y")
    assert torch.equal(total, (x.float() + res.float()).to(BF) if with_res else x)
    assert ((rstd.double() - r.squeeze(1)).abs() <= REL * r.squeeze(1)).all()
    y2, _ = lmoe.add_rmsnorm(x, gamma, res)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward_e4m3(dev, rows, cols):
    x, res = _draw(dev, rows, cols, rows), _draw(dev, rows, cols, cols)
    gamma = torch.rand(cols, device=dev) + 0.5
    _, _, y64 = _ref(x, res, gamma, 1e-6)
    codes, scales, total = lmoe.add_rmsnorm_e4m3(x, gamma, res)
    s64 = y64.abs().amax(1) / 448.0
    assert ((scales.double() - s64).abs() <= REL * s64).all()
    val = codes.view(torch.float8_e4m3fn).double() * scales.double().unsqueeze(1)
    err = (val - y64).abs()
    bound = (2.0 ** -4 + REL) * y64.abs() + (2.0 ** -10 + REL) * s64.unsqueeze(1)
    assert (err <= bound).all(), float((err / bound).max())
    assert torch.equal(total, (x.float() + res.float()).to(BF))


@pytest.mark.parametrize("ld,off", [(7176, 8), (7175, 0), (7168, 1), (8000, 16)])
@pytest.mark.parametrize("fp8", [False, True])
def test_strides_and_alignment(dev, ld, off, fp8):
    """Strided and odd-aligned rows give the bits of the same rows packed (the sums of the
    two kernels run in other orders, so within the bound where the kernel differs)."""
    rows, cols = 9, 7168
    x, res = _draw(dev, rows, cols, 1, ld, off), _draw(dev, rows, cols, 2, ld + 8, off)
    gamma = torch.rand(cols, device=dev) + 0.5
    _, _, y64 = _ref(x, res, gamma, 1e-6)
    if fp8:
        codes, scales, total = lmoe.add_rmsnorm_e4m3(x, gamma, res)
        val = codes.view(torch.float8_e4m3fn).double() * scales.double().unsqueeze(1)
        bound = (2.0 ** -4 + REL) * y64.abs() + (2.0 ** -10 + REL) * scales.double().unsqueeze(1)
        assert ((val - y64).abs() <= bound).all()
    else:
        buf = torch.full((rows, ld + 3), 7.0, dtype=BF, device=dev)
        y, total = lmoe.add_rmsnorm(x, gamma, res, y=buf[:, 1:cols + 1])
        _close(y, y64)
        assert (buf[:, 0] == 7.0).all() and (buf[:, cols + 1:] == 7.0).all()
    assert torch.equal(total, (x.float() + res.float()).to(BF))


@pytest.mark.parametrize("cols", [7168, 1001])
def test_in_place(dev, cols):
    """total over residual and y over x: the running residual stream of a decoder."""
    x, res = _draw(dev, 50, cols, 1), _draw(dev, 50, cols, 2)
    gamma = torch.rand(cols, device=dev) + 0.5
    y0, t0 = lmoe.add_rmsnorm(x, gamma, res)
    x1, r1 = x.clone(), res.clone()
    y1, t1 = lmoe.add_rmsnorm(x1, gamma, r1, y=x1, total=r1)
    assert y1.data_ptr() == x1.data_ptr() and t1.data_ptr() == r1.data_ptr()
    assert torch.equal(y0, y1) and torch.equal(t0, t1)


def test_zero_and_non_finite_rows(dev):
    gamma = torch.ones(512, device=dev)
    x = _draw(dev, 4, 512, 3).clone()
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 7] = float("inf")
    y, total = lmoe.add_rmsnorm(x, gamma)
    assert total is x
    assert (y[0] == 0).all() and torch.isnan(y[1]).all()
    assert torch.isnan(y[2, 7]) and (y[2, :7] == 0).all()   # inf * (1/inf), x * (1/inf)
    _close(y[3:], _ref(x[3:], None, gamma, 1e-6)[2])
    codes, scales, _ = lmoe.add_rmsnorm_e4m3(x, gamma)
    assert float(scales[0]) == 1.0 and (codes[0] == 0).all()
    assert torch.isnan(codes[1].view(torch.float8_e4m3fn).float()).all()


def test_no_rows(dev):
    gamma = torch.ones(64, device=dev)
    x = torch.empty(0, 64, dtype=BF, device=dev)
    y, total = lmoe.add_rmsnorm(x, gamma, x)
    assert y.shape == (0, 64) and total.shape == (0, 64)
    dx, dg = lmoe.add_rmsnorm_backward(x, x, gamma, torch.empty(0, device=dev))
    assert dx.shape == (0, 64) and (dg == 0).all()


def _bwd_ref(dy, total, gamma, rstd, dt):
    d, t, r = dy.double(), total.double(), rstd.double().unsqueeze(1)
    xh, g = t * r, d * gamma.double()
    dot = (g * xh).mean(1, keepdim=True)
    dx = (g - xh * dot) * r + (0 if dt is None else dt.double())
    mag = (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) * r
    mag = mag + (0 if dt is None else dt.double().abs())
    return dx, mag, (d * xh).sum(0), (d * xh).abs().sum(0)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("with_dt", [True, False])
def test_backward(dev, rows, cols, with_dt):
    dy, total = _draw(dev, rows, cols, 1), 2.0 * _draw(dev, rows, cols, 2)
    dt = _draw(dev, rows, cols, 3) if with_dt else None
    gamma = torch.rand(cols, device=dev) + 0.5
    rstd = (total.double().square().mean(1) + 1e-6).rsqrt().float()
    dx64, mag, dg64, dgmag = _bwd_ref(dy, total, gamma, rstd, dt)
    dx, dg = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt)
    _close(dx, dx64, extra=REL * mag, tag="dx")
    # a column's sum: at most 64 rows per chain here, then at most 64 partials and a tree
    assert ((dg.double() - dg64).abs() <= 2.0 ** -17 * dgmag + 1e-38).all()
    dx2, none = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt, want_dgamma=False)
    assert none is None and torch.equal(dx, dx2)
    again = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt)
    assert torch.equal(again[1], dg)                        # a fixed order


@pytest.mark.parametrize("cols", [1024, 1001])
def test_backward_in_place_and_strided(dev, cols):
    dy, total = _draw(dev, 600, cols, 1), _draw(dev, 600, cols, 2)
    dt = _draw(dev, 600, cols, 3)
    gamma = torch.rand(cols, device=dev) + 0.5
    rstd = (total.double().square().mean(1) + 1e-6).rsqrt().float()
    dx, dg = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt)
    for over in ("dy", "dtotal"):
        d, t = dy.clone(), dt.clone()
        o, g = lmoe.add_rmsnorm_backward(d, total, gamma, rstd, t, dx=d if over == "dy" else t)
        assert torch.equal(o, dx) and torch.equal(g, dg), over
    wide = torch.zeros(600, cols + 24, dtype=BF, device=dev)
    o, g = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt, dx=wide[:, 8:cols + 8])
    assert torch.equal(o, dx) and torch.equal(g, dg)
    assert (wide[:, :8] == 0).all() and (wide[:, cols + 8:] == 0).all()


def test_backward_is_the_slope_of_the_forward(dev):
    """dx and dgamma against central differences of the formula in 64 bits, on the device's
    own dy, along random directions."""
    rows, cols, eps = 5, 64, 1e-3
    total = _draw(dev, rows, cols, 1)
    gamma = torch.rand(cols, device=dev) + 0.5
    dy = _draw(dev, rows, cols, 2)
    rstd = lmoe.add_rmsnorm(total, gamma, eps=eps, train=True)[2]
    dx, dg = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd)

    def loss(t, g):
        return float((dy.double() * t * (t.square().mean(1, keepdim=True) + eps).rsqrt() * g).sum())

    t, g, h = total.double(), gamma.double(), 1e-4
    for seed in range(4):
        gen = torch.Generator(device=dev).manual_seed(seed)
        vt = torch.randn(rows, cols, generator=gen, device=dev, dtype=torch.float64)
        vg = torch.randn(cols, generator=gen, device=dev, dtype=torch.float64)
        for name, num, ana, mag in (
                ("dx", (loss(t + h * vt, g) - loss(t - h * vt, g)) / (2 * h),
                 (dx.double() * vt).sum(), (dx.double() * vt).abs().sum()),
                ("dgamma", (loss(t, g + h * vg) - loss(t, g - h * vg)) / (2 * h),
                 (dg.double() * vg).sum(), (dg.double() * vg).abs().sum())):
            # dx is rounded to bf16 (2^-8 of each term); the difference's own error is O(h^2)
            assert abs(num - float(ana)) <= (HALF + 1e-5) * float(mag), (name, num, float(ana))


def test_other_stream_and_graph(dev):
    """On a stream of the caller's, and captured into a CUDA graph and replayed on new data."""
    x, res = _draw(dev, 300, 1024, 1), _draw(dev, 300, 1024, 2)
    gamma = torch.rand(1024, device=dev) + 0.5
    want = lmoe.add_rmsnorm(x, gamma, res)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = lmoe.add_rmsnorm(x, gamma, res, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rstd = lmoe.add_rmsnorm(x, gamma, res, train=True)[2]
    xs, out = x.clone(), None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lmoe.add_rmsnorm(xs, gamma, res)
        grads = lmoe.add_rmsnorm_backward(xs, out[1], gamma, rstd, res)
    xs.copy_(2 * x)
    graph.replay()
    want = lmoe.add_rmsnorm(2 * x, gamma, res)
    wg = lmoe.add_rmsnorm_backward(2 * x, want[1], gamma, rstd, res)
    assert torch.equal(out[0], want[0]) and torch.equal(grads[0], wg[0])
    assert torch.equal(grads[1], wg[1])


def test_offsets_past_32_bits(dev):
    """Rows whose byte and element offsets pass 2^32 (a wide row stride over one buffer)."""
    rows, cols, ld = 3, 1024, 1 << 31
    try:
        buf = torch.empty(2 * ld + cols, dtype=BF, device=dev)
    except torch.OutOfMemoryError:
        pytest.skip("needs 9 GB")
    x = buf.as_strided((rows, cols), (ld, 1))
    x.copy_(_draw(dev, rows, cols, 5))
    gamma = torch.rand(cols, device=dev) + 0.5
    y, _ = lmoe.add_rmsnorm(x, gamma)
    want, _ = lmoe.add_rmsnorm(x.contiguous(), gamma)
    assert torch.equal(y, want)


def test_refusals(dev):
    x, gamma = _draw(dev, 4, 64, 1), torch.ones(64, device=dev)
    for bad in (lambda: lmoe.add_rmsnorm(x.float(), gamma),
                lambda: lmoe.add_rmsnorm(x, gamma.to(BF)),
                lambda: lmoe.add_rmsnorm(x, gamma[:32]),
                lambda: lmoe.add_rmsnorm(x, gamma, x[:2]),
                lambda: lmoe.add_rmsnorm(x.t(), torch.ones(4, device=dev)),
                lambda: lmoe.add_rmsnorm(x.cpu(), gamma),
                lambda: lmoe.add_rmsnorm_backward(x, x, gamma, gamma),
                lambda: lmoe.add_rmsnorm_backward(x, x[:, :32], gamma, torch.ones(4, device=dev))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lmoe.LmoeError):
        lmoe.add_rmsnorm(x, gamma, eps=-1.0)


@pytest.mark.parametrize("cols,with_dt", [(7168, True), (2048, False)])
def test_stalled_wait_reports_timeout_and_recovers(dev, monkeypatch, cols, with_dt):
    """A device-side wait that runs out (a barrier nothing arrives on): the call ends, it is reported,
    no row passes for a gradient, and the next call is correct."""
    rows = 2000
    dy, total = _draw(dev, rows, cols, 1), _draw(dev, rows, cols, 2)
    dt = _draw(dev, rows, cols, 3) if with_dt else None
    gamma = torch.rand(cols, device=dev) + 0.5
    rstd = (total.double().square().mean(1) + 1e-6).rsqrt().float()
    want = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt)
    torch.cuda.synchronize()
    assert lmoe.norm_device_error() == lmoe.LMOE_OK
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "100")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    dx, dg = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt)
    torch.cuda.synchronize()
    assert lmoe.norm_device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    assert lmoe.norm_device_error() == lmoe.LMOE_OK
    assert torch.isnan(dx.float()).all() and torch.isnan(dg).all()
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    dx, dg = lmoe.add_rmsnorm_backward(dy, total, gamma, rstd, dt)
    assert torch.equal(dx, want[0]) and torch.equal(dg, want[1])


@pytest.mark.parametrize("rows", [0, 5, 700])
@pytest.mark.parametrize("train", [False, True])
def test_y_over_x_without_a_residual(dev, rows, train):
    """The total that is returned is x as it was, not the y that lies there now."""
    x, gamma = _draw(dev, rows, 512, 1), torch.rand(512, device=dev) + 0.5
    want = lmoe.add_rmsnorm(x, gamma, train=train)
    over = x.clone()
    got = lmoe.add_rmsnorm(over, gamma, train=train, y=over)
    assert got[0] is over and len(got) == len(want)
    assert all(torch.equal(g, w) for g, w in zip(got, want)) and torch.equal(got[1], x)
