"""The layer for a few tokens in one kernel (lmoe_forward_few) against plain 64-bit arithmetic.

Routing is checked first: the logits within the derived bound of the 64-bit ones, the selection and
gates bit for bit what the routing rule gives on those logits.  With that routing the output is
held to the layer's stated tolerance (gpu_helpers): before its bf16 store, max |err| <= 2e-2 RMS
and mean relative error <= 5e-3.  e4m3 experts: an operand within ~2^-17 of a code boundary may
take the neighbouring code, which moves an output by one e4m3 step (2^-3) of that element's share:
max |err| <= 2^-3 RMS, the same mean bound.

Logits: the latent is an fp32 sum of d exact products (error <= d 2^-23 sum|x||w|), taken by the
router as two bf16 terms (2^-16 of it left), and the router's own sum is fp32 too."""
from dataclasses import replace

import numpy as np
import pytest
import torch

import gpu_helpers as H
from latent_compressed_expert_gb300 import lmoe, synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    lmoe.load()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def k3(dev):
    """K3's widths, one layer for the module: (shape, weights on the device, bf16 layer)."""
    w = synth.make_weights(synth.DECODE, seed=3, device=dev)
    return synth.DECODE, w, lmoe.Layer(synth.DECODE, w, max_tokens=64)


def _situ(g, v, c):
    g, v = c * torch.tanh(g / c), c * torch.tanh(v / c)
    return g * torch.sigmoid(g) * v


def _codes64(v):
    """Values that e4m3 codes with a scale per row stand for, from 64-bit rows."""
    s = (v.abs().amax(-1, keepdim=True) / 448).float()
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (v / s).float().to(torch.float8_e4m3fn).double() * s.double()


def _reference(sh, w, x, idx, gate, residual, fp8):
    x64 = x.double()
    lat = x64 @ w["w_down"].double().T
    a = _codes64(lat) if fp8 else lat
    z = torch.empty_like(lat)
    for t in range(x.shape[0]):
        e = idx[t].long()
        wg, wv, wd = (w[n][e] for n in ("w_gate", "w_value", "w_edown"))
        wg, wv, wd = ((_codes64(m.double()) if fp8 else m.double()) for m in (wg, wv, wd))
        h = _situ(wg @ a[t], wv @ a[t], sh.c)
        h = _codes64(h) if fp8 else h
        u = (gate[t].double()[:, None] * (wd @ h.unsqueeze(-1)).squeeze(-1)).sum(0)
        z[t] = w["gamma"].double() * u * (u.square().mean() + sh.eps).rsqrt()
    y = z @ w["w_up"].double().T
    for s in range(sh.S):
        y += _situ(x64 @ w["w_sgate"][s].double().T, x64 @ w["w_svalue"][s].double().T, sh.c) \
            @ w["w_sdown"][s].double().T
    return y if residual is None else y + residual.double()


def _check_logits(sh, w, x, logits, bias=None):
    x64, wd, wr = x.double(), w["w_down"].double(), w["w_router"].double()
    lat = x64 @ wd.T
    want = lat @ wr.T + (0 if bias is None else bias.double())
    e_lat = sh.d * 2.0 ** -23 * (x64.abs() @ wd.abs().T) + 2.0 ** -16 * lat.abs()
    bound = e_lat @ wr.abs().T + sh.L * 2.0 ** -22 * (lat.abs() @ wr.abs().T) \
        + 2.0 ** -22 * want.abs()
    assert ((logits.double() - want).abs() <= bound).all()


def _check(oracle_mod, sh, w, layer, x, tau=None, residual=None, bias=None, logits=None, tag=""):
    y, dbg = layer.forward_few(x, residual=residual, tau=tau, logit_bias=bias, logits_in=logits,
                               debug=True)
    torch.cuda.synchronize()
    assert layer.few_device_error() == lmoe.LMOE_OK and layer.last_kernel_launches == 1
    if logits is None:
        _check_logits(sh, w, x, dbg["logits"], bias)
    else:
        assert torch.equal(dbg["logits"], logits)
    r_idx, r_gate, _ = oracle_mod.route(dbg["logits"].cpu().numpy(),
                                        None if tau is None else tau.cpu().numpy(), sh.K)
    assert np.array_equal(dbg["idx"].cpu().numpy(), r_idx), tag
    assert np.array_equal(dbg["gate"].cpu().numpy().view(np.int32), r_gate.view(np.int32)), tag
    ref = _reference(sh, w, x, dbg["idx"], dbg["gate"], residual, layer.expert_fp8).cpu().numpy()
    if layer.expert_fp8:
        assert torch.equal(dbg["y_f32"].to(torch.bfloat16), y), tag
        st = H.error_stats(H._np(dbg["y_f32"]), ref)
        assert st["max_err_over_rms"] <= 2.0 ** -3 and st["mean_rel_err"] <= H.MEAN_REL_ERR, (tag, st)
    else:
        H.assert_layer_close(y, dbg["y_f32"], ref, tag)
    again = layer.forward_few(x, residual=residual, tau=tau, logit_bias=bias, logits_in=logits)
    assert torch.equal(again, y), tag      # the same bits every time, with and without debug
    return y


def _tau(sh, seed, dev):
    return torch.sigmoid(1.5 + 0.3 * torch.randn(sh.E, generator=torch.Generator().manual_seed(seed))
                         ).to(dev)


SHAPES = [
    synth.TINY,
    H.mid_shape(8),
    synth.LayerShape("noshared", T=8, d=128, L=64, E=32, K=4, I=64, S=0, Is=0),
    # widths that are no multiple of the 128-row weight tiles, one expert per token
    synth.LayerShape("odd", T=8, d=320, L=192, E=48, K=1, I=192, S=1, Is=64),
    # every expert for every token; 32 experts per token
    synth.LayerShape("all", T=8, d=256, L=128, E=16, K=16, I=64, S=1, Is=64),
    synth.LayerShape("k32", T=8, d=256, L=128, E=4096, K=32, I=128, S=2, Is=64),
]


@pytest.mark.parametrize("sh", SHAPES, ids=lambda s: s.name)
@pytest.mark.parametrize("T", [1, 2, 5, 8])
def test_small_shapes(dev, oracle_mod, sh, T):
    w = synth.make_weights(sh, seed=T, device=dev, hot_row_frac=0.01)
    w["gamma"] = torch.linspace(0.5, 1.5, sh.L, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=T, device=dev, T=T)
    _check(oracle_mod, sh, w, layer, x, tag=(sh.name, T))
    _check(oracle_mod, sh, w, layer, x, tau=_tau(sh, T, dev), residual=synth.make_x(
        sh, seed=T + 50, device=dev, T=T), bias=torch.randn(sh.E, device=dev), tag=(sh.name, T))


@pytest.mark.parametrize("sh", [H.mid_shape(8), SHAPES[5]], ids=lambda s: s.name)
@pytest.mark.parametrize("T", [1, 3, 8])
def test_small_shapes_e4m3(dev, oracle_mod, sh, T):
    w = synth.make_weights(sh, seed=T, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8, expert_fp8=True)
    x = synth.make_x(sh, seed=T, device=dev, T=T)
    _check(oracle_mod, sh, w, layer, x, tau=_tau(sh, T, dev), residual=x, tag=(sh.name, T))


@pytest.mark.parametrize("T", [1, 3, 8])
def test_k3(k3, oracle_mod, T):
    sh, w, layer = k3
    x = synth.make_x(sh, seed=T, device=layer.device, T=T)
    tau = torch.sigmoid(2.1 + 0.1 * torch.randn(sh.E, device=layer.device))
    _check(oracle_mod, sh, w, layer, x, tau=tau, residual=x, tag=("k3", T))


def test_k3_e4m3(k3, oracle_mod):
    sh, w, _ = k3
    layer = lmoe.Layer(sh, w, max_tokens=8, expert_fp8=True)
    for T in (1, 8):
        x = synth.make_x(sh, seed=T, device=layer.device, T=T)
        _check(oracle_mod, sh, w, layer, x, residual=x, tag=("k3 e4m3", T))


def test_tokens_that_share_their_experts(dev, oracle_mod):
    """Eight equal rows (every expert read once for all of them), and rows that share some."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=1, device=dev, T=1).expand(8, -1).contiguous()
    y = _check(oracle_mod, sh, w, layer, x)
    assert all(torch.equal(y[i], y[0]) for i in range(8))
    logits = synth.make_logits(8, sh.E, seed=4).to(dev)
    logits[:, :4] += 10.0
    _check(oracle_mod, sh, w, layer, synth.make_x(sh, seed=2, device=dev, T=8), logits=logits)


def test_a_token_does_not_depend_on_its_neighbours(dev):
    """A token's output is the same bits alone and among others: columns of the products are
    separate, and the split of a reduction does not depend on the batch (the order in which its
    experts are added does, so the check is on logits and on equal batches' rows)."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=3, device=dev, T=8)
    full = layer.forward_few(x, debug=True)[1]
    for t in (0, 5):
        one = layer.forward_few(x[t:t + 1].contiguous(), debug=True)[1]
        assert torch.equal(one["logits"][0], full["logits"][t])
        assert torch.equal(one["idx"][0], full["idx"][t])
        assert torch.equal(one["gate"][0], full["gate"][t])


def test_ties_and_saturated_scores(dev, oracle_mod):
    """Exact ties in the keys (all logits equal; scores at 1) go to the lower expert."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=3, device=dev, T=4)
    for value in (0.0, 40.0, -100.0):
        _check(oracle_mod, sh, w, layer, x, logits=torch.full((4, sh.E), value, device=dev))


def test_agrees_with_forward(k3):
    """lmoe_forward on the same routing (given logits): the layer's tolerance."""
    sh, w, layer = k3
    x = synth.make_x(sh, seed=9, device=layer.device, T=6)
    logits = synth.make_logits(6, sh.E, seed=9).to(layer.device)
    y0 = layer.forward(x, residual=x, logits_in=logits, balance=False)
    y1 = layer.forward_few(x, residual=x, logits_in=logits)
    H.assert_close(y1.float().cpu().numpy(), y0.float().cpu().numpy(), "few vs forward")


def test_outliers_and_zero_rows(dev, oracle_mod):
    """x with 1000x outliers (pre-activations past the cap), and a token of zeros."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=5, device=dev, hot_row_frac=0.02)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=5, device=dev, T=4, outlier_frac=0.01)
    _check(oracle_mod, sh, w, layer, x)
    x[2] = 0
    y = layer.forward_few(x, residual=x)
    assert (y[2] == 0).all() and torch.isfinite(y.float()).all()


def test_no_tokens_and_workspace_reuse(dev):
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    assert layer.forward_few(torch.empty(0, sh.d, dtype=torch.bfloat16, device=dev)).shape == (0, sh.d)
    xs = [synth.make_x(sh, seed=t, device=dev, T=t) for t in (8, 1, 5, 2, 8)]
    want = [layer.forward_few(x) for x in xs]
    for _ in range(20):     # back to back, batch sizes in turn on one workspace
        got = [layer.forward_few(x) for x in xs]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    assert layer.few_device_error() == lmoe.LMOE_OK
    assert (layer.few_ws[:256] == 0).all()


def test_stream_and_graph(dev):
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=7, device=dev, T=3)
    want = layer.forward_few(x, residual=x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer.forward_few(x, residual=x, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    xs = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(3):
            yg = layer.forward_few(xs, residual=xs)
    xs.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(yg, want) and layer.few_device_error() == lmoe.LMOE_OK


def test_stalled_wait_reports_timeout_and_recovers(dev, monkeypatch):
    """The first grid-wide barrier waits for one arrival too many: every CTA gives up within the
    limit, the call reports it, and the next call is correct."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8)
    x = synth.make_x(sh, seed=7, device=dev, T=3)
    want = layer.forward_few(x)
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "100")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    layer.forward_few(x)
    torch.cuda.synchronize()
    assert layer.few_device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    assert layer.few_device_error() == lmoe.LMOE_OK
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    assert torch.equal(layer.forward_few(x), want)


def test_refusals(dev):
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=16)
    x = synth.make_x(sh, seed=7, device=dev, T=9)
    with pytest.raises(ValueError):
        layer.forward_few(x)                                     # more than eight tokens
    for bad in (lambda: layer.forward_few(x[:2].float()), lambda: layer.forward_few(x[:2, :64]),
                lambda: layer.forward_few(x[:2], tau=torch.zeros(3, device=dev)),
                lambda: layer.forward_few(x[:2], residual=x[:3]),
                lambda: layer.forward_few(x[:2].cpu())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(lmoe.LmoeError):
        layer.forward_few(x[:2], y=x[:2])                        # y may not be x
    # operands that do not fit an SM's shared memory: fewer tokens, or none at all
    wide = replace(sh, d=16384, L=64, E=16, K=1, I=64, S=1, Is=64)
    wl = lmoe.Layer(wide, synth.make_weights(wide, seed=1, device=dev), max_tokens=8)
    with pytest.raises(ValueError):
        wl.forward_few(synth.make_x(wide, seed=1, device=dev, T=8))
    wl.forward_few(synth.make_x(wide, seed=1, device=dev, T=2))


@pytest.mark.parametrize("fp8", [False, True])
def test_nan(dev, fp8):
    """NaN in a token, in an expert's weights and in a shared expert's: the outputs that depend on
    them are NaN, as Layer.forward's are, and no others."""
    sh = H.mid_shape(8)
    clean = synth.make_weights(sh, seed=1, device=dev)
    x = synth.make_x(sh, seed=3, device=dev, T=3)
    # routing given: tokens 0 and 2 share expert 5
    logits = torch.full((3, sh.E), -8.0, device=dev)
    logits[0, 0:8] = logits[1, 8:16] = logits[2, 5:13] = 1.0
    nan = float("nan")
    layer = lmoe.Layer(sh, clean, max_tokens=8, expert_fp8=fp8)
    base = layer.forward_few(x, logits_in=logits)
    assert torch.isfinite(base.float()).all()
    bad = x.clone()
    bad[1, 7] = nan
    cases = [(clean, bad, [1])]
    for name, at, tokens in (("w_gate", (5, 3, 9), [0, 2]), ("w_value", (9, 3, 9), [1, 2]),
                             ("w_sgate", (1, 3, 9), [0, 1, 2]),
                             ("w_svalue", (0, 3, 9), [0, 1, 2])):
        w = dict(clean)
        w[name] = clean[name].clone()
        w[name][at] = nan
        cases.append((w, x, tokens))
    for i, (w, xi, tokens) in enumerate(cases):
        layer = lmoe.Layer(sh, w, max_tokens=8, expert_fp8=fp8)
        y = layer.forward_few(xi, logits_in=logits)
        full = layer.forward(xi, logits_in=logits, balance=False)
        assert torch.isnan(full[tokens].float()).all(), i
        assert torch.isnan(y[tokens].float()).all(), i
        others = [t for t in range(3) if t not in tokens]
        assert torch.equal(y[others], base[others]), i


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_an_expert_that_is_not_finite_spoils_its_own_tokens(dev, fp8, value):
    """A NaN or an infinity in an expert's down projection reaches the tokens that use the expert and
    no others of the batch, whether they share experts with those or not."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    x = synth.make_x(sh, seed=3, device=dev, T=3)
    logits = torch.full((3, sh.E), -8.0, device=dev)
    logits[0, 0:8] = logits[1, 8:16] = logits[2, 5:13] = 1.0
    base = lmoe.Layer(sh, w, max_tokens=8, expert_fp8=fp8).forward_few(x, logits_in=logits)
    for expert, tokens in ((0, [0]), (9, [1, 2])):
        bad = dict(w)
        bad["w_edown"] = w["w_edown"].clone()
        bad["w_edown"][expert, 3, 9] = value
        layer = lmoe.Layer(sh, bad, max_tokens=8, expert_fp8=fp8)
        y = layer.forward_few(x, logits_in=logits)
        full = layer.forward(x, logits_in=logits, balance=False)
        others = [t for t in range(3) if t not in tokens]
        assert torch.equal(y[others], base[others])
        assert torch.equal(y[tokens].isnan(), full[tokens].isnan())
        assert not torch.equal(y[tokens], base[tokens])


def test_two_threads_with_layers_of_different_sizes(dev):
    """Calls of different batch sizes from two host threads, each on a workspace of its own and both
    on one stream: every launch is accepted and every output right."""
    import ctypes
    import threading

    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    work = []
    for T in (1, 8):
        layer = lmoe.Layer(sh, w, max_tokens=8)
        x = synth.make_x(sh, seed=T, device=dev, T=T)
        work.append((layer, x, layer.forward_few(x), torch.empty_like(x)))
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream().cuda_stream
    codes = [[], []]

    def run(i):
        layer, x, _, y = work[i]
        lib, D = lmoe.load(), ctypes.byref(layer._few_dims[x.shape[0]])
        args = [ctypes.c_void_p(t.data_ptr()) for t in (layer.packed, x)] + [None] + \
            [ctypes.c_void_p(t.data_ptr()) for t in (y, layer.few_ws)]
        for _ in range(4000):
            codes[i].append(lib.lmoe_forward_few(D, *args, layer.few_ws.numel(), None, stream))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(c == lmoe.LMOE_OK for part in codes for c in part), [
        sum(c != 0 for c in part) for part in codes]
    for layer, _, want, y in work:
        assert torch.equal(y, want) and layer.few_device_error() == lmoe.LMOE_OK


def test_first_call_under_capture(dev):
    """It is refused, the capture goes on, and the layer works afterwards."""
    sh = H.mid_shape(8)
    layer = lmoe.Layer(sh, synth.make_weights(sh, seed=1, device=dev), max_tokens=8)
    x = synth.make_x(sh, seed=7, device=dev, T=3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(ValueError):
            layer.forward_few(x)
        twice = x + x
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(twice, 2 * x) and layer.few_ws is None
    y = layer.forward_few(x)
    torch.cuda.synchronize()
    assert layer.few_device_error() == lmoe.LMOE_OK
    assert torch.equal(layer.forward_few(x), y)


def test_a_latent_past_the_range(dev, oracle_mod):
    """One latent feature overflows to an infinity: logits of its sign, gates and values at their
    caps, finite outputs, as in Layer.forward."""
    sh = H.mid_shape(8)
    w = synth.make_weights(sh, seed=1, device=dev)
    x = synth.make_x(sh, seed=3, device=dev, T=1)
    w["w_down"] = w["w_down"].clone()
    w["w_down"][3] = 1e38 * torch.sign(x[0])
    layer = lmoe.Layer(sh, w, max_tokens=8)
    y, dbg = layer.forward_few(x, debug=True)
    assert torch.equal(dbg["logits"][0], torch.sign(w["w_router"][:, 3].float()) * float("inf"))
    idx, gate, _ = oracle_mod.route(dbg["logits"].cpu().numpy(), None, sh.K)
    assert np.array_equal(dbg["idx"].cpu().numpy(), idx)
    ref = _reference(sh, w, x, dbg["idx"], dbg["gate"], None, False).cpu().numpy()
    H.assert_layer_close(y, dbg["y_f32"], ref)
    full = layer.forward(x, logits_in=dbg["logits"], balance=False)
    H.assert_close(y.float().cpu().numpy(), full.float().cpu().numpy(), "few vs forward")


@pytest.mark.parametrize("T", [1, 8])
@pytest.mark.parametrize("sh,fp8", [
    # DOWN's experts in one part (L / 16 units fill the SMs as evenly as twice as many halves)
    (synth.LayerShape("one part", T=8, d=256, L=2048, E=32, K=4, I=64, S=1, Is=64), False),
    (synth.LayerShape("one part", T=8, d=256, L=2048, E=32, K=4, I=128, S=1, Is=64), True),
    # an expert's reduction over more than one stage: a ragged second one, two whole ones
    (synth.LayerShape("I 576", T=8, d=256, L=256, E=32, K=4, I=576, S=1, Is=64), False),
    (synth.LayerShape("I 1024", T=8, d=256, L=128, E=16, K=4, I=1024, S=0, Is=0), False),
    (synth.LayerShape("I 1152", T=8, d=256, L=256, E=32, K=4, I=1152, S=1, Is=64), True)],
    ids=lambda v: v.name if isinstance(v, synth.LayerShape) else "e4m3" if v else "bf16")
def test_parts_and_long_expert_reductions(dev, oracle_mod, sh, fp8, T):
    w = synth.make_weights(sh, seed=T, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8, expert_fp8=fp8)
    x = synth.make_x(sh, seed=T, device=dev, T=T)
    _check(oracle_mod, sh, w, layer, x, tau=_tau(sh, T, dev), residual=x, tag=(sh.name, T))


def test_stalled_wait_with_e4m3_experts(dev, monkeypatch):
    sh = H.mid_shape(8)
    layer = lmoe.Layer(sh, synth.make_weights(sh, seed=1, device=dev), max_tokens=8, expert_fp8=True)
    x = synth.make_x(sh, seed=7, device=dev, T=3)
    want = layer.forward_few(x)
    monkeypatch.setenv("LMOE_WAIT_LIMIT_MS", "100")
    monkeypatch.setenv("LMOE_FAULT_INJECT", "stall")
    layer.forward_few(x)
    torch.cuda.synchronize()
    assert layer.few_device_error() == lmoe.LMOE_ERR_DEVICE_TIMEOUT
    monkeypatch.delenv("LMOE_FAULT_INJECT")
    monkeypatch.delenv("LMOE_WAIT_LIMIT_MS")
    assert torch.equal(layer.forward_few(x), want)
    torch.cuda.synchronize()
    assert layer.few_device_error() == lmoe.LMOE_OK


def test_latent_before_its_codes(dev):
    """e4m3 experts: the fp32 latent that the codes are taken from (kept in the workspace behind the
    header, the two bf16 terms, the logits, their keys, h and u).  A box of 64 products is added
    in two chains, each of two MMAs that cut off less than 2^-23 of their sum, 2^-24 on average: up to
    2^-23 of a latent where they all point its way.  The 14 boxes of a warp and the eight warps are
    added with rounding, 2^-25 on average of sums that grow like the root of their number: below
    2^-24 sqrt(3 + 14 / 2).  In the norm both together stay below 2e-7."""
    sh = synth.LayerShape("wide", T=8, d=7168, L=3584, E=16, K=1, I=128, S=0, Is=0)
    w = synth.make_weights(sh, seed=1, device=dev)
    layer = lmoe.Layer(sh, w, max_tokens=8, expert_fp8=True)
    x = synth.make_x(sh, seed=2, device=dev, T=8)
    layer.forward_few(x)
    torch.cuda.synchronize()
    pieces = [8 * sh.L * 4, 0, 8 * sh.E * 4, 8 * sh.E * 4, 8 * sh.K * sh.I * 4, 8 * sh.L * 4]
    at = 256 + sum((n + 255) // 256 * 256 for n in pieces)
    lat = layer.few_ws[at:at + 8 * sh.L * 4].view(torch.float32).view(8, sh.L)
    want = x.double() @ w["w_down"].double().T
    assert (lat.double() - want).norm() <= 2e-7 * want.norm()
