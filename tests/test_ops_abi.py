"""Host side of the operators around the layer (RMSNorm with residual, linear layers, the layer for
a few tokens): size queries and refusals.  No call here launches a kernel."""
import ctypes

import pytest
import torch

from latent_compressed_expert_gb300 import build, lmoe, synth

# Fake device addresses that the host-side checks must turn down before any CUDA call: not on a
# machine with a GPU, where a check that let one through would touch them.
no_gpu = pytest.mark.skipif(torch.cuda.is_available(),
                            reason="fake-pointer host checks run on CPU-only machines")
OK, ARG, UNSUP, SMALL = (lmoe.LMOE_OK, lmoe.LMOE_ERR_INVALID_ARG, lmoe.LMOE_ERR_UNSUPPORTED,
                         lmoe.LMOE_ERR_WORKSPACE_TOO_SMALL)
BUF = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ("x", "residual", "gamma", "y", "scales", "total", "rstd", "dy", "dtotal", "dx", "dgamma", "ws",
     "w", "bias", "pre", "flag", "x_scales", "w_scales", "dw", "dbias", "packed"))}


@pytest.fixture(scope="module")
def lib():
    build.build()
    return lmoe.load()


def _norm(lib, **a):
    p = dict(x=BUF["x"], ldx=64, residual=BUF["residual"], ldr=64, gamma=BUF["gamma"], rows=4,
             cols=64, eps=1e-6, y=BUF["y"], ldy=64, type=lmoe.BF16, scales=None,
             total=BUF["total"], ldt=64, rstd=BUF["rstd"])
    p.update(a)
    return lib.lmoe_add_rmsnorm(*p.values(), None)


@no_gpu
@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), ARG), (dict(cols=0), ARG), (dict(eps=-1e-6), ARG),
    (dict(eps=float("nan")), ARG), (dict(type=lmoe.F32), ARG), (dict(type=7), ARG),
    (dict(rows=1 << 31), UNSUP), (dict(cols=(1 << 30) + 1), UNSUP),
    (dict(x=None), ARG), (dict(gamma=None), ARG), (dict(y=None), ARG),
    (dict(type=lmoe.E4M3), ARG),                      # codes without scales
    (dict(ldx=63), ARG), (dict(ldr=63), ARG), (dict(ldy=0), ARG), (dict(ldt=-64), ARG),
    (dict(x=BUF["x"] + 1), ARG), (dict(residual=BUF["residual"] + 1), ARG),
    (dict(y=BUF["y"] + 1), ARG), (dict(total=BUF["total"] + 1), ARG),
    (dict(gamma=BUF["gamma"] + 2), ARG), (dict(rstd=BUF["rstd"] + 2), ARG),
    (dict(type=lmoe.E4M3, scales=BUF["scales"] + 2), ARG),
    (dict(rows=0, x=None, y=None), OK),
])
def test_add_rmsnorm_refusals(lib, change, code):
    assert _norm(lib, **change) == code


def test_add_rmsnorm_backward_workspace(lib):
    q = lib.lmoe_add_rmsnorm_backward_workspace_bytes
    assert q(-1, 64) == 0 and q(4, 0) == 0 and q(1 << 31, 64) == 0 and q(4, (1 << 30) + 1) == 0
    # one fp32 row of partial sums per block: at least one, at most one per row
    assert q(0, 64) == q(1, 64) == 64 * 4
    assert q(4, 64) <= 4 * 64 * 4
    assert q(1 << 20, 7168) == q(1 << 30, 7168) <= 64 << 20


def _norm_bwd(lib, **a):
    p = dict(dy=BUF["dy"], ldy=64, total=BUF["total"], ldt=64, gamma=BUF["gamma"],
             rstd=BUF["rstd"], dtotal=BUF["dtotal"], ldd=64, rows=4, cols=64, dx=BUF["dx"], ldx=64,
             dgamma=BUF["dgamma"], ws=BUF["ws"], nb=1 << 20)
    p.update(a)
    return lib.lmoe_add_rmsnorm_backward(*p.values(), None)


@no_gpu
@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), ARG), (dict(cols=0), ARG), (dict(rows=1 << 31), UNSUP),
    (dict(cols=(1 << 30) + 1), UNSUP),
    (dict(dy=None), ARG), (dict(total=None), ARG), (dict(gamma=None), ARG), (dict(rstd=None), ARG),
    (dict(dx=None), ARG), (dict(ws=None), ARG), (dict(ws=BUF["ws"] + 8), ARG),
    (dict(ldy=63), ARG), (dict(ldt=63), ARG), (dict(ldd=63), ARG), (dict(ldx=63), ARG),
    (dict(dy=BUF["dy"] + 1), ARG), (dict(dtotal=BUF["dtotal"] + 1), ARG),
    (dict(dx=BUF["dx"] + 1), ARG), (dict(rstd=BUF["rstd"] + 1), ARG),
    (dict(dgamma=BUF["dgamma"] + 2), ARG), (dict(nb=4 * 64 * 4 - 1), SMALL),
    (dict(rows=0, dgamma=None, dy=None), OK),
])
def test_add_rmsnorm_backward_refusals(lib, change, code):
    assert _norm_bwd(lib, **change) == code


def _desc(**a):
    d = lmoe.LinearDesc()
    p = dict(M=8, N=64, K=64, act=lmoe.ACTS["none"], type=lmoe.BF16, c=100.0, x=BUF["x"], ldx=64,
             w=BUF["w"], ldw=64, bias=BUF["bias"], residual=BUF["residual"], ldr=64, y=BUF["y"],
             ldy=64, pre=BUF["pre"], ldp=128, dev_flag=BUF["flag"])
    p.update(a)
    for k, v in p.items():
        setattr(d, k, v)
    return d


E4M3 = dict(type=lmoe.E4M3, x_scales=BUF["x_scales"], w_scales=BUF["w_scales"])
SITU = dict(act=lmoe.ACTS["situ"])
SIZES = [
    (dict(M=-1), ARG), (dict(N=0), ARG), (dict(K=0), ARG), (dict(act=4), ARG), (dict(act=-1), ARG),
    (dict(type=lmoe.F32), ARG), (dict(**SITU, c=0.0), ARG), (dict(**SITU, c=float("nan")), ARG),
    (dict(N=60, ldy=64), UNSUP), (dict(K=60), UNSUP), (dict(**E4M3, K=56), UNSUP),
    (dict(**SITU, N=1 << 30), UNSUP), (dict(N=(1 << 30) + 8), UNSUP),
    (dict(M=(1 << 30) + 1), UNSUP), (dict(K=(1 << 30) + 16), UNSUP),
    (dict(M=1 << 20, N=1 << 20), UNSUP),              # tiles
    (dict(ldx=56), ARG), (dict(ldw=56), ARG), (dict(ldx=68), ARG), (dict(ldw=68), ARG),
]


@no_gpu
@pytest.mark.parametrize("change,code", SIZES + [
    (dict(x=None), ARG), (dict(w=None), ARG), (dict(y=None), ARG), (dict(dev_flag=None), ARG),
    (dict(type=lmoe.E4M3), ARG), (dict(**{**E4M3, "x_scales": None}), ARG),
    (dict(x=BUF["x"] + 8), ARG), (dict(w=BUF["w"] + 2), ARG), (dict(y=BUF["y"] + 8), ARG),
    (dict(residual=BUF["residual"] + 8), ARG), (dict(pre=BUF["pre"] + 8), ARG),
    (dict(ldy=56), ARG), (dict(ldy=68), ARG), (dict(ldr=56), ARG), (dict(ldr=68), ARG),
    (dict(ldp=56), ARG), (dict(**SITU, ldp=64), ARG), (dict(ldp=132), ARG),
    (dict(y=BUF["x"]), ARG), (dict(y=BUF["w"]), ARG), (dict(pre=BUF["y"]), ARG),
    (dict(pre=BUF["x"]), ARG), (dict(pre=BUF["w"]), ARG), (dict(pre=BUF["residual"]), ARG),
    (dict(M=0, x=None, y=None), OK),
])
def test_linear_forward_refusals(lib, change, code):
    assert lib.lmoe_linear_forward(ctypes.byref(_desc(**change)), None) == code


def test_linear_without_a_description(lib):
    assert lib.lmoe_linear_forward(None, None) == ARG
    assert lib.lmoe_linear_backward_workspace_bytes(None) == 0
    assert lib.lmoe_linear_backward(None, None, 0, None, 0, None, 0, None, None, 0, None) == ARG


def _linear_bwd(lib, d, **a):
    p = dict(dy=BUF["dy"], lddy=64, dx=BUF["dx"], lddx=64, dw=BUF["dw"], type=lmoe.F32,
             dbias=BUF["dbias"], ws=BUF["ws"], nb=1 << 30)
    p.update(a)
    return lib.lmoe_linear_backward(ctypes.byref(d), *p.values(), None)


@no_gpu
@pytest.mark.parametrize("change,code", SIZES + [(E4M3, UNSUP)])
def test_linear_backward_sizes(lib, change, code):
    d = _desc(**change)
    assert lib.lmoe_linear_backward_workspace_bytes(ctypes.byref(d)) == 0 \
        or change.get("type") == lmoe.E4M3
    assert _linear_bwd(lib, d) == code


@no_gpu
@pytest.mark.parametrize("fields,change,code", [
    ({}, dict(dy=None), ARG), ({}, dict(dy=BUF["dy"] + 8), ARG), ({}, dict(lddy=56), ARG),
    ({}, dict(lddy=68), ARG), ({}, dict(lddx=56), ARG), ({}, dict(lddx=68), ARG),
    ({}, dict(dx=BUF["dx"] + 8), ARG), ({}, dict(dw=BUF["dw"] + 4), ARG),
    ({}, dict(dbias=BUF["dbias"] + 4), ARG), ({}, dict(type=lmoe.E4M3), ARG),
    ({}, dict(dx=BUF["dy"]), ARG), ({}, dict(dx=BUF["x"]), ARG), ({}, dict(dx=BUF["w"]), ARG),
    ({}, dict(dw=BUF["dy"]), ARG), ({}, dict(dw=BUF["x"]), ARG), ({}, dict(dw=BUF["w"]), ARG),
    ({}, dict(dw=BUF["dx"]), ARG), (SITU, dict(dw=BUF["pre"]), ARG), (SITU, dict(dx=BUF["pre"]), ARG),
    (dict(x=None), {}, ARG), (dict(w=None), {}, ARG), (dict(dev_flag=None), {}, ARG),
    (dict(**SITU, pre=None), {}, ARG), (dict(**SITU, ldp=64), {}, ARG),
    (dict(**SITU, pre=BUF["pre"] + 8), {}, ARG),
    ({}, dict(ws=None), ARG), ({}, dict(ws=BUF["ws"] + 8), ARG), ({}, dict(nb=0), SMALL),
    (dict(M=0), dict(dy=None, dw=None, dbias=None), OK),
])
def test_linear_backward_refusals(lib, fields, change, code):
    assert _linear_bwd(lib, _desc(**fields), **change) == code


def test_linear_backward_workspace(lib):
    q = lambda **a: lib.lmoe_linear_backward_workspace_bytes(ctypes.byref(_desc(**a)))
    # dp as the products' operand, with an activation only, and the partial sums of dbias
    plain = q(M=4096, N=1024)
    assert 0 < plain <= 64 << 20
    assert q(M=4096, N=1024, act=lmoe.ACTS["gelu"]) == plain + 4096 * 1024 * 2
    assert q(M=4096, N=1024, **SITU) == 2 * plain + 4096 * 2048 * 2
    assert q(**E4M3) == 0


def test_few_workspace(lib):
    q = lambda sh, **a: lib.lmoe_few_workspace_bytes(ctypes.byref(lmoe.dims_of(sh, **a)))
    sizes = [q(synth.DECODE, T=t) for t in range(lmoe.FEW_MAX_TOKENS + 1)]
    assert sizes == sorted(sizes)
    assert sizes[0] > 0 and sizes[-1] < 4 << 20
    assert q(synth.DECODE, T=lmoe.FEW_MAX_TOKENS + 1) == 0
    assert q(synth.DECODE, T=-1) == 0
    assert q(synth.DECODE, T=8, expert_fp8=True) > sizes[-1]
    assert q(synth.TINY, T=4, expert_fp8=True) == 0   # e4m3 needs L and I in multiples of 128


def _few(lib, sh=synth.TINY, T=2, io=None, **a):
    p = dict(packed=BUF["packed"], x=BUF["x"], residual=BUF["residual"], y=BUF["y"], ws=BUF["ws"],
             nb=1 << 30)
    p.update(a)
    o = None
    if io is not None:
        o = lmoe.IO()
        for k, v in io.items():
            setattr(o, k, ctypes.cast(v, type(o.stage_events)) if k == "stage_events" else v)
    return lib.lmoe_forward_few(ctypes.byref(lmoe.dims_of(sh, T=T)), *p.values(),
                                None if o is None else ctypes.byref(o), None)


@no_gpu
@pytest.mark.parametrize("change,code", [
    (dict(T=lmoe.FEW_MAX_TOKENS + 1), UNSUP), (dict(T=-1), ARG),
    (dict(packed=None), ARG), (dict(x=None), ARG), (dict(y=None), ARG), (dict(ws=None), ARG),
    (dict(x=BUF["x"] + 8), ARG), (dict(y=BUF["y"] + 2), ARG), (dict(packed=BUF["packed"] + 4), ARG),
    (dict(residual=BUF["residual"] + 8), ARG), (dict(ws=BUF["ws"] + 8), ARG),
    (dict(y=BUF["x"]), ARG), (dict(y=BUF["residual"]), ARG), (dict(nb=256), SMALL),
    (dict(io=dict(balance=1)), ARG),                  # in-batch thresholds of a few tokens
    (dict(io=dict(phase=lmoe.PHASE_ROUTER)), ARG), (dict(io=dict(phase=lmoe.PHASE_EXPERTS)), ARG),
    *[(dict(io={f: 0x5000000}), ARG) for f in ("tau_out", "counts_out", "load_stats", "tau_ema",
                                               "save_pre", "save_pre_shared", "stage_events",
                                               "cand_out")],
    *[(dict(io={f: 0x5000002}), ARG) for f in ("logits_in", "logit_bias", "logits_out", "idx_out",
                                               "gate_out", "y_f32_out")],
    (dict(io=dict(balance=1, tau_in=0x5000004)), ARG),
    (dict(T=0, packed=None, x=None, y=None, ws=None), OK),
])
def test_forward_few_refusals(lib, change, code):
    assert _few(lib, **change) == code


def test_bindings_refuse_cpu_tensors(lib):
    bf = torch.bfloat16
    x, gamma, w = torch.zeros(2, 64, dtype=bf), torch.ones(64), torch.zeros(64, 64, dtype=bf)
    with pytest.raises(ValueError):
        lmoe.add_rmsnorm(x, gamma)
    with pytest.raises(ValueError):
        lmoe.add_rmsnorm_e4m3(x, gamma)
    with pytest.raises(ValueError):
        lmoe.add_rmsnorm_backward(x, x, gamma, torch.ones(2))
    with pytest.raises(ValueError):
        lmoe.Linear(w)
    with pytest.raises(ValueError):
        lmoe.Linear(w, act="relu")
    with pytest.raises(ValueError):
        lmoe.Linear(w, w_scales=torch.ones(64))


@no_gpu
@pytest.mark.parametrize("change", [
    dict(bias=BUF["bias"] + 2), dict(dev_flag=BUF["flag"] + 1),
    {**E4M3, "x_scales": BUF["x_scales"] + 2}, {**E4M3, "w_scales": BUF["w_scales"] + 1}])
def test_linear_forward_refuses_misaligned_words(lib, change):
    assert lib.lmoe_linear_forward(ctypes.byref(_desc(**change)), None) == ARG


@no_gpu
def test_linear_backward_refuses_a_misaligned_flag(lib):
    assert _linear_bwd(lib, _desc(dev_flag=BUF["flag"] + 2)) == ARG


# An output over an input at another row distance: rows would be written over before they are read.
@no_gpu
@pytest.mark.parametrize("change", [
    dict(total=BUF["x"], ldt=72), dict(total=BUF["residual"], ldr=72),
    dict(y=BUF["x"], ldx=72), dict(y=BUF["residual"], ldy=128)])
def test_add_rmsnorm_refuses_shifted_rows(lib, change):
    assert _norm(lib, **change) == ARG


@no_gpu
@pytest.mark.parametrize("change", [dict(dx=BUF["dy"], ldx=72), dict(dx=BUF["dtotal"], ldd=72)])
def test_add_rmsnorm_backward_refuses_shifted_rows(lib, change):
    assert _norm_bwd(lib, **change) == ARG


@no_gpu
@pytest.mark.parametrize("change", [dict(ldy=72), dict(ldr=72)])
def test_linear_refuses_shifted_rows(lib, change):
    assert lib.lmoe_linear_forward(ctypes.byref(_desc(y=BUF["residual"], **change)), None) == ARG


# Two outputs at one address, codes or sums over an input, scratch over an operand.
@no_gpu
@pytest.mark.parametrize("change", [
    dict(total=BUF["y"]), dict(rstd=BUF["total"]), dict(rstd=BUF["y"]), dict(rstd=BUF["x"]),
    dict(rstd=BUF["gamma"]), dict(type=lmoe.E4M3, scales=BUF["total"]),
    dict(type=lmoe.E4M3, scales=BUF["rstd"]), dict(type=lmoe.E4M3, scales=BUF["gamma"]),
    dict(type=lmoe.E4M3, scales=BUF["scales"], y=BUF["x"]),
    dict(type=lmoe.E4M3, scales=BUF["scales"], y=BUF["residual"]),
    dict(type=lmoe.E4M3, scales=BUF["y"])])
def test_add_rmsnorm_refuses_outputs_over_each_other(lib, change):
    assert _norm(lib, **change) == ARG


@no_gpu
@pytest.mark.parametrize("change", [
    *[dict(dgamma=BUF[n]) for n in ("dy", "total", "dtotal", "gamma", "rstd", "dx", "ws")],
    *[dict(ws=BUF[n]) for n in ("dy", "total", "dtotal", "gamma", "rstd", "dx")]])
def test_add_rmsnorm_backward_refuses_sums_over_operands(lib, change):
    assert _norm_bwd(lib, **change) == ARG


@no_gpu
@pytest.mark.parametrize("fields,change", [
    *[({}, dict(dbias=BUF[n])) for n in ("dx", "dw", "dy", "x", "w", "ws")],
    *[({}, dict(ws=BUF[n])) for n in ("dx", "dw", "dy", "x", "w")],
    (SITU, dict(dbias=BUF["pre"])), (SITU, dict(ws=BUF["pre"]))])
def test_linear_backward_refuses_sums_over_operands(lib, fields, change):
    assert _linear_bwd(lib, _desc(**fields), **change) == ARG


class _Placed:
    """What the binding asks of a tensor, with the device number given."""

    def __init__(self, t, number):
        self.dtype, self.shape, self.device, self._t, self._n = t.dtype, t.shape, t.device, t, number
        self.is_cuda = True

    def get_device(self):
        return self._n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x100000

    def numel(self):
        return 1 << 30


@no_gpu
@pytest.mark.parametrize("name", ["x", "residual", "y", "tau", "logits_in", "logit_bias"])
def test_forward_few_refuses_tensors_of_another_device(lib, monkeypatch, name):
    sh = synth.TINY
    layer = object.__new__(lmoe.Layer)
    layer.shape, layer.max_tokens, layer.expert_fp8 = sh, 8, False
    layer.device = torch.device("cuda:0")
    layer._few_dims = [lmoe.dims_of(sh, T=t) for t in range(3)]
    layer.few_ws = layer.packed = _Placed(torch.empty(1), 0)
    monkeypatch.setattr(lmoe, "_on", lambda dev: None)
    bf = torch.bfloat16
    shapes = {"x": ((2, sh.d), bf), "residual": ((2, sh.d), bf), "y": ((2, sh.d), bf),
              "tau": ((sh.E,), torch.float32), "logits_in": ((2, sh.E), torch.float32),
              "logit_bias": ((sh.E,), torch.float32)}
    args = {n: _Placed(torch.empty(s, dtype=t), 1 if n == name else 0)
            for n, (s, t) in shapes.items()}
    with pytest.raises(ValueError, match=name):
        layer.forward_few(**args)


def _layer_without_gpu(monkeypatch, zeros):
    """A layer whose forward_few has not been called, on a machine without a GPU; `zeros` allocates
    its workspace."""
    layer = object.__new__(lmoe.Layer)
    layer.shape, layer.max_tokens, layer.expert_fp8 = synth.TINY, 8, False
    layer.device, layer.few_ws = torch.device("cuda:0"), None
    layer.packed = _Placed(torch.empty(1), 0)
    monkeypatch.setattr(lmoe, "_on", lambda dev: None)
    monkeypatch.setattr(torch, "zeros", zeros)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)

    class Stream:
        def synchronize(self):
            pass

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    return layer


@no_gpu
def test_first_forward_few_of_two_threads(lib, monkeypatch):
    """Both threads end up with one workspace."""
    import threading
    import time

    made, used, none = [], [], torch.empty(0, synth.TINY.d, dtype=torch.bfloat16)

    def zeros(*a, **k):
        time.sleep(0.2)
        made.append(_Placed(none, 0))
        return made[-1]

    layer = _layer_without_gpu(monkeypatch, zeros)

    def first():
        layer.forward_few(_Placed(none, 0), y=_Placed(none, 0))  # no tokens: no launch
        used.append((layer.few_ws, layer._few_dims))

    threads = [threading.Thread(target=first) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(made) == 1 and len(used) == 2
    assert used[0][0] is used[1][0] is made[0] and used[0][1] is used[1][1]


@no_gpu
def test_first_forward_few_under_capture_is_refused(lib, monkeypatch):
    """Nothing is allocated from the graph's memory, and the call is made later as if it were the
    first."""
    made, none = [], torch.empty(0, synth.TINY.d, dtype=torch.bfloat16)

    def zeros(*a, **k):
        made.append(_Placed(none, 0))
        return made[-1]

    layer = _layer_without_gpu(monkeypatch, zeros)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(ValueError, match="before capturing"):
        layer.forward_few(_Placed(none, 0), y=_Placed(none, 0))
    assert not made and layer.few_ws is None
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    layer.forward_few(_Placed(none, 0), y=_Placed(none, 0))
    assert layer.few_ws is made[0] and len(made) == 1
