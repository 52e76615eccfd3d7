"""A training step of the operators together, as the example runs it, against plain 64-bit arithmetic.

Tolerances: every tensor between two operators is rounded to bf16 once, at most 2^-8 of a value and,
the values' errors being independent, less than that in the root mean square.  On its longest way a
gradient passes y and total of the last norm, d, dx of the head, dh, and in the block dp, dh and y, and
is rounded itself: 9 * 2^-8 of its root mean square bounds the error's."""
import ctypes
import importlib.util
import os
import threading

import pytest
import torch

from latent_compressed_expert_gb300 import lmoe, synth

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _load(name, *path):
    spec = importlib.util.spec_from_file_location(name, os.path.join(ROOT, *path))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    return _load("train_step", "examples", "train_step.py")


@pytest.fixture(scope="module")
def ref():
    """The update's 64-bit forms."""
    return _load("muon_reference", "tests", "test_gpu_muon.py")


def _rms(t):
    return float(t.double().square().mean().sqrt())


def _norm64(t, gamma, eps):
    return gamma * t * (t.square().mean(1, keepdim=True) + eps).rsqrt()


def _loss64(model, tokens, target, leaves):
    e, g1, up, down, g2, head = leaves
    h = e[tokens]
    y = _norm64(h, g1, model.block.eps)
    g, v = (y @ up.T).chunk(2, 1)
    g, v = 100 * torch.tanh(g / 100), 100 * torch.tanh(v / 100)
    h = h + (g * torch.sigmoid(g) * v) @ down.T
    logits = _norm64(h, g2, model.ends.eps) @ head.T
    on = target >= 0
    picked = logits[on].gather(1, target[on].unsqueeze(1)).squeeze(1)
    return (torch.logsumexp(logits[on], 1) - picked).sum() / on.sum()


@pytest.mark.parametrize("count", [5, 300])
def test_gradients_of_the_dense_model(ex, count):
    dev = torch.device("cuda:0")
    model = ex.DenseModel(777, 256, 320, dev, seed=count)
    tokens, target = ex.batch(777, count, dev, seed=count)
    loss, grads = model.gradients(tokens, target)
    leaves = [t.double().requires_grad_() for t in (
        model.ends.embedding, model.block.gamma, model.block.up.w, model.block.down.w,
        model.ends.gamma, model.ends.head.w)]
    want = _loss64(model, tokens, target, leaves)
    want.backward()
    # a logit's error: its row's y, total and h, each rounded once, of a spread of about 1 in all
    assert abs(float(loss) - float(want.detach())) <= 4 * STEP
    demb = torch.zeros_like(leaves[0]).index_add_(0, tokens, grads["dembedding"].double())
    got = (demb, grads["block"]["dgamma"], grads["block"]["dw_up"], grads["block"]["dw_down"],
           grads["dgamma"], grads["dhead"])
    for name, g, leaf in zip(("embedding", "gamma", "up", "down", "last gamma", "head"), got, leaves):
        assert _rms(g.double() - leaf.grad) <= 9 * STEP * _rms(leaf.grad), name


def test_dense_step_updates_by_the_formulas(ex, ref):
    dev = torch.device("cuda:0")
    model = ex.DenseModel(500, 256, 320, dev)
    tokens, target = ex.batch(500, 200, dev)
    for _ in range(2):
        _, grads = model.gradients(tokens, target)
        before = [m.clone() for m in model.block.masters]
        momentum = [m.clone() for m in model.momentum]
        model.step(tokens, target, rate=0.02)
        for i, (name, lin) in enumerate((("dw_up", model.block.up), ("dw_down", model.block.down))):
            m64, u, w64, step = ref._update64(model.muon, before[i], grads["block"][name], momentum[i],
                                              0.02, ex.muon_scale(before[i]))
            want, near = ref._exact(u), ref._rounded(u)
            assert (model.momentum[i].double() - m64).abs().max() <= 2.0 ** -22 * m64.abs().max()
            off = _rms(model.block.masters[i].double() - w64)
            # twice what the operands' rounding costs, and fp32's of the weights
            assert off <= step * (2 * _rms(near - want) + 1e-5 * _rms(want)) + 2.0 ** -23 * _rms(w64)
            assert torch.equal(lin.w, model.block.masters[i].bfloat16())
    for part in (model.ends.head, model.muon, model.block.up, model.block.down):
        assert part.device_error() == lmoe.LMOE_OK


def test_sparse_step_updates_by_the_formulas(ex, ref):
    """Every matrix of the layer, experts as batches, gradients as views of the backward's buffers."""
    dev = torch.device("cuda:0")
    model = ex.SparseModel(500, synth.TINY, dev)
    tokens, target = ex.batch(500, synth.TINY.T, dev)
    _, grads = model.gradients(tokens, target)
    before = {n: model.weights[n].clone() for n in ex.MATRICES}
    model.step(tokens, target, rate=0.02)
    for n in ex.MATRICES:
        g = grads["layer"]["d" + n]
        m64, u, w64, step = ref._update64(model.muon, before[n], g, torch.zeros_like(g), 0.02,
                                          ex.muon_scale(g))
        # an expert without tokens has no gradient: X is 0 / eps
        want, near = ref._exact(u), ref._rounded(u)
        off = _rms(model.weights[n].double() - w64)
        assert off <= step * (2 * _rms(near - want) + 1e-5 * _rms(want)) + STEP * _rms(w64), n
    assert model.muon.device_error() == lmoe.LMOE_OK


def test_examples_run(ex):
    dev = torch.device("cuda:0")
    for model, count in ((ex.DenseModel(300, 128, 256, dev), 100),
                         (ex.SparseModel(300, synth.TINY, dev), synth.TINY.T)):
        losses = ex.train(model, 300, count, 3, dev)
        assert len(losses) == 3 and all(l == l and abs(l) < float("inf") for l in losses)


def test_a_step_from_a_graph(ex):
    """Forward, both gradients and the update captured together: replays do what calls do."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(1)
    w0 = (torch.randn(700, 128, generator=gen, device=dev) * 0.1).bfloat16()
    x = torch.randn(90, 128, generator=gen, device=dev).bfloat16()
    t = torch.randint(0, 700, (90,), generator=gen, device=dev)
    weight = torch.full((90,), 1 / 90, device=dev)

    def make():
        return lmoe.LinearCrossEntropy(w0.clone()), lmoe.Muon(), torch.zeros(700, 128, device=dev)

    def step(head, muon, momentum):
        loss, lse = head.forward(x, t)
        g = head.backward(x, t, lse, weight)
        muon.update(head.w, g["dw"], momentum, 0.01)
        return loss, g["dx"]

    a, b = make(), make()
    want = [tuple(v.clone() for v in step(*a)) for _ in range(3)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*b)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want[i]))
    assert torch.equal(a[0].w, b[0].w) and torch.equal(a[2], b[2])


def test_first_call_of_a_host_thread(ex):
    """Calls from host threads that have used no GPU yet, with their outputs already allocated."""
    dev = torch.device("cuda:0")
    lib, stream = lmoe.load(), torch.cuda.current_stream().cuda_stream
    calls = []
    for M in (3, 2000):
        head = lmoe.LinearCrossEntropy(torch.randn(500, 64, device=dev).bfloat16())
        x, t = torch.randn(M, 64, device=dev).bfloat16(), torch.randint(0, 500, (M,), device=dev)
        want, lse = head.forward(x, t)
        loss, lse2 = torch.empty(M, device=dev), torch.empty(M, device=dev)
        d = head._desc(x, t, loss.data_ptr(), lse2.data_ptr())
        ws = torch.empty(lib.lmoe_linear_xent_workspace_bytes(d), dtype=torch.uint8, device=dev)
        calls.append((lambda d=d, ws=ws, k=(head, x, t): lib.lmoe_linear_xent_forward(
            d, ws.data_ptr(), ws.numel(), stream), loss, want))
        g = torch.ones(M, device=dev)
        ref, dx = head.backward(x, t, lse, g, want_dw=False)["dx"], torch.empty_like(x)
        b = head._desc(x, t, None, lse.data_ptr())
        wb = torch.empty(lib.lmoe_linear_xent_backward_workspace_bytes(b), dtype=torch.uint8, device=dev)
        calls.append((lambda b=b, wb=wb, g=g, dx=dx, k=(head, x, t, lse): lib.lmoe_linear_xent_backward(
            b, g.data_ptr(), dx.data_ptr(), 64, None, 0, wb.data_ptr(), wb.numel(), stream), dx, ref))
    muon = lmoe.Muon()
    for shape in ((40, 64), (300, 400)):
        g = torch.randn(*shape, device=dev)
        want, out = muon.orthogonalize(g), torch.empty(*shape, dtype=torch.bfloat16, device=dev)
        d, _ = muon._desc(g)
        d.out, d.ldo = out.data_ptr(), shape[1]
        ws = torch.empty(lib.lmoe_muon_workspace_bytes(ctypes.byref(d)), dtype=torch.uint8, device=dev)
        calls.append((lambda d=d, ws=ws, g=g: lib.lmoe_orthogonalize(
            ctypes.byref(d), ws.data_ptr(), ws.numel(), stream), out, want))
    torch.cuda.synchronize()
    for call, out, ref in calls:
        codes = []
        th = threading.Thread(target=lambda: codes.append(call()))
        th.start()
        th.join()
        torch.cuda.synchronize()
        assert codes == [lmoe.LMOE_OK]
        assert torch.equal(out, ref)


def test_first_calls_of_a_process_are_captured(ex):
    """Set-up (a kernel's shared memory, how many clusters fit) does not disturb a capture."""
    import subprocess
    import sys
    code = """
import torch
from latent_compressed_expert_gb300 import lmoe
dev = torch.device("cuda:0")
gen = torch.Generator(device=dev).manual_seed(3)
draw = lambda *s: torch.randn(*s, generator=gen, device=dev)
head, muon = lmoe.LinearCrossEntropy((draw(900, 64) * 0.2).bfloat16()), lmoe.Muon()
cases = [(draw(m, 64).bfloat16(), torch.randint(0, 900, (m,), generator=gen, device=dev),
          torch.full((m,), 1.0 / m, device=dev)) for m in (4, 1500)]
mats = [draw(60, 500), draw(700, 900), draw(3, 1000, 130)]
def everything():
    out = []
    for x, t, w in cases:
        loss, lse = head.forward(x, t)
        g = head.backward(x, t, lse, w)
        out += [loss, lse, g["dx"], g["dw"]]
    return out + [muon.orthogonalize(m) for m in mats]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = everything()
graph.replay()
torch.cuda.synchronize()
want = everything()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert head.device_error() == muon.device_error() == lmoe.LMOE_OK
print("same")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=100)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_calls_of_two_host_threads(ex):
    """Two threads on streams of their own, on the same head, weights and Muon object at once."""
    dev = torch.device("cuda:0")
    gen = torch.Generator(device=dev).manual_seed(2)
    draw = lambda *s: torch.randn(*s, generator=gen, device=dev)
    head, muon = lmoe.LinearCrossEntropy((draw(3000, 128) * 0.1).bfloat16()), lmoe.Muon()
    data = [(draw(m, 128).bfloat16(), torch.randint(0, 3000, (m,), generator=gen, device=dev),
             torch.full((m,), 1.0 / m, device=dev), draw(*s))
            for m, s in ((50, (100, 300)), (700, (400, 300)))]

    def work(d, out):
        x, t, w, g = d
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                loss, lse = head.forward(x, t)
                grads = head.backward(x, t, lse, w)
                out[:] = [loss, lse, grads["dx"], grads["dw"], muon.orthogonalize(g)]
            torch.cuda.current_stream().synchronize()

    want, got = [[], []], [[], []]
    for d, o in zip(data, want):
        work(d, o)
    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=a) for a in zip(data, got)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert len(b) == 5 and all(torch.equal(p, q) for p, q in zip(a, b))
