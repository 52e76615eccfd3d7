"""The operators together, as the example's decoder block runs them, against plain 64-bit
arithmetic.

Tolerances: every tensor between two operators is rounded to bf16 once (2^-8 of a value at most).
The dense block's branch passes three such roundings (y, h and, backwards, dh, dp, dy), the
values' errors being independent: 4 * 2^-8 of the RMS of the result bounds the RMS error of each
output and gradient, with the output's own rounding of total + branch counted in it.  e4m3 operands
round at 2^-4 at most, 2^-4 / sqrt(3) in the mean square of uniformly placed values, in four
tensors: 4 * 2^-4 of the branch's RMS."""
import importlib.util
import os

import pytest
import torch

from latent_compressed_expert_gb300 import lmoe, synth

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -8


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from latent_compressed_expert_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decoder_ffn.py")
    spec = importlib.util.spec_from_file_location("decoder_ffn", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _rms(t):
    return float(t.double().square().mean().sqrt())


def _block64(block, x, residual):
    """The dense block in 64 bits: (out, leaves)."""
    t = (x.double() + residual.double()).requires_grad_()
    gamma, up, down = (v.double().requires_grad_() for v in (block.gamma, block.up.w, block.down.w))
    y = gamma * t * (t.square().mean(1, keepdim=True) + block.eps).rsqrt()
    g, v = (y @ up.T).chunk(2, dim=1)
    g, v = 100 * torch.tanh(g / 100), 100 * torch.tanh(v / 100)
    return t + (g * torch.sigmoid(g) * v) @ down.T, (t, gamma, up, down)


@pytest.mark.parametrize("tokens", [1, 77, 600])
def test_dense_block(ex, tokens):
    block = ex.DenseFfn(512, 768, "cuda:0")
    gen = torch.Generator(device="cuda:0").manual_seed(tokens)
    x, r, dout = (torch.randn(tokens, 512, generator=gen, device="cuda:0").bfloat16()
                  for _ in range(3))
    out, saved = block.forward(x, r, train=True)
    grads = block.backward(saved, dout)
    assert torch.equal(out, block.forward(x, r))
    want, leaves = _block64(block, x, r)
    assert _rms(out.double() - want.detach()) <= 4 * STEP * _rms(want.detach())
    want.backward(dout.double())
    for name, leaf in zip(("dx", "dgamma", "dw_up", "dw_down"), leaves):
        assert _rms(grads[name].double() - leaf.grad) <= 4 * STEP * _rms(leaf.grad), name
    block.quantize()
    out8 = block.forward_e4m3(x, r)
    branch = want.detach() - leaves[0].detach()
    assert _rms(out8.double() - want.detach()) <= 4 * 2.0 ** -4 * _rms(branch) \
        + STEP * _rms(want.detach())
    assert block.up.device_error() == block.down.device_error() == lmoe.LMOE_OK


def test_training_reduces_the_loss(ex):
    losses = ex.train_dense(12)
    assert all(b < a for a, b in zip(losses, losses[1:]))


def test_decode_steps_from_a_graph(ex):
    """Every replay gives what the block gives called directly, which agrees with the layer's own
    forward on the same normalised rows (the layer's stated mean error, once for each)."""
    outs, inputs, block = ex.serve_sparse(3)
    for i, out in enumerate(outs):
        assert torch.equal(out, block.decode(inputs[i], inputs[i + 1]))
        y, total = lmoe.add_rmsnorm(inputs[i], block.gamma, inputs[i + 1])
        full = block.layer.forward(y, residual=total, tau=block.tau)
        err = (out.double() - full.double()).abs().sum() / full.double().abs().sum()
        assert err <= 2 * 5e-3
    assert block.layer.few_device_error() == lmoe.LMOE_OK


def test_decode_agrees_with_the_prompt(ex):
    shape = synth.TINY
    w = synth.make_weights(shape, seed=0, device="cuda:0")
    block = ex.SparseFfn(shape, w, torch.ones(shape.d, device="cuda:0"), max_tokens=shape.T)
    x = synth.make_x(shape, seed=5, device="cuda:0")
    out = block.prompt(x)
    got = torch.cat([block.decode(x[i:i + 8]) for i in range(0, shape.T, 8)])
    err = (got.double() - out.double()).abs().sum() / out.double().abs().sum()
    assert err <= 2 * 5e-3


def test_first_call_of_a_host_thread(ex):
    """Calls from host threads that have used no GPU yet, with their outputs already allocated."""
    import ctypes
    import threading

    dev = torch.device("cuda:0")
    lib, stream = lmoe.load(), torch.cuda.current_stream().cuda_stream
    layer = lmoe.Layer(synth.TINY, synth.make_weights(synth.TINY, seed=0, device=dev), max_tokens=8)
    x = synth.make_x(synth.TINY, seed=1, device=dev, T=2)
    y = torch.empty_like(x)
    want = layer.forward_few(x)
    calls = [(lambda: lib.lmoe_forward_few(
        ctypes.byref(layer._few_dims[2]), layer.packed.data_ptr(), x.data_ptr(), None, y.data_ptr(),
        layer.few_ws.data_ptr(), layer.few_ws.numel(), None, stream), y, want)]
    for M in (3, 9000):  # a cluster's tile, SM pairs
        xl = torch.randn(M, 256, device=dev).bfloat16()
        lin = lmoe.Linear(torch.randn(2048, 256, device=dev).bfloat16())
        out, ref = torch.empty(M, 2048, dtype=torch.bfloat16, device=dev), lin.forward(xl)
        d = lin._desc(M, xl.data_ptr(), 256, None, None, 0, out.data_ptr(), 2048, None, 0)
        calls.append((lambda d=d, keep=(lin, xl): lib.lmoe_linear_forward(d, stream), out, ref))
        dx, back = torch.empty_like(xl), lin.backward(xl, ref, want_dw=False)["dx"]
        b = lin._desc(M, xl.data_ptr(), 256, None, None, 0, None, 0, None, 0)
        calls.append((lambda b=b, r=ref, o=dx: lib.lmoe_linear_backward(
            b, r.data_ptr(), 2048, o.data_ptr(), 256, None, 0, None, None, 0, stream), dx, back))
    torch.cuda.synchronize()
    for call, out, ref in calls:
        codes = []
        t = threading.Thread(target=lambda: codes.append(call()))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert codes == [lmoe.LMOE_OK]
        assert torch.equal(out, ref)
