"""The feed-forward half of a decoder block, with the operators as a model uses them.

    total = x + residual                 (x: the attention's output, residual: the running stream)
    out   = total + FFN(rmsnorm(total))

SparseFfn puts the Stable Latent MoE layer there: prompts through Layer.forward, which solves the
thresholds and keeps their running mean, then decode steps of a few tokens through
Layer.forward_few against that mean.  DenseFfn is the dense block that precedes the sparse ones: a
gated SiTU projection and one back, with a backward pass, or with e4m3 operands for inference.

    python examples/decoder_ffn.py [--steps N]

trains a dense block towards the outputs of another one and prints the loss, then serves a prompt
and N decode steps through a sparse block, the steps replayed from one CUDA graph."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from latent_compressed_expert_gb300 import lmoe, synth  # noqa: E402


class SparseFfn:
    def __init__(self, shape, weights: dict, gamma: torch.Tensor, max_tokens: int,
                 expert_fp8: bool = False, eps: float = 1e-6):
        self.layer = lmoe.Layer(shape, weights, max_tokens=max_tokens, expert_fp8=expert_fp8)
        self.gamma, self.eps = gamma, eps
        self.tau = torch.zeros(shape.E, device=gamma.device)
        self.seen = False  # a prompt has set the thresholds

    def prompt(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        y, total = lmoe.add_rmsnorm(x, self.gamma, residual, self.eps)
        out = self.layer.forward(y, residual=total, tau_ema=self.tau, ema_first=not self.seen)
        self.seen = True
        return out

    def decode(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        y, total = lmoe.add_rmsnorm(x, self.gamma, residual, self.eps)
        return self.layer.forward_few(y, residual=total, tau=self.tau)


class DenseFfn:
    def __init__(self, d: int, width: int, device, seed: int = 0, eps: float = 1e-6):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(rows, cols):
            return torch.randn(rows, cols, generator=g, device=device) * cols ** -0.5

        self.gamma, self.eps = torch.ones(d, device=device), eps
        # fp32 masters of an optimizer; the layers multiply by their bf16 roundings
        self.masters = [draw(2 * width, d), draw(d, width)]
        self.up = lmoe.Linear(self.masters[0].bfloat16(), act="situ")  # gate rows, then value rows
        self.down = lmoe.Linear(self.masters[1].bfloat16())
        self.up8 = self.down8 = None

    def forward(self, x: torch.Tensor, residual: torch.Tensor | None = None, train: bool = False):
        """out, or with train (out, what ``backward`` needs)."""
        y, total, rstd = lmoe.add_rmsnorm(x, self.gamma, residual, self.eps, train=True)
        h, pre = self.up.forward(y, train=True) if train else (self.up.forward(y), None)
        out = self.down.forward(h, residual=total)
        return (out, (total, rstd, y, h, pre)) if train else out

    def backward(self, saved, dout: torch.Tensor) -> dict:
        """Gradients of x (and of residual, the same), gamma and both weights."""
        total, rstd, y, h, pre = saved
        down = self.down.backward(h, dout)
        up = self.up.backward(y, down["dx"], pre)
        # dout reaches total itself as well as the normalised branch
        dx, dgamma = lmoe.add_rmsnorm_backward(up["dx"], total, self.gamma, rstd, dtotal=dout)
        return {"dx": dx, "dgamma": dgamma, "dw_up": up["dw"], "dw_down": down["dw"]}

    def update(self, grads: dict, rate: float):
        self.gamma.sub_(grads["dgamma"], alpha=rate)
        for lin, master, name in zip((self.up, self.down), self.masters, ("dw_up", "dw_down")):
            master.sub_(grads[name], alpha=rate)
            lin.w.copy_(master)

    def quantize(self):
        """Lays the weights out as e4m3 codes with a scale per row, for ``forward_e4m3``."""
        (up, up_s), (down, down_s) = lmoe.quantize_e4m3(self.up.w), lmoe.quantize_e4m3(self.down.w)
        self.up8 = lmoe.Linear(up, act="situ", w_scales=up_s)
        self.down8 = lmoe.Linear(down, w_scales=down_s)

    def forward_e4m3(self, x: torch.Tensor, residual: torch.Tensor | None = None) -> torch.Tensor:
        codes, scales, total = lmoe.add_rmsnorm_e4m3(x, self.gamma, residual, self.eps)
        h = self.up8.forward(codes, x_scales=scales)
        h_codes, h_scales = lmoe.quantize_e4m3(h)
        return self.down8.forward(h_codes, residual=total, x_scales=h_scales)


def train_dense(steps: int, d: int = 512, width: int = 1024, tokens: int = 2048, rate: float = 40.0,
                device="cuda:0") -> list:
    """Losses of `steps` gradient steps of one block towards another."""
    block, teacher = (DenseFfn(d, width, device, seed) for seed in (1, 2))
    g = torch.Generator(device=device).manual_seed(3)
    x = torch.randn(tokens, d, generator=g, device=device).bfloat16()
    target = teacher.forward(x).float()
    losses = []
    for _ in range(steps):
        out, saved = block.forward(x, train=True)
        diff = out.float() - target
        losses.append(float(diff.square().mean()))
        block.update(block.backward(saved, (2.0 / diff.numel() * diff).bfloat16()), rate)
    return losses


def serve_sparse(steps: int, shape=synth.TINY, tokens: int = 4, device="cuda:0"):
    """A prompt, then decode steps from one graph; (outputs of the steps, their inputs, block)."""
    w = synth.make_weights(shape, seed=0, device=device)
    block = SparseFfn(shape, w, torch.ones(shape.d, device=device), max_tokens=shape.T)
    block.prompt(synth.make_x(shape, seed=1, device=device))
    inputs = [synth.make_x(shape, seed=2 + i, device=device, T=tokens) for i in range(steps + 1)]
    x, residual = inputs[0].clone(), torch.zeros_like(inputs[0])
    block.decode(x, residual)  # allocates the layer's workspace for a few tokens
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.decode(x, residual)
    outs = []
    for i in range(steps):
        x.copy_(inputs[i])             # here a model's attention would write
        residual.copy_(inputs[i + 1])
        graph.replay()
        outs.append(out.clone())
    return outs, inputs, block


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=20)
    steps = p.parse_args().steps
    losses = train_dense(steps)
    print(f"dense block: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    outs, _, block = serve_sparse(steps)
    assert block.layer.few_device_error() == lmoe.LMOE_OK
    print(f"sparse block: {steps} decode steps of {outs[0].shape[0]} tokens, "
          f"rms of the last {float(outs[-1].float().square().mean().sqrt()):.3f}")


if __name__ == "__main__":
    main()
