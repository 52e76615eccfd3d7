"""A whole training step: from the loss over a vocabulary back through the blocks to updated weights.

    h     = embedding[tokens]
    h     = block(h)                               (dense or sparse, examples/decoder_ffn.py)
    loss  = mean of cross entropy(rmsnorm(h) W_head^T, next tokens)

Matrices inside the model are updated by Muon, its vectors, the embedding and the head by plain gradient
steps.  DenseModel holds a dense block; SparseModel the Stable Latent MoE layer, whose experts' weights
are batches of matrices, and whose gradients go into the update as the layer's backward leaves them.

    python examples/train_step.py [--steps N]

trains both on one batch of tokens and prints their losses."""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

from decoder_ffn import DenseFfn  # noqa: E402
from latent_compressed_expert_gb300 import lmoe, synth  # noqa: E402

MATRICES = ("w_down", "w_router", "w_gate", "w_value", "w_edown", "w_up", "w_sgate", "w_svalue",
            "w_sdown")


def muon_scale(w: torch.Tensor) -> float:
    """A step of the size that Adam's have: 0.2 in the root mean square of its entries."""
    return 0.2 * max(w.shape[-2:]) ** 0.5


class Ends:
    """What stands before and after the blocks: embedding, last norm and head."""

    def __init__(self, vocabulary: int, d: int, device, seed: int = 0, eps: float = 1e-6):
        g = torch.Generator(device=device).manual_seed(seed)
        self.embedding = torch.randn(vocabulary, d, generator=g, device=device).bfloat16()
        self.gamma, self.eps = torch.ones(d, device=device), eps
        self.head = lmoe.LinearCrossEntropy(
            (torch.randn(vocabulary, d, generator=g, device=device) * d ** -0.5).bfloat16())

    def loss(self, h: torch.Tensor, target: torch.Tensor):
        """(mean loss of the rows that have a target, what ``backward`` needs)."""
        y, total, rstd = lmoe.add_rmsnorm(h, self.gamma, eps=self.eps, train=True)
        loss, lse = self.head.forward(y, target)
        weight = (target >= 0).float()
        weight /= weight.sum().clamp(min=1)
        return (loss * weight).sum(), (y, total, rstd, lse, weight, target)

    def backward(self, saved) -> dict:
        """Gradients of h, gamma and the head."""
        y, total, rstd, lse, weight, target = saved
        g = self.head.backward(y, target, lse, weight)
        dh, dgamma = lmoe.add_rmsnorm_backward(g["dx"], total, self.gamma, rstd)
        return {"dh": dh, "dgamma": dgamma, "dhead": g["dw"]}

    def update(self, grads: dict, tokens: torch.Tensor, rate: float):
        self.gamma.sub_(grads["dgamma"], alpha=rate)
        self.head.w.sub_(grads["dhead"], alpha=rate)
        self.embedding.index_add_(0, tokens, grads["dembedding"], alpha=-rate)


class DenseModel:
    def __init__(self, vocabulary: int, d: int, width: int, device, seed: int = 0):
        self.ends = Ends(vocabulary, d, device, seed)
        self.block = DenseFfn(d, width, device, seed + 1)
        self.muon = lmoe.Muon(device=device)
        self.momentum = [torch.zeros_like(m) for m in self.block.masters]

    def gradients(self, tokens: torch.Tensor, target: torch.Tensor):
        """(loss, gradients of everything)."""
        h, saved = self.block.forward(self.ends.embedding[tokens], train=True)
        loss, ends = self.ends.loss(h, target)
        grads = self.ends.backward(ends)
        block = self.block.backward(saved, grads["dh"])
        return loss, {**grads, "block": block, "dembedding": block["dx"]}

    def step(self, tokens: torch.Tensor, target: torch.Tensor, rate: float = 0.02, plain: float = 0.5):
        loss, grads = self.gradients(tokens, target)
        self.ends.update(grads, tokens, plain)
        b = grads["block"]
        self.block.gamma.sub_(b["dgamma"], alpha=plain)
        for lin, master, momentum, name in zip((self.block.up, self.block.down), self.block.masters,
                                               self.momentum, ("dw_up", "dw_down")):
            self.muon.update(lin.w, b[name], momentum, rate, muon_scale(master), master=master)
        return loss


class SparseModel:
    def __init__(self, vocabulary: int, shape, device, seed: int = 0):
        self.ends = Ends(vocabulary, shape.d, device, seed)
        self.weights = synth.make_weights(shape, seed=seed + 1, device=device)
        self.layer = lmoe.Layer(shape, self.weights, max_tokens=shape.T)
        self.layer.enable_backward(self.weights)
        self.muon = lmoe.Muon(device=device)
        self.momentum = {n: torch.zeros(self.weights[n].shape, device=device) for n in MATRICES}

    def gradients(self, tokens: torch.Tensor, target: torch.Tensor):
        x = self.ends.embedding[tokens]
        h = self.layer.forward(x, residual=x, train=True)
        loss, ends = self.ends.loss(h, target)
        grads = self.ends.backward(ends)
        layer = self.layer.backward_layer(x, grads["dh"])
        # x reaches the output through the layer and as its residual
        dx = (layer["dx"] + grads["dh"].float()).bfloat16()
        return loss, {**grads, "layer": layer, "dembedding": dx}

    def step(self, tokens: torch.Tensor, target: torch.Tensor, rate: float = 0.02, plain: float = 0.5):
        loss, grads = self.gradients(tokens, target)
        self.ends.update(grads, tokens, plain)
        g = grads["layer"]
        self.weights["gamma"].sub_(g["dgamma"], alpha=plain)
        for n in MATRICES:
            w = self.weights[n]
            self.muon.update(w, g["d" + n], self.momentum[n], rate, muon_scale(w))
        # the layer multiplies by its own layout of the weights
        self.layer.packed = lmoe.pack_weights(self.layer.dims, self.weights)
        self.layer.enable_backward(self.weights)
        return loss


def batch(vocabulary: int, count: int, device, seed: int = 0):
    """Tokens, each followed by one that it determines; every eighth has no target."""
    g = torch.Generator(device=device).manual_seed(seed)
    tokens = torch.randint(0, vocabulary, (count,), generator=g, device=device)
    target = (tokens * 7 + 3) % vocabulary
    target[::8] = -100
    return tokens, target


def train(model, vocabulary: int, count: int, steps: int, device="cuda:0") -> list:
    tokens, target = batch(vocabulary, count, device)
    return [float(model.step(tokens, target)) for _ in range(steps)]


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=10)
    steps = p.parse_args().steps
    device = torch.device("cuda:0")
    for name, model, count in (("dense", DenseModel(1000, 256, 512, device), 512),
                               ("sparse", SparseModel(1000, synth.TINY, device), synth.TINY.T)):
        losses = train(model, 1000, count, steps, device)
        print(f"{name} model: loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")


if __name__ == "__main__":
    main()
