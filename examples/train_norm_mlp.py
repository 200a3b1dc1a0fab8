#!/usr/bin/env python3
"""A residual network of layer norms and two-matrix blocks, trained data-parallel
by simulated workers on one GPU.

Every worker draws its own batch and runs its own backward pass in fp16 under a
loss scale; layer norm's forward and backward passes are the library's, and its
parameter gradients come out in the fp16 that the aggregation takes.  One
optimiser step then sums the workers' gradients, takes the global norm, clips,
and applies AdamW with moments in 32 or in 8 bits to the fp32 master weights
(fc.AdamWEngine).  A step whose gradients overflow is skipped on the device.

    python examples/train_norm_mlp.py --steps 200 --bits 8
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gradient_aggregation_gb300 import fc  # noqa: E402

EPS = 1e-5


def first_derivatives_only():
    """A second derivative through a kernel's result would leave out the kernel."""
    if torch.is_grad_enabled():
        raise RuntimeError("the kernels give first derivatives only, not create_graph=True")


class LayerNorm(torch.autograd.Function):
    """fc.fc_layernorm_forward and fc.fc_layernorm_backward as one torch function."""

    @staticmethod
    def forward(ctx, x, weight, bias):
        y = torch.empty_like(x)
        mean = torch.empty(x.shape[0], device=x.device)
        rstd = torch.empty_like(mean)
        fc.fc_layernorm_forward(x, weight, bias, EPS, y, mean, rstd)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        first_derivatives_only()
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dweight, dbias = torch.empty_like(x), torch.empty_like(weight), torch.empty_like(weight)
        workspace = torch.empty(fc.fc_layernorm_backward_workspace_size(*x.shape),
                                dtype=torch.uint8, device=x.device)
        fc.fc_layernorm_backward(dy.contiguous(), x, weight, mean, rstd, dx, dweight, dbias,
                                 workspace)
        return dx, dweight, dbias


class Model:
    """`blocks` residual blocks x + W2 relu(W1 norm(x) + b1) + b2, a norm, a readout."""

    def __init__(self, width, hidden, blocks):
        self.shapes = []
        for _ in range(blocks):
            self.shapes += [(width,), (width,), (hidden, width), (hidden,), (width, hidden),
                            (width,)]
        self.shapes += [(width,), (width,), (1, width)]
        self.blocks = blocks
        self.sizes = [torch.Size(s).numel() for s in self.shapes]

    def initial(self, generator):
        """fp32 weights in the fused layout: norms at 1 and 0, matrices scaled by their width."""
        parts = []
        for i, s in enumerate(self.shapes):
            if len(s) == 2:
                parts.append(torch.randn(s, generator=generator, device="cuda") / s[1] ** 0.5)
            else:
                norm_weight = self.shapes[i + 1:i + 2] == [s] and (i % 6 == 0)
                parts.append(torch.full(s, 1.0 if norm_weight else 0.0, device="cuda"))
        return torch.cat([p.reshape(-1) for p in parts])

    def parameters(self, fused):
        """Views of a fused vector, one a layer, that autograd can differentiate by."""
        out, at = [], 0
        for s, n in zip(self.shapes, self.sizes):
            out.append(fused[at:at + n].view(s).detach().requires_grad_())
            at += n
        return out

    def forward(self, x, p):
        for k in range(self.blocks):
            g, b, w1, b1, w2, b2 = p[6 * k:6 * k + 6]
            h = torch.relu(torch.addmm(b1, LayerNorm.apply(x, g, b), w1.t()))
            x = x + torch.addmm(b2, h, w2.t())
        g, b, w = p[6 * self.blocks:]
        return LayerNorm.apply(x, g, b) @ w.t()


def train(steps=200, workers=4, width=200, hidden=512, blocks=3, batch=64, bits=32, lr=3e-3,
          loss_scale=1024.0, max_norm=1.0, seed=0, report=None):
    """Losses of every step (mean over the workers)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(width, hidden, blocks)
    # matrices are decayed, norms and biases are not
    decay = [1.0 if len(s) == 2 else 0.0 for s in model.shapes]
    eng = fc.AdamWEngine(model.sizes, workers, model.initial(gen), lr=lr, loss_scale=loss_scale,
                         weight_decay=0.01, decay=decay, max_norm=max_norm, bits=bits,
                         low=torch.float16, seed=seed)
    teacher = torch.randn(width, 8, generator=gen, device="cuda") / width ** 0.5
    losses = []
    for step in range(steps):
        params = model.parameters(eng.weights_low)
        grads, total = [], torch.zeros((), device="cuda")
        for _ in range(workers):
            x = torch.randn(batch, width, generator=gen, device="cuda")
            target = torch.tanh(x @ teacher).sum(1, keepdim=True)
            loss = (model.forward(x.half(), params).float() - target).square().mean()
            grads.append(list(torch.autograd.grad(loss * loss_scale, params)))
            total += loss.detach()
        eng.step(grads)
        losses.append(total / workers)
        if report and (step + 1) % report == 0:
            print("step %4d  loss %.4f  gradient norm %.3f  steps applied %d"
                  % (step + 1, float(losses[-1]), float(eng.norm), int(eng.steps[0])))
    return [float(v) for v in torch.stack(losses)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--width", type=int, default=200)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--blocks", type=int, default=3)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--lr", type=float, default=3e-3)
    a = ap.parse_args()
    train(a.steps, a.workers, a.width, a.hidden, a.blocks, a.batch, a.bits, a.lr,
          report=max(1, a.steps // 10))
