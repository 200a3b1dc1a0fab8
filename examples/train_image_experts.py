#!/usr/bin/env python3
"""A small image classifier with a mixture of experts, trained data-parallel by
simulated workers on one GPU.

Images lie channels last, [samples, positions, channels], and may have fewer
positions than the batch is wide.  Residual blocks are group norm with SiLU and a
matrix; then a router scores the experts for every position, k of them work on it,
and its balance loss keeps all of them in use.  Both passes of the norms and of the
router are the library's.  One optimiser step sums the workers' fp16 gradients,
takes the global norm, clips, and applies AdamW (fc.AdamWEngine).

    python examples/train_image_experts.py --steps 200 --experts 8 --k 2
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


class GroupNormSiLU(torch.autograd.Function):
    """fc.fc_groupnorm_forward and fc.fc_groupnorm_backward as one torch function."""

    @staticmethod
    def forward(ctx, x, groups, weight, bias):
        y = torch.empty_like(x)
        mean = torch.empty(x.shape[0], groups, device=x.device)
        rstd = torch.empty_like(mean)
        workspace = torch.empty(fc.fc_groupnorm_workspace_size(*x.shape, groups),
                                dtype=torch.uint8, device=x.device)
        fc.fc_groupnorm_forward(x, groups, weight, bias, EPS, fc.FC_ACT_SILU, y, mean, rstd,
                                workspace)
        ctx.groups = groups
        ctx.save_for_backward(x, weight, bias, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        first_derivatives_only()
        x, weight, bias, mean, rstd = ctx.saved_tensors
        dx, dweight, dbias = torch.empty_like(x), torch.empty_like(weight), torch.empty_like(bias)
        workspace = torch.empty(fc.fc_groupnorm_workspace_size(*x.shape, ctx.groups),
                                dtype=torch.uint8, device=x.device)
        fc.fc_groupnorm_backward(dy.contiguous(), x, ctx.groups, weight, bias, fc.FC_ACT_SILU, mean,
                                 rstd, dx, dweight, dbias, workspace)
        return dx, None, dweight, dbias


class Router(torch.autograd.Function):
    """fc.fc_router_forward and fc.fc_router_backward: the weights of the k experts of
    each row, the two losses, the experts and how many rows chose each."""

    @staticmethod
    def forward(ctx, logits, sequences, lengths, k):
        (rows, experts), dev = logits.shape, logits.device
        chosen = torch.empty(rows, k, dtype=torch.int32, device=dev)
        weights, lse = torch.empty(rows, k, device=dev), torch.empty(rows, device=dev)
        counts = torch.empty(1, experts, dtype=torch.int32, device=dev)
        routed = torch.empty(1, dtype=torch.int32, device=dev)
        probs, loss = torch.empty(1, experts, device=dev), torch.empty(2, device=dev)
        workspace = torch.empty(fc.fc_router_workspace_size(sequences, rows // sequences, experts),
                                dtype=torch.uint8, device=dev)
        fc.fc_router_forward(logits, sequences, lengths, True, False, chosen, weights, lse, counts,
                             routed, probs, loss, workspace)
        ctx.sequences = sequences
        ctx.save_for_backward(logits, chosen, weights, lse, counts, routed)
        ctx.mark_non_differentiable(chosen, counts)
        return weights, loss, chosen, counts

    @staticmethod
    def backward(ctx, dweights, dloss, _chosen, _counts):
        first_derivatives_only()
        logits, chosen, weights, lse, counts, routed = ctx.saved_tensors
        dlogits = torch.empty_like(logits)
        fc.fc_router_backward(logits, ctx.sequences, True, False, chosen, weights, lse, counts,
                              routed, dweights.contiguous(), dloss.contiguous(), dlogits)
        return dlogits, None, None, None


class Model:
    """A stem, `blocks` residual blocks x + W silu(norm(x)), the experts, a readout of the
    mean over an image's positions."""

    def __init__(self, inputs, channels, groups, blocks, experts, k, classes):
        self.channels, self.groups, self.blocks = channels, groups, blocks
        self.experts, self.k = experts, k
        norm = [(channels,), (channels,)]
        self.shapes = [(channels, inputs)] + (norm + [(channels, channels)]) * blocks
        self.shapes += norm + [(experts, channels), (experts, channels, channels),
                               (classes, channels)]
        self.sizes = [torch.Size(s).numel() for s in self.shapes]

    def initial(self, generator):
        """fp32 weights in the fused layout: norms at 1 and 0, matrices scaled by their width."""
        parts, scale = [], True
        for s in self.shapes:
            if len(s) > 1:
                parts.append(torch.randn(s, generator=generator, device="cuda") / s[-1] ** 0.5)
            else:
                parts.append(torch.full(s, 1.0 if scale else 0.0, device="cuda"))
                scale = not scale
        return torch.cat([p.reshape(-1) for p in parts])

    def parameters(self, fused):
        """Views of a fused vector, one a layer, that autograd can differentiate by."""
        out, at = [], 0
        for s, n in zip(self.shapes, self.sizes):
            out.append(fused[at:at + n].view(s).detach().requires_grad_())
            at += n
        return out

    def forward(self, x, lengths, p):
        """Scores of the classes, the two losses of the router, the rows that each expert has."""
        samples, positions, _ = x.shape
        x = x @ p[0].t()
        for b in range(self.blocks):
            scale, shift, w = p[1 + 3 * b:4 + 3 * b]
            x = x + GroupNormSiLU.apply(x, self.groups, scale, shift) @ w.t()
        scale, shift, router, experts, readout = p[1 + 3 * self.blocks:]
        tokens = GroupNormSiLU.apply(x, self.groups, scale, shift).flatten(0, 1)
        weights, loss, chosen, counts = Router.apply(tokens @ router.t(), samples, lengths, self.k)
        # every expert on every token, of which the chosen are taken
        every = torch.einsum("rc,edc->red", tokens, experts)
        taken = every.gather(1, chosen.clamp(min=0).long()[:, :, None].expand(-1, -1, self.channels))
        mixed = (taken * weights[:, :, None].to(taken.dtype)).sum(1)  # of no routed token: 0
        x = x + mixed.view_as(x)
        inside = torch.arange(positions, device=x.device)[None, :] < lengths[:, None]
        pooled = (x.float() * inside[:, :, None]).sum(1) / lengths[:, None]
        return pooled @ readout.float().t(), loss, counts


def images(gen, batch, positions, teacher, classes):
    """Random maps of 1 to `positions` positions; the class is that of the largest mean
    projection."""
    x = torch.randn(batch, positions, teacher.shape[0], generator=gen, device="cuda")
    lengths = torch.randint(1, positions + 1, (batch,), generator=gen, device="cuda",
                            dtype=torch.int32)
    inside = torch.arange(positions, device="cuda")[None, :] < lengths[:, None]
    label = ((x @ teacher) * inside[:, :, None]).sum(1)[:, :classes].argmax(1)
    return x, lengths, label


def train(steps=200, workers=4, inputs=12, channels=64, groups=8, blocks=2, experts=8, k=2,
          classes=5, batch=16, positions=49, balance=0.01, bits=32, lr=2e-3, loss_scale=1024.0,
          max_norm=1.0, seed=0, report=None):
    """Losses of every step (mean over the workers), without the router's."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    model = Model(inputs, channels, groups, blocks, experts, k, classes)
    # matrices are decayed, norms are not
    decay = [1.0 if len(s) > 1 else 0.0 for s in model.shapes]
    eng = fc.AdamWEngine(model.sizes, workers, model.initial(gen), lr=lr, loss_scale=loss_scale,
                         weight_decay=0.01, decay=decay, max_norm=max_norm, bits=bits,
                         low=torch.float16, seed=seed)
    teacher = torch.randn(inputs, classes, generator=gen, device="cuda")
    losses = []
    for step in range(steps):
        params = model.parameters(eng.weights_low)
        grads, total = [], torch.zeros((), device="cuda")
        for _ in range(workers):
            x, lengths, label = images(gen, batch, positions, teacher, classes)
            scores, routing, counts = model.forward(x.half(), lengths, params)
            loss = torch.nn.functional.cross_entropy(scores, label)
            extra = balance * routing[0] + 0.1 * balance * routing[1]
            grad = torch.autograd.grad((loss + extra) * loss_scale, params)
            grads.append([g.contiguous() for g in grad])
            total += loss.detach()
        eng.step(grads)
        losses.append(total / workers)
        if report and (step + 1) % report == 0:
            print("step %4d  loss %.4f  balance %.3f  rows of an expert %d to %d"
                  % (step + 1, float(losses[-1]), float(routing[0]), int(counts.min()),
                     int(counts.max())))
    return [float(v) for v in torch.stack(losses)]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--workers", type=int, default=4)
    ap.add_argument("--channels", type=int, default=64)
    ap.add_argument("--groups", type=int, default=8)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--k", type=int, default=2)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--positions", type=int, default=49)
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32)
    ap.add_argument("--lr", type=float, default=2e-3)
    a = ap.parse_args()
    train(a.steps, a.workers, channels=a.channels, groups=a.groups, blocks=a.blocks,
          experts=a.experts, k=a.k, batch=a.batch, positions=a.positions, bits=a.bits, lr=a.lr,
          report=max(1, a.steps // 10))
