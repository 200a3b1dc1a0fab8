"""Group norm and the router used together: the example that trains a mixture of experts
on images, its gradients, and a captured step of both operators."""

import importlib.util
import os

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import model_ops_ref as ref
from tests.ops_ref import assert_within, rounded

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


def example():
    path = os.path.join(ROOT, "examples", "train_image_experts.py")
    spec = importlib.util.spec_from_file_location("train_image_experts", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits", [32, 8])
def test_example_runs(bits):
    losses = example().train(steps=6, workers=2, channels=40, groups=5, blocks=1, experts=6, k=3,
                             batch=7, positions=25, bits=bits)
    assert len(losses) == 6 and all(v == v and abs(v) < 100 for v in losses)


class PlainNorm:
    @staticmethod
    def apply(x, groups, weight, bias):
        c = x.shape[2]
        y = torch.nn.functional.group_norm(x.transpose(1, 2), groups, weight, bias, 1e-5)
        return torch.nn.functional.silu(y).transpose(1, 2).reshape(-1, x.shape[1], c)


def plain_router(chosen):
    """Weights and losses of a given choice, by torch's own operators."""
    class Plain:
        @staticmethod
        def apply(logits, sequences, lengths, k):
            rows, experts = logits.shape
            tokens = rows // sequences
            live = (torch.arange(tokens, device=logits.device)[None, :] < lengths[:, None]).flatten()
            lse = torch.logsumexp(logits, 1)
            p = torch.exp(logits - lse[:, None])
            w = p.gather(1, chosen.clamp(min=0).long())
            w = torch.where(live[:, None], w / w.sum(1, keepdim=True), 0.0)
            n = live.sum()
            counts = torch.zeros(experts, device=logits.device, dtype=logits.dtype)
            counts.index_add_(0, chosen[live].long().flatten(),
                              torch.ones(int(n) * k, device=logits.device, dtype=logits.dtype))
            probs = (p * live[:, None]).sum(0) / n
            loss = torch.stack([(counts * experts / (k * n) * probs).sum(),
                                (lse.square() * live).sum() / n])
            return w, loss, chosen, counts[None]
    return Plain


def test_example_gradients_match_torch():
    """The model's gradients with the library's operators, in fp32, against the same model in
    64 bits with torch's, for the experts that were chosen."""
    mod = example()
    gen = torch.Generator(device="cuda").manual_seed(4)
    model = mod.Model(12, 48, 6, 2, 8, 2, 5)
    fused = model.initial(gen)
    x = torch.randn(9, 30, 12, generator=gen, device="cuda")
    lengths = torch.tensor([30, 1, 7, 30, 22, 15, 2, 29, 30], dtype=torch.int32, device="cuda")
    seen = []

    class Watched:
        @staticmethod
        def apply(*args):
            out = router.apply(*args)
            seen.append(out[2])
            return out

    def grads(norm, route, weights, maps):
        mod.GroupNormSiLU, mod.Router = norm, route
        p = model.parameters(weights)
        scores, loss, counts = model.forward(maps, lengths, p)
        total = scores.square().mean() + 0.3 * loss[0] + 0.1 * loss[1]
        return torch.autograd.grad(total, p), counts

    norm, router = mod.GroupNormSiLU, mod.Router
    ours, counts = grads(norm, Watched, fused, x)
    # in 64 bits; only the pooled maps and the readout are rounded to fp32 on the way
    theirs, want = grads(PlainNorm, plain_router(seen[0]), fused.double(), x.double())
    assert torch.equal(counts.double(), want)
    for a, b in zip(ours, theirs):
        # fp32 on one side, through 3 norms and 5 products of 12 to 48 terms, each within
        # some 50 roundings of 2^-24
        assert float((a.double() - b).norm()) <= 1e-4 * float(b.norm()) + 1e-7


def test_second_derivatives_are_refused():
    """The kernels give first derivatives: one by these would leave out what goes through them."""
    mod, x = example(), torch.randn(2, 9, 8, device="cuda", requires_grad=True)
    weight = torch.ones(8, device="cuda", requires_grad=True)
    bias = torch.zeros(8, device="cuda", requires_grad=True)
    lengths = torch.tensor([9, 3], dtype=torch.int32, device="cuda")
    path = os.path.join(ROOT, "examples", "train_norm_mlp.py")
    spec = importlib.util.spec_from_file_location("train_norm_mlp", path)
    norms = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(norms)
    for call in (lambda: mod.GroupNormSiLU.apply(x, 2, weight, bias),
                 lambda: mod.Router.apply(x.flatten(0, 1), 2, lengths, 2)[1],
                 lambda: norms.LayerNorm.apply(x.flatten(0, 1), weight, bias)):
        loss = call().square().sum() + (x ** 3).sum()
        with pytest.raises(RuntimeError, match="first derivatives"):
            grad, = torch.autograd.grad(loss, x, create_graph=True)
            torch.autograd.grad(grad.square().sum(), x)


def test_captured_together_with_one_workspace():
    """Norm, logits, router and back, captured once and replayed on other maps: within the
    bounds of the definitions, and the bits of the calls made one by one."""
    n, s, c, groups, experts, k = 5, 36, 64, 8, 16, 2
    rows = n * s
    dev = dict(device="cuda")
    x, y, dx = (torch.empty(n, s, c, dtype=BF16, **dev) for _ in range(3))
    weight, bias = torch.linspace(0.5, 1.5, c, **dev), torch.linspace(-0.2, 0.3, c, **dev)
    mean, rstd = torch.empty(n, groups, **dev), torch.empty(n, groups, **dev)
    matrix = torch.empty(experts, c, dtype=BF16, **dev)
    logits, dlogits = (torch.empty(rows, experts, dtype=BF16, **dev) for _ in range(2))
    dy = torch.empty(n, s, c, dtype=BF16, **dev)
    dweight, dbias = torch.empty(c, **dev), torch.empty(c, **dev)
    chosen = torch.empty(rows, k, dtype=torch.int32, **dev)
    weights, lse = torch.empty(rows, k, **dev), torch.empty(rows, **dev)
    counts = torch.empty(1, experts, dtype=torch.int32, **dev)
    routed = torch.empty(1, dtype=torch.int32, **dev)
    probs, loss = torch.empty(1, experts, **dev), torch.empty(2, **dev)
    dweights, dloss = torch.empty(rows, k, **dev), torch.tensor([2.0, 0.1], **dev)
    lengths = torch.empty(n, dtype=torch.int32, **dev)
    size = max(fc.fc_groupnorm_workspace_size(n, s, c, groups),
               fc.fc_router_workspace_size(n, s, experts))
    workspace = torch.full((size,), 0xFF, dtype=torch.uint8, **dev)

    def step():
        fc.fc_groupnorm_forward(x, groups, weight, bias, 1e-5, fc.FC_ACT_SILU, y, mean, rstd,
                                workspace)
        torch.mm(y.view(rows, c), matrix.t(), out=logits)
        fc.fc_router_forward(logits, n, lengths, True, False, chosen, weights, lse, counts, routed,
                             probs, loss, workspace)
        fc.fc_router_backward(logits, n, True, False, chosen, weights, lse, counts, routed, dweights,
                              dloss, dlogits)
        torch.mm(dlogits, matrix, out=dy.view(rows, c))
        fc.fc_groupnorm_backward(dy, x, groups, weight, bias, fc.FC_ACT_SILU, mean, rstd, dx, dweight,
                                 dbias, workspace)

    def fill(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        x.copy_(torch.randn(n, s, c, generator=g, **dev))
        matrix.copy_(torch.randn(experts, c, generator=g, **dev) / 4)
        dweights.copy_(torch.randn(rows, k, generator=g, **dev))
        lengths.copy_(torch.randint(0, s + 1, (n,), generator=g, **dev))

    fill(1)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step()
    results = (y, logits, chosen, weights, lse, counts, probs, loss, dlogits, dx, dweight, dbias)
    for seed in (2, 3):
        fill(seed)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in results]
        step()
        torch.cuda.synchronize()
        for a, b in zip(replayed, results):
            assert torch.equal(a, b)
        (wy, _, _), (by, _, _) = ref.groupnorm(x, groups, weight, bias, 1e-5, fc.FC_ACT_SILU)
        assert_within("y", y, wy, rounded(by, wy, BF16))
        want, bound = ref.router(logits, n, lengths, k, True, False)
        assert torch.equal(chosen, want["chosen"]) and torch.equal(counts, want["counts"])
        assert_within("loss", loss, want["loss"], rounded(bound["loss"], want["loss"], F32))
        (wx, ww, wb), (bx, bw, bb) = ref.groupnorm_backward(dy, x, groups, weight, bias,
                                                            fc.FC_ACT_SILU, mean, rstd)
        assert_within("dx", dx, wx, rounded(bx, wx, BF16))
        assert_within("dweight", dweight, ww, rounded(bw, ww, F32))
        assert_within("dbias", dbias, wb, rounded(bb, wb, F32))
