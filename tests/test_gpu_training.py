"""The training-step operators together: the AdamW engine against its 64-bit form,
and the example that trains with layer norm, the aggregation, the norm and AdamW."""

import importlib.util
import os

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import ops_ref
from tests.conftest import ROOT
from tests.ops_ref import U, assert_within

pytestmark = pytest.mark.gpu

SIZES = [1001, 64, 3333, 2, 7000]


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


def worker_grads(W, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [[(torch.randn(n, generator=g, device="cuda") * scale).half() for n in SIZES]
            for _ in range(W)]


def initial():
    g = torch.Generator(device="cuda").manual_seed(77)
    return torch.randn(sum(SIZES), generator=g, device="cuda") * 0.05


@pytest.mark.parametrize("order", [fc.FC_ORDER_SEQUENTIAL, fc.FC_ORDER_RING])
@pytest.mark.parametrize("W", [1, 3, 8])
def test_engine_step_against_64_bits(W, order):
    S, decay = 256.0, [1.0, 0.0, 1.0, 0.0, 0.5]
    eng = fc.AdamWEngine(SIZES, W, initial(), lr=1e-2, loss_scale=S, decay=decay, max_norm=0.5,
                         low=torch.bfloat16, order=order)
    grads = worker_grads(W, 5)
    w0 = eng.weights.clone()
    eng.step(grads)
    torch.cuda.synchronize()
    mean = torch.cat([sum(grads[w][l].double() for w in range(W)) for l in range(len(SIZES))])
    mean /= S * W
    norm = float(mean.norm())
    # W - 1 sums and the unscale, of terms that may cancel
    emean = (W + 2) * U * torch.cat([sum(grads[w][l].double().abs() for w in range(W))
                                     for l in range(len(SIZES))]) / (S * W)
    assert_within("a", eng.a, mean, emean)
    assert abs(float(eng.norm) - norm) <= (W + 12) * U * W ** 0.5 * norm
    f = min(1.0, 0.5 / norm)
    assert abs(float(eng.scale) - f) <= (W + 16) * U * W ** 0.5 * f
    d = torch.repeat_interleave(torch.tensor(decay, device="cuda"),
                                torch.tensor(SIZES, device="cuda"))
    zero = torch.zeros_like(mean)
    # from the kernel's own factor and mean, so that the bound is AdamW's alone
    (w, m, v), (ew, em, ev) = ops_ref.adamw(w0, zero, zero, eng.a.double() * float(eng.scale), d,
                                            1, 1e-2, 0.9, 0.999, 1e-8, 0.01)
    assert_within("w", eng.weights, w, ew)
    assert_within("m", eng.exp_avg, m, em)
    assert_within("v", eng.exp_avg_sq, v, ev)
    assert torch.equal(eng.weights_low, eng.weights.to(torch.bfloat16))
    assert eng.steps.tolist() == [1, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_engine_skips_an_overflow_and_goes_on(bits):
    eng = fc.AdamWEngine(SIZES, 2, initial(), lr=1e-3, loss_scale=64.0, max_norm=1.0, bits=bits,
                         low=torch.float16, seed=3)
    eng.step(worker_grads(2, 1))
    torch.cuda.synchronize()
    before = eng.state_dict()
    bad = worker_grads(2, 2)
    bad[1][2][100] = float("inf")
    eng.step(bad)
    torch.cuda.synchronize()
    assert not torch.isfinite(eng.scale).any()
    for k, v in eng.state_dict().items():
        assert torch.equal(v.view(torch.uint8), before[k].view(torch.uint8)), k
    eng.step(worker_grads(2, 3))
    torch.cuda.synchronize()
    assert eng.steps.tolist() == [2, 0]


@pytest.mark.parametrize("bits", [32, 8])
def test_engine_resumes_from_its_state(bits):
    make = lambda: fc.AdamWEngine(SIZES, 2, initial(), lr=1e-3, loss_scale=64.0, bits=bits,  # noqa
                                  low=torch.float16, seed=3)
    one, two = make(), make()
    for k in range(3):
        one.step(worker_grads(2, k))
    two.load_state_dict(one.state_dict())
    assert torch.equal(two.weights_low, one.weights_low)
    for k in range(3, 6):
        one.step(worker_grads(2, k))
        two.step(worker_grads(2, k))
    torch.cuda.synchronize()
    for k, v in one.state_dict().items():
        assert torch.equal(v.view(torch.uint8), two.state_dict()[k].view(torch.uint8)), k


def test_engine_refusals():
    w = initial()
    for bad in (dict(bits=16), dict(order=fc.FC_ORDER_TREE), dict(low=torch.float32)):
        with pytest.raises(ValueError):
            fc.AdamWEngine(SIZES, 2, w, lr=1e-3, loss_scale=64.0, **bad)
    with pytest.raises(ValueError):
        fc.AdamWEngine(SIZES, 2, w[:-1], lr=1e-3, loss_scale=64.0)


def example():
    path = os.path.join(ROOT, "examples", "train_norm_mlp.py")
    spec = importlib.util.spec_from_file_location("train_norm_mlp", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits", [32, 8])
def test_example_trains(bits):
    losses = example().train(steps=120, workers=2, width=129, hidden=256, blocks=2, bits=bits)
    first, last = sum(losses[:5]) / 5, sum(losses[-10:]) / 10
    assert last < 0.5 * first, (first, last)


def test_example_gradients_match_torch():
    """The model's gradients with the library's layer norm against torch's own."""
    mod = example()
    gen = torch.Generator(device="cuda").manual_seed(4)
    model = mod.Model(100, 64, 2)
    fused = model.initial(gen)
    x = torch.randn(30, 100, generator=gen, device="cuda")

    def grads(norm):
        mod.LayerNorm.apply, keep = norm, mod.LayerNorm.apply
        try:
            p = model.parameters(fused)
            return torch.autograd.grad(model.forward(x, p).square().mean(), p)
        finally:
            mod.LayerNorm.apply = keep

    ours = grads(mod.LayerNorm.apply)
    theirs = grads(lambda v, g, b: torch.nn.functional.layer_norm(v, (v.shape[1],), g, b, mod.EPS))
    for a, b in zip(ours, theirs):
        # fp32 on both sides, through products of 100 and 64 terms
        assert float((a - b).norm()) <= 1e-4 * float(b.norm()) + 1e-7
