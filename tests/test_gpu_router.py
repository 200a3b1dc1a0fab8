"""The router of a mixture of experts on a GPU against its 64-bit form."""

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import model_ops_ref as ref
from tests.ops_ref import assert_within, rounded

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
ids = lambda t: str(t).replace("torch.", "")  # noqa: E731
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


def scores(rows, experts, dtype, pad=0, shift=0, seed=1, scale=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((shift + rows * (experts + pad) + 16,), 7.0, dtype=dtype, device="cuda")
    m = buf[shift:shift + rows * (experts + pad)].view(rows, experts + pad)[:, :experts]
    m.copy_(torch.randn(rows, experts, generator=g, device="cuda") * scale)
    return m, buf


def untouched(m, buf):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside.as_strided(m.shape, m.stride(), m.storage_offset()).fill_(True)
    return bool((buf[~inside] == 7.0).all())


def outputs(rows, experts, k, groups):
    f = dict(device="cuda", dtype=F32)
    i = dict(device="cuda", dtype=torch.int32)
    return {"chosen": torch.full((rows, k), 77, **i), "weights": torch.full((rows, k), 77.0, **f),
            "lse": torch.full((rows,), 77.0, **f), "counts": torch.full((groups, experts), 77, **i),
            "routed": torch.full((groups,), 77, **i),
            "probs": torch.full((groups, experts), 77.0, **f), "loss": torch.full((2,), 77.0, **f)}


def scratch(sequences, tokens, experts, per_sequence):
    return torch.full((fc.fc_router_workspace_size(sequences, tokens, experts, per_sequence),),
                      0xFF, dtype=torch.uint8, device="cuda")


def forward(x, sequences, lengths, k, normalise, per_sequence, stream=None):
    rows, experts = x.shape
    o = outputs(rows, experts, k, sequences if per_sequence else 1)
    ws = scratch(sequences, rows // max(1, sequences), experts, per_sequence)
    fc.fc_router_forward(x, sequences, lengths, normalise, per_sequence, o["chosen"], o["weights"],
                         o["lse"], o["counts"], o["routed"], o["probs"], o["loss"], ws, stream)
    return o


def check_forward(x, sequences, lengths, k, normalise, per_sequence):
    o = forward(x, sequences, lengths, k, normalise, per_sequence)
    torch.cuda.synchronize()
    want, bound = ref.router(x, sequences, lengths, k, normalise, per_sequence)
    for q in ("chosen", "counts", "routed"):
        assert torch.equal(o[q], want[q]), q
    live = want["lse"] > -INF
    assert bool((o["lse"][~live] == -INF).all())
    assert_within("lse", o["lse"][live], want["lse"][live], bound["lse"][live])
    over = want["loss"] > torch.finfo(F32).max  # squares of logits beyond 1.8e19
    assert bool((o["loss"][over] == INF).all())
    for q in o, want, bound:
        q["loss"] = torch.where(over, 0.0, q["loss"])
    for q in ("weights", "probs", "loss"):
        assert_within(q, o[q], want[q], rounded(bound[q], want[q], F32))
    return o


def check(sequences, tokens, experts, k, dtype, normalise=True, per_sequence=False, lengths=None,
          pad=0, shift=0, scale=1.5, mask=0.0, seed=1):
    rows = sequences * tokens
    x, _ = scores(rows, experts, dtype, pad, shift, seed, scale)
    g = torch.Generator(device="cuda").manual_seed(seed + 50)
    if mask:
        x.masked_fill_(torch.rand(rows, experts, generator=g, device="cuda") < mask, -INF)
    if lengths is not None:
        lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    o = check_forward(x, sequences, lengths, k, normalise, per_sequence)
    dw = torch.randn(rows, k, generator=g, device="cuda")
    dl = torch.tensor([0.7, 0.3], device="cuda") * rows
    for dweights, dloss in ((dw, dl), (dw, None), (None, dl)):
        dx, buf = scores(rows, experts, dtype, pad, shift, 5)
        fc.fc_router_backward(x, sequences, normalise, per_sequence, o["chosen"], o["weights"],
                              o["lse"], o["counts"], o["routed"], dweights, dloss, dx)
        torch.cuda.synchronize()
        want, bound = ref.router_backward(x, sequences, k, normalise, per_sequence, o["chosen"],
                                          o["weights"], o["lse"], o["counts"], o["routed"],
                                          dweights, dloss)
        assert_within("dlogits", dx, want, rounded(bound, want, dtype))
        assert untouched(dx, buf)
    return x, o


# both sides of every width class
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("experts,k", [
    (1, 1), (2, 1), (3, 2), (7, 7), (8, 2), (9, 3), (16, 4), (17, 2), (31, 5), (32, 8), (33, 8),
    (60, 4), (64, 6), (65, 6), (100, 8), (128, 8), (129, 8), (160, 6), (255, 8), (256, 8), (257, 10),
    (384, 8), (500, 16), (512, 32), (513, 1), (768, 8), (1000, 32), (1024, 8)])
def test_widths(experts, k, dtype):
    check(1, 131, experts, k, dtype, normalise=bool(k & 1))
    check(3, 40, experts, k, dtype, normalise=not k & 1, per_sequence=True)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("per_sequence", [False, True])
def test_padded_batches(dtype, normalise, per_sequence):
    for experts, k in ((8, 2), (60, 4), (256, 8)):
        check(6, 33, experts, k, dtype, normalise, per_sequence, lengths=[33, 0, 1, 17, 32, -4])
        check(2, 7, experts, k, dtype, normalise, per_sequence, lengths=[0, 0])
        check(2, 7, experts, k, dtype, normalise, per_sequence, lengths=[99, 3])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("pad,shift", [(0, 1), (5, 0), (8, 0), (24, 8), (3, 2), (1, 0), (2, 4)])
def test_strides_and_alignment(pad, shift, dtype):
    for experts, k in ((8, 2), (64, 4), (67, 4), (256, 8)):
        check(2, 50, experts, k, dtype, pad=pad, shift=shift)


# closed experts, up to rows that leave none open
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("mask", [0.3, 0.9, 0.995])
def test_closed_experts(mask, dtype):
    for experts, k in ((4, 2), (24, 8), (100, 8), (300, 6)):
        for normalise in (False, True):
            check(4, 60, experts, k, dtype, normalise, True, mask=mask)


def test_every_row_closed():
    x = torch.full((20, 12), -INF, device="cuda")
    for per_sequence in (False, True):
        o = check_forward(x, 4, None, 3, True, per_sequence)
        assert bool((o["loss"] == 0).all()) and bool((o["routed"] == 0).all())
        dx = torch.full_like(x, 3.0)
        fc.fc_router_backward(x, 4, True, per_sequence, o["chosen"], o["weights"], o["lse"],
                              o["counts"], o["routed"], torch.ones(20, 3, device="cuda"),
                              torch.ones(2, device="cuda"), dx)
        assert bool((dx == 0).all())


# masks of the type's lowest value are numbers like others
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_lowest_values(dtype):
    for experts in (6, 40, 200):
        x, _ = scores(50, experts, dtype)
        x[:, ::2] = torch.finfo(dtype).min
        x[3] = torch.finfo(dtype).min
        o = check_forward(x, 1, None, 4, True, False)
        assert o["chosen"][3].tolist() == [0, 1, 2, 3]
        check_backward(x, o)


def check_backward(x, o):
    rows, k = o["chosen"].shape
    dw, dl = torch.ones(rows, k, device="cuda").cumsum(1), torch.tensor([2.0, 0.0], device="cuda")
    dx = torch.empty_like(x)
    fc.fc_router_backward(x, 1, True, False, o["chosen"], o["weights"], o["lse"], o["counts"],
                          o["routed"], dw, dl, dx)
    want, bound = ref.router_backward(x, 1, k, True, False, o["chosen"], o["weights"], o["lse"],
                                      o["counts"], o["routed"], dw, dl)
    assert_within("dlogits", dx, want, rounded(bound, want, x.dtype))


# logits whose fp32 lse is coarser than what sets the probabilities apart
@pytest.mark.parametrize("shift", [30.0, 3000.0, 1e6, 1e8, -1e8, 3e38])
def test_logits_far_from_zero(shift):
    for experts in (6, 40, 200):
        x, _ = scores(50, experts, F32)
        x.add_(shift)
        check_backward(x, check_forward(x, 1, None, 3, True, False))


def check_both_ways(x, k, sequences=1):
    """Both passes, with weights normalised and as they are, balanced together and apart."""
    rows = x.shape[0]
    dw = torch.randn(rows, k, generator=torch.Generator("cuda").manual_seed(6), device="cuda")
    dl = torch.tensor([2.0, 0.0], device="cuda")
    for normalise in (False, True):
        for per_sequence in (False, True):
            o = check_forward(x, sequences, None, k, normalise, per_sequence)
            dx = torch.empty_like(x)
            fc.fc_router_backward(x, sequences, normalise, per_sequence, o["chosen"], o["weights"],
                                  o["lse"], o["counts"], o["routed"], dw, dl, dx)
            want, bound = ref.router_backward(x, sequences, k, normalise, per_sequence,
                                              o["chosen"], o["weights"], o["lse"], o["counts"],
                                              o["routed"], dw, dl)
            assert_within("dlogits", dx, want, rounded(bound, want, x.dtype))


# a softmax does not depend on what is added to all logits: neither do the weights' digits
@pytest.mark.parametrize("shift", [0.0, 30.0, 100.0, 1e3, 1e4, 1e5, 1e6, 1e8, -100.0, -1e4, -1e8])
def test_weights_of_logits_far_from_zero(shift):
    for experts in (6, 40, 60, 200, 700):
        x, _ = scores(60, experts, F32)
        x.add_(shift)
        check_both_ways(x, 4, 3)


# logits whose product with log2(e) rounds by more than fp32's exponents span
@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
@pytest.mark.parametrize("shift", [65536.0, 7e4, 3e9, 1e10, 1e15, 1e30, 9e37, -7e4, -1e10, -1e37])
def test_logits_of_any_size(shift, dtype):
    for experts in (6, 40, 60, 200, 700):
        x, _ = scores(60, experts, dtype, scale=abs(shift) / 500)
        x[::2] = scores(30, experts, dtype)[0]  # rows of either size side by side
        x[1::2] += shift
        x[3, 1:] = -INF
        x[5] = shift
        check_both_ways(x, 4, 3)


@pytest.mark.parametrize("dtype,shift", [(F16, 100.0), (F16, 3e4), (BF16, 100.0), (BF16, 5e4)])
def test_weights_of_16_bit_logits_far_from_zero(dtype, shift):
    for experts in (8, 60, 256):
        x, _ = scores(60, experts, dtype, scale=shift / 30)
        x.add_(shift)
        check_both_ways(x, 4, 3)


# ties, and zeros of both signs
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_ties_go_to_the_lowest_expert(dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    for experts, k in ((8, 4), (30, 6), (64, 8), (256, 8), (700, 12)):
        x, _ = scores(200, experts, dtype)
        x.copy_(torch.randint(-2, 3, (200, experts), generator=g, device="cuda"))
        x[:, 1::3] *= -1.0
        x[7] = 0.0
        x[8] = -0.0
        x[9, ::2], x[9, 1::2] = -0.0, 0.0
        o = check_forward(x, 2, None, k, False, True)
        for r in (7, 8, 9):
            assert o["chosen"][r].tolist() == list(range(k))


def test_large_logits():
    check(1, 64, 40, 4, F32, scale=300.0)
    check(1, 64, 40, 4, F32, scale=1e-4)
    check(1, 64, 40, 4, BF16, scale=30.0, normalise=False)


@pytest.mark.parametrize("experts", [6, 60, 256])
def test_nan_and_infinity_show(experts):
    for bad in (float("nan"), INF):
        x, _ = scores(30, experts, F32)
        clean = forward(x, 3, None, 3, True, True)
        x[4, 2] = bad
        o = forward(x, 3, None, 3, True, True)
        torch.cuda.synchronize()
        rest = [r for r in range(30) if r != 4]
        for q in ("chosen", "weights", "lse"):
            assert torch.equal(o[q][rest], clean[q][rest])
        assert not bool(torch.isfinite(o["lse"][4]))
        assert bool(torch.isnan(o["weights"][4]).any())
        assert not bool(torch.isfinite(o["loss"]).any())
        got = o["chosen"][4].tolist()
        assert len(set(got)) == 3 and all(0 <= e < experts for e in got)
        assert (2 in got) == (bad == INF)
        assert torch.equal(o["counts"][1:], clean["counts"][1:])
        dx = torch.empty_like(x)
        fc.fc_router_backward(x, 3, True, True, o["chosen"], o["weights"], o["lse"], o["counts"],
                              o["routed"], torch.ones(30, 3, device="cuda"), None, dx)
        torch.cuda.synchronize()
        assert bool(torch.isfinite(dx[rest]).all())


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_many_rows(dtype):
    check(1, 40001, 64, 4, dtype)
    check(5, 6001, 256, 8, dtype, per_sequence=True, lengths=[6001, 17, 0, 5999, 3000])
    check(9, 3001, 8, 2, dtype, normalise=False, lengths=[3001, 17, 0, 2999, 3000, 1, 2, 3, 4])
    check(1, 3000, 1000, 8, dtype)


def test_many_sequences():
    check(3000, 3, 16, 2, BF16, per_sequence=True)
    check(700, 5, 130, 4, F32, per_sequence=True, lengths=[i % 7 for i in range(700)])


def test_no_rows():
    for sequences, tokens in ((0, 0), (4, 0)):
        x = torch.empty(0, 8, device="cuda")
        for per_sequence in (False, True):
            o = forward(x, sequences, None, 2, True, per_sequence)
            torch.cuda.synchronize()
            for q in ("counts", "routed", "probs", "loss"):
                assert bool((o[q] == 0).all()), q
            fc.fc_router_backward(x, sequences, True, per_sequence, o["chosen"], o["weights"],
                                  o["lse"], o["counts"], o["routed"], o["weights"], None, x)


def test_balanced_experts_have_a_loss_of_one():
    rows, experts = 64, 16
    x = torch.zeros(rows, experts, device="cuda")
    x[torch.arange(rows), torch.arange(rows) % experts] = 1e-3
    o = forward(x, 1, None, 1, False, False)
    torch.cuda.synchronize()
    assert bool((o["counts"] == rows // experts).all())
    assert abs(float(o["loss"][0]) - 1) < 1e-5  # 60 roundings


def test_same_bits_again_and_on_another_stream():
    x, a = check(4, 500, 100, 6, BF16, per_sequence=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = forward(x, 4, None, 6, True, True)
    side.synchronize()
    c = forward(x, 4, None, 6, True, True)
    torch.cuda.synchronize()
    for q in a:
        assert torch.equal(a[q], b[q]) and torch.equal(a[q], c[q])


@pytest.mark.parametrize("rows,experts,k", [(64, 8, 2), (5000, 256, 8)])
def test_captured_and_replayed(rows, experts, k):
    x, want = check(1, rows, experts, k, F32)
    o = outputs(rows, experts, k, 1)
    ws = scratch(1, rows, experts, False)
    dw, dl = torch.randn(rows, k, device="cuda"), torch.ones(2, device="cuda")
    dx = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_router_forward(x, 1, None, True, False, o["chosen"], o["weights"], o["lse"],
                             o["counts"], o["routed"], o["probs"], o["loss"], ws)
        fc.fc_router_backward(x, 1, True, False, o["chosen"], o["weights"], o["lse"], o["counts"],
                              o["routed"], dw, dl, dx)
    for _ in range(3):
        for t in o.values():
            t.fill_(55)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for q in want:
            assert torch.equal(o[q], want[q]), q


@pytest.mark.parametrize("normalise", [False, True])
@pytest.mark.parametrize("rows,experts,k", [(64, 8, 2), (5000, 256, 8), (900, 60, 3)])
def test_gradients_captured_and_replayed(rows, experts, k, normalise):
    """A replay's gradients are those of the calls made one by one, on other logits too."""
    x, _ = scores(rows, experts, F32)
    o = outputs(rows, experts, k, 1)
    ws = scratch(1, rows, experts, False)
    dw, dl = torch.randn(rows, k, device="cuda"), torch.ones(2, device="cuda")
    dx = torch.empty_like(x)

    def step():
        fc.fc_router_forward(x, 1, None, normalise, False, o["chosen"], o["weights"], o["lse"],
                             o["counts"], o["routed"], o["probs"], o["loss"], ws)
        fc.fc_router_backward(x, 1, normalise, False, o["chosen"], o["weights"], o["lse"],
                              o["counts"], o["routed"], dw, dl, dx)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2, 3):
        x.copy_(scores(rows, experts, F32, seed=seed)[0])
        for t in (dx, *o.values()):
            t.fill_(55)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got, weights = dx.clone(), o["weights"].clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, dx) and torch.equal(weights, o["weights"])
        want, bound = ref.router_backward(x, 1, k, normalise, False, o["chosen"], o["weights"],
                                          o["lse"], o["counts"], o["routed"], dw, dl)
        assert_within("dlogits", got, want, rounded(bound, want, F32))


def test_refusals():
    x = torch.zeros(12, 8, device="cuda")
    o = outputs(12, 8, 2, 1)
    ws = scratch(3, 4, 8, False)
    good = dict(x=x, sequences=3, lengths=torch.ones(3, dtype=torch.int32, device="cuda"), ws=ws,
                **o)

    def call(**change):
        k = {**good, **change}
        fc.fc_router_forward(k["x"], k["sequences"], k["lengths"], True, False, k["chosen"],
                             k["weights"], k["lse"], k["counts"], k["routed"], k["probs"],
                             k["loss"], k["ws"])
    call()
    for change in (dict(x=x.cpu()), dict(x=x.t()), dict(x=x[0]), dict(x=x.double()),
                   dict(sequences=5), dict(sequences=0), dict(sequences=-1),
                   dict(lengths=torch.ones(3, device="cuda")),
                   dict(lengths=torch.ones(2, dtype=torch.int32, device="cuda")),
                   dict(chosen=o["chosen"].long()), dict(chosen=o["chosen"][:6]),
                   dict(chosen=torch.empty(12, 9, dtype=torch.int32, device="cuda")),
                   dict(chosen=torch.empty(12, 0, dtype=torch.int32, device="cuda")),
                   dict(weights=o["weights"][:, :1]), dict(weights=o["weights"].half()),
                   dict(lse=o["lse"][:5]), dict(counts=o["counts"].long()),
                   dict(probs=o["probs"][:, :4]), dict(loss=o["loss"][:1]), dict(ws=None),
                   dict(ws=ws.cpu()), dict(routed=torch.empty(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call(**change)
    for change in (dict(ws=ws[:128]), dict(ws=ws[4:]), dict(loss=None), dict(weights=None),
                   dict(lse=None), dict(counts=None)):
        with pytest.raises(fc.FcError):
            call(**change)
    big = torch.zeros(2, 1025, device="cuda")
    with pytest.raises(fc.FcError):
        w = outputs(2, 1025, 2, 1)
        fc.fc_router_forward(big, 1, None, True, False, w["chosen"], w["weights"], w["lse"],
                             w["counts"], w["routed"], w["probs"], w["loss"],
                             torch.zeros(1 << 20, dtype=torch.uint8, device="cuda"))
    dx = torch.empty_like(x)
    call()
    back = dict(chosen=o["chosen"], weights=o["weights"], lse=o["lse"], counts=o["counts"],
                routed=o["routed"], dw=o["weights"], dl=o["loss"], dx=dx)

    def backward(**change):
        k = {**back, **change}
        fc.fc_router_backward(x, 3, True, False, k["chosen"], k["weights"], k["lse"], k["counts"],
                              k["routed"], k["dw"], k["dl"], k["dx"])
    backward()
    for change in (dict(dx=dx.half()), dict(dx=dx[:3]), dict(dw=o["weights"][:3]),
                   dict(dl=o["loss"][:1]), dict(chosen=o["chosen"].float())):
        with pytest.raises(ValueError):
            backward(**change)
    for change in (dict(lse=None), dict(counts=None), dict(routed=None), dict(weights=None)):
        with pytest.raises(fc.FcError):
            backward(**change)
    torch.cuda.synchronize()


def test_offsets_beyond_32_bits():
    """Rows further than 2^31 elements apart."""
    ld = (1 << 30) + 8
    buf = torch.zeros(3 * ld + 64, dtype=BF16, device="cuda")
    x = buf.as_strided((4, 64), (ld, 1))
    x.copy_(torch.randn(4, 64, device="cuda"))
    o = check_forward(x, 1, None, 4, True, False)
    out = torch.zeros_like(buf)
    dx = out.as_strided((4, 64), (ld, 1))
    dw, dl = torch.randn(4, 4, device="cuda"), torch.ones(2, device="cuda")
    fc.fc_router_backward(x, 1, True, False, o["chosen"], o["weights"], o["lse"], o["counts"],
                          o["routed"], dw, dl, dx)
    want, bound = ref.router_backward(x, 1, 4, True, False, o["chosen"], o["weights"], o["lse"],
                                      o["counts"], o["routed"], dw, dl)
    assert_within("dlogits", dx, want, rounded(bound, want, BF16))
