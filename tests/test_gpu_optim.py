"""Gradient norm and AdamW on a GPU against their 64-bit forms."""

import math

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import ops_ref
from tests.ops_ref import U, assert_within

pytestmark = pytest.mark.gpu

F32, F16, BF16, E4M3 = torch.float32, torch.float16, torch.bfloat16, torch.float8_e4m3fn
TYPES = [F32, F16, BF16]
ids = lambda t: str(t).replace("torch.", "")  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


def rnd(n, seed, scale=1.0, dtype=F32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, generator=g, device="cuda") * scale).to(dtype)


def layers(sizes, dtype, shift=0, seed=1, scale=1e-3):
    """Separate tensors, each `shift` elements past a 256-byte boundary."""
    out = []
    for l, n in enumerate(sizes):
        out.append(rnd(n + shift, 1000 * seed + l, scale, dtype)[shift:])
    return out


# sizes: one element; below, at and past a unit of 256; layer boundaries inside a
# unit; empty layers; many tiny layers (more than the small table holds)
SIZES = [[1], [3], [255], [256], [257], [1728, 131072, 256], [1, 255, 256, 1, 4095, 0, 2, 70001],
         [0, 5, 0, 0, 700], [7] * 100 + [1000] + [1] * 60, [300003], [513, 511] * 40]


def norm_of(grads, loss_scale=1.0, max_norm=0.0, stream=None):
    ws = torch.zeros(fc.fc_grad_norm_workspace_size(), dtype=torch.uint8, device="cuda")
    norm, scale = torch.full((1,), -1.0, device="cuda"), torch.full((1,), -1.0, device="cuda")
    fc.fc_grad_norm(fc.LayerGrads(grads), loss_scale, max_norm, norm, scale, ws, stream)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) == 0  # the counter is back at zero
    return float(norm), float(scale)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shift", [0, 1, 3, 7])
@pytest.mark.parametrize("k", range(len(SIZES)))
def test_norm(k, shift, dtype):
    grads = layers(SIZES[k], dtype, shift, seed=k + 1)
    want, factor = ops_ref.grad_norm(grads, 128.0, 1e-4)
    got, scale = norm_of(grads, 128.0, 1e-4)
    # a square, at most 11 roundings of sums, halved by the root; root, division
    assert abs(got - want) <= 8 * U * want
    assert abs(scale - factor) <= 12 * U * factor


def test_norm_clips_only_above_the_limit_and_survives_zero():
    g = [torch.full((100,), 0.1, device="cuda")]  # norm 1
    assert norm_of(g, 1.0, 2.0)[1] == 1.0
    assert abs(norm_of(g, 1.0, 0.5)[1] - 0.5) < 1e-6
    assert norm_of(g, 4.0, 0.0)[1] == 0.25
    assert norm_of([torch.zeros(1000, device="cuda")], 1.0, 1.0) == (0.0, 1.0)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_norm_of_what_is_not_finite(bad, dtype):
    grads = layers([700, 70001, 3], dtype)
    grads[1][69999] = bad
    norm, scale = norm_of(grads, 2.0, 1.0)
    assert (math.isnan(norm) if math.isnan(bad) else norm == math.inf) and math.isnan(scale)


def test_norm_does_not_read_past_a_layer():
    """Poison right before and behind every layer, at every shift."""
    for shift in range(1, 9):
        buf = torch.full((5000,), math.nan, device="cuda", dtype=F16)
        g = buf[shift:shift + 4001]
        g.copy_(rnd(4001, shift))
        want, _ = ops_ref.grad_norm([g], 1.0, 0.0)
        assert abs(norm_of([g])[0] - want) <= 8 * U * want


def test_norm_repeats_bit_for_bit():
    grads = layers([1 << 20, 12345, 7], BF16)
    assert len({norm_of(grads, 1.0, 0.1) for _ in range(4)}) == 1


# ---- AdamW -------------------------------------------------------------------------

HYPER = dict(lr=1e-2, b1=0.9, b2=0.999, eps=1e-8, wd=0.1)


def decay_of(sizes):
    return [(0.0, 1.0, 0.5)[l % 3] for l in range(len(sizes))]


class State:
    """Weights and moments of one run, each inside a larger buffer whose ends
    must not change."""
    GUARD = 64

    def __init__(self, n, bits, low, done=0, seed=5, fresh=False):
        self.n, self.bits = n, bits
        self.guards = []
        self.w = self.room(rnd(n, seed, 0.05))
        self.low = None if low is None else self.room(torch.zeros(n, dtype=low, device="cuda"))
        m = rnd(n, seed + 1, 0.0 if fresh else 3e-4)
        r = rnd(n, seed + 2, 0.0 if fresh else 1e-3).abs()
        self.steps = torch.tensor([done, 0], dtype=torch.int32, device="cuda")
        if bits == 32:
            self.m, self.v = self.room(m), self.room(r * r)
            return
        self.m8, self.ms = self.quantised(m)
        self.r8, self.rs = self.quantised(r)

    def quantised(self, x):
        s = ops_ref.block_top(x) / 448
        full = ops_ref.spread(s, self.n)
        y = torch.where(full > 0, x / torch.where(full > 0, full, 1.0), 0.0).clamp(-448, 448)
        return self.room(y.to(E4M3)), self.room(s)

    def room(self, t):
        b = t.element_size()
        buf = torch.full((2 * self.GUARD + t.numel() * b,), 0xA5, dtype=torch.uint8, device="cuda")
        view = buf[self.GUARD:self.GUARD + t.numel() * b].view(t.dtype)
        view.copy_(t)
        self.guards.append(buf)
        return view

    def check_guards(self):
        for buf in self.guards:
            assert bool((buf[:self.GUARD] == 0xA5).all() and (buf[-self.GUARD:] == 0xA5).all())

    def moments(self):
        """(m, v) in float64."""
        if self.bits == 32:
            return self.m.double(), self.v.double()
        return (self.m8.double() * ops_ref.spread(self.ms.double(), self.n),
                (self.r8.double() * ops_ref.spread(self.rs.double(), self.n)) ** 2)

    def copies(self):
        names = ["w", "steps"] + (["m", "v"] if self.bits == 32 else ["m8", "ms", "r8", "rs"])
        return {k: getattr(self, k).clone() for k in names}

    def step(self, table, scale, h=HYPER, seed=11, stream=None):
        head = (table, scale, h["lr"], h["b1"], h["b2"], h["eps"], h["wd"], self.w, self.low)
        if self.bits == 32:
            fc.fc_adamw_step(*head, self.m, self.v, self.steps, stream)
        else:
            fc.fc_adamw8_step(*head, self.m8, self.ms, self.r8, self.rs, self.steps, seed, stream)


def check_step(grads, sizes, bits, low, done, h=HYPER, scale=0.37, fresh=False, seed=11):
    n = sum(sizes)
    st = State(n, bits, low, done, fresh=fresh)
    m0, v0 = st.moments()
    w0 = st.w.clone()
    decay = decay_of(sizes)
    s = None if scale is None else torch.tensor([scale], device="cuda")
    st.step(fc.LayerGrads(grads, decay), s, h, seed)
    torch.cuda.synchronize()
    st.check_guards()
    t = done + 1
    assert st.steps.tolist() == [t, 0]
    d = torch.repeat_interleave(torch.tensor(decay, device="cuda"),
                                torch.tensor(sizes, device="cuda"))
    f = 1.0 if scale is None else float(s)
    g = torch.cat([x.double() for x in grads]) * f
    (w, m, v), (ew, em, ev) = ops_ref.adamw(w0, m0, v0, g, d, t, **h)
    if bits == 8:
        # the moments read are products code * scale, rounded once more
        em, ev = em + U * m0.abs(), ev + 3 * U * v0
        ew = ew + (h["lr"] / (1 - h["b1"] ** t)) * U * m0.abs() / (
            torch.sqrt(v / (1 - h["b2"] ** t)) + h["eps"]) + 0.1 * ew
    assert_within("w", st.w, w, ew)
    if low is not None:
        assert torch.equal(st.low, st.w.to(low))
    if bits == 32:
        assert_within("m", st.m, m, em)
        assert_within("v", st.v, v, ev)
        return st
    check_codes(st.m8, st.ms, m, em, None)
    i = torch.arange(n, device="cuda")
    r = torch.sqrt(v)
    check_codes(st.r8, st.rs, r, 0.5 * ev / torch.where(r > 0, r, 1.0) + 2 * U * r,
                (ops_ref.random16(seed, t, i).double() + 0.5) / 65536)
    return st


def check_codes(codes, scales, x, ex, chance):
    """e4m3 codes and block scales of x, known to ex; chance None: nearest."""
    top = ops_ref.block_top(x)
    etop = ops_ref.block_top(ex)
    assert_within("scale", scales, top / 448, etop / 448 + 2 * U * top / 448)
    full = ops_ref.spread(top, x.numel())
    live = full > 0
    y = torch.where(live, x.abs() / torch.where(live, full, 1.0) * 448, 0.0)
    ey = torch.where(live, (ex + ops_ref.spread(etop, x.numel()) * y / 448)
                     / torch.where(live, full, 1.0) * 448, 0.0) + 4 * U * y
    got = codes.double()
    q = ops_ref.e4m3_quantum(y)
    if chance is None:
        assert bool(((got * x) >= 0).all())
        assert_within("codes", got.abs(), y, q / 2 + ey)
        return
    want = torch.where(y > 0, torch.clamp(torch.floor(y / q + chance) * q, min=2.0 ** -9), 0.0)
    # where the draw lies within the error of the threshold either neighbour is right
    near = ((y / q + chance) - torch.round(y / q + chance)).abs() <= ey / q + 2.0 ** -20
    assert bool((got[~near] == want[~near]).all())
    assert_within("codes", got, y, q * 1.001 + ey)
    assert float(near.double().mean()) < 0.01 or x.numel() < 1000


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("k", range(len(SIZES)))
def test_adamw_sizes(k, dtype, bits):
    sizes = SIZES[k]
    check_step(layers(sizes, dtype, seed=k + 1), sizes, bits, (None, F16, BF16)[k % 3], done=k)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shift", range(1, 8))
def test_adamw_shifted_layers(shift, dtype, bits):
    sizes = [5000, 1001, 3, 2048, 7777]
    check_step(layers(sizes, dtype, shift), sizes, bits, BF16, done=3)


# vectors long enough for the streamed kernel: whole tiles only; a ragged end; layer
# boundaries inside units, inside tiles and in the last units; many layers
LONG = [[1 << 20], [(1 << 20) + 1], [1 << 20, 3000, 77], [700001, 13, 500000, 255, 4099],
        [(1 << 21) + 2048 * 3 + 255], [9001] * 200, [1] * 300 + [1500000] + [3] * 300]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("k", range(len(LONG)))
def test_adamw_long(k, dtype, bits):
    check_step(layers(LONG[k], dtype, shift=k % 4, seed=k + 1), LONG[k], bits,
               (F16, None, BF16)[k % 3], done=k)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("low", [None, F16])
def test_adamw_long_skip(bits, low):
    sizes = [700001, 13, 500000, 255, 4099]
    grads = layers(sizes, F16)
    grads[0][5] = math.inf
    st = State(sum(sizes), bits, low, done=4)
    before = st.copies()
    st.step(fc.LayerGrads(grads), torch.tensor([math.nan], device="cuda"))
    torch.cuda.synchronize()
    after = st.copies()
    for k in before:
        assert torch.equal(before[k].view(torch.uint8), after[k].view(torch.uint8)), k
    assert low is None or torch.equal(st.low, st.w.to(low))
    st.check_guards()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_adamw_reads_no_gradient_outside_a_layer(dtype, bits):
    """NaN around every layer: none of it may reach the weights."""
    sizes = [1001, 256, 259, 4097]
    for shift in (1, 2, 3):
        grads = []
        for l, n in enumerate(sizes):
            buf = torch.full((n + 32,), math.nan, dtype=dtype, device="cuda")
            grads.append(buf[8 + shift:8 + shift + n])
            grads[-1].copy_(rnd(n, l, 1e-3))
        check_step(grads, sizes, bits, F16, done=1)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("done", [0, 1, 9, 999, 1000000])
@pytest.mark.parametrize("h", [HYPER, dict(lr=0.0, b1=0.9, b2=0.95, eps=1e-8, wd=0.1),
                               dict(lr=1e-3, b1=0.0, b2=0.0, eps=1e-6, wd=0.0),
                               dict(lr=1e-3, b1=0.99, b2=0.9999, eps=1e-12, wd=1.0)])
def test_adamw_counts_and_factors(h, done, bits):
    sizes = [3000, 1111]
    check_step(layers(sizes, F32), sizes, bits, None, done, h, scale=None)


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_from_the_start(bits):
    """All-zero moments; a layer whose gradient is zero keeps zero moments."""
    sizes = [2000, 512, 1000]
    grads = layers(sizes, F32)
    grads[1].zero_()
    st = check_step(grads, sizes, bits, None, 0, fresh=True)
    m, v = st.moments()
    assert bool((m[2000:2512] == 0).all()) and bool((v[2000:2512] == 0).all())


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_adamw_skips_an_overflowed_step(bad, bits):
    sizes = [1728, 70001, 256, 3]
    grads = layers(sizes, F16, 1)
    grads[1][5] = math.inf
    st = State(sum(sizes), bits, BF16, done=4)
    before = st.copies()
    st.step(fc.LayerGrads(grads), torch.tensor([bad], device="cuda"))
    torch.cuda.synchronize()
    after = st.copies()
    for k in before:
        assert torch.equal(before[k].view(torch.uint8), after[k].view(torch.uint8)), k
    assert torch.equal(st.low, st.w.to(BF16))
    st.check_guards()


def test_adamw8_holds_extreme_blocks():
    """Blocks of tiny, huge, zero and mixed gradients, and a block below 2^-110."""
    n = 256 * 6 + 77
    g = rnd(n, 3)
    g[:256] *= 1e-15
    g[256:512] *= 1e12
    g[512:768] = 0
    g[768:1024] *= torch.logspace(-12, 0, 256, device="cuda")
    g[1024:1280] *= 1e-18
    h = dict(HYPER, eps=1e-20)
    st = check_step([g], [n], 8, None, 0, h, scale=None, fresh=True)
    m, v = st.moments()
    assert bool((v[512:768] == 0).all()) and bool((v[:512] > 0).all())
    tiny = State(256, 8, None, fresh=True)
    tiny.step(fc.LayerGrads([torch.full((256,), 1e-34, device="cuda")]), None)
    torch.cuda.synchronize()
    assert float(tiny.ms) == 0.0 and bool((tiny.m8.float() == 0).all())


def test_adamw8_second_moment_follows_its_average():
    """Rounding by chance keeps v on its exact course over hundreds of steps,
    where rounding to nearest would not move it at all."""
    n, steps = 256 * 64, 400
    st = State(n, 8, None, fresh=True)
    h = dict(HYPER, lr=1e-3, wd=0.0)
    big, small = rnd(n, 1).sign() * 1e-2, rnd(n, 2).sign() * 1e-3
    st.step(fc.LayerGrads([big]), None, dict(h, b2=0.0), seed=3)   # v = 1e-4
    v0 = st.moments()[1].mean()
    table = fc.LayerGrads([small])
    for k in range(steps):
        st.step(table, None, h, seed=3)
    torch.cuda.synchronize()
    want = float(v0) * 0.999 ** steps + 1e-6 * (1 - 0.999 ** steps)
    got = float(st.moments()[1].mean())
    # each step leaves a value up to 1/8 apart from the exact one, by chance:
    # per element a spread of about (1/16) sqrt(steps) of its course at most,
    # averaged over 16384 elements, and the square's own bias of (1/16)^2
    assert abs(got / want - 1) < 0.02


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_many_steps_and_determinism(bits):
    sizes = [1001, 40000, 255, 3]
    runs = []
    for _ in range(2):
        st = State(sum(sizes), bits, F16, seed=9, fresh=True)
        for k in range(6):
            st.step(fc.LayerGrads(layers(sizes, BF16, seed=20 + k), decay_of(sizes)),
                    torch.tensor([0.5], device="cuda"), seed=99)
        torch.cuda.synchronize()
        assert st.steps.tolist() == [6, 0]
        runs.append(st.copies())
    for k in runs[0]:
        assert torch.equal(runs[0][k].view(torch.uint8), runs[1][k].view(torch.uint8)), k


@pytest.mark.parametrize("bits", [32, 8])
def test_norm_and_adamw_in_a_cuda_graph_and_on_another_stream(bits):
    """The pair captured once and replayed counts and moves as eager calls do."""
    sizes = [5000, 333, 64]
    grads = layers(sizes, F16, 1, scale=1.0)
    table = fc.LayerGrads(grads, decay_of(sizes))
    ws = torch.zeros(fc.fc_grad_norm_workspace_size(), dtype=torch.uint8, device="cuda")
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")

    def both(st, stream=None):
        fc.fc_grad_norm(table, 8.0, 1.0, norm, scale, ws, stream)
        st.step(table, scale, stream=stream)

    eager = State(sum(sizes), bits, F16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        both(eager, side)
    side.synchronize()
    st = State(sum(sizes), bits, F16)
    both(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(st)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    a, b = eager.copies(), st.copies()
    for k in a:
        assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k
    assert st.steps.tolist() == [4, 0]


def test_binding_checks():
    g = fc.LayerGrads([torch.zeros(300, device="cuda")])
    st = State(300, 32, None)
    with pytest.raises(ValueError):
        fc.LayerGrads([torch.zeros(4, device="cuda"), torch.zeros(4, device="cuda", dtype=F16)])
    with pytest.raises(ValueError):
        fc.LayerGrads([torch.zeros(4, 6, device="cuda")[:, ::2]])
    with pytest.raises(ValueError):
        fc.LayerGrads([torch.zeros(4, device="cuda")], decay=[1.0, 0.0])
    with pytest.raises(ValueError):
        fc.fc_adamw_step(g, None, 1e-3, .9, .99, 1e-8, 0, st.w[:299], None, st.m, st.v, st.steps)
    with pytest.raises(ValueError):
        fc.fc_adamw_step(g, None, 1e-3, .9, .99, 1e-8, 0, st.w, st.w, st.m, st.v, st.steps)
    with pytest.raises(ValueError):
        fc.fc_adamw_step(g, None, 1e-3, .9, .99, 1e-8, 0, st.w, None, st.m.cpu(), st.v, st.steps)
    with pytest.raises(ValueError):
        fc.fc_adamw8_step(g, None, 1e-3, .9, .99, 1e-8, 0, st.w, None, st.m, st.w, st.v, st.w,
                          st.steps, 1)
    with pytest.raises(fc.FcError) as e:
        fc.fc_adamw_step(g, None, -1.0, .9, .99, 1e-8, 0, st.w, None, st.m, st.v, st.steps)
    assert e.value.status == fc.FC_ERR_INVALID_ARG and "lr" in str(e.value)
