"""Group norm with an activation on a GPU against its 64-bit form."""

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import model_ops_ref as ref
from tests.ops_ref import U, assert_within, rounded

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
NONE, RELU, SILU = 0, 1, 2
ids = lambda t: str(t).replace("torch.", "")  # noqa: E731
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


def images(n, s, c, dtype, pad=0, gap=0, shift=0, seed=1, scale=1.0, mean=0.0, first=False):
    """[n, s, c], positions c + pad and samples s * (c + pad) + gap apart (or, `first`,
    positions first), `shift` elements past a boundary; and the buffer around them."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    ld, ss = c + pad, s * (c + pad) + gap
    if first:
        ss = c + pad
        ld = n * ss + gap
    buf = torch.full((shift + n * s * (c + pad) + max(n, s) * gap + 16,), 7.0, dtype=dtype,
                     device="cuda")
    m = buf.as_strided((n, s, c), (ss, ld, 1), shift)
    m.copy_(torch.randn(n, s, c, generator=g, device="cuda") * scale + mean)
    return m, buf


def untouched(m, buf):
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside.as_strided(m.shape, m.stride(), m.storage_offset()).fill_(True)
    return bool((buf[~inside] == 7.0).all())


def params(c, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(c, generator=g, device="cuda") * 0.3 + 1).to(dtype)
    return w, (torch.randn(c, generator=g, device="cuda") * 0.3).to(dtype)


def scratch(n, s, c, groups):
    return torch.full((fc.fc_groupnorm_workspace_size(n, s, c, groups),), 0xFF, dtype=torch.uint8,
                      device="cuda")


def check(n, s, c, groups, dtype, act=SILU, ptype=F32, gtype=F32, affine=True, mean=0.3,
          scale=1.0, eps=EPS, fill=None, **lay):
    x, _ = images(n, s, c, dtype, seed=1, scale=scale, mean=mean, **lay)
    if fill is not None:
        fill(x)
    y, ybuf = images(n, s, c, dtype, seed=2, **lay)
    w, b = params(c, ptype, 3) if affine else (None, None)
    mu, rs = (torch.empty(n, groups, device="cuda") for _ in range(2))
    ws = scratch(n, s, c, groups)
    fc.fc_groupnorm_forward(x, groups, w, b, eps, act, y, mu, rs, ws)
    torch.cuda.synchronize()
    (wy, wm, wr), (ey, em, er) = ref.groupnorm(x, groups, w, b, eps, act)
    assert_within("mean", mu, wm, em)
    assert_within("rstd", rs, wr, er)
    assert_within("y", y, wy, rounded(ey, wy, dtype))
    assert untouched(y, ybuf)
    # without the statistics: the same y
    y2, _ = images(n, s, c, dtype, seed=4, **lay)
    fc.fc_groupnorm_forward(x, groups, w, b, eps, act, y2, None, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)

    dy, _ = images(n, s, c, dtype, seed=5, scale=0.5, **lay)
    dx, dxbuf = images(n, s, c, dtype, seed=6, **lay)
    dw, db = (torch.full((c,), 9.0, dtype=gtype, device="cuda") for _ in range(2))
    ws.fill_(0xFF)
    fc.fc_groupnorm_backward(dy, x, groups, w, b, act, mu, rs, dx, dw, db, ws)
    torch.cuda.synchronize()
    (wdx, wdw, wdb), (edx, edw, edb) = ref.groupnorm_backward(dy, x, groups, w, b, act, mu, rs)
    assert_within("dx", dx, wdx, rounded(edx, wdx, dtype))
    assert_within("dweight", dw, wdw, rounded(edw, wdw, gtype))
    assert_within("dbias", db, wdb, rounded(edb, wdb, gtype))
    assert untouched(dx, dxbuf)
    return x, w, b, y, mu, rs, dy, dx, dw, db


# group widths that are whole vectors, parts of one, and neither; maps from one position on
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n,s,c,groups", [
    (1, 64, 256, 32), (2, 49, 96, 32), (3, 169, 384, 32), (2, 100, 320, 32), (5, 33, 64, 64),
    (2, 256, 48, 1), (2, 16, 2048, 32), (3, 7, 4096, 1), (1, 1, 512, 8), (4, 1000, 8, 2),
    (2, 300, 16, 16), (1, 2000, 128, 4), (37, 9, 40, 5), (2, 5, 1024, 1024)])
def test_aligned(n, s, c, groups, dtype):
    check(n, s, c, groups, dtype, ptype=F32 if c % 64 else dtype, gtype=dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n,s,c,groups", [
    (2, 50, 7, 7), (3, 129, 33, 3), (2, 64, 250, 10), (1, 17, 1001, 7), (2, 400, 12, 4),
    (4, 31, 6, 1), (2, 9, 514, 2), (1, 333, 129, 1), (1, 3, 2050, 5), (6, 20, 1, 1)])
def test_odd_channels(n, s, c, groups, dtype):
    check(n, s, c, groups, dtype, act=RELU, ptype=dtype, eps=1e-3)


@pytest.mark.parametrize("act", [NONE, RELU, SILU])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_activations_and_parameters(dtype, affine, act):
    check(3, 70, 96, 8, dtype, act=act, affine=affine)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("lay", [
    dict(pad=8), dict(pad=24, gap=64), dict(pad=5), dict(gap=3), dict(shift=1), dict(shift=2),
    dict(shift=8, gap=8), dict(first=True), dict(first=True, pad=8, gap=16),
    dict(first=True, pad=1, shift=3)], ids=str)
def test_strides_and_alignment(lay, dtype):
    check(3, 90, 64, 4, dtype, **lay)


# long maps: what one cluster's shared memory holds, and what it does not
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n,s,c,groups,lay", [
    (2, 4096, 320, 32, {}), (1, 20000, 64, 2, {}), (1, 65536, 32, 1, {}), (2, 16384, 128, 32, {}),
    (1, 30011, 24, 3, {}), (1, 9001, 66, 33, {}), (1, 20011, 35, 5, {}), (1, 70000, 48, 3, {}),
    (1, 5000, 96, 32, dict(shift=1)), (2, 40000, 8, 1, dict(pad=8))], ids=str)
def test_long_maps(n, s, c, groups, lay, dtype):
    check(n, s, c, groups, dtype, **lay)


# groups whose number no cut of the channels divides, so that the last slab is narrower;
# few samples of wide groups, which leave many parts to join
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n,s,c,groups,lay", [
    (40, 1352, 211, 211, dict(pad=24)), (3, 5139, 137, 137, {}), (5, 90, 83, 83, {}),
    (7, 400, 304, 19, {}), (2, 700, 176, 11, {}), (9, 333, 1112, 139, dict(pad=8)),
    (3, 129, 1982, 1, dict(pad=5)), (2, 468, 1122, 2, {}), (1, 17, 6000, 1, dict(shift=1)),
    (2, 1200, 1072, 4, {}), (2, 9001, 272, 1, {}), (4, 9001, 120, 4, {}),
    (3, 7001, 210, 35, dict(pad=1))], ids=str)
def test_uneven_slabs_and_wide_groups(n, s, c, groups, lay, dtype):
    check(n, s, c, groups, dtype, act=RELU if c % 2 else SILU, **lay)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_many_samples(dtype):
    check(700, 20, 64, 8, dtype)
    check(3000, 1, 32, 2, dtype, act=RELU)


# 16-bit rows of any alignment, several samples to a cluster, rows of threads without a
# position: what a sample's threads need of the next one has to be there when they read it
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("act", [NONE, RELU, SILU])
@pytest.mark.parametrize("n,s,c,groups,lay", [
    (700, 20, 33, 3, {}), (700, 20, 63, 7, {}), (3000, 2, 33, 3, {}), (3000, 1, 33, 3, {}),
    (5000, 3, 7, 1, {}), (700, 20, 64, 8, dict(pad=1)), (3000, 1, 32, 2, dict(shift=1, gap=3))],
    ids=str)
def test_many_samples_at_odd_places(n, s, c, groups, lay, act, dtype):
    check(n, s, c, groups, dtype, act=act, **lay)


# groups that no cluster holds, of so many samples that they are streamed in chunks
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("n,s,c,groups,lay", [
    (9000, 1, 4104, 2, {}), (20000, 2, 520, 1, dict(pad=1)), (8193, 3, 521, 1, dict(gap=3)),
    (5000, 4, 4104, 2, dict(first=True))], ids=str)
def test_samples_in_chunks(n, s, c, groups, lay, dtype):
    x, w, b, y, mu, rs, dy, dx, dw, db = check(n, s, c, groups, dtype, act=RELU if s == 2 else SILU,
                                               gtype=dtype, **lay)
    ws = scratch(n, s, c, groups)
    act = RELU if s == 2 else SILU
    for want in ((None, db), (dw, None), (None, None)):
        dx2 = torch.empty_like(dx)
        got = [None if t is None else torch.empty_like(t) for t in want]
        fc.fc_groupnorm_backward(dy, x, groups, w, b, act, mu, rs, dx2, got[0], got[1], ws)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2)
        for t, g in zip(want, got):
            assert t is None or torch.equal(t, g)


def test_chunks_captured_and_replayed():
    n, s, c, groups = 9000, 1, 4104, 2
    x, w, b, y, mu, rs, dy, dx, dw, db = check(n, s, c, groups, BF16)
    ws = scratch(n, s, c, groups)
    outs = [torch.empty_like(t) for t in (y, mu, rs, dx, dw, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_groupnorm_forward(x, groups, w, b, EPS, SILU, outs[0], outs[1], outs[2], ws)
        fc.fc_groupnorm_backward(dy, x, groups, w, b, SILU, outs[1], outs[2], outs[3], outs[4],
                                 outs[5], ws)
    for _ in range(2):
        for t in outs:
            t.fill_(5.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for t, want in zip(outs, (y, mu, rs, dx, dw, db)):
            assert torch.equal(t, want)


@pytest.mark.parametrize("gtype", TYPES, ids=ids)
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_gradient_types(dtype, gtype):
    check(4, 50, 72, 9, dtype, gtype=gtype)


def test_gradients_that_are_not_wanted():
    x, w, b, y, mu, rs, dy, dx, dw, db = check(2, 40, 64, 4, BF16)
    ws = scratch(2, 40, 64, 4)
    for want in ((None, db), (dw, None), (None, None)):
        dx2 = torch.empty_like(dx)
        got = [None if t is None else torch.empty_like(t) for t in want]
        fc.fc_groupnorm_backward(dy, x, 4, w, b, SILU, mu, rs, dx2, got[0], got[1], ws)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2)
        for t, g in zip(want, got):
            assert t is None or torch.equal(t, g)


# a mean far above the spread; a first value far from all others; values all alike
@pytest.mark.parametrize("s,c,groups", [(64, 64, 4), (4096, 64, 8), (65536, 16, 1)])
def test_hard_statistics(s, c, groups):
    check(2, s, c, groups, F32, mean=1000.0, scale=0.5, act=NONE)

    def outlier(x):
        x[:, 0, :] = 1e4
    check(2, s, c, groups, F32, act=NONE, fill=outlier)

    def alike(x):
        x.fill_(3.25)
    x, w, b, y, mu, rs, *_ = check(2, s, c, groups, F32, fill=alike)
    assert bool((mu == 3.25).all())


def test_large_values_do_not_leave_the_range():
    check(2, 50, 32, 4, F32, scale=1e15, mean=0.0, act=NONE)
    check(2, 50, 32, 4, BF16, scale=1e10, mean=0.0, act=SILU)
    check(2, 50, 32, 4, F32, scale=40.0, act=SILU, eps=1e4)


def test_nan_and_infinity_stay_in_their_group():
    for dtype in TYPES:
        x, _ = images(2, 30, 32, dtype)
        x[0, 3, 5] = float("nan")
        x[1, 7, 30] = float("inf")
        y = torch.empty_like(x)
        mu, rs = (torch.empty(2, 4, device="cuda") for _ in range(2))
        fc.fc_groupnorm_forward(x, 4, None, None, EPS, RELU, y, mu, rs, scratch(2, 30, 32, 4))
        bad = ~torch.isfinite(y.float())
        assert bool(bad[0, :, :8].all()) and not bool(bad[0, :, 8:].any())
        assert bool(bad[1, :, 24:].any()) and not bool(bad[1, :, :24].any())
        assert torch.isnan(mu[0, 0]) and bool(torch.isfinite(mu[0, 1:]).all())


def test_reads_nothing_outside_the_images():
    for lay in (dict(pad=3, gap=5, shift=1), dict(pad=8, gap=16), dict(first=True, pad=8)):
        for dtype in (F32, BF16):
            x, buf = images(3, 40, 24, dtype, **lay)
            keep = x.clone()
            buf.fill_(float("nan"))
            x.copy_(keep)
            y = torch.empty(3, 40, 24, dtype=dtype, device="cuda")
            mu, rs = (torch.empty(3, 3, device="cuda") for _ in range(2))
            ws = scratch(3, 40, 24, 3)
            fc.fc_groupnorm_forward(x, 3, None, None, EPS, SILU, y, mu, rs, ws)
            dx = torch.empty_like(y)
            dw, db = (torch.empty(24, device="cuda") for _ in range(2))
            fc.fc_groupnorm_backward(x, x, 3, None, None, SILU, mu, rs, dx, dw, db, ws)
            for t in (y, mu, rs, dx, dw, db):
                assert bool(torch.isfinite(t.float()).all())


def test_relu_side_is_exact():
    """Values at the border: z = 0 up to fp32's rounding."""
    g = torch.Generator(device="cuda").manual_seed(7)
    n, s, c, groups = 2, 512, 64, 4
    x, _ = images(n, s, c, F32, seed=8)
    mu = torch.randn(n, groups, generator=g, device="cuda")
    rs = torch.rand(n, groups, generator=g, device="cuda") + 0.5
    w, b = params(c, F32, 9)
    # x with (x - mean) rstd w = -b as nearly as fp32 holds it
    m, r = (t.double().repeat_interleave(c // groups, 1)[:, None, :] for t in (mu, rs))
    x.copy_((m - b.double() / (r * w.double())).float().expand(n, s, c))
    x.view(torch.int32).add_(torch.randint(-2, 3, (n, s, c), generator=g, device="cuda",
                                           dtype=torch.int32))
    dy = torch.randn(n, s, c, generator=g, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    fc.fc_groupnorm_backward(dy, x, groups, w, b, RELU, mu, rs, dx, dw, db,
                             scratch(n, s, c, groups))
    (wdx, wdw, wdb), (edx, edw, edb) = ref.groupnorm_backward(dy, x, groups, w, b, RELU, mu, rs)
    assert_within("dbias", db, wdb, rounded(edb, wdb, F32))
    assert_within("dweight", dw, wdw, rounded(edw, wdw, F32))
    assert_within("dx", dx, wdx, rounded(edx, wdx, F32))


@pytest.mark.parametrize("size", [2.0 ** -90, 2.0 ** -60, 2.0 ** 40])
def test_relu_side_is_exact_at_any_size(size):
    """The border again, with parameters far from 1."""
    g = torch.Generator(device="cuda").manual_seed(8)
    n, s, c, groups = 2, 256, 64, 4
    mu = torch.randn(n, groups, generator=g, device="cuda")
    rs = torch.rand(n, groups, generator=g, device="cuda") + 0.5
    w, b = (t * size for t in params(c, F32, 9))
    m, r = (t.double().repeat_interleave(c // groups, 1)[:, None, :] for t in (mu, rs))
    x = (m - b.double() / (r * w.double())).float().expand(n, s, c).contiguous()
    x.view(torch.int32).add_(torch.randint(-2, 3, (n, s, c), generator=g, device="cuda",
                                           dtype=torch.int32))
    dy = torch.randn(n, s, c, generator=g, device="cuda")
    dx, dw, db = torch.empty_like(x), torch.empty(c, device="cuda"), torch.empty(c, device="cuda")
    fc.fc_groupnorm_backward(dy, x, groups, w, b, RELU, mu, rs, dx, dw, db,
                             scratch(n, s, c, groups))
    (wdx, wdw, wdb), (edx, edw, edb) = ref.groupnorm_backward(dy, x, groups, w, b, RELU, mu, rs)
    assert_within("dbias", db, wdb, rounded(edb, wdb, F32))
    assert_within("dweight", dw, wdw, rounded(edw, wdw, F32))
    assert_within("dx", dx, wdx, rounded(edx, wdx, F32))


@pytest.mark.parametrize("scale", [2.0 ** -58, 2.0 ** -40])
@pytest.mark.parametrize("s,c,groups", [(50, 32, 4), (9001, 272, 1)])
def test_spreads_far_below_one(s, c, groups, scale):
    check(2, s, c, groups, F32, act=NONE, mean=0.0, scale=scale, eps=0.0)


def test_same_bits_again_and_on_another_stream():
    a = check(5, 300, 96, 32, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = check(5, 300, 96, 32, BF16)
    side.synchronize()
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    # a stream given by hand
    x, w, bias, y, mu, rs = a[:6]
    y2 = torch.empty_like(y)
    ws = scratch(5, 300, 96, 32)
    torch.cuda.synchronize()
    fc.fc_groupnorm_forward(x, 32, w, bias, EPS, SILU, y2, mu, rs, ws, side)
    side.synchronize()
    assert torch.equal(y, y2)


@pytest.mark.parametrize("n,s,c,groups", [(2, 64, 64, 8), (2, 20000, 64, 1), (3, 50, 33, 3)])
def test_captured_and_replayed(n, s, c, groups):
    x, w, b, y, mu, rs, dy, dx, dw, db = check(n, s, c, groups, BF16)
    ws = scratch(n, s, c, groups)
    outs = [torch.empty_like(t) for t in (y, mu, rs, dx, dw, db)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_groupnorm_forward(x, groups, w, b, EPS, SILU, outs[0], outs[1], outs[2], ws)
        fc.fc_groupnorm_backward(dy, x, groups, w, b, SILU, outs[1], outs[2], outs[3], outs[4],
                                 outs[5], ws)
    for _ in range(3):
        for t in outs:
            t.fill_(5.0)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        for t, want in zip(outs, (y, mu, rs, dx, dw, db)):
            assert torch.equal(t, want)
    # new inputs in the same places
    x.mul_(0.5)
    graph.replay()
    (wy, _, _), (ey, _, _) = ref.groupnorm(x, groups, w, b, EPS, SILU)
    torch.cuda.synchronize()
    assert_within("y", outs[0], wy, rounded(ey, wy, BF16))


def test_no_samples_and_refusals():
    x = torch.empty(0, 5, 8, device="cuda")
    ws = scratch(0, 5, 8, 2)
    mu = torch.empty(0, 2, device="cuda")
    fc.fc_groupnorm_forward(x, 2, None, None, EPS, NONE, x, mu, mu, ws)
    dw, db = torch.full((8,), 3.0, device="cuda"), torch.full((8,), 3.0, device="cuda")
    fc.fc_groupnorm_backward(x, x, 2, None, None, NONE, mu, mu, x, dw, db, ws)
    assert bool((dw == 0).all()) and bool((db == 0).all())

    x = torch.zeros(2, 5, 8, device="cuda")
    y, w = torch.empty_like(x), torch.ones(8, device="cuda")
    mu, rs = torch.empty(2, 2, device="cuda"), torch.empty(2, 2, device="cuda")
    ws = scratch(2, 5, 8, 2)
    good = dict(x=x, groups=2, w=w, b=w, eps=EPS, act=NONE, y=y, mu=mu, rs=rs, ws=ws)

    def call(**change):
        k = {**good, **change}
        fc.fc_groupnorm_forward(k["x"], k["groups"], k["w"], k["b"], k["eps"], k["act"], k["y"],
                                k["mu"], k["rs"], k["ws"])
    call()
    for change in (dict(x=x[0]), dict(x=x.transpose(1, 2)), dict(x=x.cpu()), dict(x=x.double()),
                   dict(y=y.half()), dict(y=y[:1]), dict(y=y.transpose(1, 2)), dict(groups=0),
                   dict(groups=-1), dict(w=w.half()), dict(w=w[:7]), dict(b=w.cpu()),
                   dict(mu=mu[:1]), dict(ws=None), dict(ws=ws.cpu()), dict(ws=ws[::2]),
                   dict(mu=mu.double())):
        with pytest.raises(ValueError):
            call(**change)
    for change in (dict(groups=3), dict(groups=16), dict(act=3), dict(act=-1), dict(eps=-1.0),
                   dict(eps=float("nan")), dict(mu=None), dict(ws=ws[:256]), dict(ws=ws[1:]),
                   dict(x=x[:, :1].expand(2, 5, 8)), dict(x=x[:1].expand(2, 5, 8))):
        with pytest.raises((fc.FcError, ValueError)):
            call(**change)
    torch.cuda.synchronize()
    bf = torch.zeros(2, 5, 8, device="cuda", dtype=BF16)
    with pytest.raises(ValueError):
        fc.fc_groupnorm_forward(bf, 2, w, w.to(BF16), EPS, NONE, torch.empty_like(bf), mu, rs, ws)


def test_channels_last_view():
    t = torch.randn(2, 48, 9, 11, device="cuda").to(memory_format=torch.channels_last)
    x = t.permute(0, 2, 3, 1).flatten(1, 2)
    assert x.data_ptr() == t.data_ptr()
    out = torch.empty_like(t)
    y = out.permute(0, 2, 3, 1).flatten(1, 2)
    fc.fc_groupnorm_forward(x, 6, None, None, EPS, SILU, y, None, None, scratch(2, 99, 48, 6))
    want = torch.nn.functional.silu(torch.nn.functional.group_norm(t.double(), 6, eps=EPS))
    assert float((out - want).abs().max()) < 1e-5  # 5 roundings and more of values up to 6


def test_offsets_beyond_32_bits():
    """Two samples more than 2^31 elements apart, and positions too."""
    far = (1 << 31) + 64
    for strides in ((far, 32, 1), (32, far // 63, 1)):
        n, s, c = 2, 64, 32
        buf = torch.zeros(far + 64 * 64 + far // 63, dtype=BF16, device="cuda")
        out = torch.zeros_like(buf)
        x, y = buf.as_strided((n, s, c), strides), out.as_strided((n, s, c), strides)
        if strides[1] % 8:
            pass  # rows of any alignment
        x.copy_(torch.randn(n, s, c, device="cuda"))
        mu, rs = (torch.empty(n, 4, device="cuda") for _ in range(2))
        ws = scratch(n, s, c, 4)
        fc.fc_groupnorm_forward(x, 4, None, None, EPS, SILU, y, mu, rs, ws)
        (wy, _, _), (ey, _, _) = ref.groupnorm(x, 4, None, None, EPS, SILU)
        assert_within("y", y, wy, rounded(ey, wy, BF16))
        dw, db = (torch.empty(c, device="cuda") for _ in range(2))
        fc.fc_groupnorm_backward(x, x, 4, None, None, SILU, mu, rs, y, dw, db, ws)
        (wdx, wdw, _), (edx, edw, _) = ref.groupnorm_backward(x, x, 4, None, None, SILU, mu, rs)
        assert_within("dx", y, wdx, rounded(edx, wdx, BF16))
        assert_within("dweight", dw, wdw, rounded(edw, wdw, F32))
        del buf, out, x, y
        torch.cuda.empty_cache()
    assert U == 2.0 ** -24
