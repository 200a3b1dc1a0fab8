"""Layer norm on a GPU against its 64-bit form."""

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import ops_ref
from tests.ops_ref import assert_within, rounded

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
ids = lambda t: str(t).replace("torch.", "")  # noqa: E731
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


def matrix(rows, cols, dtype, pad=0, shift=0, seed=1, scale=1.0, mean=0.0):
    """[rows, cols] whose rows are cols + pad apart, `shift` elements past a
    boundary, and the buffer around it (filled with a pattern)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    buf = torch.full((shift + rows * (cols + pad) + 16,), 7.0, dtype=dtype, device="cuda")
    m = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    m.copy_(torch.randn(rows, cols, generator=g, device="cuda") * scale + mean)
    return m, buf


def untouched(m, buf, pad, shift):
    rows, cols = m.shape
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = True
    return bool((buf[~inside] == 7.0).all())


def params(cols, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(cols, generator=g, device="cuda") * 0.3 + 1).to(dtype)
    return w, (torch.randn(cols, generator=g, device="cuda") * 0.3).to(dtype)


def check(rows, cols, dtype, pad=0, shift=0, ptype=F32, gtype=F32, affine=True, mean=0.3,
          scale=1.0, eps=EPS, pshift=0):
    x, _ = matrix(rows, cols, dtype, pad, shift, 1, scale, mean)
    y, ybuf = matrix(rows, cols, dtype, pad, shift, 2)
    w = b = None
    if affine:
        w, b = (torch.cat((p.new_zeros(pshift), p))[pshift:] for p in params(cols, ptype, 3))
    mu, rs = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    fc.fc_layernorm_forward(x, w, b, eps, y, mu, rs)
    torch.cuda.synchronize()
    (wy, wm, wr), (ey, em, er) = ops_ref.layernorm(x, w, b, eps)
    assert_within("mean", mu, wm, em + ops_ref.U * wm.abs())
    assert_within("rstd", rs, wr, er)
    assert_within("y", y, wy, rounded(ey, wy, dtype))
    assert untouched(y, ybuf, pad, shift)
    # inference: the same y without the statistics
    y2, _ = matrix(rows, cols, dtype, pad, shift, 4)
    fc.fc_layernorm_forward(x, w, b, eps, y2)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)

    dy, _ = matrix(rows, cols, dtype, pad, shift, 5, 0.5)
    dx, dxbuf = matrix(rows, cols, dtype, pad, shift, 6)
    dw, db = (torch.full((cols,), 9.0, dtype=gtype, device="cuda") for _ in range(2))
    ws = torch.full((fc.fc_layernorm_backward_workspace_size(rows, cols),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx, dw, db, ws)
    torch.cuda.synchronize()
    (wdx, wdw, wdb), (edx, edw, edb) = ops_ref.layernorm_backward(dy, x, w, mu, rs)
    assert_within("dx", dx, wdx, rounded(edx, wdx, dtype))
    assert_within("dweight", dw, wdw, rounded(edw, wdw, gtype))
    assert_within("dbias", db, wdb, rounded(edb, wdb, gtype))
    assert untouched(dx, dxbuf, pad, shift)
    return x, w, b, y, mu, rs, dy, dx, dw, db, ws


# every width class of the aligned kernels, both sides of each border, and what
# is wider than the registers hold
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [8, 64, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 2048, 2056,
                                  4096, 4104, 8192, 8200, 16384, 16392, 40000])
def test_aligned_widths(cols, dtype):
    check(37, cols, dtype, ptype=F32 if cols % 16 else dtype)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [1, 2, 3, 31, 33, 127, 129, 255, 257, 511, 513, 1001, 1023, 1025,
                                  2047, 2049, 4095, 4097, 8191, 8193, 16383, 16385, 33333])
def test_odd_widths(cols, dtype):
    check(23, cols, dtype, ptype=dtype if cols % 3 else F32, eps=1e-3)


# enough rows for the kernels that take many, at both sides of every width class, aligned
# and with rows that start anywhere
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols", [136, 256, 260, 384, 512, 520, 768, 776, 1024, 1032, 1536, 1544,
                                  2048, 2056, 3080, 4096, 4104, 6152, 8192, 8200, 12296, 16384])
def test_many_rows_aligned(cols, dtype):
    check(300000 // cols + 3, cols, dtype, ptype=dtype if cols % 3 else F32)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("cols,pad,shift", [
    (129, 0, 0), (130, 1, 3), (255, 0, 1), (257, 0, 0), (333, 2, 5), (511, 0, 7), (513, 0, 0),
    (770, 0, 0), (1001, 0, 0), (1001, 7, 0), (1025, 0, 2), (1537, 0, 0), (2049, 3, 1), (3073, 0, 0),
    (4097, 0, 0), (6145, 0, 4), (8191, 0, 0), (8193, 0, 0), (12289, 0, 6), (16381, 1, 0),
    (1000, 5, 0), (1024, 0, 1), (512, 3, 2)])
def test_many_rows_anywhere(cols, pad, shift, dtype):
    check(300000 // cols + 3, cols, dtype, pad, shift, ptype=F32 if cols % 3 else dtype,
          pshift=shift % 2)


def test_shifted_rows_read_nothing_outside_the_matrix():
    """NaN before, between and behind the rows reaches no output."""
    for dtype in TYPES:
        for cols, pad, shift, rows in ((1001, 3, 1, 400), (515, 6, 3, 700), (133, 0, 5, 9)):
            def poisoned(seed):
                buf = torch.full((shift + rows * (cols + pad) + 16,), float("nan"), dtype=dtype,
                                 device="cuda")
                m = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
                m.copy_(matrix(rows, cols, dtype, seed=seed)[0])
                return m
            x, dy = poisoned(1), poisoned(2)
            w, b = params(cols, F32, 3)
            y, dx = torch.empty_like(x.contiguous()), torch.empty_like(x.contiguous())
            mu, rs = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
            dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            ws = torch.empty(fc.fc_layernorm_backward_workspace_size(rows, cols),
                             dtype=torch.uint8, device="cuda")
            fc.fc_layernorm_forward(x, w, b, EPS, y, mu, rs)
            fc.fc_layernorm_backward(dy, x, w, mu, rs, dx, dw, db, ws)
            torch.cuda.synchronize()
            for t in (y, mu, rs, dx, dw, db):
                assert bool(t.isfinite().all())


# the backward pass's rows in halves: fewer rows than pairs of blocks, and several rounds
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols,pad", [(1, 12296, 0), (2, 16384, 0), (75, 12304, 0),
                                           (77, 16376, 8), (301, 12290, 0), (301, 16384, 0),
                                           (160, 8196, 0), (3, 12289, 0), (161, 16383, 1)])
def test_rows_in_halves(rows, cols, pad, dtype):
    x, w, b, y, mu, rs, dy, dx, dw, db, ws = check(rows, cols, dtype, pad)
    dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx2, dw2, db2, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


# few wide rows, and the last number of rows that counts as few
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,cols,pad", [(1, 16384, 0), (3, 12296, 0), (64, 16376, 0),
                                           (1, 5001, 0), (2, 8191, 0), (1, 16383, 0),
                                           (152, 9001, 0), (153, 9001, 0), (152, 12287, 2),
                                           (5, 16384, 3)])
def test_few_wide_rows(rows, cols, pad, dtype):
    check(rows, cols, dtype, pad, ptype=dtype)


# few narrow rows, whose sums are joined in the same launch, up to where that ends
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 9, 33, 64, 127, 128, 129])
@pytest.mark.parametrize("cols", [5, 40, 64, 100, 128, 130, 200, 256, 512])
def test_few_rows(rows, cols, dtype):
    check(rows, cols, dtype, gtype=dtype)


@pytest.mark.parametrize("rows", [1, 2, 3, 5, 17, 255, 1000, 5003])
@pytest.mark.parametrize("cols", [64, 257, 1024])
def test_row_counts(rows, cols):
    check(rows, cols, BF16, gtype=F16)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("pad,shift", [(8, 0), (5, 0), (0, 1), (3, 2), (1, 7), (24, 8)])
@pytest.mark.parametrize("cols", [96, 1000, 1001])
def test_strides_and_alignment(cols, pad, shift, dtype):
    check(33, cols, dtype, pad, shift, pshift=shift % 4)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("gtype", TYPES, ids=ids)
def test_types_of_the_parameter_gradients(dtype, gtype):
    check(65, 768, dtype, ptype=dtype, gtype=gtype)


@pytest.mark.parametrize("cols", [512, 515])
def test_without_parameters(cols):
    check(40, cols, F16, affine=False)


@pytest.mark.parametrize("cols", [512, 1000, 1001])
def test_rows_far_from_zero(cols):
    """A mean a thousand times the spread: a difference of squares would lose
    every digit of the variance."""
    check(50, cols, F32, mean=1000.0)
    check(50, cols, F32, mean=-3e4, scale=30.0)


@pytest.mark.parametrize("cols", [256, 257, 20000])
def test_constant_rows(cols):
    x = torch.full((9, cols), 2.5, device="cuda", dtype=BF16)
    w, b = params(cols, F32, 1)
    y, mu, rs = torch.empty_like(x), torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
    fc.fc_layernorm_forward(x, w, b, EPS, y, mu, rs)
    torch.cuda.synchronize()
    (wy, wm, wr), (ey, em, er) = ops_ref.layernorm(x, w, b, EPS)
    assert_within("y", y, wy, rounded(ey, wy, BF16))


def test_bad_values_stay_in_their_row():
    """An infinity or a NaN spoils its own row and the sums, no other row."""
    for cols in (512, 515):
        x, _ = matrix(20, cols, F16)
        w, b = params(cols, F32, 2)
        clean, dirty = torch.empty_like(x), torch.empty_like(x)
        fc.fc_layernorm_forward(x, w, b, EPS, clean)
        x[3, 7], x[11, 0] = float("inf"), float("nan")
        mu, rs = torch.empty(20, device="cuda"), torch.empty(20, device="cuda")
        fc.fc_layernorm_forward(x, w, b, EPS, dirty, mu, rs)
        torch.cuda.synchronize()
        rest = [r for r in range(20) if r not in (3, 11)]
        assert torch.equal(clean[rest], dirty[rest])
        assert bool(dirty[3].isnan().any()) and bool(dirty[11].isnan().all())


@pytest.mark.parametrize("which", ["weight", "bias", "none"])
def test_gradients_that_are_not_wanted(which):
    x, w, b, y, mu, rs, dy, dx, dw, db, ws = check(70, 320, BF16)
    dw2 = torch.empty_like(dw) if which == "weight" else None
    db2 = torch.empty_like(db) if which == "bias" else None
    dx2 = torch.empty_like(dx)
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx2, dw2, db2, None if which == "none" else ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2)
    assert dw2 is None or torch.equal(dw, dw2)
    assert db2 is None or torch.equal(db, db2)


def test_no_rows():
    x = torch.empty(0, 300, device="cuda")
    none = torch.empty(0, device="cuda")
    fc.fc_layernorm_forward(x, None, None, EPS, torch.empty_like(x), none, none)
    dw, db = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    ws = torch.empty(fc.fc_layernorm_backward_workspace_size(0, 300), dtype=torch.uint8,
                     device="cuda")
    fc.fc_layernorm_backward(x, x, None, none, none, torch.empty_like(x), dw, db, ws)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("cols", [640, 641, 20001])
def test_backward_repeats_bit_for_bit(cols):
    x, w, b, y, mu, rs, dy, dx, dw, db, ws = check(300, cols, BF16)
    for _ in range(3):
        dx2, dw2, db2 = torch.empty_like(dx), torch.empty_like(dw), torch.empty_like(db)
        fc.fc_layernorm_backward(dy, x, w, mu, rs, dx2, dw2, db2, ws)
        torch.cuda.synchronize()
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("cols", [384, 385])
def test_gradient_against_differences(cols):
    """loss(x + e d) - loss(x - e d) of the forward kernel against the gradients
    of the backward kernel, in fp32, along random directions."""
    rows, e = 12, 1e-2
    x, _ = matrix(rows, cols, F32, seed=1)
    w, b = params(cols, F32, 2)
    dy, _ = matrix(rows, cols, F32, seed=3)

    def loss(x, w, b):
        y = torch.empty_like(dy)
        fc.fc_layernorm_forward(x, w, b, EPS, y)
        return float((y.double() * dy.double()).sum())

    y, mu, rs = torch.empty_like(dy), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    fc.fc_layernorm_forward(x, w, b, EPS, y, mu, rs)
    dx, dw, db = torch.empty_like(dy), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(fc.fc_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8,
                     device="cuda")
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx, dw, db, ws)
    for seed in range(4):
        tx, _ = matrix(rows, cols, F32, seed=10 + seed)
        tw, tb = params(cols, F32, 20 + seed)
        up = loss(x + e * tx, w + e * tw, b + e * tb)
        down = loss(x - e * tx, w - e * tw, b - e * tb)
        slope = float((dx.double() * tx).sum() + (dw.double() * tw).sum() + (db.double() * tb).sum())
        # the directions' derivative is of order sqrt(rows cols) = 70; the
        # third derivative along them enters with e^2 / 6, fp32 rounding of y
        # with 1e-7 sqrt(rows cols) / e
        assert abs((up - down) / (2 * e) - slope) < 0.15, seed


def test_on_another_stream_and_in_a_graph():
    x, w, b, y, mu, rs, dy, dx, dw, db, ws = check(500, 1024, BF16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, dx2, dw2, db2 = (torch.zeros_like(t) for t in (y, dx, dw, db))
    torch.cuda.synchronize()
    fc.fc_layernorm_forward(x, w, b, EPS, y2, mu, rs, side)
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx2, dw2, db2, ws, side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    for t in (y2, dx2, dw2, db2):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fc.fc_layernorm_forward(x, w, b, EPS, y2, mu, rs)
        fc.fc_layernorm_backward(dy, x, w, mu, rs, dx2, dw2, db2, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(db, db2)


def test_binding_checks():
    x = torch.zeros(4, 8, device="cuda")
    y = torch.empty_like(x)
    stats = torch.empty(4, device="cuda")
    w = torch.ones(8, device="cuda")
    f, b = fc.fc_layernorm_forward, fc.fc_layernorm_backward
    for call in (lambda: f(x, None, None, EPS, y[:3]),
                 lambda: f(x, None, None, EPS, y.half()),
                 lambda: f(x.t(), None, None, EPS, y),
                 lambda: f(x, w[:7], None, EPS, y),
                 lambda: f(x, w.half(), None, EPS, y),
                 lambda: f(x.half(), w, w.half(), EPS, y.half()),
                 lambda: f(x, w.cpu(), None, EPS, y),
                 lambda: f(x, None, None, EPS, y, stats[:3], stats[:3]),
                 lambda: f(x.double(), None, None, EPS, y.double()),
                 lambda: b(y, x, w, stats, stats, y, w[:5], None, None),
                 lambda: b(y, x, w, stats, stats, y, w, w.half(), None)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(fc.FcError) as e:
        f(x, None, None, EPS, y, stats, None)
    assert e.value.status == fc.FC_ERR_INVALID_ARG
    with pytest.raises(fc.FcError) as e:
        b(y, x, w, stats, stats, y, w, None, None)
    assert e.value.status == fc.FC_ERR_WORKSPACE
