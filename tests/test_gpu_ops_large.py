"""The training-step operators past 2^31 elements: what lies there is checked
against the 64-bit forms."""

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import ops_ref
from tests.ops_ref import U, assert_within, rounded

pytestmark = pytest.mark.gpu

N = (1 << 31) + 5 * 256 + 77
H = dict(lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.1)


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free device memory")
    yield
    torch.cuda.empty_cache()


def windows():
    """Whole blocks at the start, around 2^31 and at the end."""
    last = (N - 1) // 256 * 256
    return [slice(0, 512), slice((1 << 31) - 256, (1 << 31) + 512), slice(last - 512, N)]


def random(n, seed, scale, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(n, dtype=dtype, device="cuda")
    for a in range(0, n, 1 << 28):
        b = min(n, a + (1 << 28))
        out[a:b] = torch.randn(b - a, generator=g, device="cuda") * scale
    return out


def test_norm_and_adamw():
    # two layers, the second from an odd element on
    first = (1 << 31) - 301
    g = random(N + 1, 1, 1e-3)
    grads = [g[:first], g[first + 1:]]
    table = fc.LayerGrads(grads, [1.0, 0.0])
    ws = torch.zeros(fc.fc_grad_norm_workspace_size(), dtype=torch.uint8, device="cuda")
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    fc.fc_grad_norm(table, 1.0, 1.0, norm, scale, ws)
    want = sum(float((x[a:a + (1 << 28)].double() ** 2).sum()) for x in grads
               for a in range(0, x.numel(), 1 << 28)) ** 0.5
    assert abs(float(norm) - want) <= 8 * U * want
    w = random(N, 2, 0.05)
    m, v = torch.zeros(N, device="cuda"), torch.zeros(N, device="cuda")
    steps = torch.zeros(2, dtype=torch.int32, device="cuda")
    parts = windows()
    w0 = [w[s].clone() for s in parts]
    fc.fc_adamw_step(table, scale, H["lr"], H["b1"], H["b2"], H["eps"], H["wd"], w, None, m, v,
                     steps)
    torch.cuda.synchronize()
    assert steps.tolist() == [1, 0]
    for s, w1 in zip(parts, w0):
        i = torch.arange(s.start, s.stop, device="cuda")
        graw = torch.where(i < first, g[i.clamp(max=first - 1)], g[(i + 1).clamp(max=N)])
        zero = torch.zeros_like(graw)
        (rw, rm, rv), (ew, em, ev) = ops_ref.adamw(
            w1, zero, zero, graw.double() * float(scale), (i < first).double(), 1, **H)
        assert_within("w", w[s], rw, ew)
        assert_within("m", m[s], rm, em)
        assert_within("v", v[s], rv, ev)


def test_adamw8():
    g = random(N, 3, 1e-3, torch.float16)
    w = random(N, 4, 0.05)
    blocks = fc.state_blocks(N)
    m8 = torch.zeros(N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    r8 = torch.zeros(N, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    ms, rs = torch.zeros(blocks, device="cuda"), torch.zeros(blocks, device="cuda")
    steps = torch.zeros(2, dtype=torch.int32, device="cuda")
    parts = windows()
    w0 = [w[s].clone() for s in parts]
    fc.fc_adamw8_step(fc.LayerGrads([g]), None, H["lr"], H["b1"], H["b2"], H["eps"], H["wd"], w,
                      None, m8, ms, r8, rs, steps, 12345)
    torch.cuda.synchronize()
    for s, w1 in zip(parts, w0):
        gd = g[s].double()
        zero, n = torch.zeros_like(gd), gd.numel()
        (rw, rm, rv), (ew, em, ev) = ops_ref.adamw(w1, zero, zero, gd, zero + 1, 1, **H)
        assert_within("w", w[s], rw, ew)
        b = slice(s.start // 256, -(-s.stop // 256))
        for codes, scales, x, ex, chance in (
                (m8, ms, rm, em, None),
                (r8, rs, rv.sqrt(), 0.5 * ev / rv.sqrt() + 2 * U * rv.sqrt(),
                 (ops_ref.random16(12345, 1, torch.arange(s.start, s.stop, device="cuda")).double()
                  + 0.5) / 65536)):
            top = ops_ref.block_top(x)
            assert_within("scale", scales[b], top / 448, (ops_ref.block_top(ex) + 2 * U * top) / 448)
            y = x.abs() / ops_ref.spread(top, n) * 448
            q = ops_ref.e4m3_quantum(y)
            err = 40 * U * y
            got = codes[s].double().abs()
            if chance is None:
                assert_within("codes", got, y, q / 2 + err)
            else:
                at = y / q + chance
                sure = (at - torch.round(at)).abs() > err / q + 2.0 ** -20
                want = torch.clamp(torch.floor(at) * q, min=2.0 ** -9)
                assert bool((got == want)[sure].all())


@pytest.mark.parametrize("cols", [8192, 8001])
def test_layernorm(cols):
    rows = (1 << 31) // cols + 40
    x = random(rows * cols, 5, 1.0, torch.bfloat16).view(rows, cols)
    dy = random(rows * cols, 6, 0.5, torch.bfloat16).view(rows, cols)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    w = random(cols, 7, 0.2) + 1
    b = random(cols, 8, 0.2)
    mu, rs = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(fc.fc_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8,
                     device="cuda")
    fc.fc_layernorm_forward(x, w, b, 1e-5, y, mu, rs)
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx, dw, db, ws)
    torch.cuda.synchronize()
    sums = torch.zeros(2, cols, dtype=torch.float64, device="cuda")
    size = torch.zeros(2, cols, dtype=torch.float64, device="cuda")
    for a in range(0, rows, 8192):
        s = slice(a, min(rows, a + 8192))
        d = dy[s].double()
        h = (x[s].double() - mu[s].double()[:, None]) * rs[s].double()[:, None]
        sums += torch.stack(((d * h).sum(0), d.sum(0)))
        size += torch.stack(((d * h).abs().sum(0), d.abs().sum(0)))
    # 3000 rows at most in a row for one thread (152 SMs, two rows at a time)
    assert_within("dweight", dw, sums[0], 3100 * U * size[0])
    assert_within("dbias", db, sums[1], 3100 * U * size[1])
    for s in (slice(0, 3), slice(rows - 60, rows)):
        (wy, wm, wr), (ey, em, er) = ops_ref.layernorm(x[s], w, b, 1e-5)
        assert_within("y", y[s], wy, rounded(ey, wy, torch.bfloat16))
        (wdx, _, _), (edx, _, _) = ops_ref.layernorm_backward(dy[s], x[s], w, mu[s], rs[s])
        assert_within("dx", dx[s], wdx, rounded(edx, wdx, torch.bfloat16))
