"""Training-step operators where their arithmetic or their launches could give way:
rows far from zero, extreme gradients and factors, several host threads."""

import threading

import pytest
import torch

from gradient_aggregation_gb300 import fc
from tests import ops_ref
from tests.ops_ref import U, assert_within, rounded
from tests.test_gpu_layernorm import matrix, params
from tests.test_gpu_optim import HYPER, State, check_codes, check_step, rnd

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
ids = lambda t: str(t).replace("torch.", "")  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _lib(fc_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield


# ---- layer norm backward ---------------------------------------------------------

def backward_with_own_bounds(dy, x, weight, mean, rstd, run=64):
    """The backward pass in 64 bits and bounds for fp32 arithmetic that follows the
    definition's order: x - mean is rounded once, and h = (x - mean) * rstd once
    more, so h is known to 3U of itself however far the row lies from zero."""
    dy, x = dy.double(), x.double()
    mean, rstd = mean.double()[:, None], rstd.double()[:, None]
    w = weight.double()
    h = (x - mean) * rstd
    q = dy * w
    s1, s2 = q.mean(1, keepdim=True), (q * h).mean(1, keepdim=True)
    dx = rstd * (q - s1 - h * s2)
    eh = 3 * U * h.abs()
    # sums of at most 2^14 terms: 32 in a row, the rest in a tree
    e1 = 45 * U * q.abs().mean(1, keepdim=True)
    e2 = 45 * U * (q * h).abs().mean(1, keepdim=True) + (q.abs() * eh).mean(1, keepdim=True)
    edx = rstd * (3 * U * (q.abs() + s1.abs() + (h * s2).abs()) + e1 + h.abs() * e2
                  + eh * s2.abs()) + 2 * U * dx.abs()
    add = (run + 24) * U
    edw = add * (dy * h).abs().sum(0) + (dy.abs() * eh).sum(0)
    return (dx, (dy * h).sum(0), dy.sum(0)), (edx, edw, add * dy.abs().sum(0))


def check_backward(x, dy, cols, eps):
    rows = x.shape[0]
    w, b = params(cols, F32, 3)
    y, dx = torch.empty(rows, cols, dtype=x.dtype, device="cuda"), torch.empty(
        rows, cols, dtype=x.dtype, device="cuda")
    mu, rs = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    ws = torch.empty(fc.fc_layernorm_backward_workspace_size(rows, cols), dtype=torch.uint8,
                     device="cuda")
    fc.fc_layernorm_forward(x, w, b, eps, y, mu, rs)
    fc.fc_layernorm_backward(dy, x, w, mu, rs, dx, dw, db, ws)
    torch.cuda.synchronize()
    (wdx, wdw, wdb), (edx, edw, edb) = backward_with_own_bounds(dy, x, w, mu, rs)
    assert_within("dx", dx, wdx, rounded(edx, wdx, x.dtype))
    assert_within("dweight", dw, wdw, rounded(edw, wdw, F32))
    assert_within("dbias", db, wdb, rounded(edb, wdb, F32))


# one width of each kernel and class: several rows a warp; vectors; rows that start
# anywhere; halves; more than the registers hold
@pytest.mark.parametrize("mean", [10.0, 1e3, -3e4])
@pytest.mark.parametrize("cols,pad", [(64, 0), (100, 1), (128, 0), (256, 0), (1000, 0), (1000, 1),
                                      (1001, 0), (2048, 0), (4096, 0), (8192, 0), (8190, 3),
                                      (12288, 0), (12290, 1), (16384, 0), (20001, 0)])
def test_backward_of_rows_far_from_zero(cols, pad, mean):
    """The gradients of a row do not depend on its distance from zero."""
    x, _ = matrix(40, cols, F32, pad, 0, 1, 1.0, mean)
    dy, _ = matrix(40, cols, F32, pad, 0, 5, 0.5)
    check_backward(x, dy, cols, 1e-5)


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids)
@pytest.mark.parametrize("cols,pad", [(512, 0), (1001, 0), (16384, 0)])
def test_backward_of_16_bit_rows_far_from_zero(cols, pad, dtype):
    x, _ = matrix(40, cols, dtype, pad, 0, 1, 30.0, 1000.0)
    dy, _ = matrix(40, cols, dtype, pad, 0, 5, 0.5)
    check_backward(x, dy, cols, 1e-5)


@pytest.mark.parametrize("cols,pad", [(64, 0), (512, 0), (1001, 0), (16384, 0), (20001, 0)])
def test_backward_of_rows_of_tiny_variance(cols, pad):
    """eps = 0 and a spread of 1e-18: rstd is 1e18 and its square times the sum of
    q h would not fit fp32, the gradient does."""
    x, _ = matrix(20, cols, F32, pad, 0, 1, 1e-18)
    dy, _ = matrix(20, cols, F32, pad, 0, 5, 1e4)
    check_backward(x, dy, cols, 0.0)


# ---- AdamW with 8-bit moments: gradients whose squares do not fit ----------------------

# below 0.9M elements the step's registers hold a unit, above they are streamed
@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
@pytest.mark.parametrize("sizes", [[256 * 5 + 77], [1 << 20, 151111, 256 + 33]], ids=len)
@pytest.mark.parametrize("size", [1e12, 2e13, 1e15, 1e18])
def test_adamw8_large_gradients(size, sizes, dtype):
    """|g| up to the square root of what fp32 holds, in blocks of their own, in blocks
    of ordinary ones and in the last block: weights, codes and scales as defined."""
    grads = [rnd(n, 3 + l) for l, n in enumerate(sizes)]
    grads[0][:256] *= size
    if len(grads) > 1:
        grads[-1][:256] *= size
    grads[0][700:703] *= size
    grads[-1][-5:] *= size
    st = check_step([g.to(dtype) for g in grads], sizes, 8, F16, 0, HYPER, scale=None, fresh=True)
    assert bool((st.rs >= 0).all())


def step_and_check_weights(st, g, k, h):
    """Step k + 1 from the moments that the state holds, 8-bit ones as they are held;
    the new moments in 64 bits and the bound on m."""
    m0, v0 = st.moments()
    w0 = st.w.clone()
    st.step(fc.LayerGrads([g]), None, h)
    torch.cuda.synchronize()
    (w, m, v), (ew, em, ev) = ops_ref.adamw(w0, m0, v0, g, torch.ones_like(w0), k + 1, **h)
    if st.bits == 8:
        em = em + U * m0.abs()
        ew = ew + (h["lr"] / (1 - h["b1"] ** (k + 1))) * U * m0.abs() / (
            torch.sqrt(v / (1 - h["b2"] ** (k + 1))) + h["eps"]) + 0.1 * ew
    assert_within("w", st.w, w, ew)
    return m, em


def test_adamw8_goes_on_after_large_gradients():
    """The blocks come back to ordinary gradients by their averages, and the state
    stays that of the definition, step after step."""
    n = 1 << 20
    st = State(n, 8, None, fresh=True)
    big, small = rnd(n, 1, 1e3), rnd(n, 2)
    big[::3000] *= 1e14
    for k, g in enumerate((big, small, small, small)):
        m, em = step_and_check_weights(st, g, k, dict(HYPER, b1=0.5, b2=0.5))
        check_codes(st.m8, st.ms, m, em, None)


@pytest.mark.parametrize("n", [1000, 1 << 20])
def test_adamw8_finite_gradients_leave_a_finite_state(n):
    """Up to the largest fp32 number: beyond 9.7e24 a gradient counts as that."""
    g = rnd(n, 5)
    g[100], g[400], g[900] = 3e38, -3e38, 1e30
    st = State(n, 8, F16, fresh=True)
    for _ in range(3):
        st.step(fc.LayerGrads([g]), None)
        torch.cuda.synchronize()
        for t in (st.w, st.ms, st.rs, st.m8.float(), st.r8.float()):
            assert bool(t.isfinite().all())
        assert bool((st.rs >= 0).all())
    assert float(st.m8[100]) * float(st.ms[0]) > 1e24
    # an element of its own block moves as one of an ordinary size does
    assert abs(float(st.w[900] - State(n, 8, F16, fresh=True).w[900])) < 4 * HYPER["lr"]
    # and one that is not finite still shows
    g[100] = float("inf")
    st.step(fc.LayerGrads([g]), None)
    torch.cuda.synchronize()
    assert not bool(st.w[100].isfinite())


# ---- AdamW: a wait that runs out ------------------------------------------------------

@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("tile", [0, 1, 100, 1 << 40])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_wait_that_runs_out(bits, tile, skip):
    """The failure path of the streamed step, without any fault: a tile that is not
    copied in.  The record stays whichever block finishes last, neither that step
    nor a later one is counted, and the tile keeps its weights; from a whole
    state the steps go on as if nothing had been."""
    n, done = 1_300_001, 7
    g = rnd(n, 1)
    table = fc.LayerGrads([g])
    scale = torch.tensor([float("nan") if skip else 1.0], device="cuda")
    st, ref = State(n, bits, BF16, done), State(n, bits, BF16, done)
    whole = st.copies()
    ref.step(table, None)
    fc.fc_test_adamw_loss(tile)
    st.step(table, scale)
    torch.cuda.synchronize()
    st.check_guards()
    assert int(st.steps[0]) == done and int(st.steps[1]) == -(1 << 31)
    same = st.w == whole["w"]
    assert bool(((st.w == ref.w) | same).all())
    # a tile, and what its block had still to do, or nothing at all
    assert bool(same.all()) if skip else 4608 <= int(same.sum()) <= 30000
    st.step(table, None)
    torch.cuda.synchronize()
    assert int(st.steps[0]) == done and int(st.steps[1]) == -(1 << 31)
    for k, v in whole.items():
        getattr(st, k).copy_(v)
    st.step(table, None)
    torch.cuda.synchronize()
    want = ref.copies()
    for k, v in st.copies().items():
        assert torch.equal(v.view(torch.uint8), want[k].view(torch.uint8)), k
    assert st.steps.tolist() == [done + 1, 0]


def test_engine_tells_of_a_wait_that_ran_out():
    sizes, W = [1_200_000], 2
    grads = [[rnd(sizes[0], w, 1.0, F16)] for w in range(W)]
    eng = fc.AdamWEngine(sizes, W, rnd(sizes[0], 9), lr=1e-3, loss_scale=64.0)
    eng.step(grads)
    assert eng.status() == fc.FC_OK
    saved = eng.state_dict()
    fc.fc_test_adamw_loss(3)
    eng.step(grads)
    assert eng.status() == fc.FC_ERR_TIMEOUT
    with pytest.raises(fc.FcError) as e:
        eng.state_dict()
    assert e.value.status == fc.FC_ERR_TIMEOUT
    eng.load_state_dict(saved)
    eng.step(grads)
    assert eng.status() == fc.FC_OK and eng.steps.tolist() == [2, 0]


def test_adamw_loss_hook_refusals():
    for limit in (0, 999_999, 2_000_000_001):
        with pytest.raises(fc.FcError):
            fc.fc_test_adamw_loss(0, limit)
    fc.fc_test_adamw_loss(-1, 0)


# ---- calls whose tensors do not fit: refused before anything is launched ---------------

def test_engine_refuses_gradients_of_another_layout():
    """The buffers of the engine hold its own sizes, no others."""
    sizes, W = [300, 77], 2
    eng = fc.AdamWEngine(sizes, W, rnd(377, 9), lr=1e-3, loss_scale=1.0)
    half = lambda *ns: [torch.zeros(n, device="cuda", dtype=F16) for n in ns]  # noqa: E731
    for grads in ([half(300, 77)], [half(300, 77)] * 3, [half(77, 300)] * 2,
                  [half(300, 77, 4000)] * 2, [half(4000, 77)] * 2, [half(300)] * 2):
        with pytest.raises(ValueError):
            eng.step(grads)
        with pytest.raises(ValueError):
            eng.step(fc.PtrTable(grads))
    eng.step([half(300, 77)] * 2)
    torch.cuda.synchronize()
    assert eng.steps.tolist() == [1, 0]


def test_workspaces_have_the_bytes_that_they_name():
    """An expanded or strided tensor has more elements than memory, or gaps."""
    g = torch.zeros(400, device="cuda")
    norm, scale = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")
    need = fc.fc_grad_norm_workspace_size()
    x = torch.zeros(8, 400, device="cuda")
    dx, w, st = torch.empty_like(x), torch.ones(400, device="cuda"), torch.zeros(8, device="cuda")
    most = max(need, fc.fc_layernorm_backward_workspace_size(8, 400))
    for ws in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(most),
               torch.zeros(2 * most, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            fc.fc_grad_norm(fc.LayerGrads([g]), 1.0, 0.0, norm, scale, ws)
        with pytest.raises(ValueError):
            fc.fc_layernorm_backward(x, x, w, st, st, dx, w.clone(), w.clone(), ws)


# ---- calls on several host threads -----------------------------------------------------

@pytest.mark.parametrize("pair", [(12291, 16383), (6152, 8192), (8200, 12288), (1537, 2047)])
def test_layernorm_widths_of_one_kernel_on_several_host_threads(pair):
    """Two widths that one kernel serves, called through the C ABI (which, unlike the
    binding, lets go of the interpreter) from four host threads on their own streams:
    no call takes away what another one's launch needs."""
    L, rows, rounds, failed = fc.lib(), 200, 2000, []

    def run(cols, seed):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            x = rnd(rows * cols, seed, 1.0, BF16).view(rows, cols)
            y, want = torch.empty_like(x), torch.empty_like(x)
            fc.fc_layernorm_forward(x, None, None, 1e-5, want)
            args = (x.data_ptr(), rows, cols, cols, fc.FC_TYPE_BF16, None, None, 0, 1e-5,
                    y.data_ptr(), cols, None, None, s.cuda_stream)
            for _ in range(rounds):
                st = L.fc_layernorm_forward(*args)
                if st:
                    failed.append((cols, st, L.fc_last_error()))
                    return
            s.synchronize()
            if not torch.equal(y, want):
                failed.append((cols, "other values"))

    threads = [threading.Thread(target=run, args=(pair[i % 2], i)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
def test_launch_sizes_are_looked_up_once_a_kernel(dtype):
    """Hundreds of widths, aligned ones and others, forward and backward: as many
    lookups as kernels at most, and none when the widths come again."""
    lookups = fc.lib().fc_test_launch_lookups
    widths = list(range(136, 16384, 96)) + list(range(131, 16384, 97))

    def all_of_them():
        for c in widths:
            rows = 300000 // c + 3
            x = torch.zeros(rows, c, dtype=dtype, device="cuda")
            mu = torch.zeros(rows, device="cuda")
            ws = torch.empty(fc.fc_layernorm_backward_workspace_size(rows, c), dtype=torch.uint8,
                             device="cuda")
            w = torch.ones(c, device="cuda")
            fc.fc_layernorm_forward(x, w, w, 1e-5, torch.empty_like(x), mu, mu.clone())
            fc.fc_layernorm_backward(x, x, w, mu, mu, torch.empty_like(x), w.clone(), w.clone(), ws)

    before = lookups()
    all_of_them()
    first = lookups()
    all_of_them()
    torch.cuda.synchronize()
    # kernels of one element type: 13 and 12 forward, 26 backward
    assert first - before <= 60
    assert lookups() == first


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-30, 1e-38, 1e-40, 2e-45])
def test_adamw_tiny_eps(bits, eps):
    """Down to the smallest fp32 number: no NaN where a gradient is and always was 0."""
    for n in (1000, 1 << 20):
        st = State(n, bits, None, fresh=True)
        w0 = st.w.clone()
        g = rnd(n, 3)
        g[:300] = 0
        g[::7] = 0
        for k in range(2):
            step_and_check_weights(st, g, k, dict(HYPER, eps=eps, wd=0.0))
        assert torch.equal(st.w[g == 0], w0[g == 0])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
@pytest.mark.parametrize("rows,cols,pad", [
    (200000, 64, 0), (200000, 61, 0), (100000, 256, 0), (60000, 257, 1), (20000, 1024, 0),
    (9000, 3000, 0), (4000, 8192, 0), (3000, 12288, 0), (3000, 12289, 0), (2000, 16384, 0),
    (2000, 16383, 1), (900, 16392, 0), (300, 70000, 0), (5, 600000, 0)])
def test_backward_keeps_to_its_scratch(rows, cols, pad, dtype):
    """Many rows of every class, with exactly the bytes asked for and a guard behind."""
    x, _ = matrix(rows, cols, dtype, pad)
    dy, _ = matrix(rows, cols, dtype, pad, seed=2)
    mu, rs = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    dw, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    need = fc.fc_layernorm_backward_workspace_size(rows, cols)
    buf = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    fc.fc_layernorm_backward(dy, x, None, mu, rs, torch.empty_like(x), dw, db, buf[:need])
    torch.cuda.synchronize()
    assert bool((buf[need:] == 0xA5).all())
    for got, terms in ((dw, lambda s: dy[s].double() * x[s].double()), (db, lambda s: dy[s].double())):
        want, size = (torch.zeros(cols, dtype=torch.float64, device="cuda") for _ in range(2))
        for a in range(0, rows, 8192):
            t = terms(slice(a, a + 8192))
            want += t.sum(0)
            size += t.abs().sum(0)
        # at worst one thread adds all rows of its block one after another
        assert_within("sums", got, want, (rows + 24) * U * size)


# ---- what 8 bits do to the moments over many steps, as include/fc.h says ---------------

def test_adamw8_second_moment_settles_above_its_average():
    """For gradients drawn anew in each step, beta2 = 0.95: 2.6 % above (a definition
    run on the CPU, 32768 elements, 200 steps: 1.0256)."""
    n = 1 << 15
    st = State(n, 8, None, fresh=True)
    h = dict(HYPER, b2=0.95, lr=0.0, wd=0.0)
    exact, got, want = torch.zeros(n, device="cuda"), 0.0, 0.0
    for t in range(400):
        g = rnd(n, 1000 + t)
        exact = 0.95 * exact + 0.05 * g * g
        st.step(fc.LayerGrads([g]), None, h)
        if t >= 200:
            got, want = got + float(st.moments()[1].mean()), want + float(exact.mean())
    # 32768 x 200 values, of which about one in 20 steps is independent
    assert abs(got / want - 1.0256) < 0.005


@pytest.mark.parametrize("spread,low,high", [(0.0, 0.2, 0.33), (0.3, 0.0, 0.03)])
def test_adamw8_first_moment_needs_gradients_that_vary(spread, low, high):
    """beta1 = 0.9, coming from another mean: where gradients hardly change m stays a
    median of 26 % off, where they spread by 0.3 of their mean it is right to 2 %."""
    n, rounds = 1 << 15, 300
    st = State(n, 8, None, seed=40)
    mean, total = rnd(n, 50, 3e-4), torch.zeros(n, dtype=torch.float64, device="cuda")
    for t in range(2 * rounds):
        g = mean * (1 + spread * rnd(n, 100 + t))
        st.step(fc.LayerGrads([g]), None, dict(HYPER, lr=0.0, wd=0.0))
        if t >= rounds:
            total += st.moments()[0]
    off = float(((total / rounds - mean) / mean).abs().median())
    assert low <= off <= high
